"""Plain forms of the calls for shared prefixes, accumulated weights and cuts by weight.

Written from the definitions, one sequence, head or slot at a time.  Test infrastructure: the
library computes nothing here.
"""
import math

import numpy as np
import torch


# ---------------------------------------------------------------- cuts by weight

def evict_row(w, pos, off, n, m, sink, recent):
    """One (layer, sequence, kv head): returns (weights, positions, [(source slot, target slot)])."""
    w_out, p_out = w.copy(), pos.copy()
    m = min(n, m)
    place = [int(pos[s]) if pos[s] >= 0 else s + off for s in range(n)]

    def order(s):
        x = float(w[s])
        return (0 if place[s] < sink or place[s] >= n + off - recent else 1, math.inf if math.isnan(x) else 0,
                0.0 if math.isnan(x) else -x, s)

    kept = sorted(range(n), key=order)[:m]
    front = set(s for s in kept if s < m)
    moves = list(zip(sorted(s for s in kept if s >= m), [s for s in range(m) if s not in front]))
    for s in front:
        p_out[s] = place[s]
    for s, d in moves:
        w_out[d], p_out[d] = w[s], place[s]
    w_out[m:n], p_out[m:n] = 0.0, -1
    return w_out, p_out, moves


def evict(w, pos, off, table, lens, new, k, v, ps, sink, recent):
    """Numpy arrays; k, v [L, P, ps, Hkv, D] are changed in place.  Returns (weights, positions, offsets)."""
    w_out, p_out = w.copy(), pos.copy()
    NL, B, H, _ = w.shape
    for layer in range(NL):
        for b in range(B):
            n, m = int(lens[b]), int(new[b])
            for h in range(H):
                w_out[layer, b, h], p_out[layer, b, h], moves = evict_row(w[layer, b, h], pos[layer, b, h], int(off[b]), n, m, sink, recent)
                for x in (k, v):
                    old = x[layer].copy() if moves else None
                    for s, d in moves:
                        x[layer, table[b, d // ps], d % ps, h] = old[table[b, s // ps], s % ps, h]
    return w_out, p_out, off + lens - np.minimum(lens, new)


# ---------------------------------------------------------------- accumulated weights

def paged_weights(q, lse, kp, table, lens, cu, w):
    """In 64 bits.  Returns the new weights, W = what each entry received and, beside it, the sum of
    weight times sum |q k| / sqrt(D) (what the rounding of the logits is relative to)."""
    Hkv, D = kp.shape[2], kp.shape[3]
    G, ps = q.shape[1] // Hkv, kp.shape[1]
    out = w.double().clone()
    got, size = torch.zeros_like(out), torch.zeros_like(out)
    for b in range(len(lens)):
        L, n = int(lens[b]), int(cu[b + 1] - cu[b])
        if n == 0 or L == 0:
            continue
        k = kp[table[b, : -(-L // ps)].long()].flatten(0, 1)[:L].double()
        rows = slice(int(cu[b]), int(cu[b + 1]))
        gone = torch.arange(L, device=q.device)[None] > (L - n + torch.arange(n, device=q.device))[:, None]
        for h in range(q.shape[1]):
            x = (q[rows, h].double() @ k[:, h // G].T) / math.sqrt(D)
            p = torch.exp(x - lse[rows, h].double()[:, None]).masked_fill(gone, 0.0)
            a = (q[rows, h].double().abs() @ k[:, h // G].abs().T) / math.sqrt(D) + lse[rows, h].double().abs()[:, None]
            got[b, h // G, :L] += p.sum(0)
            size[b, h // G, :L] += (p * a).masked_fill(gone, 0.0).sum(0)
    return out + got, got, size


def weights_bound(ref, got, size, D, rows):
    """|result - ref|: a logit is D products summed in fp32 and scaled, and its distance from the
    log-sum-exp one rounding of each: at most (D + 6) 2^-24 of |q| |k| + |lse| off, which e^x takes over as a
    relative error; 2^-21 for the exponential; `rows` additions in fp32 at most rows 2^-24 of the sum; the
    last addition and what was there before half a step of the result."""
    return (D + 6) * 2.0 ** -24 * size * 1.01 + (2.0 ** -21 + rows * 2.0 ** -24) * got + 2.0 ** -23 * ref.abs() + 1e-30
