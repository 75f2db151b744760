"""Plain 64-bit forms of the paged-cache calls, and bounds of the kernels' rounding.

Written from the definitions, one sequence and one page at a time.  Test infrastructure:
the library computes nothing here.
"""
import math

import numpy as np
import torch


def rope_angles(rot, theta, scaling="none", factor=1.0, orig=0, fast=32.0, slow=1.0):
    i = np.arange(rot // 2, dtype=np.float64)
    if scaling == "base":
        theta = theta * factor ** (rot / (rot - 2.0))
    f = theta ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        g = np.clip((orig * f / (2 * np.pi) - slow) / (fast - slow), 0.0, 1.0)
        f = f * (g + (1 - g) / factor)
    return f


def rotate(x, pos, f, layout, mscale=1.0):
    """x [n, H, D] float64 at positions pos [n]."""
    rot = 2 * len(f)
    a = np.arange(0, rot, 2) if layout == "interleaved" else np.arange(rot // 2)
    b = a + 1 if layout == "interleaved" else a + rot // 2
    ang = np.asarray(pos, np.float64)[:, None, None] * f
    c, s = np.cos(ang) * mscale, np.sin(ang) * mscale
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def attend(q, k, v, first):
    """q [n, Hq, D], k, v [L, Hkv, D] float64 tensors; row i sees keys 0 .. first + i.
    Returns o, lse, A = sum p |v| (what rounding of the weights is relative to) and
    S = the largest sum |q k| / sqrt(D) of the row (what rounding of the logits is)."""
    n, Hq, D = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    G = Hq // Hkv
    o, A = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device)
    S = torch.zeros((n, Hq), dtype=torch.float64, device=q.device)
    last = first + torch.arange(n, device=q.device)
    gone = torch.arange(L, device=q.device)[None] > last[:, None]
    rows = (last >= 0) & (L > 0)
    if L == 0 or not bool(rows.any()):
        return o, lse, A, S
    for h in range(Hq):
        x = (q[:, h] @ k[:, h // G].T) / math.sqrt(D)
        x = x.masked_fill(gone, -math.inf)
        z = torch.logsumexp(x, -1)
        p = torch.exp(x - torch.where(rows, z, 0.0)[:, None])
        o[:, h] = torch.where(rows[:, None], p @ v[:, h // G], 0.0)
        A[:, h] = torch.where(rows[:, None], p @ v[:, h // G].abs(), 0.0)
        S[:, h] = (q[:, h].abs() @ k[:, h // G].abs().T).amax(-1) / math.sqrt(D)
        lse[:, h] = torch.where(rows, z, -math.inf)
    return o, lse, A, S


def paged_attend(q, kp, vp, table, lens, cu, W_rows=None):
    """The whole call over packed rows; outputs of rows outside the sequences are NaN."""
    N, Hq, D = q.shape
    ps = kp.shape[1]
    out = [torch.full((N, Hq, D), math.nan, dtype=torch.float64, device=q.device) for _ in range(2)]
    lse, S = (torch.full((N, Hq), math.nan, dtype=torch.float64, device=q.device) for _ in range(2))
    for b in range(len(lens)):
        L, n = int(lens[b]), int(cu[b + 1] - cu[b])
        if n == 0:
            continue
        pages = table[b, : -(-L // ps)].long()
        k = kp[pages].flatten(0, 1)[:L].double()
        v = vp[pages].flatten(0, 1)[:L].double()
        sl = slice(int(cu[b]), int(cu[b + 1]))
        out[0][sl], lse[sl], out[1][sl], S[sl] = attend(q[sl].double(), k, v, L - n)
    return out[0], lse, out[1], S


def attn_bounds(ref, A, S, lse, D, L, out_half_step, p_half_step):
    """Element-wise bounds of |o - ref| and |lse - ref|.

    Logits: D products summed in fp32, scaled once: at most (D + 4) 2^-24 S off; a weight's
    relative error is twice that (its own logit and the row's maximum cancel in the
    quotient) plus 2^-21 for the exponential and its argument's rounding (|x| below 2^6),
    plus p_half_step where the weights are rounded for the product; L fp32 additions add at
    most L 2^-24 (numerator and denominator each).  Each of these is relative to A.  The
    output's rounding is relative to the output."""
    e = (D + 4) * 2.0 ** -24 * S
    weights = 2 * e + 2.0 ** -21 + p_half_step + 2 * L * 2.0 ** -24
    tol_o = out_half_step * ref.abs() + weights[..., None] * A + 1e-30
    tol_lse = e + (L + 8) * 2.0 ** -24 + 2.0 ** -22 * lse.abs()
    return tol_o, tol_lse


# ---------------------------------------------------------------- pages, one at a time

class Short(Exception):
    """The pool has too few free pages (args[0]: how many are missing)."""


def fork(ref, table, lens, parents, ps, deep):
    """Returns (ref, child table, child lens, copies [(src, dst, slots)])."""
    ref, W = ref.copy(), table.shape[1]
    free = [p for p in range(len(ref)) if ref[p] == 0]
    ct, cl, copies, taken = np.full((len(parents), W), -1, np.int32), np.zeros(len(parents), np.int32), [], 0
    for c, p in enumerate(parents):
        if p < 0:
            continue
        L = int(lens[p])
        cl[c] = L
        for e in range(-(-L // ps)):
            filled = min(ps, L - e * ps)
            if deep or filled < ps:
                if taken < len(free):
                    ct[c, e] = free[taken]
                    copies.append((int(table[p, e]), free[taken], filled))
                taken += 1
            else:
                ct[c, e] = table[p, e]
    if taken > len(free):
        raise Short(taken - len(free))
    for e in ct[ct >= 0]:
        ref[e] += 1
    return ref, ct, cl, copies


def resize(ref, table, old, new, ps):
    """Returns (ref, table, copies)."""
    ref, out, copies = ref.copy(), table.copy(), []
    B = len(old)
    for b in range(B):
        for e in range(-(-int(new[b]) // ps), -(-int(old[b]) // ps)):
            ref[table[b, e]] -= 1
    held = ref.copy()
    free = [p for p in range(len(ref)) if held[p] == 0]
    taken = 0

    def take():
        nonlocal taken
        taken += 1
        return free[taken - 1] if taken <= len(free) else -1

    for b in range(B):
        po, pn, low = -(-int(old[b]) // ps), -(-int(new[b]) // ps), min(int(old[b]), int(new[b]))
        out[b] = -1
        out[b, :min(po, pn)] = table[b, :min(po, pn)]
        if low % ps and held[table[b, low // ps]] > 1:
            src, dst = int(table[b, low // ps]), take()
            out[b, low // ps] = dst
            copies.append((src, dst, low % ps))
            if dst >= 0:
                ref[src] -= 1
                ref[dst] = 1
        for e in range(po, pn):
            out[b, e] = take()
            if out[b, e] >= 0:
                ref[out[b, e]] = 1
    if taken > len(free):
        raise Short(taken - len(free))
    return ref, out, copies


def compact(ref, table, ps):
    """Returns (ref, table, remap, n_live, copies)."""
    live = [p for p in range(len(ref)) if ref[p] > 0]
    n = len(live)
    holes = [p for p in range(n) if ref[p] == 0]
    remap = np.full(len(ref), -1, np.int32)
    copies = []
    for p in live:
        remap[p] = p if p < n else holes[len(copies)]
        if p >= n:
            copies.append((p, int(remap[p]), ps))
    out = np.zeros_like(ref)
    for p in live:
        out[remap[p]] = ref[p]
    t = np.where(table >= 0, remap[np.maximum(table, 0)], -1).astype(np.int32)
    return out, t, remap, n, copies
