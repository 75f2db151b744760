"""How many bits the few-row bf16 attention keeps of a softmax weight.

Those kernels multiply a weight as two bf16 terms, its value and the remainder.  On ordinary
data the output's own rounding to bf16 hides what the remainder adds, so the cases here make
outputs that nearly vanish beside the sum of their terms: every 16th key is zero (logit 0, the
row's maximum, weight 1, exact in bf16), the others are the first unit vector, so that all of
them have the one weight w = exp(-t / sqrt D) of a row with q[0] = -t.  Values are 1 behind the
latter and -c behind the former, with c chosen per column so that n w - m c is nearly 0 for the
row that the column belongs to (n and m keys of either kind).  t is picked where w lies far from
its bf16 neighbours, and a weight of one bf16 term then shows beyond the bound (2 to 36 times,
less over more keys, as the bound grows with the number of additions).
"""
import math

import numpy as np
import pytest
import torch

import causal_gqa_flash_attention_gb300 as ne
from causal_gqa_flash_attention_gb300 import _build

import paged_ref as ref

BF16 = torch.bfloat16
HALF = torch.finfo(BF16).eps / 2
EVERY = 16                                                 # (a step of a warp has 16 or 32 keys: a zero key in each)


def bf16(x):
    """Rounded to bf16, as float64."""
    return torch.tensor(x, dtype=torch.float64).to(BF16).double()


def queries(rows, D):
    """t of every row: bf16 values whose weight is at least 0.7 half steps from a bf16 one."""
    t = torch.arange(0.25, 8.0, 2.0 ** -6, dtype=torch.float64) * math.sqrt(D) / 8
    t = torch.unique(t.to(BF16).double())
    w = torch.exp(-t / math.sqrt(D))
    step = 2.0 ** (torch.floor(torch.log2(w)) - 8)         # half a step at w
    far = t[((w - w.to(BF16).double()).abs() > 0.7 * step) & (w > 0.3)]
    assert far.numel() >= 8
    return far[torch.arange(rows) % far.numel()]


def case(n, L, Hq, Hkv, D):
    """q [n, Hq, D] and one sequence's k, v [L, Hkv, D] (float64 of bf16 values)."""
    G = Hq // Hkv
    g = torch.Generator().manual_seed(L + D + Hq)
    q = torch.randn(n, Hq, D, generator=g).to(BF16).double()
    t = queries(n * G, D).view(n, 1, G).expand(n, Hkv, G).reshape(n, Hq)
    q[..., 0] = -t
    k, v = torch.zeros(L, Hkv, D, dtype=torch.float64), torch.ones(L, Hkv, D, dtype=torch.float64)
    zero = torch.arange(L) % EVERY == 0
    k[~zero, :, 0] = 1.0
    for d in range(D):                                     # column d belongs to row d % (n G) of each kv head
        r = d % (n * G)
        last = L - n + r // G
        m = int(zero[:last + 1].sum())
        w = math.exp(-float(t[r // G, r % G]) / math.sqrt(D))
        v[zero, :, d] = -bf16((last + 1 - m) * w / m)
    return q, k, v


def bounds(q, k, v, D, p_half_step):
    o, lse, A, S = ref.attend(q, k, v, k.shape[0] - q.shape[0])
    return (o, *ref.attn_bounds(o, A, S, lse, D, k.shape[0], HALF, p_half_step))


def with_rounded_weights(q, k, v, terms):
    """The attention with weights of `terms` bf16 terms each (relative to the row's maximum, 1)."""
    n, Hq, D = q.shape
    L, G = k.shape[0], Hq // k.shape[1]
    o = torch.zeros_like(q)
    gone = torch.arange(L)[None] > (L - n + torch.arange(n))[:, None]
    for h in range(Hq):
        p = torch.exp((q[:, h] @ k[:, h // G].T) / math.sqrt(D)).masked_fill(gone, 0.0)
        kept, rest = torch.zeros_like(p), p
        for _ in range(terms):
            kept = kept + rest.to(BF16).double()
            rest = p - kept
        o[:, h] = kept @ v[:, h // G] / p.sum(-1, keepdim=True)
    return o.to(BF16).double()


# n, L, Hq, Hkv, D, max_new: 16 rows, 32 rows, two chunks at head_dim 32, more heads than a tile has rows.
CASES = [(1, 512, 12, 4, 64, 1), (1, 3008, 8, 1, 64, 1), (2, 250, 8, 4, 128, 2), (1, 640, 32, 2, 128, 1), (8, 333, 8, 2, 64, 8),
         (1, 96, 4, 2, 32, 1), (5, 700, 12, 2, 32, 5), (70, 300, 4, 2, 32, 70), (2, 401, 130, 1, 64, 2), (3, 48, 4, 4, 64, 3)]


@pytest.mark.parametrize("n,L,Hq,Hkv,D,max_new", CASES)
def test_a_missing_remainder_exceeds_the_bound(n, L, Hq, Hkv, D, max_new):
    """No GPU: one bf16 term per weight is caught on these inputs, two are not."""
    q, k, v = case(n, L, Hq, Hkv, D)
    want, tol, _ = bounds(q, k, v, D, HALF ** 2)
    assert bool(((with_rounded_weights(q, k, v, 2) - want).abs() <= tol).all())
    worst = ((with_rounded_weights(q, k, v, 1) - want).abs() / tol).amax(-1)
    rows = min(n * Hq // Hkv, D)                           # those that a column belongs to
    hit = worst.view(n, Hkv, Hq // Hkv).transpose(1, 2).reshape(-1, Hkv)[:rows]
    assert bool((hit > 1).all()), float(hit.min())


@pytest.mark.gpu
@pytest.mark.parametrize("n,L,Hq,Hkv,D,max_new", CASES)
def test_few_row_kernels_keep_sixteen_bits_of_a_weight(n, L, Hq, Hkv, D, max_new):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    ne.load()
    q, k, v = case(n, L, Hq, Hkv, D)
    want, tol, tol_lse = bounds(q, k, v, D, HALF ** 2)
    ps = 16
    P = -(-L // ps)
    pages = torch.randperm(P, generator=torch.Generator().manual_seed(1))
    kp, vp = (torch.zeros(P, ps, Hkv, D, dtype=BF16, device="cuda") for _ in "kv")
    for pool, x in ((kp, k), (vp, v)):
        flat = torch.zeros(P * ps, Hkv, D, dtype=BF16)
        flat[:L] = x.to(BF16)
        pool[pages] = flat.view(P, ps, Hkv, D).cuda()
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
    o, lse = ne.paged_attn(q.to(BF16).cuda(), kp, vp, i32(pages[None]), i32([L]), i32([0, n]), max_new=max_new)
    torch.cuda.synchronize()
    assert ne.get_device_error() == ne.NE_OK
    e = (o.double().cpu() - want).abs()
    assert bool((e <= tol).all()), float((e / tol).max())
    assert bool(((lse.double().cpu() - ref.attend(q, k, v, L - n)[1]).abs() <= tol_lse).all())
