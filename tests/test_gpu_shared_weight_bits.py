"""How many bits the attention over shared prefixes keeps of a softmax weight: with few rows per sequence, and
at head_dim 32 with any, those of ne_paged_attn (two bf16 terms).  On the inputs of test_gpu_paged_weights, whose
outputs nearly vanish beside the sum of their terms: every sequence of a group holds the same keys and values and
asks the same, so one sequence's 64-bit result is every one's."""
import numpy as np
import pytest
import torch

import causal_gqa_flash_attention_gb300 as ne
from causal_gqa_flash_attention_gb300 import _build

import paged_ref as ref
import test_gpu_paged_weights as one

BF16 = torch.bfloat16
PS = 16

# sequences, then n, L, Hq, Hkv, D, max_new: both subtiles of a prefix's row tile and one, 32 rows a sequence, own
# positions of one key and of many, several row tiles at head_dim 32, several groups' worth of prefix tiles.
CASES = [(64, (1, 1064, 12, 4, 64, 1)), (5, (1, 517, 8, 1, 64, 1)), (7, (8, 600, 8, 2, 64, 8)), (3, (1, 2048 + 257, 6, 2, 64, 1)),
         (37, (1, 1300, 16, 4, 128, 1)), (3, (2, 900, 8, 4, 128, 2)), (20, (1, 640, 32, 2, 128, 1)),
         (6, (1, 530, 4, 2, 32, 1)), (3, (5, 700, 12, 2, 32, 5)), (3, (70, 800, 4, 2, 32, 70))]


def test_a_missing_remainder_exceeds_the_bound():
    """No GPU: one bf16 term per weight is caught on these inputs, two are not."""
    for _, c in CASES:
        one.test_a_missing_remainder_exceeds_the_bound(*c)


@pytest.mark.gpu
@pytest.mark.parametrize("B,c", CASES)
def test_shared_steps_keep_sixteen_bits_of_a_weight(B, c):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    ne.load()
    n, L, Hq, Hkv, D, max_new = c
    q, k, v = one.case(n, L, Hq, Hkv, D)
    want, tol, tol_lse = one.bounds(q, k, v, D, one.HALF ** 2)
    P = -(-L // PS)
    pages = torch.randperm(P, generator=torch.Generator().manual_seed(1))
    kp, vp = (torch.zeros(P, PS, Hkv, D, dtype=BF16, device="cuda") for _ in "kv")
    for pool, x in ((kp, k), (vp, v)):
        flat = torch.zeros(P * PS, Hkv, D, dtype=BF16)
        flat[:L] = x.to(BF16)
        pool[pages] = flat.view(P, PS, Hkv, D).cuda()
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
    W = max(P, (300 << 20) // (B * PS * Hkv * 2 * D * 2) + 1)      # (tables that could hold much: the call does share)
    table = torch.full((B, W), P + 9)
    table[:, :P] = pages
    cu = np.arange(B + 1) * n
    qs = q.to(BF16).cuda().repeat(B, 1, 1)
    o, lse = ne.paged_attn_shared(qs, kp, vp, i32(table), i32([L] * B), i32([0, B]), i32([L - n]), i32(cu), max_new=max_new)
    torch.cuda.synchronize()
    assert ne.get_device_error() == ne.NE_OK
    ratio = ((o.double().cpu().view(B, n, Hq, D) - want).abs() / tol).amax()
    assert float(ratio) <= 1, float(ratio)
    assert bool(((lse.double().cpu().view(B, n, Hq) - ref.attend(q, k, v, L - n)[1]).abs() <= tol_lse).all())
