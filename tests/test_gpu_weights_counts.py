"""Which rows the accumulated weights count, exactly: with queries of zeros a weight is 2^(-lse log2 e), 1 where the
log-sum-exp is 0 and 0 where it is large, so every entry is a whole number of rows and any row that is lost, counted
twice or taken for another shows, however many there are (a bound of rounding hides one of thousands)."""
import numpy as np
import pytest
import torch

import causal_gqa_flash_attention_gb300 as ne
from causal_gqa_flash_attention_gb300 import _build

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    ne.load()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype,Hq,Hkv,D,n,lens,max_new", [
    # One head's units over many CTAs, whole prompts and chunks.
    (BF16, 3, 1, 64, [3000], [3000], None), (BF16, 8, 1, 64, [512], [512], None), (BF16, 16, 1, 128, [700], [2000], None),
    (BF16, 16, 4, 128, [2048], [16384], None), (BF16, 12, 4, 32, [1500], [4000], None), (F32, 8, 1, 64, [200], [300], None),
    (F32, 12, 4, 64, [700], [3000], None), (F32, 4, 2, 32, [512, 77], [4000, 100], None),
    # Mixed batches, empty sequences, more heads than a tile has rows, few rows, wrong hints.
    (BF16, 12, 4, 64, [300, 1, 0, 512, 1, 77], [4096, 1000, 300, 512, 1, 900], 512), (BF16, 130, 1, 64, [40, 3], [300, 3], None),
    (F32, 70, 1, 32, [9, 40], [300, 41], None), (BF16, 12, 4, 64, [1] * 40, list(range(40, 80)), 1), (BF16, 8, 2, 128, [4, 1, 3], [700, 1, 90], 4),
    (F32, 4, 2, 32, [1, 1], [128, 65], 1), (BF16, 6, 2, 64, [60, 7], [300, 7], 1),
])
def test_every_row_counts_once(dtype, Hq, Hkv, D, n, lens, max_new):
    rng = np.random.default_rng(sum(lens) + Hq)
    ps, B, G = 16, len(n), Hq // Hkv
    cu = np.concatenate([[0], np.cumsum(n)])
    W = -(-max(lens) // ps) + 1
    table = rng.permutation(B * W).reshape(B, W)
    kp = torch.randn(B * W, ps, Hkv, D, device="cuda").to(dtype)
    take = rng.integers(0, 4, (cu[-1], Hq)) > 0             # three rows of four
    lse = torch.where(torch.tensor(take, device="cuda"), 0.0, 1e30).float()
    base = rng.integers(0, 100, (B, Hkv, W * ps)).astype(np.float32)
    want = base.copy()
    for b in range(B):
        seen = np.zeros((Hkv, lens[b] + 1))                 # rows whose last key this is
        for i in range(n[b]):
            if (t := lens[b] - n[b] + i) >= 0:
                seen[:, t] += take[cu[b] + i].reshape(Hkv, G).sum(1)
        want[b, :, :lens[b]] += seen[:, ::-1].cumsum(1)[:, ::-1][:, :lens[b]]
    q = torch.zeros(cu[-1], Hq, D, dtype=dtype, device="cuda")
    out = ne.paged_weights(q, lse, kp, i32(table), i32(lens), torch.tensor(base).cuda(), i32(cu), max_new=max_new)
    torch.cuda.synchronize()
    assert ne.get_device_error() == ne.NE_OK
    for b in range(B):
        assert np.array_equal(out[b, :, :lens[b]].cpu().numpy(), want[b, :, :lens[b]])
