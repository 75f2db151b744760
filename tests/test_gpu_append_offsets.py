"""paged_append with an offset per sequence: bit for bit what a call per sequence with that offset writes."""
import numpy as np
import pytest
import torch

import causal_gqa_flash_attention_gb300 as ne
from causal_gqa_flash_attention_gb300 import _build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    ne.load()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype,layout", [(torch.bfloat16, "interleaved"), (torch.float32, "half")])
@pytest.mark.parametrize("n,lens,offs", [([1, 1, 1], [5, 64, 33], [0, 1000003, 17]), ([7, 0, 40], [20, 3, 40], [(1 << 30) - 1, 2, 0])])
def test_offsets(dtype, layout, n, lens, offs):
    g = torch.Generator(device="cuda").manual_seed(4)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    N, Hq, Hkv, D, ps = sum(n), 4, 2, 64, 16
    cu = np.concatenate([[0], np.cumsum(n)])
    table = i32(np.arange(15)[::-1].reshape(3, 5).copy())
    q, k, v = mk(N, Hq, D), mk(N, Hkv, D), mk(N, Hkv, D)
    spec = ne.rope_spec(D, layout=layout)
    pools = [torch.zeros(15, ps, Hkv, D, dtype=dtype, device="cuda") for _ in range(4)]
    got = ne.paged_append(k, v, pools[0], pools[1], table, i32(lens), i32(cu), rope=spec, pos_offset=i32(offs), q=q)
    want = torch.zeros_like(got)
    for b in range(3):
        sl = slice(int(cu[b]), int(cu[b + 1]))
        if n[b]:
            want[sl] = ne.paged_append(k[sl], v[sl], pools[2], pools[3], table[b:b + 1], i32(lens[b:b + 1]), i32([0, n[b]]), rope=spec,
                                       pos_offset=offs[b], q=q[sl])
    torch.cuda.synchronize()
    assert ne.get_device_error() == ne.NE_OK
    assert torch.equal(got, want) and torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])


def test_bad_offset_is_reported():
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    for off in (-1, 1 << 30):
        ne.paged_append(k, k, pool, pool.clone(), i32([[0], [1]]), i32([1, 1]), rope=ne.rope_spec(64), pos_offset=i32([0, off]))
        assert ne.get_device_error() == ne.NE_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        ne.paged_append(k, k, pool, pool.clone(), i32([[0], [1]]), i32([1, 1]), rope=ne.rope_spec(64), pos_offset=i32([0]))
    assert ne.get_device_error() == ne.NE_OK
