"""Accumulated attention weights on the GPU against the 64-bit form of serving_ref, with its bounds."""
import math

import numpy as np
import pytest
import torch

import causal_gqa_flash_attention_gb300 as ne
from causal_gqa_flash_attention_gb300 import _build, synthetic

import paged_ref
import serving_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    ne.load()


def ok():
    torch.cuda.synchronize()
    assert ne.get_device_error() == ne.NE_OK, ne.last_error()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def make(dtype, Hq, Hkv, D, ps, n, lens, seed, hnd=False, tail=0, lead=0, sigma=2.0):
    """Inputs of a call; what it must not read is NaN, table entries in nobody's use lie outside the pool."""
    rng = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(n)]) + lead
    N, B = int(cu[-1]) + tail, len(lens)
    W = max(1, max(-(-x // ps) for x in lens)) + 1
    P = sum(-(-x // ps) for x in lens) + 2
    table, perm, at = np.full((B, W), P + 9, np.int32), rng.permutation(P), 0
    for b, x in enumerate(lens):
        table[b, :-(-x // ps)] = perm[at:at - (-x // ps)]
        at += -(-x // ps)
    kp = synthetic.randn((P, Hkv, ps, D) if hnd else (P, ps, Hkv, D), seed + 1, 1.0, dtype).cuda()
    kp = kp.transpose(1, 2) if hnd else kp
    used = torch.zeros(P, ps, dtype=torch.bool)
    for b, x in enumerate(lens):
        for e in range(-(-x // ps)):
            used[table[b, e], :min(ps, x - e * ps)] = True
    kp.masked_fill_(~used.cuda()[:, :, None, None], math.nan)
    q = synthetic.randn((N, Hq, D), seed + 2, sigma, dtype).cuda()
    outside = torch.ones(N, dtype=torch.bool, device="cuda")
    outside[int(cu[0]):int(cu[-1])] = False
    q[outside] = math.nan
    t = i32(np.where(table > P, 0, table))
    _, lse, _, _ = paged_ref.paged_attend(q, kp, kp, t, lens, cu)
    w = torch.rand((B, Hkv, W * ps), generator=torch.Generator().manual_seed(seed)).cuda()
    return q, lse.float(), kp, i32(table), i32(lens), w, i32(cu), t, cu, outside


def check(dtype, Hq, Hkv, D, ps, n, lens, seed=1, max_new=None, mode="new", **kw):
    q, lse, kp, table, ln, w, dcu, t, cu, _ = make(dtype, Hq, Hkv, D, ps, n, lens, seed, **kw)
    base = torch.zeros_like(w) if mode == "none" else w
    want, got, size = ref.paged_weights(q, lse, kp, t, lens, cu, base)
    out = w if mode == "same" else torch.full_like(w, 7.0)
    keep = out.clone()
    res = ne.paged_weights(q, lse, kp, table, ln, None if mode == "none" else w, dcu, max_new=max_new, weights_out=out)
    ok()
    assert res is out
    live = torch.arange(w.shape[-1], device="cuda") < ln[:, None, None]
    live = live.expand_as(w)
    assert torch.equal(out[~live], keep[~live])
    G = Hq // Hkv
    tol = ref.weights_bound(want, got, size, D, G * max(1, max(n)))
    err = (out.double() - want).abs()
    assert bool(torch.isfinite(out[live]).all())
    assert bool((err <= tol)[live].all()), f"{int((err > tol)[live].sum())} of {int(live.sum())}, worst ratio {float((err / tol)[live].max())}"
    return out


@pytest.mark.parametrize("dtype,Hq,Hkv,D,ps,lens", [
    (BF16, 12, 4, 64, 16, [1, 2, 31, 32, 33, 127, 128, 129, 1000]),
    (BF16, 16, 4, 128, 64, [1, 63, 64, 65, 700]),
    (BF16, 8, 8, 32, 8, [5, 8, 9, 33]),
    (BF16, 10, 2, 64, 256, [4097, 31]),
    (BF16, 22, 2, 64, 16, [77, 513]),
    (BF16, 40, 2, 128, 16, [77, 0, 213]),
    (BF16, 71, 1, 64, 128, [130, 1, 999]),
    (F32, 4, 2, 32, 16, [1, 128, 64, 100]),
    (F32, 12, 4, 64, 8, [7, 8, 9, 1025]),
    (F32, 20, 2, 64, 16, [40, 300]),
    (F32, 70, 1, 32, 16, [40, 300]),
])
def test_one_token(dtype, Hq, Hkv, D, ps, lens):
    check(dtype, Hq, Hkv, D, ps, [min(1, x) for x in lens], lens, max_new=1)


# (new tokens, lengths): ragged, empty sequences, sequences without new tokens, prompts, more rows than positions
BATCHES = [
    ([5, 1, 0, 130, 33], [700, 129, 64, 130, 1000]),
    ([300, 0, 2], [300, 0, 500]),
    ([257, 41, 85], [128, 41, 4100]),
]


@pytest.mark.parametrize("n,lens", BATCHES)
@pytest.mark.parametrize("dtype,Hq,Hkv,D,ps", [
    (BF16, 12, 4, 64, 16), (BF16, 8, 2, 128, 64), (BF16, 6, 2, 32, 8), (BF16, 5, 1, 64, 256), (BF16, 160, 1, 64, 32), (BF16, 4, 4, 128, 128),
    (F32, 12, 4, 64, 16), (F32, 4, 2, 32, 8), (F32, 70, 1, 64, 64),
])
def test_chunks(dtype, Hq, Hkv, D, ps, n, lens):
    check(dtype, Hq, Hkv, D, ps, n, lens, seed=3)


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (BF16, 32), (F32, 64), (F32, 32)])
@pytest.mark.parametrize("max_new", [1, 4, 8, 1000])
def test_any_max_new_is_right(dtype, D, max_new):
    check(dtype, 6, 2, D, 16, [7, 1, 60, 0], [300, 1, 61, 20], max_new=max_new, seed=5)


@pytest.mark.parametrize("dtype,D,n", [(BF16, 64, [1, 1]), (BF16, 128, [50, 3]), (F32, 32, [1, 1]), (F32, 64, [50, 3])])
@pytest.mark.parametrize("mode", ["same", "none", "new"])
def test_padding_layouts_and_outputs(dtype, D, n, mode):
    check(dtype, 8, 4, D, 16, n, [130, 77], hnd=True, tail=5, lead=3, mode=mode, max_new=max(n), seed=7)


def test_without_row_offsets():
    q, lse, kp, table, ln, w, cu, *_ = make(BF16, 12, 4, 64, 16, [1, 1, 1], [40, 1, 300], 9)
    a = ne.paged_weights(q, lse, kp, table, ln, w, cu, max_new=1)
    b = ne.paged_weights(q, lse, kp, table, ln, w)
    ok()
    assert torch.equal(a, b)


def test_no_rows_at_all_copies():
    kp = torch.zeros(4, 16, 2, 64, dtype=BF16, device="cuda")
    w = torch.rand(2, 2, 32, device="cuda")
    e = torch.zeros(0, 4, 64, dtype=BF16, device="cuda")
    out = ne.paged_weights(e, torch.zeros(0, 4, device="cuda"), kp, i32([[0, 1], [2, 3]]), i32([20, 32]), w, i32([0, 0, 0]))
    ok()
    assert torch.equal(out[0, :, :20], w[0, :, :20]) and torch.equal(out[1], w[1]) and bool((out[0, :, 20:] == 0).all())


@pytest.mark.parametrize("dtype,n", [(BF16, 1), (BF16, 20), (F32, 1), (F32, 20)])
def test_many_sequences(dtype, n):
    """More than one pass of the search for the shares."""
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 60, 1000)
    lens[[0, 999]] = 0
    check(dtype, 4, 2, 32 if dtype == F32 else 64, 8, [int(min(n, x)) for x in lens], [int(x) for x in lens], max_new=n, seed=11)


@pytest.mark.parametrize("dtype,Hq,D,n,L", [(BF16, 8, 64, 512, 512), (BF16, 16, 128, 700, 2000), (F32, 8, 64, 200, 300), (BF16, 3, 64, 3000, 3000)])
def test_units_cut_over_many_ctas(dtype, Hq, D, n, L):
    """One kv head: a unit's query tiles lie on many CTAs; the same call gives the same bits."""
    a = check(dtype, Hq, 1, D, 16, [n], [L], seed=13)
    b = check(dtype, Hq, 1, D, 16, [n], [L], seed=13)
    assert torch.equal(a, b)


def test_sums_to_the_rows():
    """Every row's weights sum to one: over all positions the entries receive rows times heads."""
    q, lse, kp, table, ln, w, cu, *_ = make(BF16, 12, 4, 64, 16, [100, 1], [400, 90], 15)
    got = ne.paged_weights(q, lse, kp, table, ln, None, cu).double().sum(-1)
    ok()
    want = torch.tensor([[300.0] * 4, [3.0] * 4], dtype=torch.float64, device="cuda")
    assert bool(((got - want).abs() < 1e-4 * want).all())


def test_bad_device_arguments_are_reported():
    for bad in ("len", "cu", "page"):
        for n in ([1, 1], [40, 40]):
            q, lse, kp, table, ln, w, cu, *_ = make(BF16, 12, 4, 64, 16, n, [64, 64], 17)
            if bad == "len":
                ln[0] = 10000
                table[0] = 0
            if bad == "cu":
                cu[0] = -4
            if bad == "page":
                table[0, 0] = 1 << 22
            good = w.clone()
            out = ne.paged_weights(q, lse, kp, table, ln, w, cu, max_new=max(n))
            torch.cuda.synchronize()
            assert ne.get_device_error() == ne.NE_ERR_INVALID_ARG, bad
            assert bool(torch.isfinite(out[1, :, :64]).all()) and bool((out[1, :, :64] >= good[1, :, :64]).all())
    ok()


def test_captured_and_on_another_stream():
    for n in (1, 60):
        q, lse, kp, table, ln, w, cu, *_ = make(BF16, 12, 4, 64, 16, [n, n], [300, 120], 19)
        want = ne.paged_weights(q, lse, kp, table, ln, w, cu, max_new=n)
        out, ws = torch.zeros_like(w), ne.alloc_weights_workspace()
        torch.cuda.synchronize()
        side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(g, stream=side):
                ne.paged_weights(q, lse, kp, table, ln, w, cu, max_new=n, weights_out=out, workspace=ws)
            g.replay()
            g.replay()
        side.synchronize()
        ok()
        live = torch.arange(w.shape[-1], device="cuda") < ln[:, None, None]
        assert torch.equal(out[live.expand_as(out)], want[live.expand_as(out)])


def test_offsets_beyond_32_bits():
    P, ps, H, D = 70000, 64, 4, 128                         # 9.2 GB
    kp = torch.empty(P, ps, H, D, dtype=BF16, device="cuda")
    ids = [P - 1, 5, P - 2, 3]
    kp[ids] = torch.randn(4, ps, H, D, device="cuda").to(BF16)
    small = kp[ids].clone()
    for n in (1, 30):
        q = synthetic.randn((n, 8, D), 3, 1.0, BF16).cuda()
        lse = torch.full((n, 8), 5.0, device="cuda")
        a = ne.paged_weights(q, lse, kp, i32([ids]), i32([256]), None, i32([0, n]), max_new=n)
        b = ne.paged_weights(q, lse, small, i32([[0, 1, 2, 3]]), i32([256]), None, i32([0, n]), max_new=n)
        ok()
        assert torch.equal(a, b) and float(a.abs().sum()) > 0
