"""Cuts by accumulated weight on the GPU, bit for bit against the plain form of serving_ref."""
import math

import numpy as np
import pytest
import torch

import causal_gqa_flash_attention_gb300 as ne
from causal_gqa_flash_attention_gb300 import _build

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


def state(lens, fresh, NL, H, D, ps, dtype, seed, hnd=False, extra=0, kind="exp"):
    """A pool, tables, weights and positions as earlier calls leave them; entries behind the lengths 7 and 9."""
    rng = np.random.default_rng(seed)
    B, W = len(lens), max(1, max(-(-x // ps) for x in lens)) + extra
    T, P = W * ps, B * W + 2
    table = rng.permutation(P)[: B * W].reshape(B, W).astype(np.int32)
    w = rng.exponential(size=(NL, B, H, T)).astype(np.float32)
    if kind == "ties":
        w = np.round(w).astype(np.float32)
    if kind == "equal":
        w[:] = 0.25
    if kind == "odd":
        w = rng.choice(np.array([0.0, -0.0, math.nan, math.inf, -math.inf, 1e-40, -1.0, 1.0, 3.4e38], np.float32), size=w.shape)
    off = rng.integers(0, 100, B).astype(np.int32)
    pos = np.full((NL, B, H, T), 9, np.int32)
    for b, n in enumerate(lens):
        placed = n - fresh[b]
        for i in range(NL):
            for h in range(H):
                pos[i, b, h, :placed] = rng.permutation(placed + off[b])[:placed]
        pos[:, b, :, placed:n] = -1
        w[:, b, :, n:] = 7.0
    shape = (NL, P, H, ps, D) if hnd else (NL, P, ps, H, D)
    k, v = (torch.randn(shape, generator=torch.Generator().manual_seed(seed + i)).to(dtype).cuda() for i in range(2))
    if hnd:
        k, v = k.transpose(2, 3), v.transpose(2, 3)
    return table, w, pos, off, k, v


def bits(x):
    return x.view(np.uint32) if x.dtype == np.float32 else x


def check(lens, new, fresh, NL=2, H=2, D=64, ps=16, dtype=BF16, sink=2, recent=5, seed=1, same=False, **kw):
    table, w, pos, off, k, v = state(lens, fresh, NL, H, D, ps, dtype, seed, **kw)
    kr, vr = k.float().cpu().numpy(), v.float().cpu().numpy()
    w_ref, p_ref, o_ref = ref.evict(w, pos, off, table, np.array(lens), np.array(new), kr, vr, ps, sink, recent)
    dw, dp, do = torch.tensor(w).cuda(), i32(pos), i32(off)
    outs = (dw, dp, do) if same else (dw.clone(), dp.clone(), torch.zeros_like(do))
    if not same:                                            # what a call must write is not there yet
        for x, fill in zip(outs[:2], (3.0, 5)):
            for b, n in enumerate(lens):
                x[:, b, :, :n] = fill
    got = ne.pages_evict(dw, dp, do, i32(table), i32(lens), i32(new), k, v, sink=sink, recent=recent, weights_out=outs[0],
                         positions_out=outs[1], pos_offset_out=outs[2])
    ok()
    assert all(a is b for a, b in zip(got, outs))
    assert np.array_equal(bits(got[0].cpu().numpy()), bits(w_ref))
    assert np.array_equal(got[1].cpu().numpy(), p_ref)
    assert np.array_equal(got[2].cpu().numpy(), o_ref)
    assert np.array_equal(k.float().cpu().numpy(), kr) and np.array_equal(v.float().cpu().numpy(), vr)
    if not same:
        assert np.array_equal(bits(dw.cpu().numpy()), bits(w)) and np.array_equal(dp.cpu().numpy(), pos)
    return got


@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("lens,new,fresh", [
    ([65, 65, 65], [64, 64, 64], [1, 1, 1]),               # a step of a full cache
    ([1, 2, 31, 32, 33, 64, 200], [1, 1, 30, 16, 32, 1, 100], [0, 1, 31, 0, 5, 64, 7]),
    ([40, 0, 40, 40, 40], [0, 0, 40, 99, 39], [40, 0, 3, 4, 0]),   # nothing, all, more than all
    ([700, 513], [256, 511], [700, 2]),
])
def test_lengths(lens, new, fresh, same):
    check(lens, new, fresh, same=same)


@pytest.mark.parametrize("kind", ["ties", "equal", "odd"])
@pytest.mark.parametrize("same", [False, True])
def test_ties_and_odd_values(kind, same):
    check([300, 97, 64, 1], [123, 50, 60, 1], [10, 0, 64, 1], kind=kind, same=same, seed=5)


@pytest.mark.parametrize("sink,recent", [(0, 0), (0, 40), (40, 0), (100, 100), (1 << 30, 0), (0, 1 << 30), (3, 1)])
@pytest.mark.parametrize("kind", ["exp", "ties"])
def test_guarded_slots(sink, recent, kind):
    check([150, 80, 33], [60, 79, 5], [20, 1, 33], sink=sink, recent=recent, kind=kind, seed=7)


@pytest.mark.parametrize("dtype,D,ps,H,NL,hnd,extra", [
    (BF16, 32, 8, 1, 1, False, 0), (BF16, 128, 64, 4, 1, True, 2), (F32, 32, 256, 3, 2, False, 1), (F32, 64, 16, 1, 3, True, 0),
    (BF16, 64, 128, 5, 1, False, 3),
])
def test_types_and_layouts(dtype, D, ps, H, NL, hnd, extra):
    check([130, 77, 256], [64, 76, 129], [30, 77, 0], NL=NL, H=H, D=D, ps=ps, dtype=dtype, hnd=hnd, extra=extra, seed=9)


@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("n,m", [(50000, 20000), (50001, 50000), (60003, 30001), (70000, 100)])
def test_long_rows(n, m, same):
    """Rows whose keys fit into shared memory, and rows whose keys do not."""
    check([n], [m], [n // 3], NL=1, H=1, D=32, ps=64, recent=1000, sink=4, kind="ties" if n % 2 else "exp", same=same, seed=11)


@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("n", [1000, 1024, 1030, 2048, 2056, 4096, 4100, 8192, 8200, 16384, 16400])
@pytest.mark.parametrize("gone", [1, 3, 4, 5, 400])
def test_few_and_many_go(n, gone, same):
    """On either side of every width of the kernels, and of the count from which on a threshold is searched."""
    check([n], [n - gone], [n // 2], NL=1, H=2, D=32, ps=8, recent=7, sink=3, kind="ties" if gone % 2 else "exp", same=same, seed=n + gone)


@pytest.mark.parametrize("gone", [2, 300])
@pytest.mark.parametrize("n", [900, 3000, 9000])
def test_a_crowd_of_guarded_slots(n, gone):
    """More guarded slots than stay: they compete among themselves, and all others go."""
    check([n], [n - 100 - gone], [n], NL=1, H=2, D=32, ps=8, recent=n - 100, sink=0, kind="ties", seed=n + gone)


def test_fresh_outputs_and_one_layer_pools():
    table, w, pos, off, k, v = state([90, 40], [90, 40], 1, 2, 64, 16, BF16, 13)
    w[:, 0, :, 90:], w[:, 1, :, 40:] = 0, 0
    pos[:] = -1
    kr, vr = k.float().cpu().numpy(), v.float().cpu().numpy()
    w_ref, p_ref, o_ref = ref.evict(w, pos, off, table, np.array([90, 40]), np.array([50, 50]), kr, vr, 16, 1, 8)
    got = ne.pages_evict(torch.tensor(w[0]).cuda(), i32(pos[0]), i32(off), i32(table), i32([90, 40]), i32([50, 50]), k[0], v[0],
                         sink=1, recent=8)
    ok()
    for x, r in zip(got, (w_ref[0], p_ref[0], o_ref)):
        assert np.array_equal(x.cpu().numpy(), r)
    assert np.array_equal(k.float().cpu().numpy(), kr)


def test_the_binding_refuses():
    table, w, pos, off, k, v = state([64], [64], 2, 2, 64, 16, BF16, 29)
    good = [torch.tensor(w).cuda(), i32(pos), i32(off), i32(table), i32([64]), i32([32]), k, v]
    for kw in (dict(sink=1 << 32), dict(recent=-(1 << 40)), dict(workspace=torch.zeros(256, dtype=torch.uint8)),
               dict(weights_out=torch.zeros(2, 1, 2, 32, device="cuda")), dict(pos_offset_out=i32([0, 0]))):
        with pytest.raises(ValueError):
            ne.pages_evict(*good, **kw)
    for i, bad in ((0, good[0][:1]), (0, good[0].double()), (1, good[1].long()), (1, good[1].cpu()), (2, i32([0, 0])), (3, good[3][0]), (4, i32([64, 1])),
                   (6, k[0])):
        args = list(good)
        args[i] = bad
        with pytest.raises(ValueError):
            ne.pages_evict(*args)
    for kw in (dict(sink=-1), dict(recent=(1 << 30) + 1), dict(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ne.NeError):
            ne.pages_evict(*good, **kw)
    ok()


def test_nothing_to_do():
    k = torch.zeros(1, 4, 16, 2, 64, dtype=BF16, device="cuda")
    e = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    got = ne.pages_evict(torch.zeros(1, 0, 2, 48, device="cuda"), e(1, 0, 2, 48), e(0), e(0, 3), e(0), e(0), k, k.clone())
    ok()
    assert [tuple(x.shape) for x in got] == [(1, 0, 2, 48), (1, 0, 2, 48), (0,)]


def test_repeated_cuts_keep_what_one_cut_by_the_same_weights_keeps():
    """Positions survive cuts: the kept set after two cuts is the best of the first cut's kept set."""
    table, w, pos, off, k, v = state([400], [400], 1, 1, 32, 16, F32, 17)
    off[:] = 0
    k[0, torch.tensor(table[0]).long().cuda()] = torch.arange(400, device="cuda").float().view(25, 16, 1, 1).expand(25, 16, 1, 32)
    dw, dp, do = torch.tensor(w).cuda(), i32(pos), i32(off)
    ln = i32([400])
    for m in (250, 249, 100):
        new = i32([m])
        ne.pages_evict(dw, dp, do, i32(table), ln, new, k, v, sink=4, recent=20, weights_out=dw, positions_out=dp, pos_offset_out=do)
        ln = new
    ok()
    score = w[0, 0, 0, :400].copy()
    guard = np.r_[0:4, 380:400]
    rest = [s for s in sorted(range(400), key=lambda s: (-score[s], s)) if s not in guard][:76]
    kept = dp[0, 0, 0, :100].cpu().numpy()
    assert sorted(kept) == sorted(list(guard) + rest) and int(do[0]) == 300
    rows = k[0, torch.tensor(table[0]).long().cuda()].flatten(0, 1)[:100, 0, 0].cpu().numpy()
    assert np.array_equal(rows, kept)                       # each row moved with its position
    assert np.array_equal(dw[0, 0, 0, :100].cpu().numpy(), score[kept])
    assert bool((dp[0, 0, 0, 100:] == -1).all()) and bool((dw[0, 0, 0, 100:] == 0).all())


def test_bad_lengths_offsets_and_pages_are_reported():
    for bad in ("len", "new", "offset", "page"):
        table, w, pos, off, k, v = state([64, 64], [64, 64], 1, 1, 64, 16, BF16, 19)
        lens, new = [64, 64], [32, 32]
        if bad == "len":
            lens[0] = 65
        if bad == "new":
            new[0] = -1
        if bad == "offset":
            off[0] = -5
        if bad == "page":
            table[0] = 1 << 20
        kr, vr = k.float().cpu().numpy(), v.float().cpu().numpy()
        w_ref, p_ref, _ = ref.evict(w, pos, off, table, np.array([0, 64]), np.array([0, 32]), kr, vr, 16, 0, 4)
        got = ne.pages_evict(torch.tensor(w).cuda(), i32(pos), i32(off), i32(table), i32(lens), i32(new), k, v, recent=4)
        torch.cuda.synchronize()
        assert ne.get_device_error() == ne.NE_ERR_INVALID_ARG
        assert np.array_equal(got[0][0, 1, 0, :64].cpu().numpy(), w_ref[0, 1, 0, :64])   # the other sequence is right
        assert np.array_equal(got[1][0, 1, 0, :64].cpu().numpy(), p_ref[0, 1, 0, :64])
    ok()


def test_captured_and_on_another_stream():
    table, w, pos, off, k, v = state([300, 120], [300, 120], 2, 2, 64, 16, BF16, 23)
    args = lambda kk, vv: (torch.tensor(w).cuda(), i32(pos), i32(off), i32(table), i32([300, 120]), i32([100, 60]), kk, vv)  # noqa: E731
    k0, v0 = k.clone(), v.clone()
    want = ne.pages_evict(*args(k0, v0), sink=1, recent=9)
    a = args(k.clone(), v.clone())
    out = [torch.zeros_like(x) for x in want]
    ws = ne.alloc_evict_workspace(2, 2, 2, w.shape[-1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            ne.pages_evict(*a, sink=1, recent=9, weights_out=out[0], positions_out=out[1], pos_offset_out=out[2], workspace=ws)
        g.replay()
        g.replay()                                          # (the same again: sources stay, targets get what they have)
    side.synchronize()
    ok()
    for x, y, n in zip(out[:2], want[:2], (None, None)):
        for b, L in enumerate((300, 120)):
            assert torch.equal(x[:, b, :, :L], y[:, b, :, :L])
    assert torch.equal(out[2], want[2]) and torch.equal(a[6], k0) and torch.equal(a[7], v0)


def test_offsets_beyond_32_bits():
    """Rows that lie behind 2^32 bytes in a pool."""
    P, ps, H, D = 70000, 64, 4, 128                         # 9.2 GB each
    k, v = (torch.empty(1, P, ps, H, D, dtype=BF16, device="cuda") for _ in range(2))
    table = np.array([[P - 1, 5, P - 2, 3]], np.int32)
    live = torch.tensor(table[0]).long().cuda()
    for x in (k, v):
        x[0, live] = torch.randn(4, ps, H, D, device="cuda").to(BF16)
    small = [x[:, live].clone() for x in (k, v)]
    rng = np.random.default_rng(3)
    w = rng.exponential(size=(1, 1, H, 256)).astype(np.float32)
    pos = np.full((1, 1, H, 256), -1, np.int32)
    a = (torch.tensor(w).cuda(), i32(pos), i32([0]))
    ne.pages_evict(*a, i32(table), i32([256]), i32([100]), k, v, recent=10)
    ne.pages_evict(*a, i32([[0, 1, 2, 3]]), i32([256]), i32([100]), *small, recent=10)
    ok()
    for x, y in zip((k, v), small):
        assert torch.equal(x[:, live], y)
