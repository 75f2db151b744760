"""Attention over shared prefixes on the GPU against the plain 64-bit attention of every sequence for
itself (paged_ref), with its bounds."""
import math

import numpy as np
import pytest
import torch

import causal_gqa_flash_attention_gb300 as ne
from causal_gqa_flash_attention_gb300 import _build, synthetic

import paged_ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: torch.finfo(BF16).eps / 2, F32: torch.finfo(F32).eps / 2}


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


def make(dtype, Hq, Hkv, D, ps, groups, shared, n, lens, seed=1, hnd=False, tail=0, lead=0, copies=False, wide=True):
    """Sequences of a group hold the same shared positions, in the same pages (or, copies, in their
    own); everything that no sequence holds is NaN, unused table entries lie outside the pool."""
    rng = np.random.default_rng(seed)
    B, W = len(lens), max(1, max(-(-x // ps) for x in lens)) + 1
    if wide:                                                # (tables that could hold much: the call does share)
        W = max(W, (300 << 20) // (B * ps * Hkv * 2 * D * (2 if dtype == BF16 else 4)) + 1)
    cu = np.concatenate([[0], np.cumsum(n)]) + lead
    N = int(cu[-1]) + tail
    P = sum(-(-x // ps) for x in lens) + 2
    perm, at = rng.permutation(P), 0
    table = np.full((B, W), P + 9, np.int64)
    kp, vp = (synthetic.randn((P, Hkv, ps, D) if hnd else (P, ps, Hkv, D), seed + i, 1.0, dtype).cuda() for i in (1, 2))
    if hnd:
        kp, vp = kp.transpose(1, 2), vp.transpose(1, 2)
    used = torch.zeros(P, ps, dtype=torch.bool)
    for b, x in enumerate(lens):
        pages = -(-x // ps)
        table[b, :pages] = perm[at:at + pages]
        at += pages
        r = int(np.searchsorted(groups, b, side="right")) - 1
        if 0 <= r < len(shared) and b > groups[r]:
            lead_row, S = table[groups[r]], min(shared[r], x)
            if not copies:
                table[b, :S // ps] = lead_row[:S // ps]
            for e in range(-(-S // ps)):
                m = min(ps, S - e * ps)
                for y in (kp, vp):
                    y[int(table[b, e]), :m] = y[int(lead_row[e]), :m].clone()
        for e in range(pages):
            used[table[b, e], :min(ps, x - e * ps)] = True
    for y in (kp, vp):
        y.masked_fill_(~used.cuda()[:, :, None, None], math.nan)
    q = synthetic.randn((N, Hq, D), seed + 3, 1.5, dtype).cuda()
    outside = torch.ones(N, dtype=torch.bool, device="cuda")
    outside[int(cu[0]):int(cu[-1])] = False
    q[outside] = math.nan
    return q, kp, vp, i32(table), i32(lens), i32(groups), i32(shared), i32(cu), table, cu, outside


def check(dtype, Hq, Hkv, D, ps, groups, shared, n, lens, max_new=None, **kw):
    q, kp, vp, table, ln, gr, sh, cu, t, cu_h, outside = make(dtype, Hq, Hkv, D, ps, groups, shared, n, lens, **kw)
    o = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    ws = ne.alloc_paged_shared_workspace(len(lens), q.shape[0], Hq, Hkv, D)
    ws.fill_(255)                                           # (NaN, and records of no CTA)
    got = ne.paged_attn_shared(q, kp, vp, table, ln, gr, sh, cu, max_new=max_new, o=o, lse=lse, workspace=ws)
    ok()
    assert got[0] is o and got[1] is lse
    safe = torch.where(table >= kp.shape[0], 0, table)
    o_ref, lse_ref, A, S = paged_ref.paged_attend(q, kp, vp, safe, lens, cu_h)
    live = ~torch.isnan(lse_ref)
    # Half a step of bf16 where a tile kernel rounds the weights; none in fp32.
    tol_o, tol_lse = paged_ref.attn_bounds(o_ref, A, S, torch.where(torch.isinf(lse_ref), 0.0, lse_ref), D, max(1, max(lens)), HALF[dtype],
                                           HALF[BF16] if dtype == BF16 else 0.0)
    assert bool(torch.isfinite(o[live].double()).all())
    err = (o.double() - o_ref).abs()
    bad = (err > tol_o)[live]
    assert not bool(bad.any()), f"o: {int(bad.sum())} of {bad.numel()}, worst ratio {float((err / tol_o)[live].max())}"
    fin = live & ~torch.isinf(lse_ref)
    e2 = (lse.double() - lse_ref).abs()
    assert bool((e2 <= tol_lse)[fin].all()), float((e2 / tol_lse)[fin].max())
    empty = torch.isinf(lse_ref)
    assert bool((lse[empty] == -math.inf).all()) and bool((o[empty] == 0).all())
    assert bool((o[outside] == 7).all()) and bool((lse[outside] == 7).all())
    return o, lse


HEADS = [(BF16, 12, 4, 64, 16), (BF16, 8, 2, 128, 64), (BF16, 6, 2, 32, 8), (BF16, 20, 1, 64, 256), (BF16, 4, 4, 128, 16),
         (F32, 12, 4, 64, 16), (F32, 4, 2, 32, 8), (F32, 9, 1, 64, 64)]


@pytest.mark.parametrize("dtype,Hq,Hkv,D,ps", HEADS)
@pytest.mark.parametrize("copies", [False, True])
def test_one_token(dtype, Hq, Hkv, D, ps, copies):
    lens = [600, 513, 700, 1025, 530]
    check(dtype, Hq, Hkv, D, ps, [0, 5], [512], [1] * 5, lens, max_new=1, copies=copies)


# groups, shared, new tokens, lengths
BATCHES = [
    # three groups (one of a single sequence), sequences of their own in front and behind, odd shared lengths
    ([1, 4, 5, 8], [700, 300, 257], [1, 1, 1, 1, 1, 1, 1, 1, 1, 1], [40, 701, 900, 750, 301, 258, 600, 300, 1, 511]),
    # sequences without new tokens, shared positions up to the new ones, nothing shared, less than a step
    ([0, 3, 6, 8], [512, 255, 0], [3, 0, 5, 1, 2, 0, 4, 6], [515, 512, 900, 256, 300, 255, 4, 90]),
    # chunks of odd lengths, an empty sequence in a group
    ([0, 4], [1024], [20, 1, 33, 7], [1100, 1025, 1057, 2000]),
    ([0, 2, 4], [0, 256], [9, 0, 17, 1], [9, 0, 300, 257]),
]


@pytest.mark.parametrize("batch", range(len(BATCHES)))
@pytest.mark.parametrize("dtype,Hq,Hkv,D,ps", HEADS)
def test_groups(dtype, Hq, Hkv, D, ps, batch):
    groups, shared, n, lens = BATCHES[batch]
    check(dtype, Hq, Hkv, D, ps, groups, shared, n, lens, max_new=max(n) if batch != 3 else None, seed=3 + batch)


@pytest.mark.parametrize("dtype,Hq,Hkv,D", [(BF16, 12, 4, 64), (BF16, 8, 2, 128), (BF16, 4, 2, 32), (F32, 4, 2, 32), (F32, 8, 2, 64)])
def test_many_sequences_and_cut_units(dtype, Hq, Hkv, D):
    """Fifty sequences over a prefix of many tiles: its units lie on many CTAs, own ones on one or two."""
    rng = np.random.default_rng(5)
    lens = [int(x) for x in 4100 + rng.integers(1, 400, 50)]
    check(dtype, Hq, Hkv, D, 16, [0, 50], [4100], [1] * 50, lens, max_new=1, seed=7)


@pytest.mark.parametrize("dtype,D,n", [(BF16, 64, 1), (BF16, 128, 3), (F32, 32, 1)])
def test_many_groups(dtype, D, n):
    """Hundreds of groups of two: many whole units per CTA, more sequences than a pass of the search."""
    rng = np.random.default_rng(6)
    R = 240
    shared = [int(x) for x in rng.integers(0, 520, R)]
    lens = [shared[b // 2] + n + int(x) for b, x in enumerate(rng.integers(0, 60, 2 * R))]
    check(dtype, 4, 2, D, 8, list(range(0, 2 * R + 1, 2)), shared, [n] * (2 * R), lens, max_new=n, seed=9)


@pytest.mark.parametrize("max_new", [1, 8, 22, 4000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_any_max_new_is_right(dtype, max_new):
    """A hint, and no more: too small, too large."""
    check(dtype, 12, 1, 64, 16, [0, 3], [512], [25, 1, 70], [600, 513, 700], max_new=max_new, seed=11)


@pytest.mark.parametrize("dtype,Hq,Hkv,D,ps", [(BF16, 12, 4, 64, 16), (BF16, 8, 2, 128, 64), (BF16, 6, 2, 32, 8), (BF16, 5, 5, 64, 32),
                                                (F32, 6, 2, 64, 16), (F32, 2, 2, 32, 64)])
@pytest.mark.parametrize("n", [[200, 1, 130, 77, 256], [90] * 5, [0, 300, 2, 0, 85]])
def test_chunks_of_several_row_tiles(dtype, Hq, Hkv, D, ps, n):
    """Sequences of more rows than a tile, rows of several in the tiles of their prefix."""
    lens = [1000 + x + y for x, y in zip(n, [0, 300, 5, 128, 51])]
    check(dtype, Hq, Hkv, D, ps, [0, 3, 5], [1000, 520], n, lens, max_new=max(n), seed=17)


@pytest.mark.parametrize("D,n", [(64, [64] * 8), (128, [60, 64, 64, 3, 64, 17, 64, 64])])
def test_chunks_that_fill_their_tiles(D, n):
    """The first runs as paged_attn, whatever the groups say."""
    lens = [700 + x for x in n]
    check(BF16, 4, 1, D, 16, [0, 8], [700], n, lens, max_new=64, seed=18)
    if n == [64] * 8:
        q, kp, vp, table, ln, gr, sh, cu, *_ = make(BF16, 4, 1, D, 16, [0, 8], [700], n, lens)
        a = ne.paged_attn_shared(q, kp, vp, table, ln, i32([5, 2]), sh, cu, max_new=64)
        b = ne.paged_attn(q, kp, vp, table, ln, cu, max_new=64)
        ok()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_more_than_128_query_heads():
    check(BF16, 130, 1, 64, 16, [0, 3], [512], [1, 1, 1], [600, 513, 700], max_new=1, seed=12)
    check(F32, 130, 1, 32, 16, [0, 3], [512], [1, 1, 1], [600, 513, 700], max_new=1, seed=12)


@pytest.mark.parametrize("dtype,n", [(BF16, [1, 1, 1]), (BF16, [14, 2, 9]), (F32, [1, 1, 1]), (F32, [14, 2, 9])])
def test_padding_and_layouts(dtype, n):
    check(dtype, 8, 4, 64, 32, [0, 3], [300], n, [400, 302, 310], hnd=True, tail=5, lead=3, max_new=max(n), seed=13)


def test_small_caches_run_as_paged_attn():
    for dtype, D in ((BF16, 64), (F32, 32)):
        q, kp, vp, table, ln, gr, sh, cu, *_ = make(dtype, 12, 4, D, 16, [0, 3], [512], [1, 2, 3], [600, 514, 700], wide=False)
        a = ne.paged_attn_shared(q, kp, vp, table, ln, gr, sh, cu, max_new=3)
        b = ne.paged_attn(q, kp, vp, table, ln, cu, max_new=3)
        ok()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        check(dtype, 12, 4, D, 16, [0, 3], [512], [1, 2, 3], [600, 514, 700], max_new=3, wide=False)


def test_negative_positions():
    """More new tokens than positions in a sequence of its own: rows without keys."""
    check(BF16, 12, 4, 64, 16, [0, 2], [256], [1, 1, 9], [300, 257, 4], seed=15)
    check(F32, 4, 2, 32, 16, [0, 2], [256], [1, 1, 9], [300, 257, 4], seed=15)


def test_without_row_offsets_and_without_groups():
    q, kp, vp, table, ln, gr, sh, cu, *_ = make(BF16, 12, 4, 64, 16, [0, 3], [512], [1] * 3, [600, 513, 700])
    a = ne.paged_attn_shared(q, kp, vp, table, ln, gr, sh, cu, max_new=1)
    b = ne.paged_attn_shared(q, kp, vp, table, ln, gr, sh)
    c = ne.paged_attn_shared(q, kp, vp, table, ln, i32([0]), i32([]))
    d = ne.paged_attn(q, kp, vp, table, ln)
    ok()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(c[0], d[0]) and torch.equal(c[1], d[1])


def test_same_bits_captured_and_on_another_stream():
    rng = np.random.default_rng(8)
    lens = [int(x) for x in 2100 + rng.integers(1, 300, 20)]
    q, kp, vp, table, ln, gr, sh, cu, *_ = make(BF16, 12, 4, 64, 16, [0, 12, 20], [2100, 1000], [1] * 20, lens)
    want = ne.paged_attn_shared(q, kp, vp, table, ln, gr, sh, cu, max_new=1)
    ws = ne.alloc_paged_shared_workspace(20, 20, 12, 4, 64)
    o, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    torch.cuda.synchronize()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            ne.paged_attn_shared(q, kp, vp, table, ln, gr, sh, cu, max_new=1, o=o, lse=lse, workspace=ws)
        for _ in range(3):
            o.zero_()
            g.replay()
            side.synchronize()
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    ok()


def test_bad_groups_are_reported_and_others_right():
    base = ([0, 2, 4], [512, 256], [1, 1, 1, 1], [600, 513, 300, 257])
    for groups, shared in (([0, 2, 5], [512, 256]), ([-1, 2, 4], [512, 256]), ([0, 2, 1], [512, 256]), ([0, 2, 4], [512, -7]),
                           ([0, 2, 4], [512, 768]), ([0, 2, 4], [640, 256]), ([0, 4], [512])):
        q, kp, vp, table, ln, gr, sh, cu, *_ = make(BF16, 12, 4, 64, 16, *base)
        want = ne.paged_attn(q, kp, vp, table, ln)
        o, _ = ne.paged_attn_shared(q, kp, vp, table, ln, i32(groups), i32(shared))
        torch.cuda.synchronize()
        bad = groups != base[0] or shared[1] == -7
        # (768 positions of a group whose first sequence holds 300: the whole steps that it holds are taken,
        # 256, behind which the second sequence of 257 has its new token.  640 counts as 512.)
        assert ne.get_device_error() == (ne.NE_ERR_INVALID_ARG if bad else ne.NE_OK)
        if groups == base[0] and shared[0] == 512:          # the first group is what it was
            assert bool(((o[:2] - want[0][:2]).float().abs() < 0.02).all())
    ok()


def test_offsets_beyond_32_bits():
    P, ps, H, D = 70000, 64, 4, 128                         # 9.2 GB each
    kp, vp = (torch.empty(P, ps, H, D, dtype=BF16, device="cuda") for _ in range(2))
    ids = torch.arange(P - 40, P, device="cuda")
    for x in (kp, vp):
        x[ids] = torch.randn(40, ps, H, D, device="cuda").to(BF16)
    small = [x[ids].clone() for x in (kp, vp)]
    row = np.arange(P - 40, P - 20)
    table = np.stack([row, np.concatenate([row[:8], row[8:] + 20])])
    table = np.concatenate([table, np.full((2, 500), P + 9)], 1)       # (of 67 MB: the call does share)
    q = synthetic.randn((2, 8, D), 3, 1.0, BF16).cuda()
    a = ne.paged_attn_shared(q, kp, vp, i32(table), i32([1200, 700]), i32([0, 2]), i32([512]))
    b = ne.paged_attn_shared(q, *small, i32(table - (P - 40)), i32([1200, 700]), i32([0, 2]), i32([512]))
    ok()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
