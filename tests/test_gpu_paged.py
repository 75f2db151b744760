"""The paged cache on the GPU against the plain 64-bit forms of paged_ref.

Outputs of the attention and of the rotation are held to bounds computed from the data
(paged_ref.attn_bounds; see there); page ids, counts, tables, copied slots and everything
that a call must leave alone are compared bit for bit.
"""
import math
import random

import numpy as np
import pytest
import torch

import causal_gqa_flash_attention_gb300 as ne
from causal_gqa_flash_attention_gb300 import _build, synthetic

import paged_ref as ref

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


def pool(P, ps, Hkv, D, dtype, seed, hnd=False, L=None, fill=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    shape = (P, Hkv, ps, D) if hnd else (P, ps, Hkv, D)
    x = torch.empty(shape if L is None else (L, *shape), device="cuda", dtype=dtype)
    x.normal_(generator=g) if fill is None else x.fill_(fill)
    return x.transpose(-3, -2) if hnd else x


def tables(lens, ps, seed, spare=3):
    """Random distinct pages for every sequence; unused entries hold an id outside the pool."""
    rng = np.random.default_rng(seed)
    W = max(1, max(-(-int(x) // ps) for x in lens)) + 1
    P = sum(-(-int(x) // ps) for x in lens) + spare
    perm = rng.permutation(P)
    t = np.full((len(lens), W), P + 7, np.int32)
    at = 0
    for b, x in enumerate(lens):
        k = -(-int(x) // ps)
        t[b, :k] = perm[at:at + k]
        at += k
    return t, P


def poison(kp, vp, table, lens, value):
    """Slots at or behind a sequence's length, and pages of nobody, hold `value`."""
    ps = kp.shape[-3]
    used = torch.zeros(kp.shape[-4], ps, dtype=torch.bool, device="cuda")
    for b, x in enumerate(lens):
        for e in range(-(-int(x) // ps)):
            used[int(table[b, e]), :min(ps, int(x) - e * ps)] = True
    for p in (kp, vp):
        p.masked_fill_(~used[:, :, None, None], value)


def check_attn(q, kp, vp, table, lens, cu, o, lse, dtype, p_half_step):
    o_ref, lse_ref, A, S = ref.paged_attend(q, kp, vp, table, lens, cu)
    live = ~torch.isnan(lse_ref)
    tol_o, tol_lse = ref.attn_bounds(o_ref, A, S, torch.where(torch.isinf(lse_ref), 0.0, lse_ref), q.shape[-1],
                                     max(1, int(max(lens))), HALF[dtype], p_half_step)
    err = (o.double() - o_ref).abs()
    assert bool(torch.isfinite(o[live].double()).all())
    bad = (err > tol_o)[live]
    assert not bool(bad.any()), f"o: {int(bad.sum())} of {bad.numel()}, worst ratio {float((err / tol_o)[live].max())}"
    fin = live & ~torch.isinf(lse_ref)
    e2 = (lse.double() - lse_ref).abs()
    assert bool((e2 <= tol_lse)[fin].all()), float((e2 / tol_lse)[fin].max())
    empty = torch.isinf(lse_ref)
    assert bool((lse[empty] == -math.inf).all()) and bool((o[empty] == 0).all())


def attn_case(dtype, Hq, Hkv, D, ps, n, lens, seed, hnd=False, tail=0, max_new=None, value=math.nan, lead=0):
    cu = np.concatenate([[0], np.cumsum(n)]) + lead
    N = int(cu[-1]) + tail
    t, P = tables(lens, ps, seed)
    kp, vp = pool(P, ps, Hkv, D, dtype, seed + 1, hnd), pool(P, ps, Hkv, D, dtype, seed + 2, hnd)
    poison(kp, vp, t, lens, value)
    q = synthetic.randn((N, Hq, D), seed + 3, 1.0, dtype).cuda()
    o = torch.full((N, Hq, D), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((N, Hq), 7.0, dtype=F32, device="cuda")
    table = i32(t)
    ne.paged_attn(q, kp, vp, table, i32(lens), i32(cu), max_new=max_new, o=o, lse=lse)
    ok()
    # bf16 weights: a product of 128-row tiles rounds them to bf16 (half a step), the kernels
    # for few rows keep a second bf16 term (a half step of a half step).
    check_attn(q, kp, vp, table, lens, cu, o, lse, dtype, HALF[BF16] if dtype == BF16 else 0.0)
    outside = torch.ones(N, dtype=torch.bool, device="cuda")
    outside[int(cu[0]):int(cu[-1])] = False
    assert bool((o[outside] == 7).all()) and bool((lse[outside] == 7).all())
    return q, kp, vp, table, i32(lens), i32(cu), o, lse


# ---------------------------------------------------------------- attention: one token

@pytest.mark.parametrize("dtype,Hq,Hkv,D,ps,lens", [
    (BF16, 12, 4, 64, 16, [1, 2, 15, 16, 17, 127, 128, 129, 300, 1000]),
    (BF16, 16, 4, 128, 64, [1, 63, 64, 65, 700]),
    (BF16, 8, 8, 32, 8, [5, 8, 9, 33]),
    (BF16, 4, 2, 32, 256, [255, 256, 257, 1]),
    (BF16, 10, 2, 64, 32, [4097, 31]),
    (BF16, 40, 2, 64, 16, [77, 513]),            # 20 query heads per kv head: two head groups
    (BF16, 71, 1, 64, 128, [130, 1, 999]),       # 71: five groups, the last of seven heads
    (F32, 4, 2, 32, 16, [1, 128, 64, 100]),
    (F32, 12, 4, 64, 8, [7, 8, 9, 1025]),
    (F32, 20, 2, 64, 16, [40, 300]),
])
def test_attn_one_token(dtype, Hq, Hkv, D, ps, lens):
    attn_case(dtype, Hq, Hkv, D, ps, [1] * len(lens), lens, 11 + D + len(lens), max_new=1)


def test_attn_one_token_without_row_offsets_and_head_major_pages():
    lens = [33, 1, 200]
    q, kp, vp, table, ln, cu, o, lse = attn_case(BF16, 12, 4, 64, 16, [1] * 3, lens, 5, hnd=True, max_new=1)
    o2, lse2 = ne.paged_attn(q, kp, vp, table, ln)
    ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_attn_long_sequence_beside_short_ones():
    """One sequence holds nearly all the work: it is cut over all CTAs and joined."""
    attn_case(BF16, 12, 4, 64, 16, [1] * 6, [20011, 3, 1, 16, 250, 17], 21, max_new=1)
    attn_case(F32, 4, 1, 64, 32, [1] * 3, [9001, 3, 64], 22, max_new=1)


def test_attn_many_sequences():
    """More sequences than a CTA has threads: the split runs over them in passes."""
    rng = random.Random(3)
    lens = [rng.choice([0, 1, rng.randint(1, 60)]) for _ in range(700)]
    n = [rng.choice([0, 1, 1]) for _ in lens]
    attn_case(BF16, 4, 2, 64, 16, n, lens, 31, max_new=1)


# ---------------------------------------------------------------- attention: chunks

CHUNKS = [
    (12, 4, 64, 16, [5, 1, 40, 0, 3], [300, 17, 40, 90, 3]),       # prompt, chunk, single tokens, an idle sequence
    (16, 4, 128, 64, [130, 7], [513, 7]),
    (16, 4, 128, 16, [300, 1, 1], [300, 2000, 65]),
    (6, 6, 64, 32, [257], [1025]),
    (8, 1, 64, 128, [33, 64], [129, 64]),
    (8, 2, 32, 8, [20, 9], [77, 200]),
    (10, 2, 64, 16, [51, 100], [1000, 100]),                       # five heads: 125 of 128 rows
    (71, 1, 64, 64, [3, 5], [500, 5]),
    (12, 4, 64, 256, [600], [600]),
    (40, 1, 128, 16, [19, 2], [400, 1111]),
    (130, 1, 64, 32, [2, 3], [300, 3]),                            # more heads than a tile has rows
    (12, 4, 64, 8, [300, 1], [555, 130]),                          # sixteen pages to a tile
]


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (F32, 64)])
@pytest.mark.parametrize("ps", [8, 64, 256])
def test_attn_head_major_pages(dtype, D, ps):
    for mn in (1, None):
        attn_case(dtype, 12, 4, D, ps, [70, 1, 5], [333, 500, 5], 87, hnd=True, max_new=mn)


@pytest.mark.parametrize("dtype,n,max_new", [(BF16, 1, 1), (BF16, 16, None), (F32, 1, 1), (F32, 2, 2), (F32, 4, 4),
                                             (F32, 16, None)])
def test_attn_one_unit_over_many_ctas(dtype, n, max_new):
    """One kv head and few rows: a single unit is cut into dozens or hundreds of parts."""
    attn_case(dtype, 4, 1, 64, 64, [n], [40003], 95, max_new=max_new)


def test_attn_many_sequences_of_chunks():
    """More sequences than one warp looks through at once, for the tile kernel."""
    rng = random.Random(5)
    lens = [rng.choice([0, 1, rng.randint(1, 300)]) for _ in range(460)]
    n = [rng.choice([0, 1, min(x, 20)]) if x else 0 for x in lens]
    for D in (64, 128):
        attn_case(BF16, 4, 2, D, 16, n, lens, 97, max_new=None, tail=1)
    attn_case(F32, 4, 2, 64, 16, n, lens, 98, max_new=None, tail=1)


def test_attn_contexts_too_short_to_cut():
    """Tables of at most 256 positions: whole units only, no join."""
    for dtype in (BF16, F32):
        for mn in (1, None):
            attn_case(dtype, 12, 4, 64, 16, [1, 3, 0, 60, 1, 9], [239, 3, 17, 200, 1, 5], 91, max_new=mn, tail=1)


@pytest.mark.parametrize("Hq,Hkv,D,ps,n,lens", CHUNKS)
@pytest.mark.parametrize("max_new", [1, 4, None])
def test_attn_chunks_bf16(Hq, Hkv, D, ps, n, lens, max_new):
    """max_new chooses a kernel and nothing else: every choice is right for every chunk."""
    attn_case(BF16, Hq, Hkv, D, ps, n, lens, 41 + Hq, max_new=max_new, tail=3, lead=2)


@pytest.mark.parametrize("Hq,Hkv,D,ps,n,lens", [c for c in CHUNKS if c[2] < 128])
@pytest.mark.parametrize("max_new", [1, None])
def test_attn_chunks_f32(Hq, Hkv, D, ps, n, lens, max_new):
    attn_case(F32, Hq, Hkv, D, ps, n, lens, 51 + Hq, max_new=max_new, tail=3, lead=2)


@pytest.mark.parametrize("Hq,Hkv,D,ps,n,lens", [c for c in CHUNKS if c[2] < 128])
@pytest.mark.parametrize("max_new", [2, 4, 6])
def test_attn_chunks_f32_by_few_rows(Hq, Hkv, D, ps, n, lens, max_new):
    attn_case(F32, Hq, Hkv, D, ps, n, lens, 61 + Hq, max_new=max_new, tail=1)


@pytest.mark.parametrize("hnd", [False, True])
@pytest.mark.parametrize("D,G,n", [(32, 3, 1), (32, 7, 1), (32, 4, 4), (64, 1, 1), (64, 5, 1), (64, 3, 10), (64, 9, 3)])
def test_attn_few_tokens_f32(D, G, n, hnd):
    """Lengths around the 32 keys of a warp and the 256 of a tile, every page size."""
    for ps in (8, 16, 32, 128):
        lens = [n, 31, 32, 33, 255, 256, 257, 289, 511, 1500]
        attn_case(F32, 2 * G, 2, D, ps, [min(n, x) for x in lens], lens, ps + D + G, hnd=hnd, max_new=n)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("max_new", [1, None])
def test_attn_rows_without_keys(dtype, max_new):
    """More new tokens than positions: the first rows have nothing to attend to."""
    attn_case(dtype, 12, 4, 64, 16, [9, 70, 1, 2, 300], [4, 33, 0, 2, 1], 61, max_new=max_new, tail=2)


def test_attn_large_logits():
    """sigma 3 queries and keys: the running maximum moves and rows rescale."""
    n, lens = [200, 1], [900, 3000]
    t, P = tables(lens, 16, 1)
    kp, vp = pool(P, 16, 4, 128, BF16, 2) * 3, pool(P, 16, 4, 128, BF16, 3)
    q = synthetic.randn((201, 16, 128), 4, 3.0, BF16).cuda()
    cu = [0, 200, 201]
    for mn in (1, None):
        o, lse = ne.paged_attn(q, kp, vp, i32(t), i32(lens), i32(cu), max_new=mn)
        ok()
        check_attn(q, kp, vp, i32(t), lens, cu, o, lse, BF16, HALF[BF16])


def test_attn_queries_from_a_fused_projection_and_side_by_side_pools():
    """Row slices of one projection, and a pool that holds keys and values side by side."""
    ps, Hq, Hkv, D, lens, n = 16, 12, 4, 64, [100, 40], [3, 20]
    t, P = tables(lens, ps, 7)
    kv = pool(P * 2, ps, Hkv, D, BF16, 8).view(P, 2, ps, Hkv, D)
    kp, vp = kv[:, 0], kv[:, 1]
    qkv = synthetic.randn((23, Hq + 2 * Hkv, D), 9, 1.0, BF16).cuda()
    q, cu = qkv[:, :Hq], [0, 3, 23]
    for mn in (1, None):
        o, lse = ne.paged_attn(q, kp, vp, i32(t), i32(lens), i32(cu), max_new=mn)
        ok()
        check_attn(q.contiguous(), kp, vp, i32(t), lens, cu, o, lse, BF16, HALF[BF16])


@pytest.mark.parametrize("dtype,mn", [(BF16, 1), (BF16, None), (F32, 1), (F32, 8), (F32, None)])
def test_attn_pages_beyond_32_bit_offsets(dtype, mn):
    """Pages 2^30 elements apart: the last starts at element 2^32 of its pool."""
    ps, Hkv, D, P = 16, 2, 64, 5
    flat = [torch.empty((P - 1) * 2 ** 30 + ps * Hkv * D, dtype=dtype, device="cuda") for _ in range(2)]
    kp, vp = (x.as_strided((P, ps, Hkv, D), (2 ** 30, Hkv * D, D, 1)) for x in flat)
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    kp.copy_(torch.randn(P, ps, Hkv, D, generator=g, device="cuda"))
    vp.copy_(torch.randn(P, ps, Hkv, D, generator=g, device="cuda"))
    n, lens, t = [20, 1], [30, 39], np.array([[4, 1, 0], [3, 0, 2]], np.int32)
    q = synthetic.randn((21, 6, D), 4, 1.0, dtype).cuda()
    cu = [0, 20, 21]
    k = synthetic.randn((21, Hkv, D), 5, 1.0, dtype).cuda()
    ne.paged_append(k, k, kp, vp, i32(t), i32(lens), i32(cu))
    o, lse = ne.paged_attn(q, kp, vp, i32(t), i32(lens), i32(cu), max_new=mn)
    ok()
    check_attn(q, kp, vp, i32(t), lens, cu, o, lse, dtype, HALF[BF16] if dtype == BF16 else 0.0)
    assert torch.equal(kp[4, 10:], k[:6]) and torch.equal(vp[2, 6], k[20])
    # A copy from the last page to the first free one.
    refc = np.array([2, 1, 1, 0, 1], np.int32)
    ref4 = kp[4].clone()
    out = ne.pages_fork(i32(refc), i32([[4, 1]]), i32([10]), i32([0]), kp, vp)
    ok()
    assert out[1].tolist() == [[3, -1]] and torch.equal(kp[3, :10], ref4[:10])


@pytest.mark.parametrize("dtype,mn", [(BF16, 1), (BF16, None), (F32, 1), (F32, 8), (F32, None)])
def test_attn_nan_in_a_key_in_use_shows(dtype, mn):
    """A NaN key in front of a row's position makes that row NaN (o and lse) and no row that
    does not see it, in its own or another sequence."""
    ps, lens, n = 16, [300, 90], [40, 1]
    t, P = tables(lens, ps, 3)
    kp, vp = pool(P, ps, 4, 64, dtype, 4), pool(P, ps, 4, 64, dtype, 5)
    at = 280                                               # the 20th new token's own key
    kp[t[0, at // ps], at % ps, 2] = math.nan
    q = synthetic.randn((41, 12, 64), 6, 1.0, dtype).cuda()
    o, lse = ne.paged_attn(q, kp, vp, i32(t), i32(lens), i32([0, 40, 41]), max_new=mn)
    ok()
    hit = torch.zeros(41, 12, dtype=torch.bool, device="cuda")
    hit[20:40, 6:9] = True                                 # kv head 2
    assert bool(torch.isnan(lse)[hit].all()) and bool(torch.isnan(o.float())[hit].all())
    assert bool(torch.isfinite(lse)[~hit].all()) and bool(torch.isfinite(o.float())[~hit].all())


@pytest.mark.parametrize("dtype,mn", [(BF16, 1), (BF16, None), (F32, 1), (F32, 8), (F32, None)])
def test_attn_same_bits_every_time(dtype, mn):
    q, kp, vp, t, ln, cu, o, lse = attn_case(dtype, 12, 4, 64, 16, [64, 1, 1, 33], [3000, 5000, 17, 900], 71, max_new=mn)
    ws = ne.alloc_paged_workspace(4, 99, 12, 4, 64)
    for _ in range(5):
        ws.fill_(255)                                      # whatever the workspace held
        o2, lse2 = ne.paged_attn(q, kp, vp, t, ln, cu, max_new=mn, workspace=ws)
        ok()
        assert torch.equal(o2, o) and torch.equal(lse2, lse)


@pytest.mark.parametrize("mn", [1, None])
def test_attn_captured_and_replayed_on_other_lengths(mn):
    """A graph reads lengths, tables and offsets at replay, and two graphs may share a
    workspace on one stream."""
    ps, lens = 16, [500, 30]
    t, P = tables([600, 600], ps, 5)
    kp, vp = pool(P, ps, 4, 64, BF16, 6), pool(P, ps, 4, 64, BF16, 7)
    q = synthetic.randn((41, 12, 64), 8, 1.0, BF16).cuda()
    table, ln, cu = i32(t), i32(lens), i32([0, 40, 41])
    ws = ne.alloc_paged_workspace(2, 41, 12, 4, 64)
    outs = [(torch.zeros_like(q), torch.zeros(41, 12, device="cuda")) for _ in range(2)]
    ne.paged_attn(q, kp, vp, table, ln, cu, max_new=mn, o=outs[0][0], lse=outs[0][1], workspace=ws)
    ok()
    graphs = []
    for o, lse in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ne.paged_attn(q, kp, vp, table, ln, cu, max_new=mn, o=o, lse=lse, workspace=ws)
        graphs.append(g)
    for lens, rows in (([500, 30], [0, 40, 41]), ([600, 1], [0, 1, 2]), ([37, 599], [0, 20, 41])):
        ln.copy_(i32(lens))
        cu.copy_(i32(rows))
        for g in graphs:
            g.replay()
        ok()
        m = rows[-1]
        for o, lse in outs:
            check_attn(q[:m], kp, vp, table, lens, rows, o[:m], lse[:m], BF16, HALF[BF16])


def test_attn_two_streams_with_a_workspace_each():
    a = attn_case(BF16, 12, 4, 64, 16, [1] * 4, [4000, 300, 5000, 2], 81, max_new=1)
    b = attn_case(BF16, 16, 4, 128, 64, [200, 1], [1500, 900], 82)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        for st, c in zip(streams, (a, b)):
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(st):
                got.append((ne.paged_attn(*c[:6]), c))
    torch.cuda.synchronize()
    ok()
    for (o, lse), c in got:
        m = int(c[5][-1])
        if c is b:
            assert torch.equal(o[:m], c[6][:m]) and torch.equal(lse[:m], c[7][:m])
        else:
            check_attn(c[0], c[1], c[2], c[3], c[4].tolist(), c[5].tolist(), o, lse, BF16, HALF[BF16])


@pytest.mark.parametrize("dtype,mn", [(BF16, 1), (BF16, None), (F32, 1)])
def test_attn_bad_device_arguments_are_reported(dtype, mn):
    """Ids, lengths and offsets outside their ranges never reach memory: the call reports
    them and the other sequences are right."""
    ps, lens, n = 16, [40, 300, 20], [2, 3, 1]
    t, P = tables(lens, ps, 3)
    kp, vp = pool(P, ps, 4, 64, dtype, 4), pool(P, ps, 4, 64, dtype, 5)
    q = synthetic.randn((6, 12, 64), 6, 1.0, dtype).cuda()
    cu = [0, 2, 5, 6]

    def run(t, lens, cu):
        r = ne.paged_attn(q, kp, vp, i32(t), i32(lens), i32(cu), max_new=mn)
        torch.cuda.synchronize()
        return r

    good_o, good_lse = run(t, lens, cu)
    ok()
    for change, word in (("page", "page id"), ("neg", "page id"), ("len", "length"), ("cu", "cu_new"), ("huge", "page id")):
        t2, l2, c2 = t.copy(), list(lens), list(cu)
        if change == "page":
            t2[1, 3] = P
        if change == "huge":
            t2[1, 0] = 2 ** 31 - 1
        if change == "neg":
            t2[1, 18] = -5
        if change == "len":
            l2[1] = 10 ** 6
            t2[1] = t2[1, 0]
        if change == "cu":
            c2[2] = 1
            c2[1] = 2
        o, lse = run(t2, l2, c2)
        assert ne.get_device_error() == ne.NE_ERR_INVALID_ARG and word in ne.last_error()
        # Row 1 belongs to two sequences under the bad offsets.  The others' key axis may be
        # cut elsewhere, so they agree to the rounding of two bf16 results at most.
        keep = [0] if change == "cu" else [0, 1, 5]
        assert torch.allclose(o[keep].float(), good_o[keep].float(), rtol=2 * HALF[BF16], atol=2 * HALF[BF16])
        assert bool(torch.isfinite(o.float()).all())
    ok()


# ---------------------------------------------------------------- append

def append_case(dtype, Hq, Hkv, D, ps, n, lens, seed, hnd=False, tail=0, lead=0, off=0, with_q=True, inplace=False, **rope):
    cu = np.concatenate([[0], np.cumsum(n)]) + lead
    N = int(cu[-1]) + tail
    t, P = tables(lens, ps, seed)
    kp, vp = pool(P, ps, Hkv, D, dtype, seed + 1, hnd), pool(P, ps, Hkv, D, dtype, seed + 2, hnd)
    k0, v0 = kp.clone(), vp.clone()
    qkv = synthetic.randn((N, Hq + 2 * Hkv, D), seed + 3, 1.0, dtype).cuda()
    src = qkv.clone()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    spec = ne.rope_spec(D, **rope) if rope else None
    q_out = q if inplace else torch.full((N, Hq, D), 7.0, dtype=dtype, device="cuda")
    got = ne.paged_append(k, v, kp, vp, i32(t), i32(lens), i32(cu), rope=spec, pos_offset=off, q=q if with_q else None,
                          q_out=q_out if with_q else None)
    ok()
    f = ref.rope_angles(rope.get("rot_dim", D), rope.get("theta", 10000.0), rope.get("scaling", "none"), rope.get("factor", 1.0),
                        rope.get("orig_len", 0)) if rope else np.zeros(0)
    ms = rope.get("mscale", 1.0)
    x = src.double().cpu().numpy()
    want_k, want_v = k0.double().cpu().numpy(), v0.clone()
    size_k = np.zeros_like(want_k)                         # |x0| + |x1| of the pair behind a value; 0: must be left as is
    want_q, size_q = np.full((N, Hq, D), 7.0), np.zeros((N, Hq, D))
    if inplace:
        want_q = x[:, :Hq].copy()
    for b in range(len(lens)):
        for i in range(n[b]):
            row, p = int(cu[b]) + i, int(lens[b]) - n[b] + i
            if p < 0:
                want_q[row] = 0
                continue
            y = ref.rotate(x[row:row + 1], [p + off], f, rope.get("layout", "interleaved"), ms)[0] if rope else x[row]
            m = ref.rotate(np.abs(x[row:row + 1]), [0], f * 0, rope.get("layout", "interleaved"))[0] if rope else np.abs(x[row])
            rot = 2 * len(f)
            lay = rope.get("layout", "interleaved")
            a = np.arange(0, rot, 2) if lay == "interleaved" else np.arange(rot // 2)
            c = a + 1 if lay == "interleaved" else a + rot // 2
            if rot:
                m = m.copy()
                m[..., a] = m[..., c] = m[..., a] + m[..., c]
            want_q[row], size_q[row] = y[:Hq], m[:Hq]
            page, slot = t[b, p // ps], p % ps
            want_k[page, slot], size_k[page, slot] = y[Hq:Hq + Hkv], m[Hq:Hq + Hkv]
            want_v[page, slot] = v[row] if not inplace else src[row, Hq + Hkv:]
    # The angle: one rounding of the fraction of a turn to fp32 (2^-25 turns = 2 pi 2^-25
    # rad), sin and cos 2^-22 absolute, mscale, two products and a sum: each 2^-24 of |x0| + |x1|;
    # then the output's half step.
    rel = (2 * math.pi * 2.0 ** -25 + 2.0 ** -22 + 4 * 2.0 ** -24) * max(1.0, abs(ms)) if rope else 0.0
    for name, have, want, size in (("k", kp, want_k, size_k), ("q", q_out, want_q, size_q))[:2 if with_q else 1]:
        e = np.abs(have.double().cpu().numpy() - want)
        tol = rel * size * (1 + HALF[dtype]) + HALF[dtype] * np.abs(want) * (size > 0) * (1 if rope else 0)
        assert np.all(e <= tol), (name, float(np.max(e - tol)))
    assert torch.equal(vp, want_v)
    if not inplace:
        assert torch.equal(qkv, src)
    return got


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("rot", [64, 32, 18, 2])
def test_append_layouts_and_partial_heads(dtype, layout, rot):
    append_case(dtype, 12, 4, 64, 16, [3, 1, 0, 20], [40, 17, 5, 20], 1 + rot, layout=layout, rot_dim=rot, tail=2, lead=1)


@pytest.mark.parametrize("Hq,Hkv,D,ps,n,lens,hnd", [
    (16, 4, 128, 64, [130, 5, 1], [130, 900, 64], False), (4, 2, 32, 8, [1, 1, 1], [1, 8, 9], False),
    (5, 5, 64, 256, [300], [301], True), (8, 1, 128, 16, [17, 33], [33, 33], True),
    (12, 4, 64, 16, [700, 1000, 2100], [700, 1001, 4000], False),            # several tokens per CTA
])
def test_append_shapes(Hq, Hkv, D, ps, n, lens, hnd):
    append_case(BF16, Hq, Hkv, D, ps, n, lens, 3 * D, hnd=hnd, layout="half" if hnd else "interleaved")


@pytest.mark.parametrize("N", [600, 1100, 2400, 5000])     # eight, four, two warps and one to a token
@pytest.mark.parametrize("dtype,Hq,Hkv,D,layout,rot,inplace", [
    (F32, 3, 1, 64, "half", 48, True), (BF16, 5, 1, 32, "half", 16, False), (F32, 2, 2, 32, "interleaved", 30, True),
    (BF16, 3, 3, 128, "half", 100, True)])
def test_append_every_share_of_a_token(N, dtype, Hq, Hkv, D, layout, rot, inplace):
    n = [N // 3, N - N // 3 - 1, 1]
    append_case(dtype, Hq, Hkv, D, 16, n, [x + 11 for x in n], N, layout=layout, rot_dim=rot, inplace=inplace, tail=3)


@pytest.mark.parametrize("rope", [dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0, layout="half"),
                                  dict(scaling="parts", factor=8.0, orig_len=2048, mscale=1.2079441541679836),
                                  dict(theta=500000.0)])
def test_append_scaled_and_far_positions(rope):
    """Positions up to 2^30 + 2^20: the angle is exact there too."""
    for off in (0, 131072, (1 << 30) - 1):
        append_case(F32, 4, 2, 64, 16, [5, 9], [100, 9], 7, off=off, **rope)


def test_append_without_rotation_without_queries_and_in_place():
    append_case(BF16, 12, 4, 64, 16, [3, 1], [40, 17], 1)
    assert append_case(BF16, 12, 4, 64, 16, [3, 1], [40, 17], 2, with_q=False, theta=10000.0) is None
    for layout in ("interleaved", "half"):
        for rot in (64, 18):
            append_case(BF16, 12, 4, 64, 16, [30, 1], [40, 17], 3, inplace=True, layout=layout, rot_dim=rot)


def test_append_more_tokens_than_positions():
    """Rows at negative positions are not stored; their queries are zero."""
    append_case(BF16, 12, 4, 64, 16, [9, 4], [4, 0], 5, tail=1, layout="half")


def test_append_many_sequences_finds_every_row():
    rng = random.Random(1)
    n = [rng.choice([0, 0, 1, 2, 5]) for _ in range(1500)]
    append_case(BF16, 4, 2, 32, 8, n, [x + rng.randint(0, 9) for x in n], 6, layout="interleaved")


def test_append_bad_device_arguments_are_reported():
    ps, lens = 16, [40, 30]
    t, P = tables(lens, ps, 3)
    kp, vp = pool(P, ps, 4, 64, BF16, 4), pool(P, ps, 4, 64, BF16, 5)
    k = synthetic.randn((5, 4, 64), 6, 1.0, BF16).cuda()
    for change, word in (("page", "page id"), ("len", "length"), ("cu", "cu_new")):
        t2, l2, c2 = t.copy(), list(lens), [0, 2, 5]
        if change == "page":
            t2[1, 1] = P
        if change == "len":
            l2[1] = -3
        if change == "cu":
            c2[2] = 6
        k0, v0 = kp.clone(), vp.clone()
        ne.paged_append(k, k, kp, vp, i32(t2), i32(l2), i32(c2))
        torch.cuda.synchronize()
        assert ne.get_device_error() == ne.NE_ERR_INVALID_ARG and word in ne.last_error()
        if change != "cu":
            live = torch.zeros(P, ps, dtype=torch.bool, device="cuda")
            for p in (38, 39):
                live[t[0, p // ps], p % ps] = True
            if change == "page":
                for p in (27, 28, 29):
                    live[t[1, p // ps], p % ps] = p // ps != 1
            assert torch.equal(kp[~live], k0[~live]) and torch.equal(vp[~live], v0[~live])
    ok()


# ---------------------------------------------------------------- pages

def state(B, W, P, ps, seed, share=True, shuffle=True):
    """Tables of random lengths; every third sequence shares whole pages with the one before."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, W * ps + 1, B)
    lens[0] = W * ps
    t, at = np.full((B, W), -1, np.int32), 0
    perm = rng.permutation(P) if shuffle else np.arange(P)
    for b in range(B):
        k = -(-int(lens[b]) // ps)
        s = min(int(lens[b]) // ps, int(lens[b - 1]) // ps) if share and b % 3 == 2 else 0
        if at + k - s > P:
            lens[b] = 0
            continue
        t[b, :s] = t[b - 1, :s]
        t[b, s:k] = perm[at:at + k - s]
        at += k - s
    refc = np.bincount(t[t >= 0], minlength=P).astype(np.int32)
    return lens.astype(np.int32), t, refc


def check_pools(kp, vp, k0, v0, copies):
    for src, dst, slots in copies:
        k0[:, dst, :slots] = k0[:, src, :slots]
        v0[:, dst, :slots] = v0[:, src, :slots]
    assert torch.equal(kp, k0) and torch.equal(vp, v0)


SHAPES = [  # B, W, P, ps, L, Hkv, D, dtype, hnd
    (5, 4, 40, 16, 3, 4, 64, BF16, False), (1, 1, 1, 8, 1, 1, 32, BF16, False), (7, 9, 63, 64, 2, 2, 64, F32, True),
    (40, 20, 1000, 8, 2, 3, 128, BF16, True), (300, 33, 9001, 16, 1, 1, 64, BF16, False), (3, 5, 17, 256, 1, 5, 32, F32, False),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[str(s[:4]) for s in SHAPES])
@pytest.mark.parametrize("deep", [False, True])
@pytest.mark.parametrize("inplace", [False, True])
def test_fork(shape, deep, inplace):
    B, W, P, ps, L, Hkv, D, dtype, hnd = shape
    lens, t, refc = state(B, W, P, ps, 1)
    rng = np.random.default_rng(2)
    kp, vp = pool(P, ps, Hkv, D, dtype, 3, hnd, L), pool(P, ps, Hkv, D, dtype, 4, hnd, L)
    k0, v0 = kp.clone(), vp.clone()
    C = max(1, B // 2)
    parents = rng.integers(-1, B, C).astype(np.int32)
    rc = i32(refc)
    got = ne.pages_fork(rc, i32(t), i32(lens), i32(parents), kp, vp, deep=deep, refcount_out=rc if inplace else None)
    ok()
    try:
        want = ref.fork(refc, t, lens, parents, ps, deep)
        short = 0
    except ref.Short as e:
        want, short = (refc, np.full((C, W), -1), np.zeros(C), []), e.args[0]
    for g, w in zip(got, want[:3]):
        assert np.array_equal(g.cpu().numpy(), w)
    assert int(got[3]) == short
    check_pools(kp, vp, k0, v0, want[3])


def run_resize(lens, t, refc, new, kp, vp, ps, inplace):
    k0, v0 = kp.clone(), vp.clone()
    rc, tab = i32(refc), i32(t)
    got = ne.pages_resize(rc, tab, i32(lens), i32(new), kp, vp, refcount_out=rc if inplace else None,
                          table_out=tab if inplace else None)
    ok()
    try:
        want, short = ref.resize(refc, t, lens, new, ps), 0
    except ref.Short as e:
        want, short = (refc, t, []), e.args[0]
    assert int(got[2]) == short
    assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy(), want[1])
    check_pools(kp, vp, k0, v0, want[2])
    return short


@pytest.mark.parametrize("shape", SHAPES, ids=[str(s[:4]) for s in SHAPES])
@pytest.mark.parametrize("inplace", [False, True])
def test_resize(shape, inplace):
    B, W, P, ps, L, Hkv, D, dtype, hnd = shape
    kp, vp = pool(P, ps, Hkv, D, dtype, 3, hnd, L), pool(P, ps, Hkv, D, dtype, 4, hnd, L)
    shorts = 0
    for seed, kind in enumerate(("step", "free", "cut", "any", "any", "same", "grow")):
        lens, t, refc = state(B, W, P, ps, 10 + seed)
        rng = np.random.default_rng(20 + seed)
        cap = W * ps
        new = {"step": np.minimum(lens + 1, cap), "free": np.where(rng.random(B) < 0.5, 0, lens),
               "cut": rng.integers(0, lens + 1), "any": rng.integers(0, cap + 1, B), "same": lens,
               "grow": np.full(B, cap)}[kind].astype(np.int32)
        shorts += run_resize(lens, t, refc, new, kp, vp, ps, inplace) > 0
    print("short:", shorts)


@pytest.mark.parametrize("inplace", [False, True])
def test_resize_short_changes_nothing(inplace):
    """Nine free pages after the releases, twelve wanted."""
    ps, W, P = 16, 8, 20
    t = np.full((3, W), -1, np.int32)
    t[0, :8], t[1, :3], t[2, :2] = np.arange(8), np.arange(8, 11), np.arange(11, 13)
    refc = np.bincount(t[t >= 0], minlength=P).astype(np.int32)
    lens, new = np.array([128, 48, 32], np.int32), np.array([96, 128, 128 - 1], np.int32)
    kp, vp = pool(P, ps, 2, 32, BF16, 3, L=2), pool(P, ps, 2, 32, BF16, 4, L=2)
    assert run_resize(lens, t, refc, new, kp, vp, ps, inplace) == 2


@pytest.mark.parametrize("inplace", [False, True])
def test_resize_unshares_a_page_that_is_cut_into(inplace):
    """Two sequences share pages 4 and 5; both are cut into page 5 and get a copy each, and
    the page they leave is free afterwards."""
    ps, W, P = 8, 4, 12
    t = np.full((3, W), -1, np.int32)
    t[0, :3], t[1, :2], t[2, :1] = [4, 5, 7], [4, 5], [4]
    refc = np.bincount(t[t >= 0], minlength=P).astype(np.int32)
    kp, vp = pool(P, ps, 2, 64, F32, 3, L=2), pool(P, ps, 2, 64, F32, 4, L=2)
    lens, new = np.array([20, 16, 8], np.int32), np.array([13, 9, 30], np.int32)
    assert run_resize(lens, t, refc, new, kp, vp, ps, inplace) == 0


@pytest.mark.parametrize("shape", SHAPES, ids=[str(s[:4]) for s in SHAPES])
@pytest.mark.parametrize("inplace", [False, True])
def test_compact(shape, inplace):
    B, W, P, ps, L, Hkv, D, dtype, hnd = shape
    for seed, shuffle in ((1, True), (2, False), (3, True)):
        lens, t, refc = state(B, W, P, ps, seed, shuffle=shuffle)
        if seed == 3:
            t[:], refc[:] = -1, 0                          # an empty pool
        kp, vp = pool(P, ps, Hkv, D, dtype, 3, hnd, L), pool(P, ps, Hkv, D, dtype, 4, hnd, L)
        k0, v0 = kp.clone(), vp.clone()
        rc, tab = i32(refc), i32(t)
        got = ne.pages_compact(rc, tab, kp, vp, refcount_out=rc if inplace else None, table_out=tab if inplace else None)
        ok()
        want = ref.compact(refc, t, ps)
        assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy(), want[1])
        assert np.array_equal(got[2].cpu().numpy(), want[2]) and int(got[3]) == want[3]
        check_pools(kp, vp, k0, v0, want[4])


def test_pages_report_bad_ids():
    ps, P, W = 16, 20, 4
    kp, vp = pool(P, ps, 2, 64, BF16, 3, L=1), pool(P, ps, 2, 64, BF16, 4, L=1)
    lens, t, refc = state(3, W, P, ps, 1, share=False)
    for what in ("parent", "page", "len"):
        t2, l2, par = t.copy(), lens.copy(), np.array([0, 1], np.int32)
        if what == "parent":
            par[1] = 3
        if what == "page":
            t2[0, 0] = P
        if what == "len":
            l2[0] = W * ps + 1
        k0 = kp.clone()
        ne.pages_fork(i32(refc), i32(t2), i32(l2), i32(par), kp, vp)
        torch.cuda.synchronize()
        assert ne.get_device_error() == ne.NE_ERR_INVALID_ARG
        word = {"parent": "parent", "page": "page id", "len": "length"}[what]
        assert word in ne.last_error()
        k0[:, refc == 0] = kp[:, refc == 0]
        assert torch.equal(kp, k0)                         # pages in use are never written
    ok()


def test_pages_captured():
    """A scheduling step in a graph: the lengths are read at replay."""
    ps, W, P, B = 16, 8, 64, 4
    lens, t, refc = state(B, W, P, ps, 5)
    kp, vp = pool(P, ps, 2, 64, BF16, 3, L=2), pool(P, ps, 2, 64, BF16, 4, L=2)
    rc, tab, old, new = i32(refc), i32(t), i32(lens), i32(lens)
    ws = ne.alloc_pages_workspace(P, B, W)
    outs = [torch.empty_like(rc), torch.empty_like(tab), torch.empty(1, dtype=torch.int32, device="cuda")]
    ne.pages_resize(rc, tab, old, new, kp, vp, *outs, workspace=ws)
    ok()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ne.pages_resize(rc, tab, old, new, kp, vp, *outs, workspace=ws)
    rng = np.random.default_rng(1)
    for _ in range(4):
        want_new = rng.integers(0, W * ps + 1, B).astype(np.int32)
        new.copy_(i32(want_new))
        g.replay()
        ok()
        try:
            want = ref.resize(refc, t, lens, want_new, ps)
        except ref.Short:
            continue
        assert np.array_equal(outs[0].cpu().numpy(), want[0]) and np.array_equal(outs[1].cpu().numpy(), want[1])


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype,Hq,Hkv,D", [(BF16, 12, 4, 64), (F32, 4, 2, 32), (BF16, 16, 4, 128)])
def test_a_serving_run(dtype, Hq, Hkv, D):
    """Sequences take pages, prompts go in by chunks, one is forked, all generate, one ends
    early, the pool is compacted, and every step's attention equals plain attention over
    all tokens so far (keys rotated in 64 bits from the same inputs)."""
    ps, W, P, layers = 16, 12, 80, 2
    rng = np.random.default_rng(1)
    f = ref.rope_angles(D, 10000.0)
    spec = ne.rope_spec(D)
    kp, vp = pool(P, ps, Hkv, D, dtype, 1, L=layers), pool(P, ps, Hkv, D, dtype, 2, L=layers)
    kp.fill_(math.nan), vp.fill_(math.nan)
    refc = torch.zeros(P, dtype=torch.int32, device="cuda")
    table = torch.full((3, W), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    hist = [[] for _ in range(3)]                          # per sequence: (k, v) rows [layers, Hkv, D], fp64 rotated keys

    def step(n):
        nonlocal refc, table, lens
        new = lens + i32(n)
        refc, table, short = ne.pages_resize(refc, table, lens, new, kp, vp)
        assert int(short) == 0
        cu = np.concatenate([[0], np.cumsum(n)])
        N = int(cu[-1])
        starts, lens = lens.tolist(), new
        for l in range(layers):
            qkv = synthetic.randn((N, Hq + 2 * Hkv, D), int(rng.integers(1 << 30)), 1.0, dtype).cuda()
            k, v = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
            q = ne.paged_append(k, v, kp[l], vp[l], table, lens, i32(cu), rope=spec, q=qkv[:, :Hq])
            o, lse = ne.paged_attn(q, kp[l], vp[l], table, lens, i32(cu), max_new=int(max(n)))
            ok()
            x = qkv.double().cpu().numpy()
            for b in range(len(n)):
                pos = np.arange(starts[b], starts[b] + n[b])
                y = ref.rotate(x[cu[b]:cu[b + 1]], pos, f, "interleaved")
                for i in range(n[b]):
                    if l == 0:
                        hist[b].append([])
                    hist[b][starts[b] + i].append((y[i, Hq:Hq + Hkv], x[cu[b] + i, Hq + Hkv:]))
                if n[b] == 0:
                    continue
                kk = torch.from_numpy(np.stack([h[l][0] for h in hist[b]]))
                vv = torch.from_numpy(np.stack([h[l][1] for h in hist[b]]))
                o_ref, lse_ref, A, S = ref.attend(torch.from_numpy(y[:, :Hq]), kk, vv, starts[b])
                # Queries and keys were rounded once more than in the reference (half a step of
                # the rotated value each): logits off by 2 half steps of S on top of the bounds.
                tol_o, tol_lse = ref.attn_bounds(o_ref, A, S, lse_ref, D, len(hist[b]), HALF[dtype],
                                                 (HALF[BF16] if dtype == BF16 else 0.0))
                extra = 2 * HALF[dtype] * (1 + HALF[dtype]) * S + (0 if dtype == BF16 else 2.0 ** -20 * S)
                e = (o[cu[b]:cu[b + 1]].double().cpu() - o_ref).abs()
                grow = torch.expm1(2 * extra)[..., None] * A   # every weight off by a factor e^(+-2 extra) at most
                assert bool((e <= tol_o + grow).all())
                e = (lse[cu[b]:cu[b + 1]].double().cpu() - lse_ref).abs()
                assert bool((e <= tol_lse + extra).all())

    step([40, 7, 0])
    step([1, 33, 5])                                       # a chunk beside a single token
    # The third sequence ends; its place is taken by a fork of the second.
    refc, table, short = ne.pages_resize(refc, table, lens, lens * i32([1, 1, 0]), kp, vp)
    refc, child, cl, short = ne.pages_fork(refc, table, lens * i32([1, 1, 0]), i32([1]), kp, vp)
    table[2], lens = child[0], torch.cat((lens[:2], cl))
    hist[2] = [list(x) for x in hist[1]]
    for _ in range(3):
        step([1, 1, 1])
    refc, table, remap, n_live = ne.pages_compact(refc, table, kp, vp)
    assert int(n_live) == int((refc > 0).sum()) and bool((refc[int(n_live):] == 0).all())
    step([1, 1, 20])
    # Speculative tokens taken back, then other ones.
    back = lens - i32([0, 0, 9])
    refc, table, short = ne.pages_resize(refc, table, lens, back, kp, vp)
    lens, hist[2] = back, hist[2][:-9]
    step([1, 1, 1])
    refc, table, short = ne.pages_resize(refc, table, lens, lens * 0, kp, vp)
    ok()
    assert not bool(refc.any()) and bool((table == -1).all())


def test_whole_prompt_equals_the_training_attention():
    """Rotation, cache and attention of a whole prompt against attn_fwd on the same tokens."""
    B, T, Hq, Hkv, D, ps = 2, 200, 12, 4, 64, 16
    q, k, v, _ = (x.cuda() for x in synthetic.make_custom(B, T, Hq, Hkv, D, BF16, seed=3))
    o, lse = ne.attn_fwd(q, k, v)
    t, P = tables([T] * B, ps, 1)
    kp, vp = pool(P, ps, Hkv, D, BF16, 1), pool(P, ps, Hkv, D, BF16, 2)
    table, ln, cu = i32(t), i32([T] * B), i32([0, T, 2 * T])
    qr = ne.paged_append(k.flatten(0, 1), v.flatten(0, 1), kp, vp, table, ln, cu, rope=ne.rope_spec(D), q=q.flatten(0, 1))
    o2, lse2 = ne.paged_attn(qr, kp, vp, table, ln, cu)
    ok()
    # attn_fwd keeps rotated values in fp16 (half step 2^-11) where the cache holds bf16
    # (2^-8), so a logit differs by at most x = 2 (2^-8 + 2^-11) S and a weight by a factor of
    # e^(2x); the weights of the products and the outputs are rounded to bf16 on both sides.
    x = 2 * (2.0 ** -8 + 2.0 ** -11)
    for b in range(B):
        o_ref, _, A, S = ref.attend(q[b].double(), k[b].double(), v[b].double(), 0)
        # (S of the unrotated rows; a rotated pair's magnitudes add up to at most sqrt 2 times as
        # much on either side.)
        d = (o[b].double() - o2[b * T:(b + 1) * T].double()).abs()
        assert bool((d <= torch.expm1(2 * x * 2 * S)[..., None] * A + 2 * 2.0 ** -8 * (A + o_ref.abs()) + 2.0 ** -7 * A).all())
        e = (lse[b].T.double() - lse2[b * T:(b + 1) * T].double()).abs()
        assert bool((e <= x * 2 * S + 2.0 ** -10).all())
