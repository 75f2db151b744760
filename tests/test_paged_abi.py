"""The paged-cache calls without a GPU: refusals before any device work, the rope spec
against its formulas, workspace sizes, and a model of how the attention's work is split."""
import ctypes
import math
import random

import numpy as np
import pytest
import torch

import causal_gqa_flash_attention_gb300 as ne
from causal_gqa_flash_attention_gb300 import _build

import paged_ref as ref

vp = ctypes.c_void_p
P, NULL = vp(4096), vp(0)
WS = 1 << 34


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ne.load()


def cache(**kw):
    c = dict(k=4096, v=4096, elem_bytes=2, layers=1, n_pages=8, page_size=16, Hkv=2, D=64, layer_stride=0,
             page_stride=16 * 128, tok_stride=128, head_stride=64)
    c.update(kw)
    return ctypes.byref(ne.PagedCache(*[c[n] for n, _ in ne.PagedCache._fields_]))


def attn(lib, c=None, q=P, table=P, lens=P, cu=P, o=vp(1 << 20), lse=vp(2 << 20), q_ld=256, B=2, N=5, Hq=4, W=4, max_new=3, ws=P, nb=WS, f32=False):
    fn = lib.ne_paged_attn_f32 if f32 else lib.ne_paged_attn
    return fn(q, cache() if c is None else c, table, lens, cu, o, lse, q_ld, B, N, Hq, W, max_new, ws, nb, NULL)


def append(lib, c=None, q=P, k=vp(1 << 20), v=vp(2 << 20), table=P, lens=P, cu=P, spec=None, off=0, qo=vp(3 << 20), lds=(256, 128, 128, 256), B=2, N=5,
           Hq=4, W=4):
    return lib.ne_paged_append(q, k, v, cache() if c is None else c, table, lens, cu, spec, off, qo, *lds, B, N, Hq, W, NULL)


BAD_CACHES = [
    (dict(elem_bytes=8), ne.NE_ERR_INVALID_ARG, "elem_bytes"),
    (dict(elem_bytes=4), ne.NE_ERR_INVALID_ARG, "element"),                  # f32 pools, bf16 call
    (dict(layers=2, layer_stride=1 << 20), ne.NE_ERR_INVALID_ARG, "layer"),
    (dict(n_pages=1 << 24), ne.NE_ERR_INVALID_ARG, "n_pages"),
    (dict(page_size=24), ne.NE_ERR_UNSUPPORTED, "page_size"),
    (dict(page_size=4), ne.NE_ERR_UNSUPPORTED, "page_size"),
    (dict(page_size=512), ne.NE_ERR_UNSUPPORTED, "page_size"),
    (dict(D=96), ne.NE_ERR_UNSUPPORTED, "head_dim"),
    (dict(k=None), ne.NE_ERR_INVALID_ARG, "null"),
    (dict(v=4104), ne.NE_ERR_INVALID_ARG, "aligned"),
    (dict(tok_stride=132), ne.NE_ERR_INVALID_ARG, "stride"),                 # not 16 bytes
    (dict(head_stride=32), ne.NE_ERR_INVALID_ARG, "stride"),                 # heads overlap
    (dict(page_stride=1 << 39), ne.NE_ERR_INVALID_ARG, "stride"),
]


@pytest.mark.parametrize("kw,status,word", BAD_CACHES, ids=[str(k) for k, _, _ in BAD_CACHES])
def test_attn_and_append_refuse_bad_caches(lib, kw, status, word):
    for st in (attn(lib, cache(**kw)), append(lib, cache(**kw))):
        assert st == status and word in lib.ne_last_error().decode()


@pytest.mark.parametrize("kw,word", [
    (dict(Hq=5), "Hkv"), (dict(Hq=0), "Hkv"), (dict(B=-1), "B and N"), (dict(N=-1), "B and N"), (dict(cu=NULL), "N == B"),
    (dict(W=0), "max_pages"), (dict(W=1 << 27), "max_pages"), (dict(table=NULL), "page_table"), (dict(lens=vp(4098)), "4-byte"),
    (dict(cu=vp(4097)), "4-byte"), (dict(max_new=0), "max_new"), (dict(q=NULL), "q must"), (dict(q=vp(4104)), "aligned"),
    (dict(q_ld=255), "rows"), (dict(q_ld=260), "rows"), (dict(o=NULL), "null"), (dict(lse=vp(4100)), "aligned"),
    (dict(ws=NULL), "workspace"), (dict(ws=vp(4112)), "workspace"), (dict(nb=1024), "too small"), (dict(N=1 << 24), "2^31"),
    (dict(o=vp(4096 + 512)), "overlap"), (dict(lse=vp(1 << 20)), "overlap"), (dict(lse=vp(4096 + 64)), "overlap"),
])
def test_attn_refuses_bad_arguments(lib, kw, word):
    assert attn(lib, **kw) == ne.NE_ERR_INVALID_ARG and word in lib.ne_last_error().decode()


def test_f32_attn_refuses_head_dim_128_and_bf16_pools(lib):
    assert attn(lib, cache(elem_bytes=4, D=128, head_stride=128, tok_stride=256), f32=True) == ne.NE_ERR_UNSUPPORTED
    assert attn(lib, cache(), f32=True) == ne.NE_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,word", [
    (dict(q=NULL), "together"), (dict(qo=NULL), "together"), (dict(k=NULL), "k must"), (dict(v=vp(4104)), "v must"),
    (dict(lds=(256, 64, 128, 256)), "k rows"), (dict(lds=(256, 128, 132, 256)), "v rows"), (dict(lds=(248, 128, 128, 256)), "q rows"),
    (dict(lds=(256, 128, 128, 128)), "q_out rows"), (dict(qo=P, lds=(256, 128, 128, 512)), "same row stride"),
    (dict(qo=vp(4096 + 256)), "q_out"), (dict(qo=vp((1 << 20) + 64)), "k or v"),
    (dict(off=-1), "pos_offset"), (dict(off=1 << 30), "pos_offset"), (dict(cu=NULL), "N == B"), (dict(N=1 << 25), "2^31"),
])
def test_append_refuses_bad_arguments(lib, kw, word):
    assert append(lib, **kw) == ne.NE_ERR_INVALID_ARG and word in lib.ne_last_error().decode()


def test_append_refuses_a_spec_of_another_head_dim(lib):
    assert append(lib, spec=ctypes.byref(ne.rope_spec(128))) == ne.NE_ERR_INVALID_ARG
    assert append(lib, spec=ctypes.byref(ne.RopeSpec())) == ne.NE_ERR_INVALID_ARG


def test_empty_calls_are_no_ops(lib):
    assert attn(lib, q=NULL, table=NULL, lens=NULL, cu=NULL, o=NULL, lse=NULL, B=0, N=0, ws=NULL, nb=0) == ne.NE_OK
    assert append(lib, q=NULL, qo=NULL, k=NULL, v=NULL, table=NULL, lens=NULL, cu=NULL, B=0, N=0) == ne.NE_OK


def pages(lib, op, c=None, ref=vp(1 << 20), table=vp(2 << 20), lens=vp(3 << 20), other=vp(4 << 20), ro=vp(5 << 20), to=vp(6 << 20),
          lo=vp(7 << 20), one=vp(8 << 20), B=4, n=3, W=4, ws=vp(9 << 20), nb=1 << 20):
    c = cache(layers=2, layer_stride=1 << 16) if c is None else c
    if op == "fork":
        return lib.ne_pages_fork(c, ref, table, lens, other, 0, ro, to, lo, one, B, n, W, ws, nb, NULL)
    if op == "resize":
        return lib.ne_pages_resize(c, ref, table, lens, other, ro, to, one, B, W, ws, nb, NULL)
    return lib.ne_pages_compact(c, ref, table, ro, to, lo, one, B, W, ws, nb, NULL)


@pytest.mark.parametrize("op", ["fork", "resize", "compact"])
@pytest.mark.parametrize("kw,word", [
    (dict(ref=NULL), "null"), (dict(table=NULL), "null"), (dict(ro=vp(4104)), "aligned"), (dict(to=NULL), "null"),
    (dict(one=NULL), "null"), (dict(table=vp(4098)), "aligned"), (dict(one=vp(1 << 20)), "overlap"),
    (dict(to=vp(5 << 20)), "overlap"), (dict(B=-1), ">= 0"), (dict(W=0), "max_pages"), (dict(W=1 << 27), "max_pages"),
    (dict(ro=vp((1 << 20) + 16)), "refcount_out"), (dict(to=vp((2 << 20) + 16)), "table_out"), (dict(ws=NULL), "workspace"),
    (dict(nb=512), "too small"),
])
def test_pages_calls_refuse_bad_arguments(lib, op, kw, word):
    assert pages(lib, op, **kw) == ne.NE_ERR_INVALID_ARG and word in lib.ne_last_error().decode()


def test_a_fork_refuses_its_own_table_and_lengths_as_outputs(lib):
    assert pages(lib, "fork", to=vp(2 << 20)) == ne.NE_ERR_INVALID_ARG
    for other in (3 << 20, (4 << 20) + 8):                 # seq_lens; inside parents
        assert pages(lib, "fork", lo=vp(other)) == ne.NE_ERR_INVALID_ARG and "child_lens" in lib.ne_last_error().decode()
    assert pages(lib, "fork", other=NULL) == ne.NE_ERR_INVALID_ARG
    assert pages(lib, "resize", lens=NULL) == ne.NE_ERR_INVALID_ARG
    assert pages(lib, "compact", lo=NULL) == ne.NE_ERR_INVALID_ARG


def test_workspace_sizes(lib):
    assert lib.ne_paged_attn_workspace_size(4, 8, 12, 5, 64) == 0                   # Hq % Hkv
    assert lib.ne_paged_attn_workspace_size(4, 8, 12, 4, 96) == 0
    assert lib.ne_paged_attn_workspace_size(4, 8, 12, 4, 64) % 256 == 0
    assert lib.ne_pages_workspace_size(0, 4, 4) == 0
    # Header, two offsets per sequence, free ids and (source, target, slots, 0) of every listed
    # page: min(pages, entries) when pages are taken, half of the pool when they are moved.
    r = lambda x: -(-x // 256) * 256  # noqa: E731
    assert lib.ne_pages_workspace_size(1000, 10, 8) == 256 + r(10 * 8) + r(501 * 4) + r(501 * 16)
    assert lib.ne_pages_workspace_size(100, 10, 80) == 256 + r(10 * 8) + r(100 * 4) + r(100 * 16)


# ---------------------------------------------------------------- rope spec

@pytest.mark.parametrize("kw", [dict(), dict(rot_dim=18), dict(theta=500000.0), dict(scaling="linear", factor=4.0),
                                dict(scaling="base", factor=8.0), dict(scaling="parts", factor=8.0, orig_len=2048),
                                dict(scaling="parts", factor=4.0, orig_len=128, beta_fast=4.0, beta_slow=0.5)])
def test_rope_spec_angles(lib, kw):
    """turns / 2^64 is f / (2 pi) to the rounding of fp64 (f and the division) and of the
    64-bit fraction itself: a number on a grid of 2^-64 is at most 2^-65 from its value."""
    s = ne.rope_spec(64, **kw)
    f = ref.rope_angles(kw.get("rot_dim", 64), kw.get("theta", 10000.0), kw.get("scaling", "none"), kw.get("factor", 1.0),
                        kw.get("orig_len", 0), kw.get("beta_fast", 32.0), kw.get("beta_slow", 1.0))
    got = np.array([s.turns[i] for i in range(len(f))], np.float64) / 2.0 ** 64
    assert np.all(np.abs(got - f / (2 * np.pi)) <= 16 * 2.0 ** -53 * f + 2.0 ** -65)
    assert all(s.turns[i] == 0 for i in range(len(f), 64))


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=66), dict(rot_dim=3), dict(theta=0.0), dict(theta=math.inf),
                                dict(scaling="linear", factor=0.0), dict(scaling="base", factor=2.0, rot_dim=2),
                                dict(scaling="parts", factor=2.0), dict(mscale=math.nan),
                                dict(scaling="parts", factor=2.0, orig_len=8, beta_fast=1.0, beta_slow=1.0)])
def test_rope_spec_refusals(lib, kw):
    with pytest.raises(ne.NeError):
        ne.rope_spec(64, **kw)


def test_rope_spec_names(lib):
    with pytest.raises(ValueError, match="layout"):
        ne.rope_spec(64, layout="quarter")
    with pytest.raises(ValueError, match="scaling"):
        ne.rope_spec(64, scaling="yes")
    with pytest.raises(ne.NeError):
        ne.rope_spec(256)


# ---------------------------------------------------------------- binding

def test_binding_refuses_host_tensors_and_mismatches(lib):
    kp = torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16)
    t = torch.zeros(2, 4, dtype=torch.int32)
    ln = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ne.paged_attn(q, kp, kp, t, ln)
    with pytest.raises(ValueError, match="page_size"):
        ne.paged_attn(q, kp[0], kp[0], t, ln)
    with pytest.raises(ValueError, match="CUDA"):
        ne.paged_append(q[:, :2], q[:, :2], kp, kp, t, ln)
    with pytest.raises(ValueError, match="CUDA"):
        ne.pages_fork(torch.zeros(8, dtype=torch.int32), t, ln, ln, kp, kp)


# ---------------------------------------------------------------- the split of the work

class Split:
    """How the attention kernels cut a call, step by step as in paged_sched.cuh."""

    def __init__(self, n, lens, Hkv, G, rows, bn, C, ovh=384, min_work=128, w_full=1, w_part=1, sub=0, snap=0, snap_shift=0):
        self.n, self.lens, self.bn, self.ovh = n, lens, bn, ovh
        self.gs = min(G, rows)
        self.tpt = rows // self.gs
        self.hg = Hkv * -(-G // self.gs)
        units = []
        for b, (nb, L) in enumerate(zip(n, lens)):
            for hg in range(self.hg):
                for r in range(-(-nb // self.tpt)):
                    kv = L if r == -(-nb // self.tpt) - 1 else max(0, L - nb + (r + 1) * self.tpt)
                    units.append((b, hg, r, kv, w_full if min(self.tpt, nb - r * self.tpt) > sub else w_part))
        self.units = units
        self.start = np.concatenate([[0], np.cumsum([ovh + u[3] * u[4] for u in units])]).astype(object)
        W = int(self.start[-1])
        self.C = C
        self.snap = min(snap, (W * ((2 ** 64 - 1) // C) >> 64) >> snap_shift)
        if W < C * min_work:
            self.w = [min(c * min_work, W) for c in range(C + 1)]
        else:
            self.w = [W * (c * ((2 ** 64 - 1) // C)) >> 64 for c in range(C)] + [W]

    def parts(self, c):
        out = []
        for (b, hg, r, kv, weight), u0 in zip(self.units, self.start):
            cost, nt = self.ovh + kv * weight, -(-kv // self.bn)
            w0, w1 = self.w[c], self.w[c + 1]
            if u0 + cost <= w0 or u0 >= w1:
                continue
            per = np.float32(nt) / np.float32(cost)

            def cut(x):
                c = min(nt, int(np.rint(np.float32(x) * per)))
                return 0 if c <= self.snap else nt if nt - c <= self.snap else c
            t0 = 0 if w0 <= u0 else cut(w0 - u0)
            t1 = nt if w1 >= u0 + cost else cut(w1 - u0)
            if t0 < t1 or (nt == 0 and w0 <= u0):
                out.append((b, hg, r, t0, t1, nt))
        return out


@pytest.mark.parametrize("seed", range(40))
def test_split_covers_every_key_tile_once_and_parts_can_be_joined(seed):
    rng = random.Random(seed)
    G, Hkv = rng.choice([1, 2, 3, 5, 8, 20]), rng.choice([1, 2, 4])
    rows, bn, C, more = rng.choice([(16, 64, 304, dict(snap=3, snap_shift=8)), (32, 128, 304, dict(snap=3, snap_shift=9)), (8, 256, 152, {}), (64, 32, 304, {}),
                                    (256, 128, 152, dict(ovh=1024, min_work=2048, w_full=5, w_part=4, sub=128 // G, snap=1))])
    B = rng.randint(1, 9)
    n = [rng.choice([0, 1, 1, rng.randint(1, 60)]) for _ in range(B)]
    lens = [rng.choice([0, 1, rng.randint(1, 200), rng.randint(1, 9000)]) for _ in range(B)]
    s = Split(n, lens, Hkv, G, rows, bn, C, **more)
    seen, records = {}, {}
    for c in range(s.C):
        heads = tails = 0
        for b, hg, r, t0, t1, nt in s.parts(c):
            seen.setdefault((b, hg, r), []).append((t0, t1, nt))
            if (t0, t1) != (0, nt):
                slot = 1 if t0 == 0 else 0
                heads, tails = heads + slot, tails + 1 - slot
                records[2 * c + slot] = ((b, hg, r), 2 if t1 == nt else 1)
        assert heads <= 1 and tails <= 1                   # one slot of each kind per CTA
    assert set(seen) == {u[:3] for u in s.units}
    for parts in seen.values():
        parts.sort()
        assert parts[0][0] == 0 and parts[-1][1] == parts[-1][2]
        assert all(a[1] == b[0] for a, b in zip(parts, parts[1:]))
    # The join's walk: from every slot-1 record over the following slot-0 records to a last one.
    joined = 0
    for c in range(s.C):
        if 2 * c + 1 not in records:
            continue
        unit, found = records[2 * c + 1][0], 1
        for d in range(c + 1, s.C):
            if 2 * d in records:
                assert records[2 * d][0] == unit
                found += 1
                if records[2 * d][1] == 2:
                    break
        else:
            raise AssertionError("a cut unit without an end")
        assert found == len(seen[unit])
        joined += found
    assert joined == len(records)
