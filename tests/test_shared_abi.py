"""ne_paged_attn_shared and ne_paged_weights without a GPU: refusals before any device work, workspace sizes,
and what the binding refuses."""
import ctypes

import pytest
import torch

import causal_gqa_flash_attention_gb300 as ne
from causal_gqa_flash_attention_gb300 import _build

vp = ctypes.c_void_p
MB = 1 << 20
NULL = vp(0)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ne.load()


def cache(**kw):
    c = dict(k=4096, v=4096, elem_bytes=2, layers=1, n_pages=8, page_size=16, Hkv=2, D=64, layer_stride=0,
             page_stride=16 * 128, tok_stride=128, head_stride=64)
    c.update(kw)
    return ctypes.byref(ne.PagedCache(*[c[n] for n, _ in ne.PagedCache._fields_]))


A = dict(q=vp(1 * MB), table=vp(2 * MB), lens=vp(3 * MB), cu=vp(4 * MB), groups=vp(5 * MB), shared=vp(6 * MB), R=1, o=vp(7 * MB),
         lse=vp(8 * MB), q_ld=256, B=2, N=5, Hq=4, W=4, max_new=3, ws=vp(16 * MB), nb=1 << 34)


def attn(lib, c=None, f32=False, **kw):
    a = A | kw
    fn = lib.ne_paged_attn_shared_f32 if f32 else lib.ne_paged_attn_shared
    return fn(a["q"], cache() if c is None else c, a["table"], a["lens"], a["cu"], a["groups"], a["shared"], a["R"], a["o"], a["lse"], a["q_ld"],
              a["B"], a["N"], a["Hq"], a["W"], a["max_new"], a["ws"], a["nb"], NULL)


@pytest.mark.parametrize("kw,text", [
    (dict(groups=NULL), "groups"), (dict(groups=vp(5 * MB + 2)), "groups"), (dict(shared=NULL), "shared"), (dict(R=-1), "R"), (dict(R=3), "R"),
    (dict(q=NULL), "q"), (dict(q_ld=200), "q"), (dict(o=vp(1 * MB)), "overlap"), (dict(lse=vp(7 * MB)), "overlap"), (dict(Hq=5), "Hq"),
    (dict(max_new=0), "max_new"), (dict(W=0), "max_pages"), (dict(table=NULL), "page_table"), (dict(cu=NULL), "N == B"),
    (dict(ws=NULL), "workspace"), (dict(ws=vp(16 * MB + 32)), "workspace"), (dict(nb=1 << 20), "too small"),
])
def test_shared_refusals(lib, kw, text):
    assert attn(lib, **kw) == ne.NE_ERR_INVALID_ARG
    assert text in ne.last_error()


def test_shared_bad_caches_and_empty_calls(lib):
    assert attn(lib, cache(layers=2, layer_stride=1 << 20)) == ne.NE_ERR_INVALID_ARG
    assert attn(lib, cache(elem_bytes=4)) == ne.NE_ERR_INVALID_ARG and attn(lib, f32=True) == ne.NE_ERR_INVALID_ARG
    assert attn(lib, cache(D=96)) == ne.NE_ERR_UNSUPPORTED
    assert attn(lib, B=0, R=0) == ne.NE_OK and attn(lib, N=0, q=NULL) == ne.NE_OK


def test_shared_workspace(lib):
    """Two workspaces of ne_paged_attn (of the tile kernel's at head_dim 32), and rows and records of two lines."""
    r256 = lambda x: -(-x // 256) * 256  # noqa: E731
    for N, Hq, Hkv, D in ((64, 12, 4, 64), (5, 8, 2, 128)):
        rows = N * Hq
        want = 2 * (lib.ne_paged_attn_workspace_size(1, N, Hq, Hkv, D) + r256(rows * D * 4) + 2 * r256(rows * 8))
        assert lib.ne_paged_attn_shared_workspace_size(1, N, Hq, Hkv, D) == want
    parts = r256(304 * 256 * (32 * 4 + 8) + 304 * 16)
    assert lib.ne_paged_attn_shared_workspace_size(1, 4, 4, 2, 32) == 2 * (parts + r256(16 * 128) + 2 * r256(16 * 8))
    assert lib.ne_paged_attn_shared_workspace_size(1, 4, 5, 2, 32) == 0


WT = dict(q=vp(1 * MB), lse=vp(2 * MB), table=vp(3 * MB), lens=vp(4 * MB), cu=vp(5 * MB), w=vp(6 * MB), out=vp(7 * MB), q_ld=256, B=2, N=5,
          Hq=4, W=4, max_new=30, ws=vp(16 * MB), nb=1 << 34)


def weights(lib, c=None, f32=False, **kw):
    a = WT | kw
    fn = lib.ne_paged_weights_f32 if f32 else lib.ne_paged_weights
    return fn(a["q"], a["lse"], cache() if c is None else c, a["table"], a["lens"], a["cu"], a["w"], a["out"], a["q_ld"], a["B"], a["N"],
              a["Hq"], a["W"], a["max_new"], a["ws"], a["nb"], NULL)


@pytest.mark.parametrize("kw,text", [
    (dict(q=NULL), "q"), (dict(q_ld=260), "q"), (dict(lse=NULL), "lse"), (dict(out=NULL), "weights_out"), (dict(w=vp(6 * MB + 2)), "weights"),
    (dict(out=vp(6 * MB + 64)), "overlap"), (dict(out=vp(1 * MB)), "overlap"), (dict(out=vp(2 * MB)), "overlap"), (dict(B=-1), "B"),
    (dict(N=-1), "N"), (dict(max_new=0), "max_new"), (dict(Hq=5), "Hq"), (dict(W=0), "max_pages"), (dict(cu=NULL), "N == B"),
    (dict(cu=vp(5 * MB + 2)), "cu_new"), (dict(cu=vp(5 * MB + 2), N=0), "cu_new"), (dict(table=NULL, N=0), "page_table"),
    (dict(max_new=40, N=50, ws=NULL), "workspace"), (dict(max_new=40, N=50, ws=vp(16 * MB + 8)), "workspace"), (dict(max_new=40, N=50, nb=1000), "too small"),
])
def test_weights_refusals(lib, kw, text):
    assert weights(lib, **kw) == ne.NE_ERR_INVALID_ARG
    assert text in ne.last_error()


def test_weights_bad_caches_and_empty_calls(lib):
    assert weights(lib, cache(layers=2, layer_stride=1 << 20)) == ne.NE_ERR_INVALID_ARG
    assert weights(lib, cache(elem_bytes=4)) == ne.NE_ERR_INVALID_ARG and weights(lib, f32=True) == ne.NE_ERR_INVALID_ARG
    assert weights(lib, B=0) == ne.NE_OK
    assert lib.ne_paged_weights_workspace_size() == 304 * (256 * 4 + 16)


def test_the_binding_refuses_what_is_not_on_a_gpu():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, 2, dtype=torch.int32)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ne.paged_attn_shared(q, k, k, i, i[0], i[0], i[0, :1])
    with pytest.raises(ValueError):
        ne.paged_weights(q, torch.zeros(2, 4), k, i, i[0])
    with pytest.raises(ValueError):
        ne.pages_evict(torch.zeros(2, 2, 32), torch.zeros(2, 2, 32, dtype=torch.int32), i[0], i, i[0], i[0], k, k)
    with pytest.raises(ValueError):
        ne.paged_attn_shared(q, k, k, i, i[0], i[0], i[0, :1], max_new=1 << 40)
    with pytest.raises(ValueError):
        ne.paged_weights(q, torch.zeros(2, 4), k, i, i[0], max_new=1 << 40)
