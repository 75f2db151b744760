"""ne_pages_evict and ne_paged_append_at without a GPU: refusals before any device work, workspace sizes."""
import ctypes

import pytest

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


ARGS = dict(w=vp(1 * MB), pos=vp(2 * MB), off=vp(3 * MB), table=vp(4 * MB), lens=vp(5 * MB), new=vp(6 * MB), sink=0, recent=0,
            w_out=vp(7 * MB), pos_out=vp(8 * MB), off_out=vp(9 * MB), B=2, W=4, ws=vp(16 * MB), nb=1 << 34)


def evict(lib, c=None, **kw):
    a = ARGS | kw
    return lib.ne_pages_evict(cache() if c is None else c, a["w"], a["pos"], a["off"], a["table"], a["lens"], a["new"], a["sink"],
                              a["recent"], a["w_out"], a["pos_out"], a["off_out"], a["B"], a["W"], a["ws"], a["nb"], NULL)


@pytest.mark.parametrize("kw,text", [
    (dict(w=NULL), "weights"), (dict(pos=vp(2 * MB + 2)), "positions"), (dict(w=vp(MB + 8)), "aligned"), (dict(pos_out=vp(8 * MB + 8)), "aligned"), (dict(off=NULL), "pos_offset"), (dict(table=NULL), "page_table"),
    (dict(lens=NULL), "seq_lens"), (dict(new=NULL), "new_lens"), (dict(w_out=NULL), "weights_out"), (dict(pos_out=NULL), "positions_out"),
    (dict(off_out=NULL), "pos_offset_out"), (dict(sink=-1), "sink"), (dict(recent=(1 << 30) + 1), "recent"), (dict(B=-1), "B"),
    (dict(W=0), "max_pages"), (dict(W=(1 << 26) + 1), "max_pages"), (dict(B=1 << 30), "layers"), (dict(ws=NULL), "workspace"),
    (dict(ws=vp(16 * MB + 16)), "workspace"), (dict(nb=100), "too small"),
    (dict(w_out=vp(1 * MB + 64)), "overlap"),              # shifted onto its own input
    (dict(w_out=vp(2 * MB)), "overlap"), (dict(pos_out=vp(1 * MB)), "overlap"), (dict(off_out=vp(5 * MB)), "overlap"),
    (dict(pos_out=vp(7 * MB + 4)), "overlap"), (dict(off_out=vp(3 * MB + 4)), "overlap"),
])
def test_evict_refusals(lib, kw, text):
    assert evict(lib, **kw) == ne.NE_ERR_INVALID_ARG
    assert text in ne.last_error()


def test_evict_takes_its_inputs_as_outputs(lib):
    """In place passes the argument checks: what stops it here is the missing device."""
    got = evict(lib, w_out=ARGS["w"], pos_out=ARGS["pos"], off_out=ARGS["off"])
    assert got != ne.NE_ERR_INVALID_ARG or "overlap" not in ne.last_error()


def test_evict_bad_cache_and_empty_call(lib):
    assert evict(lib, cache(page_size=24)) == ne.NE_ERR_UNSUPPORTED
    assert evict(lib, cache(tok_stride=132)) == ne.NE_ERR_INVALID_ARG
    assert evict(lib, B=0, w=NULL, lens=NULL) == ne.NE_OK


def test_evict_workspace(lib):
    assert lib.ne_pages_evict_workspace_size(16, 16, 4, 528) == 4096 + 1024 * 528 * 4
    assert lib.ne_pages_evict_workspace_size(1, 0, 1, 16) == 0
    for bad in ((0, 1, 1, 16), (1, -1, 1, 16), (1, 1, 0, 16), (1, 1, 1, 0), (1 << 12, 1 << 12, 1 << 10, 16)):
        assert lib.ne_pages_evict_workspace_size(*bad) == 0


def test_append_at_needs_offsets(lib):
    for fn, eb in ((lib.ne_paged_append_at, 2), (lib.ne_paged_append_at_f32, 4)):
        for off in (NULL, vp(3 * MB + 2)):
            got = fn(NULL, vp(1 * MB), vp(2 * MB), cache(elem_bytes=eb), vp(4 * MB), vp(5 * MB), vp(6 * MB), None, off, NULL, 0, 128, 128, 0, 2,
                     5, 0, 4, NULL)
            assert got == ne.NE_ERR_INVALID_ARG and "pos_offsets" in ne.last_error()
