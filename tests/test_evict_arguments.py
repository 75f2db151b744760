"""What ne_pages_evict refuses of its arrays and pools, and that its in-place form is none of it.  No call here gets as
far as a device: the addresses are made up, and every call ends in a refusal."""
import pytest

import causal_gqa_flash_attention_gb300 as ne

from test_evict_abi import ARGS, MB, cache, evict, lib, vp  # noqa: F401

POOLS = dict(k=64 * MB, v=96 * MB)


def test_one_pool_for_both_is_refused(lib):  # noqa: F811
    """k and v are both written: with one address behind both they are one output twice."""
    assert evict(lib, cache(k=64 * MB, v=64 * MB)) == ne.NE_ERR_INVALID_ARG
    assert "pool" in ne.last_error()


@pytest.mark.parametrize("same", [("w",), ("pos",), ("off",), ("w", "pos", "off")])
def test_outputs_may_be_their_inputs(lib, same):  # noqa: F811
    """Shown by the refusal that comes behind the one of overlaps: a workspace of 100 bytes."""
    assert evict(lib, cache(**POOLS), nb=100, **{x + "_out": ARGS[x] for x in same}) == ne.NE_ERR_INVALID_ARG
    assert "too small" in ne.last_error()


@pytest.mark.parametrize("name", ["w", "pos", "off", "table", "lens", "new", "w_out", "pos_out", "off_out"])
def test_a_workspace_on_an_array_is_refused(lib, name):  # noqa: F811
    """Its lists are written while rows are still read: at the array's address, and where only its end reaches into it."""
    need = lib.ne_pages_evict_workspace_size(1, 2, 2, 64)
    for at in (ARGS[name].value, ARGS[name].value - need + 256):
        assert evict(lib, cache(**POOLS), ws=vp(at)) == ne.NE_ERR_INVALID_ARG
        assert "overlap" in ne.last_error() and "workspace" in ne.last_error()
    assert evict(lib, cache(**POOLS), ws=vp(ARGS[name].value - need), nb=100) == ne.NE_ERR_INVALID_ARG
    assert "too small" in ne.last_error()                  # (in front of it: no overlap)
