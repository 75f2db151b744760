"""Page ids outside the pool in the tables of pages_resize, pages_compact and a short fork:
reported whichever entry holds them, and everything else as if the entry were not there."""
import numpy as np
import pytest
import torch

import causal_gqa_flash_attention_gb300 as ne
from causal_gqa_flash_attention_gb300 import _build

pytestmark = pytest.mark.gpu

PS, P, W = 16, 20, 4
TABLE = np.array([[0, 1, 2, -1], [3, 4, 5, -1], [6, -1, -1, -1]], np.int32)
LENS = np.array([40, 33, 16], np.int32)
REF = np.bincount(TABLE[TABLE >= 0], minlength=P).astype(np.int32)
BAD = [P, -2, 2 ** 31 - 1, -2 ** 31]


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    ne.load()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def pools():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    return [torch.empty((2, P, PS, 2, 32), dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in "kv"]


def reported():
    torch.cuda.synchronize()
    status = ne.get_device_error()
    assert status in (ne.NE_OK, ne.NE_ERR_INVALID_ARG)
    if status != ne.NE_OK:
        assert "page id" in ne.last_error()
    return status != ne.NE_OK


def resize(table, new, ref=REF):
    kp, vp = pools()
    k0, v0 = kp.clone(), vp.clone()
    got = ne.pages_resize(i32(ref), i32(table), i32(LENS), i32(new), kp, vp)
    bad = reported()
    assert torch.equal(kp, k0) and torch.equal(vp, v0)         # (no page of these cases is shared)
    return [x.cpu().numpy() for x in got] + [bad]


def changed(at, bad):
    t = TABLE.copy()
    t[at] = bad
    return t


@pytest.mark.parametrize("new", [[41, 33, 16], [10, 33, 0], [40, 64, 17], [0, 0, 0]])
def test_resize_reports_nothing_in_a_good_table(new):
    assert not resize(TABLE, np.array(new, np.int32))[3]


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("at", [(0, 0), (0, 1), (0, 2)])       # whole pages, and the partly filled last one
def test_resize_reports_and_keeps_a_kept_page(at, bad):
    ref, table, short, seen = resize(changed(at, bad), LENS + 1)
    want = changed(at, bad)
    want[2, 1] = 7                                             # (16 -> 17: the one new page)
    assert seen and short[0] == 0 and np.array_equal(table, want)
    counts = REF.copy()
    counts[7] = 1
    assert np.array_equal(ref, counts)


@pytest.mark.parametrize("bad", BAD)
def test_resize_reports_a_page_that_is_given_back(bad):
    ref, table, short, seen = resize(changed((0, 1), bad), np.array([10, 33, 16], np.int32))
    counts = REF.copy()
    counts[2] = 0                                              # page 1 is nobody's: its count stays
    assert seen and short[0] == 0 and np.array_equal(ref, counts) and table[0].tolist() == [0, -1, -1, -1]


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("at,new", [((0, 0), [41, 33, 17]), ((0, 2), [41, 33, 17]), ((1, 2), [40, 32, 64])])
def test_a_short_resize_reports_too_and_changes_nothing(at, new, bad):
    full = np.where(REF == 0, 1, REF).astype(np.int32)         # no free page
    t = changed(at, bad)
    ref, table, short, seen = resize(t, np.array(new, np.int32), full)
    assert seen and short[0] > 0 and np.array_equal(ref, full) and np.array_equal(table, t)


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("deep", [False, True])
@pytest.mark.parametrize("at", [(0, 0), (0, 2)])
@pytest.mark.parametrize("full", [False, True])
def test_fork_reports_whether_short_or_not(full, at, deep, bad):
    counts = np.where(REF == 0, 1, REF).astype(np.int32) if full else REF
    kp, vp = pools()
    k0 = kp.clone()
    ref, child, lens, short = ne.pages_fork(i32(counts), i32(changed(at, bad)), i32(LENS), i32([0, -1]), kp, vp, deep=deep)
    assert reported() and (int(short) > 0) == full
    assert torch.equal(kp[:, counts > 0], k0[:, counts > 0])
    if full:
        assert bool((child == -1).all()) and not bool(lens.any()) and np.array_equal(ref.cpu().numpy(), counts)
    else:
        e = at[1]
        fresh = deep or e == 2                                 # a copy of nothing, or a page that is not there
        assert lens.tolist() == [40, 0] and (int(child[0, e]) >= 7 if fresh else int(child[0, e]) == -1)


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("at", [(0, 0), (0, 2), (2, 3)])
def test_compact_reports_every_entry_but_minus_one(at, bad):
    kp, vp = pools()
    rc = np.zeros(P, np.int32)
    rc[[0, 1, 2, 9, 4, 5, 6]] = 1                              # page 3 became 9
    t = TABLE.copy()
    t[1, 0] = 9
    got = ne.pages_compact(i32(rc), i32(t), kp, vp)
    assert not reported() and got[1].cpu().numpy().tolist() == TABLE.tolist()
    t[at] = bad
    kp, vp = pools()
    ref, table, remap, n_live = ne.pages_compact(i32(rc), i32(t), kp, vp)
    want = TABLE.copy()
    want[at] = -1
    assert reported() and int(n_live) == 7 and np.array_equal(table.cpu().numpy(), want)
