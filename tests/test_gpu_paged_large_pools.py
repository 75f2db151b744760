"""Pools and batches beyond one pass of the page plan's loops.

A CTA of its cluster of eight lists 16 pages per thread and pass (a second pass from 131073
pages on), moves 4 (from 32769) and places one sequence (from 8193): three passes each here,
with free pages in all of them.  Ids, counts, tables and page contents bit for bit.
"""
import numpy as np
import pytest
import torch

import causal_gqa_flash_attention_gb300 as ne
from causal_gqa_flash_attention_gb300 import _build

import paged_ref as ref

pytestmark = pytest.mark.gpu

PS, W, B, P = 8, 4, 20003, 300007
SHARE = (-(-P // 8) + 3) // 4 * 4                          # a CTA's pages


def every_pass(pages):
    """Some of the pages fall into each pass of some CTA's list of free ones."""
    return set(np.unique(np.asarray(pages) % SHARE // (16 * 1024))) == {0, 1, 2}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    ne.load()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def pools(n_pages):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    return [torch.empty((1, n_pages, PS, 1, 32), dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in "kv"]


def tables(rng, n_pages, sequences):
    """Random lengths and pages, every third sequence on the whole pages of the one before."""
    lens = rng.integers(0, W * PS + 1, sequences).astype(np.int32)
    t, at, perm = np.full((sequences, W), -1, np.int32), 0, rng.permutation(n_pages)
    for b in range(sequences):
        k = -(-int(lens[b]) // PS)
        s = min(int(lens[b]) // PS, int(lens[b - 1]) // PS) if b % 3 == 2 else 0
        t[b, :s] = t[b - 1, :s]
        t[b, s:k] = perm[at:at + k - s]
        at += k - s
    return lens, t, np.bincount(t[t >= 0], minlength=n_pages).astype(np.int32)


def leave_free(rng, counts, free, n):
    """Counts with all but n pages of `free` held by somebody else."""
    counts = counts.copy()
    counts[rng.permutation(free)[n:]] = 1
    return counts


def check(got, want, kp, vp, k0, v0, copies):
    torch.cuda.synchronize()
    assert ne.get_device_error() == ne.NE_OK
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy().reshape(np.shape(w)), w)
    copies = np.array(copies, np.int64).reshape(-1, 3)
    for slots in np.unique(copies[:, 2]):
        src, dst = (torch.from_numpy(copies[copies[:, 2] == slots, i]).cuda() for i in (0, 1))
        for x in (k0, v0):
            x[:, dst, :slots] = x[:, src, :slots]
    assert torch.equal(kp, k0) and torch.equal(vp, v0)


@pytest.mark.parametrize("deep", [False, True])
@pytest.mark.parametrize("spare", [0, 5, -1])
def test_fork(deep, spare):
    rng = np.random.default_rng(1)
    lens, t, counts = tables(rng, P, B)
    parents = rng.integers(-1, B, B).astype(np.int32)
    ln = np.where(parents >= 0, lens[np.maximum(parents, 0)], 0)
    need = int((-(-ln // PS)).sum() if deep else (ln % PS > 0).sum())
    counts = leave_free(rng, counts, np.flatnonzero(counts == 0), need + spare)
    kp, vp = pools(P)
    k0, v0 = kp.clone(), vp.clone()
    got = ne.pages_fork(i32(counts), i32(t), i32(lens), i32(parents), kp, vp, deep=deep)
    if spare < 0:
        check(got, (counts, np.full((B, W), -1), np.zeros(B), 1), kp, vp, k0, v0, [])
        return
    r, ct, cl, copies = ref.fork(counts, t, lens, parents, PS, deep)
    assert every_pass([c[1] for c in copies])
    check(got, (r, ct, cl, 0), kp, vp, k0, v0, copies)


@pytest.mark.parametrize("spare", [0, 5, -1])
def test_resize(spare):
    rng = np.random.default_rng(2)
    lens, t, counts = tables(rng, P, B)
    new = rng.integers(0, W * PS + 1, B).astype(np.int32)
    out = ref.resize(counts, t, lens, new, PS)[1]
    taken = int(((out != t) & (out >= 0)).sum())
    po, pn = -(-lens // PS), -(-new // PS)
    e = np.arange(W)
    dropped = t[(e >= pn[:, None]) & (e < po[:, None])]
    back = counts - np.bincount(dropped, minlength=P).astype(np.int32)
    free = np.flatnonzero(counts == 0)
    returned = int((back == 0).sum()) - len(free)          # free once the cut sequences gave theirs back
    counts = leave_free(rng, counts, free, taken + spare - returned)
    kp, vp = pools(P)
    k0, v0 = kp.clone(), vp.clone()
    got = ne.pages_resize(i32(counts), i32(t), i32(lens), i32(new), kp, vp)
    if spare < 0:
        check(got, (counts, t, 1), kp, vp, k0, v0, [])
        return
    r, out, copies = ref.resize(counts, t, lens, new, PS)
    assert len(copies) > 100 and every_pass(out[(out != t) & (out >= 0)])
    check(got, (r, out, 0), kp, vp, k0, v0, copies)


@pytest.mark.parametrize("n_pages", [70001, 300007])
def test_compact(n_pages):
    rng = np.random.default_rng(3)
    _, t, counts = tables(rng, n_pages, B)
    free = np.flatnonzero(counts == 0)
    counts = leave_free(rng, counts, free, len(free) // 2)
    kp, vp = pools(n_pages)
    k0, v0 = kp.clone(), vp.clone()
    got = ne.pages_compact(i32(counts), i32(t), kp, vp)
    r, out, remap, n_live, copies = ref.compact(counts, t, PS)
    assert len(copies) > 3000
    check(got, (r, out, remap, n_live), kp, vp, k0, v0, copies)
