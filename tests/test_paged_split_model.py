"""A model of how a CTA of the paged attention finds its place in the line of work units and
walks on from there (paged_locate, PagedWalk::init and ::next of csrc/paged_sched.cuh), and of
calls whose units are not cut (contexts of at most 256 positions, after which no join runs).

Costs are integers as in the kernels; the head group is found by an fp32 quotient that may be
off by two units in the last place and is corrected by one step, the tile by bisection over
the sum of the costs in front of it.  The line itself, unit by unit, is built beside it without
any of that.  Kept in step with the kernels by hand.
"""
import random

import numpy as np
import pytest


class Shape:
    """PagedSplit: what a kernel makes of Hkv kv heads with G query heads each."""

    def __init__(self, kind, Hkv, G, D=64, cap=1 << 30):
        rows, bn, C, snap, shift = {"few16": (16, 64 if D == 128 else 128, 304, 3, 9), "few32": (32, 64 if D == 128 else 128, 304, 3, 9),
                                    "f32_few": (8, 256, 152, 0, 0), "f32_many": (64, 32, 304, 0, 0),
                                    "tiles": (256, 128, 152, 1, 0)}[kind]
        self.ovh, self.w_full, self.w_part, self.min_shift, self.sub = 384, 1, 1, 7, 0
        self.gs = min(G, rows)
        self.tpt = rows // self.gs
        self.hg = Hkv * -(-G // self.gs)
        if kind == "tiles":
            self.sub = 128 // G
            self.gs, self.tpt, self.hg = G, 2 * self.sub, Hkv
            self.ovh, self.w_full, self.w_part, self.min_shift = 1024, 5, 4, 11
        self.bn, self.C, self.snap, self.snap_shift = bn, C, snap, shift
        self.inv_C = (2 ** 64 - 1) // C
        self.nocut = cap <= 256

    def weight(self, ntok):
        return self.w_full if ntok > self.sub else self.w_part

    def tiles(self, n):
        return -(-n // self.tpt)

    def prefix(self, r, base):
        """Cost of tiles 0 .. r-1, all of them full."""
        if r == 0:
            return 0
        r0 = min(r, -base // self.tpt) if base < 0 else 0  # tiles without a key
        return r * self.ovh + self.w_full * ((r - r0) * base + self.tpt * ((r * (r + 1) - r0 * (r0 + 1)) // 2))

    def group_cost(self, n, L):
        if n == 0:
            return 0
        last = self.tiles(n) - 1
        return self.prefix(last, L - n) + self.ovh + self.weight(n - last * self.tpt) * L

    def interval(self, total, c):
        if total < self.C << self.min_shift:
            return min(c << self.min_shift, total), min((c + 1) << self.min_shift, total)
        at = lambda x: total * (self.inv_C * x) >> 64  # noqa: E731
        return at(c), total if c + 1 == self.C else at(c + 1)

    def least(self, total):
        return min(self.snap, (total * self.inv_C >> 64) >> self.snap_shift)


def line(s, n, lens):
    """Every unit: (sequence, head group, tile, keys, tokens, start, cost)."""
    out, at = [], 0
    for b, (nb, L) in enumerate(zip(n, lens)):
        for hg in range(s.hg):
            for r in range(s.tiles(nb)):
                end = min((r + 1) * s.tpt, nb)
                ntok = end - r * s.tpt
                kv = max(0, L - nb + end)
                cost = s.ovh + s.weight(ntok) * kv
                out.append((b, hg, r, kv, ntok, at, cost))
                at += cost
    return out, at


def start(s, n, lens, w0, ulps):
    """Sequence, head group, tile and start of the unit that w0 falls into."""
    at = 0
    for b, (nb, L) in enumerate(zip(n, lens)):             # paged_locate
        mine = s.group_cost(nb, L) * s.hg
        if mine > 0 and at <= w0 < at + mine:
            break
        at += mine
    else:
        raise AssertionError("no sequence holds the start")
    S, off, base = s.group_cost(nb, L), w0 - at, L - nb
    q = np.float32(off) / np.float32(S)
    for _ in range(abs(ulps)):
        q = np.nextafter(q, np.float32(np.inf if ulps > 0 else 0))
    hg = min(s.hg - 1, int(q))
    x = off - hg * S
    if x < 0:
        hg, x = hg - 1, x + S
    elif x >= S:
        hg, x = hg + 1, x - S
    lo, hi = 0, s.tiles(nb) - 1
    while lo < hi:
        mid = (lo + hi + 1) >> 1
        if s.prefix(mid, base) <= x:
            lo = mid
        else:
            hi = mid - 1
    return b, hg, lo, at + hg * S + s.prefix(lo, base)


def walk(s, n, lens, total, c, ulps=0):
    """The parts of CTA c: (sequence, head group, tile, t0, t1, key tiles)."""
    w0, w1 = s.interval(total, c)
    if w0 >= w1:
        return
    b, hg, r, cur = start(s, n, lens, w0, ulps)
    snap = s.least(total)
    while cur < w1:
        nb, L, nt = n[b], lens[b], s.tiles(n[b])
        base = L - nb
        kv = L if r == nt - 1 else max(0, base + (r + 1) * s.tpt)
        cost = s.ovh + s.weight(min(s.tpt, nb - r * s.tpt)) * kv
        ntk = -(-kv // s.bn)
        per = np.float32(ntk) / np.float32(cost)

        def cut(x):
            if s.nocut:
                return ntk if 2 * x >= cost else 0
            k = min(ntk, int(np.rint(np.float32(x) * per)))
            return 0 if k <= snap else ntk if ntk - k <= snap else k
        t0 = 0 if w0 <= cur else cut(w0 - cur)
        t1 = ntk if w1 >= cur + cost else cut(w1 - cur)
        if t0 < t1 or (ntk == 0 and w0 <= cur):
            yield b, hg, r, t0, t1, ntk
        cur += cost
        r += 1
        if r == nt:
            r, hg = 0, hg + 1
            if hg == s.hg:
                hg, b = 0, b + 1
                while b < len(n) and n[b] == 0:
                    b += 1
                if b >= len(n):
                    cur = max(cur, w1)


def draw(rng, cap):
    """New tokens and lengths: idle, single, chunks, more new tokens than positions."""
    B = rng.choice([1, 2, rng.randint(3, 12), rng.randint(30, 80)])
    lens = [rng.choice([0, 1, rng.randint(1, min(cap, 200)), rng.randint(1, min(cap, 9000))]) for _ in range(B)]
    n = [rng.choice([0, 1, 1, rng.randint(1, 70), L, L + rng.randint(0, 40)]) if L < 1000 else rng.choice([1, rng.randint(1, 300)]) for L in lens]
    n[rng.randrange(B)] = rng.randint(1, 90)
    return n, lens


KINDS = ["few16", "few32", "f32_few", "f32_many", "tiles"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seed", range(12))
def test_every_cta_begins_in_the_unit_that_holds_its_start(kind, seed):
    rng = random.Random(seed)
    G = rng.choice([1, 2, 3, 5, 8, 20, 71])
    s = Shape(kind, rng.choice([1, 2, 4]), G)
    n, lens = draw(rng, 9000)
    units, total = line(s, n, lens)
    assert total == sum(s.group_cost(a, b) * s.hg for a, b in zip(n, lens))
    starts = [u[5] for u in units]
    for c in range(s.C):
        w0, w1 = s.interval(total, c)
        if w0 < w1:
            u = units[int(np.searchsorted(np.array(starts, dtype=np.int64), w0, side="right")) - 1]
            for ulps in (-2, 0, 2):
                assert start(s, n, lens, w0, ulps) == (u[0], u[1], u[2], u[5])


@pytest.mark.parametrize("G,Hkv,n,L", [(32768, 32, 1, 40), (32768, 32, 2, 1), (1 << 20, 1, 1, 100), (1, 1024, 3, 5000), (4096, 4, 9, 4)])
def test_the_quotient_finds_one_of_many_head_groups(G, Hkv, n, L):
    """Up to 65536 head groups of a sequence, as many as 2^20 heads make."""
    rng = random.Random(G + n)
    for kind in ("few16", "f32_many"):
        s = Shape(kind, Hkv, G)
        S = s.group_cost(n, L)
        for hg in [0, 1, s.hg - 1] + [rng.randrange(s.hg) for _ in range(300)]:
            for off in (0, S - 1, rng.randrange(S)):
                for ulps in (-2, 0, 2):
                    assert start(s, [n], [L], hg * S + off, ulps)[:2] == (0, hg)


def check(s, n, lens):
    units, total = line(s, n, lens)
    seen, records = {}, {}
    for c in range(s.C):
        for b, hg, r, t0, t1, nt in walk(s, n, lens, total, c):
            seen.setdefault((b, hg, r), []).append((t0, t1))
            if (t0, t1) != (0, nt):
                slot = 2 * c + (t0 == 0)
                assert slot not in records                 # one part of each kind per CTA
                records[slot] = (b, hg, r)
    for b, hg, r, kv, *_ in units:
        parts = sorted(seen.pop((b, hg, r)))
        assert parts[0][0] == 0 and parts[-1][1] == -(-kv // s.bn)
        assert all(x[1] == y[0] for x, y in zip(parts, parts[1:]))
    assert not seen
    return records


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("seed", range(12))
def test_walks_cover_every_key_tile_once(kind, seed):
    rng = random.Random(100 + seed)
    check(Shape(kind, rng.choice([1, 2, 4]), rng.choice([1, 2, 3, 5, 8, 20, 71])), *draw(rng, 9000))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cap", [8, 64, 256])
@pytest.mark.parametrize("seed", range(8))
def test_units_of_short_contexts_stay_whole(kind, cap, seed):
    """No join runs behind them: every unit is one part, of one CTA, and no record is left."""
    rng = random.Random(200 + seed)
    s = Shape(kind, rng.choice([1, 2, 4]), rng.choice([1, 2, 3, 5, 8, 20, 71]), cap=cap)
    n, lens = draw(rng, cap)
    if seed == 0:                                          # many sequences, so that the shares are large
        lens = [rng.randint(0, cap) for _ in range(3000)]
        n = [rng.choice([0, 1, 5]) for _ in lens]
    assert s.nocut and max(lens) <= cap
    assert check(s, n, lens) == {}


def test_a_middle_that_two_shares_meet_in_shows_the_rule():
    """Seventy units of 512 in shares of 128: a share ends in the middle of every unit.  The rule
    at both ends of a share (a planted > at one of them) gives the unit to one CTA (to two)."""
    s = Shape("few16", 1, 1, cap=256)
    n, lens = [1] * 70, [128] * 70
    units, total = line(s, n, lens)
    assert units[0][6] == 512 and s.interval(total, 2) == (256, 384)
    assert check(s, n, lens) == {}
    taken = [0] * len(n)
    for c in range(s.C):
        w0, w1 = s.interval(total, c)
        for b, *_, at, cost in units:
            if w0 < w1 and at < w1 and w0 < at + cost:
                before = w0 > at and 2 * (w0 - at) > cost
                taken[b] += (w1 >= at + cost or 2 * (w1 - at) >= cost) and not before
    assert set(taken) == {2}
