"""A model of how the accumulated-weights kernels for many rows cut their work (WeightWalk of
csrc/paged_weights.cu): every query tile of every unit in exactly one part, whatever the lengths; of the
parts that a CTA leaves to the join at most one begins inside a unit and one leaves a unit's end to others, and
the join's walk over the records finds all parts of a unit.  Kept in step with the kernels by hand.
"""
import random

import numpy as np
import pytest

C = 152


def prefix(n, L, k, ovh, shift):
    base, out = L - n, k * (ovh + n)
    k1 = 0 if base < 0 else (base >> shift) + 1
    return out if k <= k1 else out - ((((k * (k - 1) - k1 * (k1 - 1)) >> 1) << shift) - base * (k - k1))


def parts_of(n, lens, Hkv, G, rt, shift):
    gs = min(G, rt)
    ngrp, sub = -(-G // gs), rt // gs
    ovh = 2 * sub
    nk = [-(-L // (1 << shift)) for L in lens]
    cost = [prefix(nb, L, k, ovh, shift) for nb, L, k in zip(n, lens, nk)]
    total = sum(cost) * Hkv
    at = lambda c: total if c == C else total * (((1 << 64) - 1) // C + 1) * c >> 64  # noqa: E731
    out = []
    for c in range(C):
        w0, w1 = at(c), at(c + 1)
        mine = []
        if w0 < w1:
            start, b = 0, 0
            while not start <= w0 < start + cost[b] * Hkv:
                start += cost[b] * Hkv
                b += 1
            h, x = divmod(w0 - start, cost[b])
            kt = max(k for k in range(nk[b]) if prefix(n[b], lens[b], k, ovh, shift) <= x)
            cur = start + h * cost[b] + prefix(n[b], lens[b], kt, ovh, shift)
            while cur < w1:
                first = max(0, (kt << shift) - (lens[b] - n[b]))
                unit = ovh + n[b] - first
                tf, nt = first // sub * ngrp, -(-n[b] // sub) * ngrp
                tiles = nt - tf

                def cut(x):
                    return tf + min(tiles, int(np.rint(np.float32(np.float32(x) * np.float32(tiles)) / np.float32(unit))))

                t0, t1 = tf if w0 <= cur else cut(w0 - cur), nt if w1 >= cur + unit else cut(w1 - cur)
                if t0 < t1 or (tiles == 0 and w0 <= cur):
                    mine.append((b, h, kt, t0, t1, tf, nt))
                cur += unit
                kt += 1
                if kt == nk[b]:
                    kt, h = 0, h + 1
                    if h == Hkv:
                        h, b = 0, b + 1
                        while b < len(lens) and nk[b] == 0:
                            b += 1
                        if b == len(lens):
                            break
        out.append(mine)
    return out, (nk, sub, ngrp)


def batch(rng):
    B = rng.choice([1, 2, 3, 12, 60])
    lens = [rng.choice([0, 1, 127, 128, 129, 256, 257, rng.randint(1, 5000), rng.randint(1, 100)]) for _ in range(B)]
    n = [rng.choice([0, 1, L, rng.randint(0, max(1, L)), rng.randint(0, 2 * L + 3)]) for L in lens]
    return n, lens


@pytest.mark.parametrize("seed", range(60))
def test_every_tile_once_and_every_cut_joined(seed):
    rng = random.Random(seed)
    n, lens = batch(rng)
    Hkv, G = rng.choice([1, 2, 4, 5]), rng.choice([1, 3, 4, 7, 8, 130])
    rt, shift = rng.choice([(128, 8), (64, 7)])
    if sum(lens) == 0:
        return
    ctas, (nk, sub, ngrp) = parts_of(n, lens, Hkv, G, rt, shift)
    seen, info, where = {}, [[None, None] for _ in range(C)], {}
    for c, mine in enumerate(ctas):
        for b, h, kt, t0, t1, tf, nt in mine:
            seen.setdefault((b, h, kt), []).append((t0, t1, tf, nt))
            if not (t0 == tf and t1 == nt):
                slot = 1 if t0 == tf else 0
                assert info[c][slot] is None, "two parts for one slot"
                info[c][slot] = (2 if t1 == nt else 1, (b, h, kt))
                where.setdefault((b, h, kt), []).append((c, slot))
    units = {(b, h, k) for b in range(len(lens)) for h in range(Hkv) for k in range(nk[b])}
    assert set(seen) == units
    for (b, h, kt), ps in seen.items():
        tf, nt = ps[0][2:]
        assert ps[0][0] == tf and ps[-1][1] == nt and all(x[1] == y[0] for x, y in zip(ps, ps[1:]))
        # The tiles that a unit leaves out hold no token that sees its first key.
        assert all(lens[b] - n[b] + i < (kt << shift) for i in range(tf // ngrp * sub))
    for c in range(C):                                      # the join of CTA c's slot 1
        if info[c][1] is None:
            continue
        unit, found = info[c][1][1], [(c, 1)]
        for d in range(c + 1, C):
            if info[d][0] is not None:
                found.append((d, 0))
                if info[d][0][0] == 2:
                    break
        assert found == where[unit]
    assert sum(1 for c in range(C) if info[c][1]) == len(where)


def test_shares_are_alike():
    """No CTA's tiles exceed the mean by more than a unit's rounding."""
    ctas, _ = parts_of([2048], [16384], 4, 4, 128, 8)
    tiles = [sum(p[4] - p[3] for p in mine) for mine in ctas]
    assert max(tiles) <= np.mean(tiles) + 4
