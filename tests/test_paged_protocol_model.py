"""A model of the barrier protocol of the paged attention's tile kernel
(csrc/paged_tiles.cu), run on the CPU over many sequences of parts.

Roles: the warp that finds the CTA's parts and queues them (four places), the TMA producer
(one Q pair, a ring of K and V tiles), the UMMA issuers, and the eight softmax warps, four to
a subtile, some of them without live rows.  At head_dim 64 P has columns of its own and each
subtile its issuer; the second also zeroes V rows behind a sequence's length for both, and in
a part with one subtile does nothing else.  At head_dim 128 P lies over S, one issuer serves
both subtiles, and a warp of its own zeroes V (and releases every slot along with the
issuer).  Each role is a coroutine of waits and arrivals; MMAs and copies complete at once, in
the order of their issue, but for Q's.  A run fails on a deadlock, on parity aliasing, on an
arrival that lands in another phase, and on data that is overwritten before it is read (S, P,
O, Q, ring slots).  Kept in step with the kernel by hand.
"""
import random

import pytest

QUEUE = 4


class ProtocolError(Exception):
    pass


class Bar:
    def __init__(self, name, count):
        self.name, self.count, self.arr, self.phase = name, count, 0, 0

    def arrive(self, phase):
        if phase != self.phase:
            raise ProtocolError(f"arrival for phase {phase} of {self.name} in phase {self.phase}")
        self.arr += 1
        if self.arr == self.count:
            self.arr = 0
            self.phase += 1


class Cell:
    """A buffer: written for a tag, read under it."""

    def __init__(self, name):
        self.name, self.tag = name, None

    def read(self, tag):
        if self.tag != tag:
            raise ProtocolError(f"{self.name} holds {self.tag}, {tag} was expected")


def simulate(parts, sep, NS, rng, both_release=True, dead_waits=True, two_fix_bars=True, both_see_q=True):
    """parts: (tiles, subtiles, fix, live warps of subtile 0, of subtile 1); tiles 0: no keys."""
    bars = {}

    def bar(name, count=1):
        return bars.setdefault(name, Bar(name, count))

    ring = [Cell(f"slot {s}") for s in range(NS)]
    Q, S, P, O = Cell("Q"), [Cell("S0"), Cell("S1")], [Cell("P0"), Cell("P1")], [Cell("O0"), Cell("O1")]
    q_full, q_empty, q_issued = bar("q_full"), bar("q_empty", 2 if sep else 1), bar("q_issued")
    full = [bar(f"full{s}") for s in range(NS)]
    empty = [bar(f"empty{s}", 2 if both_release else 1) for s in range(NS)]
    seg_full, seg_empty = [bar(f"seg_full{s}") for s in range(QUEUE)], [bar(f"seg_empty{s}", 11) for s in range(QUEUE)]
    s_full, o_full = [bar(f"s_full{u}") for u in range(2)], [bar(f"o_full{u}") for u in range(2)]
    p_ready, s_free = [bar(f"p_ready{u}", 4) for u in range(2)], [bar(f"s_free{u}", 4) for u in range(2)]
    vfix = [bar(f"vfix{k}") for k in range(2)]
    p_parts = [{}, {}]                                     # (tag: warps that wrote P)
    s_reads = [{}, {}]

    def finder():
        for k in range(len(parts) + 1):
            if k >= QUEUE:
                yield seg_empty[k % QUEUE], k // QUEUE - 1, f"finder: place for part {k}"
            seg_full[k % QUEUE].arrive(k // QUEUE)

    def queue():
        """The parts as a reader sees them, up to and without the end mark."""
        for k in range(len(parts) + 1):
            yield seg_full[k % QUEUE], k // QUEUE, f"reader: part {k}"
            seg_empty[k % QUEUE].arrive(k // QUEUE)
            yield None, k, None

    def walk(body):
        """Runs body(part, its index) for every part, after fetching it from the queue."""
        gen = queue()
        for b, n, what in gen:
            if b is not None:
                yield b, n, what
            elif n < len(parts):
                yield from body(parts[n], n)

    def producer():
        st = {"seg": 0, "item": 0}

        def body(part, k):
            nt = part[0]
            if nt == 0:
                return
            if st["seg"] > 0:
                yield q_empty, st["seg"] - 1, "producer: Q free"
            q_issued.arrive(st["seg"])
            st["seg"] += 1
            for t in range(nt):
                for kv in "KV":
                    i = st["item"]
                    if i >= NS:
                        yield empty[i % NS], i // NS - 1, f"producer: slot for item {i}"
                    ring[i % NS].tag = (k, t, kv, "raw")
                    full[i % NS].arrive(i // NS)
                    st["item"] += 1
        return walk(body)

    def q_copy():
        """The Q copies take their time: the K and V tiles behind them may land first."""
        for n, k in enumerate(k for k, part in enumerate(parts) if part[0]):
            yield q_issued, n, "copy of Q"
            Q.tag = k
            q_full.arrive(n)

    def issuer(u):
        st = {"seg": 0, "item": 0, "fix": 0, "p": 0, "s": 0}

        def release(i):
            if both_release or u == 0:
                empty[i % NS].arrive(i // NS)

        def v_tile(k, t, i, fix):
            yield full[i % NS], i // NS, f"issuer {u}: V"
            if not fix:
                return
            f = st["fix"]
            st["fix"] += 1
            b, n = (vfix[f & 1], f >> 1) if two_fix_bars else (vfix[0], f)
            if u == 0:
                yield b, n, "issuer 0: V zeroed"
            else:
                ring[i % NS].read((k, t, "V", "raw"))
                ring[i % NS].tag = (k, t, "V", "zeroed")
                b.arrive(n)

        def s_mma(k, t, i, nt):
            if st["s"]:
                yield s_free[u], st["s"] - 1, f"issuer {u}: S free"
            Q.read(k)
            ring[i % NS].read((k, t, "K", "raw"))
            if st["s"] and (s_reads[u].get(st["s"] - 1, 0) != 4):
                raise ProtocolError(f"S{u} overwritten before it was read")
            S[u].tag = (k, t)
            s_full[u].arrive(st["s"])
            st["s"] += 1
            release(i)
            if t + 1 == nt:
                q_empty.arrive(st["seg"])

        def body(part, k):
            nt, n_sub, fix = part[:3]
            if nt == 0:
                return
            item = st["item"]
            if both_see_q or u < n_sub:
                yield q_full, st["seg"], f"issuer {u}: Q"
            if u >= n_sub:
                for i in range(item, item + 2 * nt):
                    t = (i - item) // 2
                    if (i - item) % 2:
                        yield from v_tile(k, t, i, fix and t == nt - 1)
                    else:
                        yield full[i % NS], i // NS, f"issuer {u}: K"
                    release(i)
                    if i == item:
                        q_empty.arrive(st["seg"])
            else:
                yield full[item % NS], item // NS, f"issuer {u}: first K"
                yield from s_mma(k, 0, item, nt)
                for t in range(nt):
                    vi, kn, more = item + 2 * t + 1, item + 2 * t + 2, t + 1 < nt
                    if more:
                        yield full[kn % NS], kn // NS, f"issuer {u}: K"
                        yield from s_mma(k, t + 1, kn, nt)
                    yield from v_tile(k, t, vi, fix and t == nt - 1)
                    yield p_ready[u], st["p"], f"issuer {u}: P"
                    st["p"] += 1
                    ring[vi % NS].read((k, t, "V", "zeroed" if fix and t == nt - 1 else "raw"))
                    if p_parts[u].get((k, t), 0) != part[3 + u]:
                        raise ProtocolError(f"PV{u} of {(k, t)} without all of P")
                    P[u].tag = None
                    O[u].tag = (k, t)
                    o_full[u].arrive(st["p"] - 1)
                    release(vi)
            st["item"] += 2 * nt
            st["seg"] += 1
        return walk(body)

    def issuer_of_both():
        st = {"seg": 0, "item": 0, "fix": 0, "p": [0, 0], "s": [0, 0], "o": [0, 0]}

        def s_mma(u, k, t, i):
            Q.read(k)
            ring[i % NS].read((k, t, "K", "raw"))
            if st["s"][u] and (s_reads[u].get(st["s"][u] - 1, 0) != 4):
                raise ProtocolError(f"S{u} overwritten before it was read")
            S[u].tag = (k, t)
            s_full[u].arrive(st["s"][u])
            st["s"][u] += 1

        def body(part, k):                                 # (P over S: no S is waited for)
            nt, n_sub, fix = part[:3]
            if nt == 0:
                return
            item = st["item"]
            yield q_full, st["seg"], "issuer: Q"
            yield full[item % NS], item // NS, "issuer: first K"
            for u in range(n_sub):
                s_mma(u, k, 0, item)
            empty[item % NS].arrive(item // NS)
            if nt == 1:
                q_empty.arrive(st["seg"])
            for t in range(nt):
                vi, kn, more = item + 2 * t + 1, item + 2 * t + 2, t + 1 < nt

                def s_done():
                    empty[kn % NS].arrive(kn // NS)
                    if t + 2 == nt:
                        q_empty.arrive(st["seg"])
                yield full[vi % NS], vi // NS, "issuer: V"
                if fix and t == nt - 1:
                    f = st["fix"]
                    yield (vfix[f & 1], f >> 1, "issuer: V zeroed") if two_fix_bars else (vfix[0], f, "issuer: V zeroed")
                    st["fix"] += 1
                if more:
                    yield full[kn % NS], kn // NS, "issuer: K"
                for u in range(n_sub):
                    yield p_ready[u], st["p"][u], f"issuer: P{u}"
                    st["p"][u] += 1
                    ring[vi % NS].read((k, t, "V", "zeroed" if fix and t == nt - 1 else "raw"))
                    live = part[3 + u]
                    if p_parts[u].get((k, t), 0) != live:
                        raise ProtocolError(f"PV{u} of {(k, t)} without all of P")
                    P[u].tag = None
                    O[u].tag = (k, t)
                    if not more:
                        o_full[u].arrive(st["o"][u])
                        st["o"][u] += 1
                    if more:
                        s_mma(u, k, t + 1, kn)
                    if u == n_sub - 1:
                        empty[vi % NS].arrive(vi // NS)
                        if more:
                            s_done()
            st["item"] += 2 * nt
            st["seg"] += 1
        return walk(body)

    def fixer():
        st = {"item": 0, "fix": 0}

        def body(part, k):
            nt, _, fix = part[:3]
            for j in range(2 * nt):
                i = st["item"]
                yield full[i % NS], i // NS, f"zeroing: item {i}"
                if fix and j == 2 * nt - 1:
                    ring[i % NS].read((k, nt - 1, "V", "raw"))
                    ring[i % NS].tag = (k, nt - 1, "V", "zeroed")
                    f = st["fix"]
                    (vfix[f & 1].arrive(f >> 1) if two_fix_bars else vfix[0].arrive(f))
                    st["fix"] += 1
                if both_release:
                    empty[i % NS].arrive(i // NS)
                st["item"] += 1
        return walk(body)

    def softmax(u, wq):
        st = {"tiles": 0, "parts": 0}

        def body(part, k):
            nt, n_sub = part[:2]
            if u >= n_sub or nt == 0:
                return
            live = wq < part[3 + u]
            for t in range(nt):
                n = st["tiles"]
                yield s_full[u], n, f"softmax {u}.{wq}: S"
                if live:
                    S[u].read((k, t))
                s_reads[u][n] = s_reads[u].get(n, 0) + 1
                if sep:
                    s_free[u].arrive(n)
                    if n and (live or dead_waits):
                        yield o_full[u], n - 1, f"softmax {u}.{wq}: PV before"
                if live:
                    p_parts[u][(k, t)] = p_parts[u].get((k, t), 0) + 1
                p_ready[u].arrive(n)
                st["tiles"] += 1
            n = st["tiles"] - 1 if sep else st["parts"]
            yield o_full[u], n, f"softmax {u}.{wq}: last PV"
            st["parts"] += 1
            if live:
                O[u].read((k, nt - 1))
        return walk(body)

    roles = {"finder": finder(), "producer": producer(), "q": q_copy(), **({"issuer0": issuer(0), "issuer1": issuer(1)} if sep else {"issuer": issuer_of_both(), "fixer": fixer()})}
    for u in range(2):
        for wq in range(4):
            roles[f"softmax{u}{wq}"] = softmax(u, wq)
    pending = {}
    for name in list(roles):
        try:
            pending[name] = next(roles[name])
        except StopIteration:
            del roles[name]
    while roles:
        names = list(roles)
        rng.shuffle(names)
        for name in names:
            b, n, _ = pending[name]
            if b.phase not in (n, n + 1):
                raise ProtocolError(f"parity aliasing: {b.name} waited for phase {n} in phase {b.phase}")
            if b.phase == n + 1:
                try:
                    pending[name] = next(roles[name])
                except StopIteration:
                    del roles[name], pending[name]
                break
        else:
            raise ProtocolError("deadlock: " + "; ".join(pending[nm][2] for nm in roles))


def draw_parts(rng):
    out = []
    for _ in range(rng.randint(0, 7)):
        n_sub = rng.choice([1, 2])
        nt = rng.choice([0, 1, 1, 2, 3, 7])
        out.append((nt, n_sub, rng.random() < 0.5 and nt > 0, rng.randint(1, 4), rng.randint(1, 4) if n_sub == 2 else 0))
    return out


@pytest.mark.parametrize("sep,NS", [(False, 5), (True, 12)])
@pytest.mark.parametrize("seed", range(150))
def test_tile_kernel_protocol(sep, NS, seed):
    rng = random.Random(seed)
    simulate(draw_parts(rng), sep, NS, rng)


def finds(match, tries=400, **kw):
    """Some schedule of some parts shows the fault."""
    for seed in range(tries):
        rng = random.Random(seed)
        try:
            simulate(draw_parts(rng), kw.get("sep", True), kw.get("NS", 12), rng,
                     **{k: v for k, v in kw.items() if k not in ("sep", "NS")})
        except ProtocolError as e:
            if match in str(e):
                return True
    return False


def test_the_model_finds_a_zeroing_warp_that_falls_behind():
    assert finds("aliasing", sep=False, NS=5, both_release=False)


def test_the_model_finds_slots_that_one_issuer_releases_for_both():
    assert finds("slot", both_release=False) or finds("aliasing", both_release=False)


def test_the_model_finds_an_issuer_that_does_not_look_at_every_q():
    assert finds("aliasing", both_see_q=False)


def test_the_model_finds_warps_without_rows_that_run_ahead():
    assert finds("p_ready", dead_waits=False)


def test_the_model_finds_one_barrier_for_every_fix():
    assert finds("aliasing", two_fix_bars=False)
