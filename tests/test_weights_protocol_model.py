"""A model of the barrier protocol of the accumulated-weights kernel for many rows (weights_many_kernel of
csrc/paged_weights.cu), run on the CPU over random lists of parts.

Roles: the part finder, which also loads the log-sum-exps (a ring of their own; part k + 1 is queued before
those of part k), the TMA producer (keys of a part, then query tiles through a ring), a UMMA issuer per key
tile, which waits for a query tile's log-sum-exps before it commits its products, and four groups of
exponential warps: key tile u, query tiles of one parity.  Each role is a coroutine of its waits and arrivals (a
group arrives as one; products and copies complete at once).  A run fails on a deadlock, on parity aliasing, or on
an arrival that lands in another phase.  Kept in step with the kernel by hand.
"""
import random

import pytest

PARTS = 4


class ProtocolError(Exception):
    pass


class Bar:
    def __init__(self, name, count):
        self.name, self.count, self.arr, self.phase = name, count, 0, 0

    def arrive(self, phase):
        if phase != self.phase:
            raise ProtocolError(f"early arrival: {self.name} for phase {phase} in phase {self.phase}")
        self.arr += 1
        if self.arr > self.count:
            raise ProtocolError(f"too many arrivals: {self.name}")
        if self.arr == self.count:
            self.arr = 0
            self.phase += 1


def simulate(parts, NK, NS, NL, rng, follow_absent_keys=True):
    """parts: (key tiles 1 or 2, query tiles) of the CTA in order.  follow_absent_keys: the warps of a key tile
    that a part lacks still count its query tiles."""
    bars = {}

    def bar(name, count=1):
        return bars.setdefault(name, Bar(name, count))

    k_full, k_empty = [bar(f"k_full{i}") for i in range(NK)], [bar(f"k_empty{i}") for i in range(NK)]
    q_full, q_empty = [bar(f"q_full{i}") for i in range(NS)], [bar(f"q_empty{i}", 2) for i in range(NS)]
    l_full, l_empty = [bar(f"l_full{i}") for i in range(NL)], [bar(f"l_empty{i}", 2) for i in range(NL)]
    s_full, s_free = [bar(f"s_full{i}") for i in range(4)], [bar(f"s_free{i}") for i in range(4)]
    # Seven read the parts: the producer, the issuers and the exponentials.
    part_full, part_empty = [bar(f"part_full{i}") for i in range(PARTS)], [bar(f"part_empty{i}", 7) for i in range(PARTS)]
    sum_full, sum_free = [bar(f"sum_full{i}", 2) for i in range(2)], [bar(f"sum_free{i}", 2) for i in range(2)]
    done = []

    def finder():
        def queue(k):                                       # (the last: the end)
            if k >= PARTS:
                yield part_empty[k % PARTS], k // PARTS - 1, f"finder: part {k}"
            part_full[k % PARTS].arrive(k // PARTS)

        yield from queue(0)
        item = 0
        for k, (_, n) in enumerate(parts):
            yield from queue(k + 1)
            for _ in range(n):
                if item >= NL:
                    yield l_empty[item % NL], item // NL - 1, f"finder: lse {item}"
                l_full[item % NL].arrive(item // NL)
                item += 1

    def each_part(name):
        for k in range(len(parts) + 1):
            yield part_full[k % PARTS], k // PARTS, f"{name}: part {k}"
            part_empty[k % PARTS].arrive(k // PARTS)
            if k < len(parts):
                yield None, k, parts[k]

    def role(name, body):
        """body(k, nu, n): a generator of waits for part k."""
        for x in each_part(name):
            if x[0] is not None:
                yield x
            else:
                yield from body(x[1], *x[2])

    class State:
        pass

    p = State()
    p.keys = p.item = 0

    def producer(k, nu, n):
        if n == 0:
            return
        for _ in range(nu):
            if p.keys >= NK:
                yield k_empty[p.keys % NK], p.keys // NK - 1, f"producer: key tile {p.keys}"
            k_full[p.keys % NK].arrive(p.keys // NK)
            p.keys += 1
        for _ in range(n):
            if p.item >= NS:
                yield q_empty[p.item % NS], p.item // NS - 1, f"producer: query tile {p.item}"
            q_full[p.item % NS].arrive(p.item // NS)
            p.item += 1

    def issuer(u):
        st = State()
        st.keys = st.item = 0
        st.uses = [0, 0]

        def body(k, nu, n):
            if n == 0:
                return
            ks = st.keys + u
            if u < nu:
                yield k_full[ks % NK], ks // NK, f"issuer {u}: keys {ks}"
            for t in range(n):
                it, odd = st.item, st.item & 1
                yield q_full[it % NS], it // NS, f"issuer {u}: query tile {it}"
                if u < nu:
                    s = 2 * u + odd
                    if st.uses[odd] >= 1:
                        yield s_free[s], st.uses[odd] - 1, f"issuer {u}: S {s}"
                    yield l_full[it % NL], it // NL, f"issuer {u}: lse {it}"
                    s_full[s].arrive(st.uses[odd])
                    st.uses[odd] += 1
                    if t + 1 == n:
                        k_empty[ks % NK].arrive(ks // NK)
                q_empty[it % NS].arrive(it // NS)
                st.item += 1
            st.keys += nu
        return body

    def exps(u, half):
        st = State()
        st.item = st.uses = 0

        def body(k, nu, n):
            for j in range((st.item ^ half) & 1, n, 2):
                it = st.item + j
                if u >= nu and follow_absent_keys:
                    yield l_full[it % NL], it // NL, f"exps {u}{half}: lse {it}"
                if u < nu:
                    yield s_full[2 * u + half], st.uses, f"exps {u}{half}: S of {it}"
                    s_free[2 * u + half].arrive(st.uses)
                    st.uses += 1
                    done.append((k, u, j))
                if u < nu or follow_absent_keys:
                    l_empty[it % NL].arrive(it // NL)
            st.item += n
            if half == 1:
                if k >= 2:
                    yield sum_free[k & 1], k // 2 - 1, f"exps {u}1: sums of part {k}"
                sum_full[k & 1].arrive(k // 2)
            else:
                yield sum_full[k & 1], k // 2, f"exps {u}0: sums of part {k}"
                sum_free[k & 1].arrive(k // 2)
        return body

    roles = {"finder": finder(), "producer": role("producer", producer)}
    for u in range(2):
        roles[f"issuer{u}"] = role(f"issuer{u}", issuer(u))
        for half in range(2):
            roles[f"exps{u}{half}"] = role(f"exps{u}{half}", exps(u, half))
    slow = {name: rng.choice([1, 1, 1, 20]) for name in roles}   # some roles lag behind
    pending = {}
    for name in list(roles):
        try:
            pending[name] = next(roles[name])
        except StopIteration:
            del roles[name]
    while roles:
        names = sorted(roles, key=lambda name: rng.random() * slow[name])
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
    assert sorted(done) == sorted((k, u, j) for k, (nu, n) in enumerate(parts) for u in range(nu) for j in range(n))


def test_the_model_finds_queries_that_run_ahead_of_their_log_sum_exps():
    """The ring of queries is no longer than that of the log-sum-exps: an issuer without keys does not look at them."""
    with pytest.raises(ProtocolError):
        for seed in range(300):
            rng = random.Random(seed)
            simulate([(rng.choice([1, 2]), rng.choice([1, 2, 5, 17])) for _ in range(9)], 4, 12, 2, rng)


@pytest.mark.parametrize("NK,NS", [(4, 8), (3, 3)])
def test_weights_protocol(NK, NS):
    for seed in range(300):
        rng = random.Random(seed)
        parts = [(rng.choice([1, 2, 2]), rng.choice([0, 1, 1, 2, 3, 5, 8, 17, 30])) for _ in range(rng.randint(0, 9))]
        simulate(parts, NK, NS, 8, rng)


def test_the_model_finds_warps_that_do_not_follow():
    """Were the warps of an absent key tile to skip its query tiles, their places in the ring would never be free."""
    with pytest.raises(ProtocolError):
        simulate([(1, 30), (2, 3)], 4, 8, 8, random.Random(0), follow_absent_keys=False)
