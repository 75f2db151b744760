"""What orders the log-sum-exps that one warp of the accumulated-weights kernel for many rows stores in shared memory
before the loads of the exponential warps: a model of happens-before, run on the CPU, and the waits that the source has.

Every role carries the set of stores and loads that happen before its next step.  A wait on a barrier takes over what
its arrivals released: an ordinary arrival all that its thread knows, the arrival of a tcgen05 commit nothing of
it (it stands for the completion of its thread's asynchronous products alone).
"""
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "causal_gqa_flash_attention_gb300", "csrc",
                      "paged_weights.cu")


class Unordered(Exception):
    pass


class Bar:
    def __init__(self, count):
        self.count, self.arrived, self.phases = count, 0, []
        self.now = set()

    def arrive(self, knows):
        self.now |= knows
        self.arrived += 1
        if self.arrived == self.count:
            self.phases.append(self.now)
            self.arrived, self.now = 0, set()


def simulate(items, NL, rng, looks):
    """looks: the exponential warps wait for the log-sum-exps themselves."""
    l_full, l_empty, s_full, s_free = [Bar(1) for _ in range(NL)], [Bar(2) for _ in range(NL)], [Bar(1) for _ in range(4)], [Bar(1) for _ in range(4)]
    reads = {}                                              # item: loads of its place so far

    def finder(knows):
        for n in range(items):
            if n >= NL:
                yield l_empty[n % NL], n // NL - 1
                if not reads[n - NL] <= knows:
                    raise Unordered(f"store of {n} over loads of {n - NL}")
            knows.add(("store", n))
            l_full[n % NL].arrive(set(knows))

    def issuer(u, knows):
        for n in range(items):
            s, use = 2 * u + n % 2, n // 2
            if use:
                yield s_free[s], use - 1
            yield l_full[n % NL], n // NL
            s_full[s].arrive(set())                         # (by a commit)

    def exps(u, half, knows):
        for use, n in enumerate(range(half, items, 2)):
            yield s_full[2 * u + half], use
            if looks:
                yield l_full[n % NL], n // NL
            if ("store", n) not in knows:
                raise Unordered(f"load of {n}")
            knows.add(("load", n, u))
            reads.setdefault(n, set()).add(("load", n, u))
            s_free[2 * u + half].arrive(set(knows))
            l_empty[n % NL].arrive(set(knows))

    roles = []
    for f, args in [(finder, ())] + [(issuer, (u,)) for u in range(2)] + [(exps, (u, h)) for u in range(2) for h in range(2)]:
        knows = set()
        roles.append([f(*args, knows), knows, None])
    for r in roles:
        r[2] = next(r[0], None)
    while any(r[2] for r in roles):
        ready = [r for r in roles if r[2] and len(r[2][0].phases) > r[2][1]]
        assert ready, "deadlock"
        r = rng.choice(ready)
        r[1] |= r[2][0].phases[r[2][1]]
        r[2] = next(r[0], None)


@pytest.mark.parametrize("items", [1, 2, 8, 9, 40])
def test_the_waits_order_every_load(items):
    for seed in range(40):
        simulate(items, 8, random.Random(seed), True)


def test_a_commit_alone_orders_nothing():
    with pytest.raises(Unordered):
        simulate(1, 8, random.Random(0), False)


def test_the_kernel_waits_as_modelled():
    """In the exponential warps' loop over query tiles the wait for the log-sum-exps stands under no condition."""
    with open(SOURCE) as f:
        text = f.read()
    body = text[text.index("---- exponentials\n"):]
    loop = body[body.index("for (int j = skip; j < n; j += 2) {"):body.index("const float4* nl")]
    assert re.search(r"const bool there = mbar_test\(smem_u32\(&bar_l_full\[i\]\)", loop)
    assert re.search(r"if \(!__all_sync\(0xffffffffu, there\) &&\s*!\(ok = mbar_wait_warp\(smem_u32\(&bar_l_full\[i\]\)", loop)
    assert not re.search(r"mine[^;]*bar_l_full", loop)
