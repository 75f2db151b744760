"""What orders the log-sum-exps that one warp of the accumulated-weights kernel for many rows stores in shared memory
before the loads of the exponential warps: a model of happens-before, run on the CPU, and the arrivals that the source has.

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


def simulate(items, NL, rng, passes_on):
    """passes_on: the issuer, which waited for the log-sum-exps, arrives for S beside its commit."""
    l_full, l_empty = [Bar(1) for _ in range(NL)], [Bar(2) for _ in range(NL)]
    s_full, s_free = [Bar(2 if passes_on else 1) for _ in range(4)], [Bar(1) for _ in range(4)]
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
            if passes_on:
                s_full[s].arrive(set(knows))

    def exps(u, half, knows):
        for use, n in enumerate(range(half, items, 2)):
            yield s_full[2 * u + half], use
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


def test_the_kernel_arrives_as_modelled():
    """Behind its wait for the log-sum-exps the issuer arrives on the scores' barrier, which counts that arrival."""
    with open(SOURCE) as f:
        text = f.read()
    assert re.search(r"mbar_init\(smem_u32\(&bar_s_full\[i\]\), 2\);", text)
    issuer = text[text.index("---- UMMA issuer of key tile u\n"):text.index("---- the CTA's parts, and their log-sum-exps\n")]
    wait = issuer.index("mbar_wait_warp(smem_u32(&bar_l_full[item % C::NL])")
    arrive, commit = issuer.index("mbar_arrive(smem_u32(&bar_s_full[s]))"), issuer.index("umma_commit(smem_u32(&bar_s_full[s]))")
    assert wait < arrive and wait < commit
