"""The calls for shared prefixes, accumulated weights and cuts together, as a server with a bounded cache uses
them: a prompt once, children that share it, then private copies that keep a budget of positions each.

The reference keeps, for every layer, sequence and kv head, the list of rows that should be in the
cache, each with its position: keys and values as they were stored (what rotation makes of a position is
tested elsewhere), cut by the plain form on the weights that the library had summed, after those were
held to the plain sums.
"""
import math

import numpy as np
import pytest
import torch

import causal_gqa_flash_attention_gb300 as ne
from causal_gqa_flash_attention_gb300 import _build

import paged_ref
import serving_ref as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    ne.load()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Server:
    def __init__(self, dtype, D, Hq, Hkv, layers, ps, pages, W, seed):
        self.dtype, self.D, self.Hq, self.Hkv, self.layers, self.ps, self.W = dtype, D, Hq, Hkv, layers, ps, W
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.k, self.v = (torch.full((layers, pages, ps, Hkv, D), math.nan, dtype=dtype, device="cuda") for _ in "kv")
        self.count = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.spec = ne.rope_spec(D)

    def randn(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda").to(self.dtype)

    def stored(self, layer, table, b, slots):
        """K and V rows [slots, Hkv, D] of a sequence, in 64 bits."""
        at = torch.as_tensor(slots, device="cuda")
        page = table[b].long()[at // self.ps]
        return self.k[layer, page, at % self.ps].double(), self.v[layer, page, at % self.ps].double()


def check_rows(q, o, lse, keys, vals, n_new, half, p_half):
    """o [n, Hq, D] against attention over the rows of each head (the last n_new of them the new tokens' own)."""
    n, Hq, D = q.shape
    Hkv = len(keys)
    G = Hq // Hkv
    for h in range(Hkv):
        hs = slice(h * G, (h + 1) * G)
        o_ref, lse_ref, A, S = paged_ref.attend(q[:, hs].double(), keys[h][:, None], vals[h][:, None], len(keys[h]) - n_new)
        tol_o, tol_lse = paged_ref.attn_bounds(o_ref, A, S, lse_ref, D, len(keys[h]), half, p_half)
        assert bool(((o[:, hs].double() - o_ref).abs() <= tol_o).all())
        assert bool(((lse[:, hs].double() - lse_ref).abs() <= tol_lse).all())


@pytest.mark.parametrize("dtype,D,Hq,Hkv", [(BF16, 64, 12, 4), (F32, 32, 4, 2)])
def test_a_server_with_a_budget(dtype, D, Hq, Hkv):
    layers, ps, prompt, C, budget, sink, recent = 2, 16, 600, 3, 200, 2, 24
    W = (300 << 20) // (C * ps * Hkv * 2 * D * dtype.itemsize) + 1          # (tables of long sequences: the children's calls share)
    s = Server(dtype, D, Hq, Hkv, layers, ps, 256, W, 1)
    half = torch.finfo(dtype).eps / 2
    p_half = torch.finfo(BF16).eps / 2 if dtype == BF16 else 0.0
    ok = lambda: (torch.cuda.synchronize(), ne.get_device_error() == ne.NE_OK)[1]  # noqa: E731

    # The prompt, once.
    table = torch.full((1, W), -1, dtype=torch.int32, device="cuda")
    s.count, table, short = ne.pages_resize(s.count, table, i32([0]), i32([prompt]), s.k, s.v)
    for la in range(layers):
        q = s.randn(prompt, Hq, D)
        ne.paged_append(s.randn(prompt, Hkv, D), s.randn(prompt, Hkv, D), s.k[la], s.v[la], table, i32([prompt]), i32([0, prompt]), rope=s.spec, q=q,
                        q_out=q)
        ne.paged_attn(q, s.k[la], s.v[la], table, i32([prompt]), i32([0, prompt]), max_new=prompt)
    assert int(short) == 0 and ok()

    # Children share its pages and take a few tokens each.
    s.count, table, lens, short = ne.pages_fork(s.count, table, i32([prompt]), i32([0] * C), s.k, s.v)
    n = [5, 1, 9]
    cu = np.concatenate([[0], np.cumsum(n)])
    new = [prompt + x for x in n]
    s.count, table, short = ne.pages_resize(s.count, table, lens, i32(new), s.k, s.v)
    assert int(short) == 0
    for la in range(layers):
        q = ne.paged_append(s.randn(sum(n), Hkv, D), s.randn(sum(n), Hkv, D), s.k[la], s.v[la], table, i32(new), i32(cu), rope=s.spec,
                            q=s.randn(sum(n), Hq, D))
        o, lse = ne.paged_attn_shared(q, s.k[la], s.v[la], table, i32(new), i32([0, C]), i32([prompt]), i32(cu), max_new=max(n))
        assert ok()
        for b in range(C):
            k, v = s.stored(la, table, b, np.arange(new[b]))
            rows = slice(int(cu[b]), int(cu[b + 1]))
            check_rows(q[rows], o[rows], lse[rows], [k[:, h] for h in range(Hkv)], [v[:, h] for h in range(Hkv)], n[b], half, p_half)

    # Private copies, and the weights of their last tokens: from here on each keeps `budget` positions.
    s.count, table, lens, short = ne.pages_fork(s.count, table, i32(new), i32([0, 1, 2]), s.k, s.v, deep=True)
    assert int(short) == 0
    T = W * ps
    w = torch.zeros(layers, C, Hkv, T, device="cuda")
    pos = torch.full((layers, C, Hkv, T), -1, dtype=torch.int32, device="cuda")
    off = i32([0] * C)
    held = {}                                               # (layer, sequence, head): rows as [position, K, V] in slot order
    for la in range(layers):
        for b in range(C):
            k, v = s.stored(la, table, b, np.arange(new[b]))
            for h in range(Hkv):
                held[la, b, h] = [(p, k[p, h], v[p, h]) for p in range(new[b])]
    length, ends = list(new), list(new)
    for step in range(6):
        n = [40, 33, 21] if step == 0 else [1, 1, 1] if step != 3 else [1, 0, 4]
        cu = np.concatenate([[0], np.cumsum(n)])
        grown = [a + x for a, x in zip(length, n)]
        s.count, table, short = ne.pages_resize(s.count, table, i32(length), i32(grown), s.k, s.v)
        assert int(short) == 0
        for la in range(layers):
            q = ne.paged_append(s.randn(sum(n), Hkv, D), s.randn(sum(n), Hkv, D), s.k[la], s.v[la], table, i32(grown), i32(cu), rope=s.spec,
                                pos_offset=off, q=s.randn(sum(n), Hq, D))
            o, lse = ne.paged_attn(q, s.k[la], s.v[la], table, i32(grown), i32(cu), max_new=max(n))
            before = w[la].clone()
            ne.paged_weights(q, lse, s.k[la], table, i32(grown), w[la], i32(cu), max_new=max(n), weights_out=w[la])
            assert ok()
            safe = table.clamp(min=0)
            want, got, size = ref.paged_weights(q, lse, s.k[la], safe, grown, cu, before)
            tol = ref.weights_bound(want, got, size, D, Hq // Hkv * max(n))
            live = (torch.arange(T, device="cuda") < i32(grown)[:, None, None]).expand_as(want)
            assert bool(((w[la].double() - want).abs() <= tol)[live].all())
            for b in range(C):
                k, v = s.stored(la, table, b, np.arange(length[b], grown[b]))
                for h in range(Hkv):
                    held[la, b, h] += [(ends[b] + i, k[i, h], v[i, h]) for i in range(n[b])]
                rows = slice(int(cu[b]), int(cu[b + 1]))
                if n[b]:
                    check_rows(q[rows], o[rows], lse[rows], [torch.stack([x[1] for x in held[la, b, h]]) for h in range(Hkv)],
                               [torch.stack([x[2] for x in held[la, b, h]]) for h in range(Hkv)], n[b], half, p_half)
        # Back to the budget: the reference cuts by the same weights.
        cut = [min(budget, x) for x in grown]
        w_h, pos_h, off_h = w.cpu().numpy(), pos.cpu().numpy(), off.cpu().numpy()
        ne.pages_evict(w, pos, off, table, i32(grown), i32(cut), s.k, s.v, sink=sink, recent=recent, weights_out=w, positions_out=pos,
                       pos_offset_out=off)
        assert ok()
        for la in range(layers):
            for b in range(C):
                for h in range(Hkv):
                    w_ref, p_ref, moves = ref.evict_row(w_h[la, b, h], pos_h[la, b, h], int(off_h[b]), grown[b], cut[b], sink, recent)
                    rows = held[la, b, h]
                    for src, dst in moves:
                        rows[dst] = rows[src]
                    del rows[cut[b]:]
                    assert np.array_equal(w[la, b, h].cpu().numpy(), w_ref) and np.array_equal(pos[la, b, h].cpu().numpy(), p_ref)
                    assert [x[0] for x in rows] == list(p_ref[:cut[b]])     # what is held is what the positions say
                    assert set(range(sink)) <= set(p_ref[:cut[b]]) and set(range(ends[b] + n[b] - recent, ends[b] + n[b])) <= set(p_ref[:cut[b]])
                    k, v = s.stored(la, table, b, np.arange(cut[b]))
                    assert torch.equal(k[:, h], torch.stack([x[1] for x in rows])) and torch.equal(v[:, h], torch.stack([x[2] for x in rows]))
        s.count, table, short = ne.pages_resize(s.count, table, i32(grown), i32(cut), s.k, s.v)
        ends = [e + x for e, x in zip(ends, n)]
        length = cut
        assert [int(x) for x in off] == [e - c for e, c in zip(ends, cut)]
    # All is given back: the parents' and the children's shared pages are still held, the private ones free.
    s.count, table, short = ne.pages_resize(s.count, table, i32(length), i32([0] * C), s.k, s.v)
    assert ok() and bool((table == -1).all())


def test_a_step_of_all_calls_captured():
    """One generation step at the budget, every call in one graph, replayed: as the same calls one by one."""
    def make():
        s = Server(BF16, 64, 12, 4, 2, 16, 64, 16, 3)
        B, L = 4, 100
        table = torch.full((B, 16), -1, dtype=torch.int32, device="cuda")
        s.count, table, _ = ne.pages_resize(s.count, table, i32([0] * B), i32([L] * B), s.k, s.v)
        for la in range(2):
            x = s.randn(B * L, 4, 64), s.randn(B * L, 4, 64)
            ne.paged_append(*x, s.k[la], s.v[la], table, i32([L] * B), i32(np.arange(B + 1) * L), rope=s.spec)
        st = dict(s=s, table=table, w=torch.rand(2, B, 4, 256, generator=torch.Generator().manual_seed(1)).cuda(),
                  pos=torch.full((2, B, 4, 256), -1, dtype=torch.int32, device="cuda"), off=i32([0] * B), L=i32([L] * B), L1=i32([L + 1] * B),
                  x=[(s.randn(B, 4, 64), s.randn(B, 4, 64), s.randn(B, 12, 64)) for _ in range(2)],
                  q=[torch.zeros(B, 12, 64, dtype=BF16, device="cuda") for _ in range(2)],
                  o=[torch.zeros(B, 12, 64, dtype=BF16, device="cuda") for _ in range(2)], lse=[torch.zeros(B, 12, device="cuda") for _ in range(2)],
                  ws=ne.alloc_paged_workspace(B, B, 12, 4, 64), pw=ne.alloc_pages_workspace(64, B, 16), ew=ne.alloc_evict_workspace(2, B, 4, 256),
                  short=i32([0]))
        st["w"][..., L:] = 0
        torch.cuda.synchronize()
        return st

    def step(t):
        s = t["s"]
        ne.pages_resize(s.count, t["table"], t["L"], t["L1"], s.k, s.v, refcount_out=s.count, table_out=t["table"], short=t["short"], workspace=t["pw"])
        for la in range(2):
            k, v, q = t["x"][la]
            ne.paged_append(k, v, s.k[la], s.v[la], t["table"], t["L1"], rope=s.spec, pos_offset=t["off"], q=q, q_out=t["q"][la])
            ne.paged_attn(t["q"][la], s.k[la], s.v[la], t["table"], t["L1"], o=t["o"][la], lse=t["lse"][la], workspace=t["ws"])
            ne.paged_weights(t["q"][la], t["lse"][la], s.k[la], t["table"], t["L1"], t["w"][la], weights_out=t["w"][la])
        ne.pages_evict(t["w"], t["pos"], t["off"], t["table"], t["L1"], t["L"], s.k, s.v, sink=1, recent=8, weights_out=t["w"],
                       positions_out=t["pos"], pos_offset_out=t["off"], workspace=t["ew"])
        ne.pages_resize(s.count, t["table"], t["L1"], t["L"], s.k, s.v, refcount_out=s.count, table_out=t["table"], short=t["short"], workspace=t["pw"])

    a, b = make(), make()
    for _ in range(5):
        step(a)
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        step(b)
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    assert ne.get_device_error() == ne.NE_OK
    for k in ("table", "w", "pos", "off"):
        assert torch.equal(a[k], b[k]), k
    assert int(a["off"][0]) == 5
    assert torch.equal(a["o"][1], b["o"][1]) and torch.equal(a["s"].k.nan_to_num(), b["s"].k.nan_to_num())
