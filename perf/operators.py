"""The paged key/value cache operators, as a serving program calls them.

Three families over one cache (pages of ``ps`` positions, [P, ps, Hkv, D] each for keys
and values, page tables [B, W], reference counts [P]):

- ``append``: rotate the new tokens' queries and keys at their positions, write keys and
  values into their pages;
- ``attn``: attention of the new tokens (a chunk each, or one token each) over the pages;
- ``fork``, ``resize``, ``compact``: sequences that share or copy pages, pages taken and
  given back as lengths change, and the live pages moved together.

``run`` computes them in elementary torch operations (``own`` false) or calls the library
(``own`` true).  Page ids, counts and tables are int32 and have one right answer: the
lowest free page goes first.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    rope = dict(layout="interleaved", rot=64, theta=10000.0, scaling="none", factor=1.0, orig=0, mscale=1.0)
    return [
        # The write half of one generation step of the GPU-pipeline model, 16 sequences: latency.
        dict(name="append_step_b16", op="append", dtype="bf16", B=16, n_max=1, L=512, Hq=12, Hkv=4, D=64, ps=16,
             ragged=0, far=0, hnd=False, tail=0, shape_seed=1, **rope),
        # A prompt chunk of eight sequences with D 128 heads: half-split rotation of half the
        # head, positions past the trained context (scaled by parts).
        dict(name="append_chunk_d128", op="append", dtype="bf16", B=8, n_max=2048, L=16384, Hq=16, Hkv=4, D=128, ps=64,
             ragged=1, far=1, hnd=False, tail=3, shape_seed=2, layout="half", rot=64, theta=10000.0, scaling="parts",
             factor=8.0, orig=2048, mscale=1.2079441541679836),
        # One generation step of the small fp32 model: two short sequences, latency alone.
        dict(name="attn_step_f32_small", op="attn", dtype="f32", B=2, n_max=1, L=128, Hq=4, Hkv=2, D=32, ps=16,
             ragged=1, hnd=False, tail=0, shape_seed=3),
        # One generation step over eight long sequences: the read of the cache.
        dict(name="attn_step_b8_l16384", op="attn", dtype="bf16", B=8, n_max=1, L=16384, Hq=12, Hkv=4, D=64, ps=16,
             ragged=0, hnd=False, tail=0, shape_seed=4),
        # A serving batch in flight: sequences with one new token beside prompt chunks of up
        # to 512, odd lengths, a padded row tail.
        dict(name="attn_mixed_b12", op="attn", dtype="bf16", B=12, n_max=512, L=4096, Hq=12, Hkv=4, D=64, ps=16,
             ragged=2, hnd=False, tail=5, shape_seed=5),
        # A long prompt's next chunk: 2048 new tokens over 16384 positions, D 128.
        dict(name="attn_chunk_2048_l16384", op="attn", dtype="bf16", B=1, n_max=2048, L=16384, Hq=16, Hkv=4, D=128,
             ps=64, ragged=0, hnd=False, tail=0, shape_seed=6),
        # Beam search / parallel sampling: 16 sequences forked to 64, whole pages shared,
        # the partial last page copied over 16 layers.
        dict(name="fork_share_64", op="fork", dtype="bf16", B=16, C=64, L=512, layers=16, Hkv=4, D=64, ps=16, P=4096,
             deep=False, hnd=False, shape_seed=7),
        # Private copies of eight long sequences (a prefix that is going to be edited).
        dict(name="fork_deep_8", op="fork", dtype="bf16", B=8, C=8, L=2048, layers=16, Hkv=4, D=64, ps=16, P=4096,
             deep=True, hnd=False, shape_seed=8),
        # Before a generation step: 64 sequences one token longer, a few need a page.
        dict(name="resize_step_64", op="resize", dtype="bf16", B=64, L=512, layers=2, Hkv=4, D=64, ps=16, P=4096,
             mode="step", hnd=False, shape_seed=9),
        # A scheduler's sweep over a thousand sequences: some end, some are cut back, some grow.
        dict(name="resize_sweep_1024", op="resize", dtype="bf16", B=1024, L=2048, layers=1, Hkv=1, D=64, ps=16, P=131072,
             mode="sweep", hnd=False, shape_seed=10),
        # A small pool with holes, moved together.
        dict(name="compact_512", op="compact", dtype="f32", B=16, L=256, layers=2, Hkv=2, D=32, ps=16, P=512,
             hnd=False, shape_seed=11),
        # A pool of 16 layers, half of it free, moved together before it shrinks.
        dict(name="compact_4096", op="compact", dtype="bf16", B=32, L=1024, layers=16, Hkv=4, D=64, ps=16, P=4096,
             hnd=False, shape_seed=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "attn", "fork", "resize", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    Hkv = rng.choice([1, 2, 4, 4, 5, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    D = rng.choice([32, 64, 128]) if dtype == "bf16" else rng.choice([32, 64])
    ps = rng.choice([8, 16, 32, 64, 128])
    case = dict(op=op, dtype=dtype, Hkv=Hkv, D=D, ps=ps, hnd=rng.random() < 0.3, shape_seed=rng.randrange(1 << 30))
    if op in ("append", "attn"):
        Hq = Hkv * G
        B = _log_int(rng, 1, 48)
        L = _log_int(rng, 1, 16384)
        n_max = 1 if rng.random() < 0.4 else _log_int(rng, 1, min(L, 2048))
        most = 1 << (28 if dtype == "bf16" else 26)         # scores of a padded batch
        while B > 1 and B * n_max * Hq * L > most:
            B -= 1
        while n_max > 1 and B * n_max * Hq * L > most:
            n_max = max(1, n_max // 2)
        case |= dict(B=B, n_max=n_max, L=L, Hq=Hq, ragged=rng.choice([0, 1, 2]), tail=rng.choice([0, 0, 1, 7]))
    if op == "append":
        scaling = rng.choice(["none", "linear", "base", "parts"])
        case |= dict(layout=rng.choice(["interleaved", "half"]), rot=rng.choice([D, D, D // 2, D // 4 + 2]),
                     theta=rng.choice([10000.0, 500000.0]), scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 8.0]),
                     orig=2048 if scaling == "parts" else 0, mscale=1.0 if scaling != "parts" else 1.1, far=rng.choice([0, 0, 1]))
    if op in ("fork", "resize", "compact"):
        B = _log_int(rng, 1, 512)
        L = _log_int(rng, 1, 1024)
        layers = _log_int(rng, 1, 8)
        per = -(-L // ps)
        P = 2 * B * per + rng.randrange(1, 64)
        size = layers * P * ps * Hkv * D * (2 if dtype == "bf16" else 4)
        while size > (1 << 28) and B > 1:
            B = B // 2
            P = 2 * B * per + rng.randrange(1, 64)
            size = layers * P * ps * Hkv * D * (2 if dtype == "bf16" else 4)
        case |= dict(B=B, L=L, layers=layers, P=P)
        if op == "fork":
            case |= dict(C=_log_int(rng, 1, 2 * B), deep=rng.random() < 0.3)
        if op == "resize":
            case |= dict(mode=rng.choice(["step", "sweep"]))
    return case


def _lengths(case):
    """(new tokens, cached positions) of every sequence of an append or attn case."""
    rng = random.Random(case["shape_seed"])
    B, n_max, L = case["B"], case["n_max"], case["L"]
    n, ln = [], []
    for b in range(B):
        if case["ragged"] == 0 or (b == 0 and case["ragged"] == 1):
            nb, lb = n_max, L
        elif case["ragged"] == 1:
            nb, lb = rng.randint(1, n_max), rng.randint(max(1, L // 4), L)
        else:                                       # every second sequence adds one token
            nb, lb = (1 if b % 2 else rng.randint(1, n_max)), rng.randint(max(1, L // 8), L)
        n.append(min(nb, lb))
        ln.append(lb)
    return n, ln


def _page_lens(case):
    """(length, next length) of every sequence of a fork, resize or compact case."""
    rng = random.Random(case["shape_seed"])
    L, out = case["L"], []
    for b in range(case["B"]):
        ln = L if b == 0 else rng.randint(1, L)
        if case.get("mode") == "sweep":
            kind = rng.random()
            new = 0 if kind < 0.3 else rng.randint(0, ln) if kind < 0.5 else min(2 * L, ln + rng.randint(0, L))
        else:
            new = ln + 1
        out.append((ln, new))
    return out


# ---------------------------------------------------------------- inputs

def _randn(shape, gen, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _pool(case, layers, P, gen, dtype):
    """A pool whose pages hold older values; `hnd` keeps each head's positions together."""
    H, ps, D = case["Hkv"], case["ps"], case["D"]
    x = torch.empty((layers, P, H, ps, D) if case["hnd"] else (layers, P, ps, H, D), device="cuda", dtype=dtype)
    x.normal_(generator=gen)
    return x.transpose(2, 3) if case["hnd"] else x


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DT[case["dtype"]]
    dev = "cuda"
    s = {"case": case}
    ps = case["ps"]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    if case["op"] in ("append", "attn"):
        n, ln = _lengths(case)
        B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
        N = sum(n) + case["tail"]
        far = 1 << 17 if case.get("far") else 0           # far positions: a table that starts late
        W = -(-(max(ln)) // ps)
        P = B * W + 3
        s["n"], s["len"] = n, ln
        s["cu"] = i32(np.concatenate([[0], np.cumsum(n)]).astype(np.int32))
        s["seq"] = i32(ln)
        s["table"] = torch.randperm(P, generator=gen, device=dev).to(torch.int32)[: B * W].view(B, W).contiguous()
        s["kp"] = _pool(case, 1, P, gen, dt)[0]
        s["vp"] = _pool(case, 1, P, gen, dt)[0]
        s["q"] = _randn((N, Hq, D), gen, dt)
        if case["op"] == "append":
            # One projection's output: queries, keys and values of a token side by side.
            qkv = _randn((N, Hq + 2 * Hkv, D), gen, dt)
            s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
            s["pos0"] = far
            s["q_out"] = torch.zeros((N, Hq, D), device=dev, dtype=dt)
        else:
            s["o"] = torch.zeros((N, Hq, D), device=dev, dtype=dt)
            s["lse"] = torch.zeros((N, Hq), device=dev, dtype=torch.float32)
        return s
    lens = _page_lens(case)
    B, P, L = case["B"], case["P"], case["L"]
    cap = 2 * L if case.get("mode") == "sweep" else L + 1
    W = -(-cap // ps)
    per = np.array([-(-a // ps) for a, _ in lens])
    perm = torch.randperm(P, generator=gen, device=dev).cpu().numpy().astype(np.int32)
    table = np.full((B, W), -1, np.int32)
    at = 0
    for b in range(B):
        if case["op"] == "resize" and b % 4 == 3:         # a fork of the sequence before: whole pages shared
            k = min(per[b], lens[b - 1][0] // ps, lens[b][0] // ps)
            table[b, :k] = table[b - 1, :k]
        else:
            k = 0
        table[b, k:per[b]] = perm[at:at + per[b] - k]
        at += int(per[b]) - k
    ref = np.bincount(table[table >= 0].ravel(), minlength=P).astype(np.int32)
    s["k_all"] = _pool(case, case["layers"], P + 1, gen, dt)  # one page more than the pool uses
    s["v_all"] = _pool(case, case["layers"], P + 1, gen, dt)
    s["kp"], s["vp"] = s["k_all"][:, :P], s["v_all"][:, :P]
    s["ref"], s["table"] = i32(ref), i32(table)
    s["seq"], s["new"] = i32([a for a, _ in lens]), i32([c for _, c in lens])
    if case["op"] == "fork":
        s["parents"] = torch.randint(0, B, (case["C"],), generator=gen, device=dev, dtype=torch.int32)
    return s


# ---------------------------------------------------------------- plain forms

def _freqs(case):
    """Angle per position of every pair (float64, numpy)."""
    R, th, f = case["rot"], case["theta"], case["factor"]
    i = np.arange(R // 2, dtype=np.float64)
    if case["scaling"] == "base":
        th = th * f ** (R / (R - 2.0))
    w = th ** (-2.0 * i / R)
    if case["scaling"] == "linear":
        w = w / f
    if case["scaling"] == "parts":
        g = np.clip((case["orig"] * w / (2 * np.pi) - 1.0) / 31.0, 0.0, 1.0)
        w = w * (g + (1.0 - g) / f)
    return w


def _rotate(x, pos, case):
    """x [N, H, D] rotated at pos [N]: angles in 64 bits, products in 32."""
    R = case["rot"]
    w = torch.from_numpy(_freqs(case)).to(x.device)
    ang = pos.double()[:, None, None] * w
    c = (torch.cos(ang) * case["mscale"]).float()
    s = (torch.sin(ang) * case["mscale"]).float()
    xf = x.float()
    if case["layout"] == "interleaved":
        a, b = xf[..., 0:R:2], xf[..., 1:R:2]
        y = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    else:
        a, b = xf[..., : R // 2], xf[..., R // 2: R]
        y = torch.cat((a * c - b * s, a * s + b * c), -1)
    return torch.cat((y, xf[..., R:]), -1).to(x.dtype)


def _tokens(s):
    """Sequence, index within the sequence's new tokens and validity of every row."""
    N = s["q"].shape[0]
    t = torch.arange(N, device="cuda", dtype=torch.int32)
    b = (torch.searchsorted(s["cu"], t, right=True) - 1).clamp(max=s["cu"].numel() - 2)
    return b, t - s["cu"][b], t < s["cu"][-1]


def _append_plain(s):
    case = s["case"]
    b, i, ok = _tokens(s)
    n = s["cu"][1:] - s["cu"][:-1]
    pos = s["seq"][b] - n[b] + i
    q = _rotate(s["q"], pos + s["pos0"], case)
    s["q_out"].copy_(torch.where(ok[:, None, None], q, s["q_out"]))
    k = _rotate(s["k"], pos + s["pos0"], case)
    m = sum(s["n"])                                       # the rows behind the last sequence stay out
    page, slot = s["table"][b, (pos // case["ps"]).clamp(0, s["table"].shape[1] - 1)][:m].long(), (pos % case["ps"])[:m].long()
    s["kp"][page, slot] = k[:m]
    s["vp"][page, slot] = s["v"][:m]
    return {"q": s["q_out"], "k_pages": s["kp"], "v_pages": s["vp"]}


def _attn_plain(s):
    case = s["case"]
    Hq, Hkv, D, B = case["Hq"], case["Hkv"], case["D"], case["B"]
    G, nm = Hq // Hkv, max(s["n"])
    N = s["q"].shape[0]
    cu, seq = s["cu"], s["seq"]
    idx = (cu[:-1, None] + torch.arange(nm, device="cuda", dtype=torch.int32)).clamp(max=N - 1).long()
    q = s["q"][idx].float().view(B, nm, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * nm, D)
    page = s["table"].long()
    k = s["kp"][page].flatten(1, 2).float()               # [B, W ps, Hkv, D]
    v = s["vp"][page].flatten(1, 2).float()
    T = k.shape[1]
    j = torch.arange(T, device="cuda", dtype=torch.int32)
    v = torch.where((j < seq[:, None])[:, :, None, None], v, 0.0)
    sc = torch.matmul(q, k.permute(0, 2, 3, 1)).view(B, Hkv, G, nm, T) * (1.0 / math.sqrt(D))
    n = cu[1:] - cu[:-1]
    pos = seq[:, None] - n[:, None] + torch.arange(nm, device="cuda", dtype=torch.int32)
    keep = (j <= pos[:, :, None]) & (j < seq[:, None, None])
    sc = torch.where(keep[:, None, None], sc, -math.inf)
    mx = sc.amax(-1, keepdim=True)
    ref = torch.where(mx == -math.inf, 0.0, mx)
    p = torch.exp(sc - ref)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, Hkv, G * nm, T), v.permute(0, 2, 1, 3)).view(B, Hkv, G, nm, D)
    o = torch.where(l > 0, o / l, 0.0).permute(0, 3, 1, 2, 4).reshape(B, nm, Hq, D)
    lse = (ref + torch.log(l)).squeeze(-1).permute(0, 3, 1, 2).reshape(B, nm, Hq)
    b, i, ok = _tokens(s)
    i = i.clamp(max=nm - 1).long()
    s["o"].copy_(torch.where(ok[:, None, None], o[b, i].to(s["o"].dtype), s["o"]))
    s["lse"].copy_(torch.where(ok[:, None], lse[b, i], s["lse"]))
    return {"o": s["o"], "lse": s["lse"]}


def _free_list(ref):
    """The free pages in ascending order (the rest behind them) and how many there are."""
    used = ref > 0
    return torch.argsort(used.to(torch.int32), stable=True).to(torch.int32), (~used).sum(dtype=torch.int32)


def _copy_rows(s, src, dst, rows):
    """Copies the first rows[j] positions of page src[j] to page dst[j]; src < 0 copies nothing."""
    r = torch.arange(s["case"]["ps"], device="cuda", dtype=torch.int32)
    live = ((src >= 0)[:, None] & (r < rows[:, None]))[None, :, :, None, None]
    frm = src.clamp(min=0).long()
    to = torch.where(src >= 0, dst, s["kp"].shape[1]).long()   # the spare page behind the pool takes the rest
    k, v = s["k_all"], s["v_all"]
    k.index_copy_(1, to, torch.where(live, k[:, frm], k[:, to]))
    v.index_copy_(1, to, torch.where(live, v[:, frm], v[:, to]))


def _fork_plain(s):
    case = s["case"]
    ps, C = case["ps"], case["C"]
    ref, par = s["ref"], s["parents"].long()
    W = s["table"].shape[1]
    ln = s["seq"][par]
    full, pages = ln // ps, (ln + ps - 1) // ps
    i = torch.arange(W, device="cuda", dtype=torch.int32)
    old = s["table"][par]
    fresh = (i < pages[:, None]) & ((i >= full[:, None]) | case["deep"])
    share = (i < full[:, None]) & (not case["deep"])
    free, n_free = _free_list(ref)
    rank = (torch.cumsum(fresh.flatten().to(torch.int32), 0, dtype=torch.int32) - 1).view(C, W)
    need = fresh.sum(dtype=torch.int32)
    short = (need - n_free).clamp(min=0)
    ok = short == 0
    got = free[rank.clamp(0, ref.numel() - 1).long()]
    child = torch.where(ok, torch.where(fresh, got, torch.where(share, old, -1)), -1)
    add = torch.zeros_like(ref).index_add_(0, child.clamp(min=0).flatten().long(), (child >= 0).flatten().to(torch.int32))
    src = torch.where(fresh & ok, old, -1).flatten()
    if not case["deep"]:                                  # at most the partial last page of a child
        last = (full.clamp(max=W - 1))[:, None].long()
        src = torch.gather(src.view(C, W), 1, last).flatten()
        dst, rows = torch.gather(child, 1, last).flatten(), ln % ps
    else:
        dst, rows = child.flatten(), (ln[:, None] - i * ps).clamp(max=ps).flatten()
    _copy_rows(s, src, dst, rows)
    return {"refcount": ref + add, "table": child, "lens": torch.where(ok, ln, 0), "short": short.view(1),
            "k_pages": s["kp"], "v_pages": s["vp"]}


def _resize_plain(s):
    case = s["case"]
    ps = case["ps"]
    ref, tab, old, new = s["ref"], s["table"], s["seq"], s["new"]
    B, W = tab.shape
    i = torch.arange(W, device="cuda", dtype=torch.int32)
    po, pn = ((old + ps - 1) // ps)[:, None], ((new + ps - 1) // ps)[:, None]
    low = torch.minimum(old, new)
    drop = (i >= pn) & (i < po) & (tab >= 0)
    at = tab.clamp(min=0).flatten().long()
    left = ref - torch.zeros_like(ref).index_add_(0, at, drop.flatten().to(torch.int32))
    part = (i == (low // ps)[:, None]) & (low % ps != 0)[:, None]
    split = part & (tab >= 0) & (left[tab.clamp(min=0).long()] > 1)
    grow = (i >= po) & (i < pn)
    fresh = split | grow
    free, n_free = _free_list(left)
    rank = (torch.cumsum(fresh.flatten().to(torch.int32), 0, dtype=torch.int32) - 1).view(B, W)
    short = (fresh.sum(dtype=torch.int32) - n_free).clamp(min=0)
    ok = short == 0
    got = free[rank.clamp(0, ref.numel() - 1).long()]
    out = torch.where(ok, torch.where(fresh, got, torch.where((i < pn) & (i < po), tab, -1)), tab)
    gone = torch.zeros_like(ref).index_add_(0, at, split.flatten().to(torch.int32))
    more = torch.zeros_like(ref).index_add_(0, got.flatten().long(), fresh.flatten().to(torch.int32))
    e = (low // ps).clamp(max=W - 1)[:, None].long()
    src = torch.where(ok, torch.gather(torch.where(split, tab, -1), 1, e).flatten(), -1)
    _copy_rows(s, src, torch.gather(out, 1, e).flatten(), low % ps)
    return {"refcount": torch.where(ok, left - gone + more, ref), "table": out, "short": short.view(1),
            "k_pages": s["kp"], "v_pages": s["vp"]}


def _compact_plain(s):
    ref, tab = s["ref"], s["table"]
    P = ref.numel()
    live = ref > 0
    n_live = live.sum(dtype=torch.int32)
    ids = torch.arange(P, device="cuda", dtype=torch.int32)
    move = live & (ids >= n_live)
    hole = (~live) & (ids < n_live)
    holes = torch.argsort((~hole).to(torch.int32), stable=True).to(torch.int32)   # ascending, then the rest
    rank = torch.cumsum(move.to(torch.int32), 0, dtype=torch.int32) - 1
    remap = torch.where(live, torch.where(move, holes[rank.clamp(min=0).long()], ids), -1)
    movers = torch.argsort((~move).to(torch.int32), stable=True)
    half = P // 2 + 1                                      # at most that many pages move
    src = torch.where(move[movers[:half]], movers[:half].to(torch.int32), -1)
    dst = remap[movers[:half]]
    _copy_rows(s, src, dst, torch.full_like(src, s["case"]["ps"]))
    at = torch.where(live, remap, P).long()
    out = torch.zeros(P + 1, dtype=torch.int32, device="cuda").index_copy_(0, at, ref)[:P]
    out = torch.where(ids < n_live, out, 0)
    t = torch.where(tab >= 0, remap[tab.clamp(min=0).long()], -1)
    return {"refcount": out, "table": t, "remap": remap, "n_live": n_live.view(1), "k_pages": s["kp"], "v_pages": s["vp"]}


# ---------------------------------------------------------------- one pass

def _run_own(s):
    import causal_gqa_flash_attention_gb300 as ne
    case = s["case"]
    op = case["op"]
    if op == "append":
        if "spec" not in s:
            s["spec"] = ne.rope_spec(case["D"], rot_dim=case["rot"], theta=case["theta"], layout=case["layout"],
                                     scaling=case["scaling"], factor=case["factor"], orig_len=case["orig"],
                                     mscale=case["mscale"])
        ne.paged_append(s["k"], s["v"], s["kp"], s["vp"], s["table"], s["seq"], s["cu"], rope=s["spec"],
                        pos_offset=s["pos0"], q=s["q"], q_out=s["q_out"])
        return {"q": s["q_out"], "k_pages": s["kp"], "v_pages": s["vp"]}
    if op == "attn":
        if "ws" not in s:
            s["ws"] = ne.alloc_paged_workspace(case["B"], s["q"].shape[0], case["Hq"], case["Hkv"], case["D"])
        ne.paged_attn(s["q"], s["kp"], s["vp"], s["table"], s["seq"], s["cu"], max_new=max(s["n"]), o=s["o"],
                      lse=s["lse"], workspace=s["ws"])
        return {"o": s["o"], "lse": s["lse"]}
    if "ws" not in s:
        s["ws"] = ne.alloc_pages_workspace(case["P"], max(case["B"], case.get("C", 0)), s["table"].shape[1])
    if op == "fork":
        ref, tab, ln, short = ne.pages_fork(s["ref"], s["table"], s["seq"], s["parents"], s["kp"], s["vp"],
                                            deep=case["deep"], workspace=s["ws"])
        return {"refcount": ref, "table": tab, "lens": ln, "short": short, "k_pages": s["kp"], "v_pages": s["vp"]}
    if op == "resize":
        ref, tab, short = ne.pages_resize(s["ref"], s["table"], s["seq"], s["new"], s["kp"], s["vp"], workspace=s["ws"])
        return {"refcount": ref, "table": tab, "short": short, "k_pages": s["kp"], "v_pages": s["vp"]}
    ref, tab, remap, n_live = ne.pages_compact(s["ref"], s["table"], s["kp"], s["vp"], workspace=s["ws"])
    return {"refcount": ref, "table": tab, "remap": remap, "n_live": n_live, "k_pages": s["kp"], "v_pages": s["vp"]}


def run(state):
    if own:
        return _run_own(state)
    return {"append": _append_plain, "attn": _attn_plain, "fork": _fork_plain, "resize": _resize_plain,
            "compact": _compact_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("append", "attn"):
        n, ln = _lengths(case)
        N, Hq, Hkv, D = sum(n), case["Hq"], case["Hkv"], case["D"]
        small = 4 * (2 * case["B"] + 1)
        if case["op"] == "append":
            return {"bytes": 2 * N * (Hq + 2 * Hkv) * D * e + small + 4 * N, "flops": 6 * N * (Hq + Hkv) * case["rot"] // 2}
        pairs = sum(c * (b - c) + c * (c + 1) // 2 for c, b in zip(n, ln))
        pages = sum(-(-b // case["ps"]) for b in ln)
        return {"bytes": sum(ln) * 2 * Hkv * D * e + 2 * N * Hq * D * e + 4 * N * Hq + 4 * pages + small,
                "flops": 4 * D * Hq * pairs}
    ps, lens = case["ps"], _page_lens(case)
    row = case["layers"] * 2 * case["Hkv"] * case["D"] * e   # one position, keys and values, every layer
    pages = sum(-(-a // ps) for a, _ in lens)
    book = 8 * case["P"] + 8 * pages
    if case["op"] == "fork":
        mean = sum((a if case["deep"] else a % ps) for a, _ in lens) / len(lens)
        return {"bytes": int(2 * case["C"] * mean * row) + book, "flops": 0}
    if case["op"] == "resize":
        return {"bytes": book, "flops": 0}
    holes = pages * (1.0 - pages / case["P"])                # random places: that many live pages lie too high
    return {"bytes": int(2 * holes * ps * row) + book, "flops": 0}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_append(case, s):
    w = _freqs(case)
    n, ln = s["n"], s["len"]
    R, ps = case["rot"], case["ps"]
    x = {k: s[k].double().cpu().numpy() for k in ("q", "k")}
    q_out, kp = s["q_out"].double().cpu().numpy(), s["kp"].double().cpu().numpy()
    tab = s["table"].cpu().numpy()
    first = np.arange(0, R, 2) if case["layout"] == "interleaved" else np.arange(R // 2)
    second = first + (1 if case["layout"] == "interleaved" else R // 2)
    at = 0
    for b, (nb, lb) in enumerate(zip(n, ln)):
        pos = np.arange(lb - nb, lb)
        z = np.exp(1j * ((pos + s["pos0"])[:, None] * w)) * case["mscale"]
        for name in ("q", "k"):
            y = x[name][at:at + nb]
            t = (y[..., first] + 1j * y[..., second]) * z[:, None]
            y = y.copy()
            y[..., first], y[..., second] = t.real, t.imag
            if name == "q":
                q_out[at:at + nb] = y
            else:
                kp[tab[b, pos // ps], pos % ps] = y
        at += nb
    return {"q": q_out, "k_pages": kp, "v_pages": None}


def _exact_attn(case, s):
    n, ln, ps = s["n"], s["len"], case["ps"]
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    o, lse = s["o"].double(), s["lse"].double()
    at = 0
    for b, (nb, lb) in enumerate(zip(n, ln)):
        pages = s["table"][b, : -(-lb // ps)].long()
        k = s["kp"][pages].reshape(-1, Hkv, D)[:lb].double()
        v = s["vp"][pages].reshape(-1, Hkv, D)[:lb].double()
        for i0 in range(0, nb, 512):
            i1 = min(nb, i0 + 512)
            last = lb - nb + torch.arange(i0, i1, device="cuda")
            gone = torch.arange(lb, device="cuda")[None] > last[:, None]
            for h in range(Hq):
                x = (s["q"][at + i0:at + i1, h].double() @ k[:, h // G].T) * D ** -0.5
                x.masked_fill_(gone, -math.inf)
                z = torch.logsumexp(x, -1)
                lse[at + i0:at + i1, h] = z
                o[at + i0:at + i1, h] = torch.exp(x - z[:, None]) @ v[:, h // G]
        at += nb
    return {"o": o, "lse": lse}


def exact(case, seed):
    if case["op"] not in ("append", "attn"):
        return None                                          # whole numbers and copies
    s = prepare(case, seed)
    return _exact_append(case, s) if case["op"] == "append" else _exact_attn(case, s)
