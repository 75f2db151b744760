"""Operators over the paged cache for batches that share a prefix and for caches of a fixed size.

- ``shared``: attention of the new tokens of sequences that share a long prefix (children of one
  fork, questions about one document), the prefix read and multiplied once for all of a group;
- ``weights``: the attention weight that every cached position has received, summed over the new
  tokens and the query heads of its kv head and added to what it had before;
- ``evict``: sequences cut to fewer positions, those with the least accumulated weight given up
  per layer and kv head, the first and the newest positions kept, the kept rows moved together.

``run`` computes them in elementary torch operations (``own`` false) or calls the library (``own``
true).  Which positions are kept has one right answer: ties go to the lowest slot.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One generation step of the small fp32 model: four samples of one short prompt.  Latency.
        dict(name="shared_step_f32_small", op="shared", dtype="f32", B=4, R=1, alone=0, P=512, own=48, n_max=1, Hq=4,
             Hkv=2, D=32, ps=16, ragged=1, shape_seed=1),
        # One generation step of 64 samples of one long prompt, the GPU-pipeline model's heads.
        dict(name="shared_step_b64_p16384", op="shared", dtype="bf16", B=64, R=1, alone=0, P=16384, own=512, n_max=1, Hq=12,
             Hkv=4, D=64, ps=16, ragged=1, shape_seed=2),
        # A serving batch in flight: four groups of different prefixes, five sequences of their own.
        dict(name="shared_step_b37_groups", op="shared", dtype="bf16", B=37, R=4, alone=5, P=8192, own=1024, n_max=1, Hq=16,
             Hkv=4, D=128, ps=64, ragged=1, shape_seed=3),
        # Questions of up to 256 tokens about one document of 8192.
        dict(name="shared_chunk_b16_p8192", op="shared", dtype="bf16", B=16, R=1, alone=0, P=8192, own=300, n_max=256, Hq=12,
             Hkv=4, D=64, ps=16, ragged=1, shape_seed=4),
        # The weights of one generation step of the small fp32 model.  Latency.
        dict(name="weights_step_f32_small", op="weights", dtype="f32", B=2, n_max=1, L=128, Hq=4, Hkv=2, D=32, ps=16,
             ragged=1, shape_seed=5),
        # One generation step over eight long sequences: the read of the keys.
        dict(name="weights_step_b8_l16384", op="weights", dtype="bf16", B=8, n_max=1, L=16384, Hq=12, Hkv=4, D=64, ps=16,
             ragged=0, shape_seed=6),
        # Single tokens beside prompt chunks of up to 512, odd lengths.
        dict(name="weights_mixed_b12", op="weights", dtype="bf16", B=12, n_max=512, L=4096, Hq=12, Hkv=4, D=64, ps=16,
             ragged=2, shape_seed=7),
        # A long prompt's chunk: 2048 new tokens over 16384 positions.
        dict(name="weights_chunk_2048_l16384", op="weights", dtype="bf16", B=1, n_max=2048, L=16384, Hq=16, Hkv=4, D=128,
             ps=64, ragged=0, shape_seed=8),
        # After a generation step at the cache's full size: one position of every layer and head goes.
        dict(name="evict_step_b16", op="evict", dtype="bf16", B=16, layers=16, L=513, keep=512, mode="step", Hkv=4, D=64, ps=16,
             sink=4, recent=64, shape_seed=9),
        # The small fp32 model's cache, two sequences.  Latency.
        dict(name="evict_step_f32_small", op="evict", dtype="f32", B=2, layers=2, L=65, keep=64, mode="step", Hkv=2, D=32, ps=16,
             sink=2, recent=8, shape_seed=10),
        # Eight prompts of up to 16384 positions cut to a quarter, four layers.
        dict(name="evict_prompt_b8_l16384", op="evict", dtype="bf16", B=8, layers=4, L=16384, keep=4096, mode="prompt", Hkv=4,
             D=64, ps=16, sink=4, recent=256, shape_seed=11),
        # A scheduler under pressure: 48 sequences of all lengths, cut to between none and all of them.
        dict(name="evict_ragged_b48", op="evict", dtype="bf16", B=48, layers=4, L=2048, keep=1024, mode="ragged", Hkv=4, D=128,
             ps=64, sink=1, recent=33, shape_seed=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "weights", "weights", "evict"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    Hkv = rng.choice([1, 2, 4, 4, 5, 8])
    D = rng.choice([32, 64, 128]) if dtype == "bf16" else rng.choice([32, 64])
    case = dict(op=op, dtype=dtype, Hkv=Hkv, D=D, ps=rng.choice([8, 16, 32, 64, 128]), shape_seed=rng.randrange(1 << 30))
    if op == "evict":
        B, layers, L = _log_int(rng, 1, 48), _log_int(rng, 1, 16), _log_int(rng, 2, 16384)
        while layers * B * L * Hkv * D > 1 << 25 and B * layers > 1:
            B, layers = max(1, B // 2), max(1, layers * 3 // 4)
        mode = rng.choice(["step", "prompt", "ragged"])
        keep = L - 1 if mode == "step" else rng.randint(1, L)
        return case | dict(B=B, layers=layers, L=L, keep=keep, mode=mode, sink=rng.choice([0, 1, 4]),
                           recent=min(keep, rng.choice([0, 1, 16, 33, 128])))
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    B = _log_int(rng, 1, 64)
    n_max = 1 if rng.random() < 0.5 else _log_int(rng, 1, 512)
    most = 1 << (27 if dtype == "bf16" else 25)             # scores of a padded batch
    case |= dict(Hq=Hkv * G, n_max=n_max)
    if op == "shared":
        P, own_len = _log_int(rng, 1, 16384), n_max + _log_int(rng, 1, 1024)
        while B > 1 and B * n_max * Hkv * G * (P + own_len) > most:
            B -= 1
        R = rng.randint(1, min(B, 4))
        return case | dict(B=B, R=R, alone=rng.choice([0, 0, 1, 3]) if B - R >= 3 else 0, P=P, own=own_len,
                           ragged=rng.choice([0, 1]))
    L = max(n_max, _log_int(rng, 1, 16384))
    while B > 1 and B * n_max * Hkv * G * L > most:
        B -= 1
    while n_max > 1 and B * n_max * Hkv * G * L > most:
        n_max = max(1, n_max // 2)
    return case | dict(B=B, n_max=n_max, L=L, ragged=rng.choice([0, 1, 2]))


def _shared_shape(case):
    """Groups [R + 1], shared positions [R], (new tokens, length) of every sequence."""
    rng = random.Random(case["shape_seed"])
    B, R, in_groups = case["B"], case["R"], case["B"] - case["alone"]
    cuts = sorted(rng.sample(range(1, in_groups), R - 1)) if R > 1 else []
    groups = [0, *cuts, in_groups]
    shared = [case["P"] if r == 0 or not case["ragged"] else rng.randint(max(1, case["P"] // 4), case["P"]) for r in range(R)]
    n, ln = [], []
    for b in range(B):
        r = sum(1 for g in groups[1:] if g <= b)
        first = shared[r] if r < R else rng.randint(0, case["P"] // 4)
        nb = case["n_max"] if not case["ragged"] or b == 0 else rng.randint(1, case["n_max"])
        n.append(nb)
        ln.append(first + (case["own"] if not case["ragged"] or b == 0 else rng.randint(nb, case["own"])))
    return groups, shared, n, ln


def _lengths(case):
    """(new tokens, cached positions) of every sequence of a weights case."""
    rng = random.Random(case["shape_seed"])
    n_max, L, n, ln = case["n_max"], case["L"], [], []
    for b in range(case["B"]):
        if case["ragged"] == 0 or (b == 0 and case["ragged"] == 1):
            nb, lb = n_max, L
        elif case["ragged"] == 1:
            nb, lb = rng.randint(1, n_max), rng.randint(max(1, L // 4), L)
        else:                                               # every second sequence adds one token
            nb, lb = (1 if b % 2 else rng.randint(1, n_max)), rng.randint(max(1, L // 8), L)
        n.append(min(nb, lb))
        ln.append(lb)
    return n, ln


def _evict_lens(case):
    """(length, next length, positions given up before, slots new since then) of every sequence."""
    rng = random.Random(case["shape_seed"])
    L, keep, out = case["L"], case["keep"], []
    for b in range(case["B"]):
        if case["mode"] == "step":
            out.append((L, keep, 300 + 7 * b, 1))
        elif case["mode"] == "prompt":
            ln = L if b == 0 else rng.randint(max(1, L // 2), L)
            out.append((ln, min(ln, keep), 0, ln))
        else:
            ln = L if b == 0 else rng.randint(1, L)
            new = rng.choice([0, ln, rng.randint(0, ln), min(ln, keep), min(ln, keep)])
            out.append((ln, new, rng.randint(0, 500), rng.randint(0, ln)))
    return out


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, gen, dtype, sigma=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * sigma).to(dtype)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(n):
    out = [0]
    for x in n:
        out.append(out[-1] + x)
    return out


def prepare(case, seed):
    s = {"shared": _prepare_shared, "weights": _prepare_weights, "evict": _prepare_evict}[case["op"]](case, _gen(seed))
    s["case"] = case
    return s


def _prepare_shared(case, gen):
    groups, shared, n, ln = _shared_shape(case)
    Hq, Hkv, D, ps, B, dt = case["Hq"], case["Hkv"], case["D"], case["ps"], case["B"], DT[case["dtype"]]
    N, W = sum(n), -(-max(ln) // ps)
    need = sum(-(-x // ps) for x in ln)
    perm = torch.randperm(need + 3, generator=gen, device="cuda").to(torch.int32).cpu()
    kp, vp = _randn((need + 3, ps, Hkv, D), gen, dt), _randn((need + 3, ps, Hkv, D), gen, dt)
    table = torch.full((B, W), -1, dtype=torch.int32)
    at, src, dst, rows = 0, [], [], []
    for b in range(B):
        r = sum(1 for g in groups[1:] if g <= b)
        k = 0
        if r < case["R"] and b > groups[r]:                 # a child: whole pages shared, the partial one copied
            k = shared[r] // ps
            table[b, :k] = table[groups[r], :k]
        pages = -(-ln[b] // ps)
        table[b, k:pages] = perm[at:at + pages - k]
        at += pages - k
        if k and shared[r] % ps or (r < case["R"] and b > groups[r] and shared[r] < ps):
            src.append(int(table[groups[r], k]))
            dst.append(int(table[b, k]))
            rows.append(shared[r] % ps)
    if src:
        live = torch.arange(ps, device="cuda") < torch.tensor(rows, device="cuda")[:, None]
        a, c = torch.tensor(src, device="cuda"), torch.tensor(dst, device="cuda")
        for x in (kp, vp):
            x[c] = torch.where(live[:, :, None, None], x[a], x[c])
    return {"q": _randn((N, Hq, D), gen, dt, 2.0), "kp": kp, "vp": vp, "table": table.cuda(), "seq": _i32(ln), "cu": _i32(_cu(n)),
            "groups": _i32(groups), "shared": _i32(shared), "shape": (groups, shared, n, ln),
            "o": torch.zeros((N, Hq, D), device="cuda", dtype=dt), "lse": torch.zeros((N, Hq), device="cuda")}


def _prepare_weights(case, gen):
    n, ln = _lengths(case)
    Hq, Hkv, D, ps, B, dt = case["Hq"], case["Hkv"], case["D"], case["ps"], case["B"], DT[case["dtype"]]
    N, W = sum(n), -(-max(ln) // ps)
    s = {"case": case, "n": n, "len": ln, "cu": _i32(_cu(n)), "seq": _i32(ln)}
    s["table"] = torch.randperm(B * W + 3, generator=gen, device="cuda").to(torch.int32)[: B * W].view(B, W).contiguous()
    s["kp"] = _randn((B * W + 3, ps, Hkv, D), gen, dt)
    s["q"] = _randn((N, Hq, D), gen, dt, 2.0)
    old = -torch.log1p(-torch.rand((B, Hkv, W * ps), generator=gen, device="cuda")) * 4.0
    s["weights"] = torch.where(torch.arange(W * ps, device="cuda") < s["seq"][:, None, None], old, 0.0)
    s["out"] = torch.zeros_like(s["weights"])
    sc, _ = _scores(s)                                      # the attention's own log-sum-exp of every row
    lse = torch.logsumexp(sc, -1).permute(0, 3, 1, 2).reshape(B, max(n), Hq)
    b, i = _rows_of(s)
    s["lse"] = lse[b, i].contiguous()
    return s


def _prepare_evict(case, gen):
    lens = _evict_lens(case)
    NL, B, Hkv, D, ps, dt = case["layers"], case["B"], case["Hkv"], case["D"], case["ps"], DT[case["dtype"]]
    W = -(-max(a for a, _, _, _ in lens) // ps)
    T, P = W * ps, B * W + 3
    s = {"seq": _i32([x[0] for x in lens]), "new": _i32([x[1] for x in lens]), "offset": _i32([x[2] for x in lens])}
    s["table"] = torch.randperm(P, generator=gen, device="cuda").to(torch.int32)[: B * W].view(B, W).contiguous()
    s["k_all"] = torch.empty((NL, P + 1, ps, Hkv, D), device="cuda", dtype=dt)   # one page more than the pool uses
    s["v_all"] = torch.empty((NL, P + 1, ps, Hkv, D), device="cuda", dtype=dt)
    s["k_all"].normal_(generator=gen)
    s["v_all"].normal_(generator=gen)
    s["kp"], s["vp"] = s["k_all"][:, :P], s["v_all"][:, :P]
    slot = torch.arange(T, device="cuda")
    live = slot < s["seq"][:, None, None]
    # Accumulated weights: a few positions take most; far positions are cut to a grid, so that ties occur.
    w = torch.exp(torch.randn((NL, B, Hkv, T), generator=gen, device="cuda") * 2.0)
    w = torch.where(w < 1.0, torch.round(w * 256.0) / 256.0, w)
    s["weights"] = torch.where(live, w, 0.0)
    # Positions of the slots that an earlier call has placed: any of those in front of the new ones.
    placed = torch.tensor([x[0] - x[3] for x in lens], device="cuda")[:, None, None]
    reach = placed + s["offset"][:, None, None]
    M = int(max(x[0] - x[3] + x[2] for x in lens))
    pos = torch.full((NL, B, Hkv, T), -1, dtype=torch.int32, device="cuda")
    if M > 0:
        key = torch.rand((NL, B, Hkv, M), generator=gen, device="cuda")
        key = torch.where(torch.arange(M, device="cuda") < reach, key, 2.0)
        any_order = torch.argsort(key, dim=-1).to(torch.int32)[..., :T]
        k = any_order.shape[-1]
        pos[..., :k] = torch.where(slot[:k] < placed, any_order, -1)
    s["positions"] = pos
    s["w_out"], s["p_out"] = torch.zeros_like(s["weights"]), torch.full_like(pos, -1)
    s["o_out"] = torch.zeros_like(s["offset"])
    return s


# ---------------------------------------------------------------- plain forms

def _rows_of(s):
    """Sequence of every packed row and its index within the sequence's new tokens."""
    N = s["q"].shape[0]
    t = torch.arange(N, device="cuda", dtype=torch.int32)
    b = (torch.searchsorted(s["cu"], t, right=True) - 1).clamp(max=s["cu"].numel() - 2)
    return b, (t - s["cu"][b]).long()


def _padded_q(s, nm):
    """[B, Hkv, G, nm, D] in 32 bits."""
    case = s["case"]
    Hkv, G, D = case["Hkv"], case["Hq"] // case["Hkv"], case["D"]
    idx = (s["cu"][:-1, None] + torch.arange(nm, device="cuda", dtype=torch.int32)).clamp(max=s["q"].shape[0] - 1).long()
    return s["q"][idx].float().view(-1, nm, Hkv, G, D).permute(0, 2, 3, 1, 4)


def _part(q, k, v, keep, scale):
    """Softmax statistics of one part of the keys: maximum, sum and unnormalised output."""
    sc = torch.matmul(q, k.transpose(-1, -2)) * scale
    if keep is not None:
        sc = torch.where(keep, sc, -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(m == -math.inf, 0.0, m))
    return m, p.sum(-1, keepdim=True), torch.matmul(p, v)


def _shared_plain(s):
    case = s["case"]
    groups, shared, n, ln = s["shape"]
    Hq, Hkv, D, ps, B = case["Hq"], case["Hkv"], case["D"], case["ps"], case["B"]
    G, N, nm, scale = Hq // Hkv, s["q"].shape[0], max(n), 1.0 / math.sqrt(D)
    cu = _cu(n)
    # The prefixes, once per group: [Hkv, rows G, positions].
    m1 = torch.full((N, Hkv, G, 1), -math.inf, device="cuda")
    l1, o1 = torch.zeros((N, Hkv, G, 1), device="cuda"), torch.zeros((N, Hkv, G, D), device="cuda")
    for r, P in enumerate(shared):
        lo, hi = cu[groups[r]], cu[groups[r + 1]]
        pages = s["table"][groups[r], : -(-P // ps)].long()
        k, v = (x[pages].flatten(0, 1)[:P].float().transpose(0, 1) for x in (s["kp"], s["vp"]))
        q = s["q"][lo:hi].float().view(hi - lo, Hkv, G, D).transpose(0, 1).reshape(Hkv, -1, D)
        for dst, x in zip((m1, l1, o1), _part(q, k, v, None, scale)):
            dst[lo:hi] = x.view(Hkv, hi - lo, G, -1).transpose(0, 1)
    # Every sequence's own positions.
    first = torch.zeros(B, dtype=torch.int32, device="cuda")
    for r in range(case["R"]):
        first[groups[r]:groups[r + 1]] = s["shared"][r]
    T = max(x - (shared[sum(1 for g in groups[1:] if g <= b)] if b < groups[-1] else 0) for b, x in enumerate(ln))
    pos = first[:, None] + torch.arange(T, device="cuda", dtype=torch.int32)
    page = torch.gather(s["table"], 1, (pos // ps).clamp(max=s["table"].shape[1] - 1).long()).clamp(min=0).long()
    k, v = (x[page, (pos % ps).long()].float().permute(0, 2, 1, 3) for x in (s["kp"], s["vp"]))
    nb = s["cu"][1:] - s["cu"][:-1]
    at = (s["seq"] - nb)[:, None] + torch.arange(nm, device="cuda", dtype=torch.int32)
    keep = (pos[:, None] <= at[:, :, None]) & (pos < s["seq"][:, None])[:, None]
    q = _padded_q(s, nm).reshape(B, Hkv, G * nm, D)
    own_part = _part(q, k, v, keep[:, None, None].expand(B, 1, G, nm, T).reshape(B, 1, G * nm, T), scale)
    b, i = _rows_of(s)
    m2, l2, o2 = (x.view(B, Hkv, G, nm, -1)[b, :, :, i] for x in own_part)
    m = torch.maximum(m1, m2)
    ref = torch.where(m == -math.inf, 0.0, m)
    w1, w2 = torch.exp(m1 - ref), torch.exp(m2 - ref)
    l = l1 * w1 + l2 * w2
    o = (o1 * w1 + o2 * w2) / l
    s["o"].copy_(torch.where(l > 0, o, 0.0).reshape(N, Hq, D))
    s["lse"].copy_((ref + torch.log(l)).reshape(N, Hq))
    return {"o": s["o"], "lse": s["lse"]}


def _scores(s):
    """Logits [B, Hkv, G, nm, T] of padded rows, -inf where a row does not see a position, and which do."""
    case = s["case"]
    B, nm = case["B"], max(s["n"])
    q = _padded_q(s, nm)
    k = s["kp"][s["table"].long()].flatten(1, 2).float().permute(0, 2, 3, 1)
    sc = torch.matmul(q.flatten(2, 3), k).view(*q.shape[:4], k.shape[-1]) * (1.0 / math.sqrt(case["D"]))
    nb = s["cu"][1:] - s["cu"][:-1]
    i = torch.arange(nm, device="cuda", dtype=torch.int32)
    at = torch.where(i < nb[:, None], (s["seq"] - nb)[:, None] + i, -1)
    keep = torch.arange(k.shape[-1], device="cuda", dtype=torch.int32) <= at[:, :, None]
    return torch.where(keep[:, None, None], sc, -math.inf), keep


def _weights_plain(s):
    case = s["case"]
    Hkv, G, nm = case["Hkv"], case["Hq"] // case["Hkv"], max(s["n"])
    sc, _ = _scores(s)
    idx = (s["cu"][:-1, None] + torch.arange(nm, device="cuda", dtype=torch.int32)).clamp(max=s["q"].shape[0] - 1).long()
    lse = s["lse"][idx].view(-1, nm, Hkv, G).permute(0, 2, 3, 1)[..., None]
    got = s["weights"] + torch.exp(sc - lse).sum((2, 3))
    T = got.shape[-1]
    live = torch.arange(T, device="cuda", dtype=torch.int32) < s["seq"][:, None, None]
    s["out"].copy_(torch.where(live, got, s["out"]))
    return {"weights": s["out"]}


def _evict_plain(s):
    case = s["case"]
    ps, T = case["ps"], s["weights"].shape[-1]
    w, old, new = s["weights"], s["seq"][:, None, None], s["new"][:, None, None]
    off = s["offset"][:, None, None]
    m = torch.minimum(old, new)
    slot = torch.arange(T, device="cuda", dtype=torch.int32)
    live = (slot < old).expand_as(w)
    pos = torch.where(s["positions"] < 0, slot + off, s["positions"])
    guarded = live & ((pos < case["sink"]) | (pos >= old + off - case["recent"]))
    # Guarded ones first, then by weight, ties by slot.
    order = torch.argsort(w, dim=-1, descending=True, stable=True)
    rank = torch.where(guarded, 0, torch.where(live, 1, 2))
    order = torch.gather(order, -1, torch.argsort(torch.gather(rank, -1, order), dim=-1, stable=True))
    place = torch.empty_like(order).scatter_(-1, order, torch.arange(T, device="cuda").expand_as(order))
    keep = place < m
    hole, move = (slot < m) & ~keep, (slot >= m) & keep
    movers = torch.argsort((~move).to(torch.int32), dim=-1, stable=True)
    nth = (torch.cumsum(hole.to(torch.int32), -1) - 1).clamp(min=0)
    src = torch.where(hole, torch.gather(movers, -1, nth), slot.long())
    s["w_out"].copy_(torch.where(slot < m, torch.gather(w, -1, src), torch.where(live, 0.0, s["w_out"])))
    s["p_out"].copy_(torch.where(slot < m, torch.gather(pos, -1, src), torch.where(live, -1, s["p_out"])))
    s["o_out"].copy_(s["offset"] + s["seq"] - m[:, 0, 0])
    heads = torch.arange(case["Hkv"], device="cuda")[:, None]
    spare = s["kp"].shape[1]                                # the page behind the pool takes what does not move
    to = torch.where(hole, torch.gather(s["table"], 1, (slot // ps).expand(case["B"], T).long())[:, None], spare).long()
    for x in (s["k_all"], s["v_all"]):
        for i in range(case["layers"]):
            page = torch.gather(s["table"], 1, (src[i] // ps).flatten(1)).view(src[i].shape).clamp(min=0).long()
            x[i, to[i], (slot % ps).long(), heads] = x[i, page, src[i] % ps, heads]
    return {"weights": s["w_out"], "positions": s["p_out"], "pos_offset": s["o_out"], "k_pages": s["kp"], "v_pages": s["vp"]}


# ---------------------------------------------------------------- one pass

def _run_own(s):
    import causal_gqa_flash_attention_gb300 as ne
    case = s["case"]
    if case["op"] == "shared":
        if "ws" not in s:
            s["ws"] = ne.alloc_paged_shared_workspace(case["B"], s["q"].shape[0], case["Hq"], case["Hkv"], case["D"])
        ne.paged_attn_shared(s["q"], s["kp"], s["vp"], s["table"], s["seq"], s["groups"], s["shared"], s["cu"],
                             max_new=case["n_max"], o=s["o"], lse=s["lse"], workspace=s["ws"])
        return {"o": s["o"], "lse": s["lse"]}
    if case["op"] == "weights":
        ne.paged_weights(s["q"], s["lse"], s["kp"], s["table"], s["seq"], s["weights"], s["cu"], max_new=case["n_max"],
                         weights_out=s["out"])
        return {"weights": s["out"]}
    if "ws" not in s:
        s["ws"] = ne.alloc_evict_workspace(case["layers"], case["B"], case["Hkv"], s["weights"].shape[-1])
    ne.pages_evict(s["weights"], s["positions"], s["offset"], s["table"], s["seq"], s["new"], s["kp"], s["vp"],
                   sink=case["sink"], recent=case["recent"], weights_out=s["w_out"], positions_out=s["p_out"],
                   pos_offset_out=s["o_out"], workspace=s["ws"])
    return {"weights": s["w_out"], "positions": s["p_out"], "pos_offset": s["o_out"], "k_pages": s["kp"], "v_pages": s["vp"]}


def run(state):
    if own:
        return _run_own(state)
    return {"shared": _shared_plain, "weights": _weights_plain, "evict": _evict_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    e, ps = (2 if case["dtype"] == "bf16" else 4), case["ps"]
    Hkv, D, B = case["Hkv"], case["D"], case["B"]
    if case["op"] == "evict":
        heads, total, moved = case["layers"] * Hkv, 0, 0.0
        for a, b, _, fresh in _evict_lens(case):
            b = min(a, b)
            total += a
            # Kept rows behind the new length: the newest, and of the others as many as kept ones are of all.
            guard = min(b, case["recent"])
            moved += min(a - b, guard if fresh else 0) + max(0, a - b - guard) * (b - guard) / max(1, a - guard)
        return {"bytes": int(heads * (16 * total + 4 * moved * D * e)) + 16 * B + 4 * sum(-(-x[0] // ps) for x in _evict_lens(case)),
                "flops": 0}
    Hq = case["Hq"]
    if case["op"] == "shared":
        groups, shared, n, ln = _shared_shape(case)
        first = [shared[sum(1 for g in groups[1:] if g <= b)] if b < groups[-1] else 0 for b in range(B)]
        N, cached = sum(n), sum(shared) + sum(x - f for x, f in zip(ln, first))
        pairs = sum(c * (x - c) + c * (c + 1) // 2 for c, x in zip(n, ln))
        return {"bytes": cached * 2 * Hkv * D * e + 2 * N * Hq * D * e + 4 * N * Hq + 4 * (cached // ps + 3 * B),
                "flops": 4 * D * Hq * pairs}
    n, ln = _lengths(case)
    N = sum(n)
    pairs = sum(c * (x - c) + c * (c + 1) // 2 for c, x in zip(n, ln))
    return {"bytes": sum(ln) * Hkv * (D * e + 8) + N * Hq * (D * e + 4) + 4 * (sum(ln) // ps + 3 * B), "flops": 2 * D * Hq * pairs}


# ---------------------------------------------------------------- the definition in 64 bits

def _sequence(case, s, b, n, ln, at, what):
    """Per head, 512 rows at a time: (row range, head, logits in 64 bits with -inf for unseen positions)."""
    ps, D, G = case["ps"], case["D"], case["Hq"] // case["Hkv"]
    k = s["kp"][s["table"][b, : -(-ln // ps)].long()].reshape(-1, case["Hkv"], D)[:ln].double()
    for i0 in range(0, n, 512):
        i1 = min(n, i0 + 512)
        gone = torch.arange(ln, device="cuda")[None] > (ln - n + torch.arange(i0, i1, device="cuda"))[:, None]
        for h in range(case["Hq"]):
            x = (s["q"][at + i0:at + i1, h].double() @ k[:, h // G].T) * D ** -0.5
            what(slice(at + i0, at + i1), h, x.masked_fill_(gone, -math.inf))


def exact(case, seed):
    if case["op"] == "evict":
        return None                                         # whole numbers, choices and copies
    s = prepare(case, seed)
    G, ps = case["Hq"] // case["Hkv"], case["ps"]
    n, ln = s["shape"][2:] if case["op"] == "shared" else (s["n"], s["len"])
    o, lse = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    got = s["out"].double() if case["op"] == "weights" else None
    at = 0
    for b in range(case["B"]):
        if case["op"] == "shared":
            v = s["vp"][s["table"][b, : -(-ln[b] // ps)].long()].reshape(-1, case["Hkv"], case["D"])[:ln[b]].double()

            def what(rows, h, x):
                z = torch.logsumexp(x, -1)
                lse[rows, h] = z
                o[rows, h] = torch.exp(x - z[:, None]) @ v[:, h // G]
        else:
            got[b, :, :ln[b]] = s["weights"][b, :, :ln[b]].double()

            def what(rows, h, x):
                got[b, h // G, :ln[b]] += torch.exp(x - s["lse"][rows, h].double()[:, None]).sum(0)
        _sequence(case, s, b, n[b], ln[b], at, what)
        at += n[b]
    return {"o": o, "lse": lse} if case["op"] == "shared" else {"weights": got}
