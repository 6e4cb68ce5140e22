"""Workloads of the cache operators: drafted-token (tree) attention over a
key/value cache, appending accepted drafts to it, accumulated attention weight
per cached key, and eviction by that weight.

`own` chooses between the plain form (elementary torch operations in 32 bits)
and this library's calls; both take what prepare() made."""

import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
LOG2E = 1.4426950408889634


def _tree(name, B, Hq, Hkv, T, Lk, D, dtype="bf16", ragged=False, chain=False):
    return {"name": name, "op": "tree", "B": B, "Hq": Hq, "Hkv": Hkv, "T": T, "Lk": Lk, "D": D, "dtype": dtype,
            "ragged": ragged, "chain": chain}


def _weight(name, B, Hq, Hkv, T, Lk, D, dtype="bf16", prompt=False):
    return {"name": name, "op": "weight", "B": B, "Hq": Hq, "Hkv": Hkv, "T": T, "Lk": Lk, "D": D, "dtype": dtype,
            "prompt": prompt}


def _append(name, B, Hkv, T, Lk, D, dtype="bf16", tree=False):
    return {"name": name, "op": "append", "B": B, "Hkv": Hkv, "T": T, "Lk": Lk, "D": D, "dtype": dtype, "tree": tree}


def _evict(name, B, Hkv, Lk, keep, recent, D, dtype="bf16", ragged=False):
    return {"name": name, "op": "evict", "B": B, "Hkv": Hkv, "Lk": Lk, "keep": keep, "recent": recent, "D": D,
            "dtype": dtype, "ragged": ragged}


def listed():
    return [
        # one interactive user: a draft tree of 8 tokens over a short context (latency)
        _tree("tree_b1_t8_k1000", 1, 32, 8, 8, 1000, 128),
        # four sequences, 8 drafts each, 8192 keys of context: the decode workload of the benchmark
        _tree("tree_b4_t8_k8192", 4, 32, 8, 8, 8192, 128),
        # a serving batch of unequal contexts and wide trees (an odd draft count, padded per sequence)
        _tree("tree_b16_t61_ragged", 16, 32, 8, 61, 8192, 128, ragged=True),
        # plain decode, one token, over a long context, head dimension 256
        _tree("decode_b2_t1_k131072_d256", 2, 16, 2, 1, 131072, 256, dtype="fp16", chain=True),
        # weights that one step's accepted drafts gave a short context (latency)
        _weight("weight_b1_t8_k1000", 1, 32, 8, 8, 1000, 128),
        # the same over 8192 keys for four sequences
        _weight("weight_b4_t8_k8192", 4, 32, 8, 8, 8192, 128),
        # a whole prompt's weights, before its cache is compressed for the first time
        _weight("weight_prompt_l8192", 1, 32, 8, 8192, 8192, 128, prompt=True),
        # a ragged prompt of equal head counts, head dimension 96
        _weight("weight_prompt_q1777_k2111_d96", 2, 16, 16, 1777, 2111, 96, dtype="fp16", prompt=True),
        # accepted drafts of a tree go into the cache (latency)
        _append("append_b4_t8", 4, 8, 8, 8192, 128, tree=True),
        # a prompt's keys and values go into the cache
        _append("append_prompt_b2_l2048", 2, 8, 2048, 2304, 128),
        # steady state: every 256 tokens a cache of 8448 slots goes back to 8192
        _evict("evict_b4_8448_to_8192", 4, 8, 8448, 8192, 512, 128),
        # a long prompt's cache is compressed to an eighth
        _evict("evict_b1_32768_to_4096", 1, 8, 32768, 4096, 256, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "weight", "weight", "append", "evict"])
    D = rng.choice([64, 96, 128, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 8])
    B = _log(rng, 1, 16)
    if op == "tree":
        T = _log(rng, 1, 64)
        most = min(131072, 536870912 // (4 * D * B * Hkv), 8_000_000_000 // (4 * B * Hkv * G * T))
        Lk = _log(rng, 64, most)
        return {k: v for k, v in _tree("", B, Hkv * G, Hkv, T, Lk, D, dtype, rng.random() < 0.6, T == 1 or rng.random() < 0.3).items() if k != "name"}
    if op == "weight":
        if rng.random() < 0.5:
            B = _log(rng, 1, 4)
            T = _log(rng, 100, min(8192, int(math.sqrt(2_000_000_000 / (B * Hkv * G)) * 0.8)))
            Lk = T + rng.choice([0, 0, rng.randrange(1, T)]) if T < 4000 else T
            return {k: v for k, v in _weight("", B, Hkv * G, Hkv, T, Lk, D, dtype, True).items() if k != "name"}
        T = _log(rng, 1, 64)
        most = min(131072, 536870912 // (4 * D * B * Hkv), 8_000_000_000 // (4 * B * Hkv * G * T))
        Lk = _log(rng, 64, most)
        return {k: v for k, v in _weight("", B, Hkv * G, Hkv, min(T, Lk), Lk, D, dtype).items() if k != "name"}
    if op == "append":
        tree = rng.random() < 0.5
        T = _log(rng, 1, 64) if tree else _log(rng, 1, 4096)
        return {k: v for k, v in _append("", B, Hkv, T, T + _log(rng, 64, 16384), D, dtype, tree).items() if k != "name"}
    Lk = _log(rng, 256, min(131072, 268435456 // (4 * D * B * Hkv)))
    keep = max(1, int(Lk * rng.choice([0.1, 0.25, 0.5, 0.9, 0.97])))
    return {k: v for k, v in _evict("", B, Hkv, Lk, keep, int(keep * rng.choice([0.0, 0.05, 0.3])), D, dtype, rng.random() < 0.5).items() if k != "name"}


def _trees(gen, B, T):
    """Ancestor masks (uint8 [B, T, T], a draft sees itself too) of random trees: each draft's parent is an earlier draft or the context."""
    parent = (torch.rand(B, T, generator=gen) * (torch.arange(T) + 1)).long() - 1
    mask = torch.zeros(B, T, T, dtype=torch.uint8)
    rows = torch.arange(B)
    for t in range(T):
        p = parent[:, t]
        mask[:, t] = mask[rows, p.clamp(min=0)] * (p >= 0).to(torch.uint8)[:, None]
        mask[:, t, t] = 1
    return mask, parent


def _lens(gen, c, room=0):
    """Tokens in the cache: all of it, or spread between an eighth of it and all of it."""
    n = c["Lk"] - room
    if not c.get("ragged"):
        return torch.full((c["B"],), n, dtype=torch.int32)
    lo = max(1, n // 8)
    return torch.randint(lo, n + 1, (c["B"],), generator=gen).to(torch.int32)


def prepare(case, seed):
    c = case
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, B, Hkv, D, Lk = _DT[c["dtype"]], c["B"], c["Hkv"], c["D"], c["Lk"]
    s = dict(c)

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dt)

    if c["op"] in ("tree", "weight"):
        s["scale"] = float(np.float32(1.0 / math.sqrt(D)))
    if c["op"] == "tree":
        T = c["T"]
        s["q"], s["k"], s["v"] = rand(B, c["Hq"], T, D), rand(B, Hkv, Lk, D), rand(B, Hkv, Lk, D)
        s["k_new"], s["v_new"] = rand(B, Hkv, T, D), rand(B, Hkv, T, D)
        s["cache_len"] = _lens(cpu, c).cuda()
        tl = torch.full((B,), T, dtype=torch.int32)
        if c["ragged"]:
            tl = torch.randint(max(1, T // 2), T + 1, (B,), generator=cpu).to(torch.int32)
        s["tree_len"] = tl.cuda()
        s["mask"] = None if c["chain"] else _trees(cpu, B, T)[0].cuda()
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(B, c["Hq"], T, device="cuda")
    elif c["op"] == "weight":
        T = c["T"]
        s["q"], s["k"] = rand(B, c["Hq"], T, D), rand(B, Hkv, Lk, D)
        if c["prompt"]:
            s["limit"] = None
            lim = (torch.arange(T, device="cuda") + (Lk - T + 1)).expand(B, T)
        else:  # the drafts on an accepted path see the context and the path before them; the others are rejected
            depth = torch.zeros(B, T, dtype=torch.int32)
            for b in range(B):
                n = int(torch.randint(1, T + 1, (1,), generator=cpu))
                on = torch.randperm(T, generator=cpu)[:n].sort().values
                depth[b, on] = torch.arange(Lk - n + 1, Lk + 1, dtype=torch.int32)
            s["limit"] = lim = depth.cuda()
        # the log-sum-exp that the attention over the same keys gave
        qf, kf = s["q"].float().view(B, Hkv, -1, D), s["k"].float()
        sc = qf @ kf.transpose(-1, -2)
        sc *= s["scale"] * LOG2E
        see = torch.arange(Lk, device="cuda")[None, None, :] < lim[:, :, None].clamp(min=1)
        sc.view(B, c["Hq"], T, Lk).masked_fill_(~see[:, None], float("-inf"))
        top = sc.amax(-1, keepdim=True)
        sc -= top
        lse = torch.log2(sc.exp2_().sum(-1)) + top[..., 0]
        s["lse"] = lse.view(B, c["Hq"], T).contiguous()
        del sc
        s["weight"] = torch.rand(B, Hkv, Lk, generator=gen, device="cuda") * 4
        s["weight_out"] = torch.empty_like(s["weight"])
    elif c["op"] == "append":
        T = c["T"]
        s["k"], s["v"], s["k_new"], s["v_new"] = rand(B, Hkv, Lk, D), rand(B, Hkv, Lk, D), rand(B, Hkv, T, D), rand(B, Hkv, T, D)
        s["cache_len"] = torch.randint(0, Lk - T + 1, (B,), generator=cpu).to(torch.int32).cuda()
        s["seen"] = s["cache_len"] + 1000
        path = torch.zeros(B, T, dtype=torch.int32)
        n = torch.full((B,), T, dtype=torch.int32)
        if c["tree"]:
            for b in range(B):
                n[b] = int(torch.randint(1, T + 1, (1,), generator=cpu))
                path[b, : n[b]] = torch.randperm(T, generator=cpu)[: n[b]].sort().values.to(torch.int32)
        s["path"] = path.cuda() if c["tree"] else None
        s["accept_len"] = n.cuda()
        s["pos"] = torch.zeros(B, Hkv, Lk, dtype=torch.int32, device="cuda")
        s["limit"] = torch.empty(B, T, dtype=torch.int32, device="cuda")
        s["cache_len_out"], s["seen_out"] = torch.empty_like(s["cache_len"]), torch.empty_like(s["seen"])
    else:
        s["k"], s["v"] = rand(B, Hkv, Lk, D), rand(B, Hkv, Lk, D)
        s["cache_len"] = _lens(cpu, c).cuda()
        s["seen"] = s["cache_len"] + 5000
        # accumulated weights are heavy-tailed: a few keys draw most of the attention
        s["weight"] = torch.randn(B, Hkv, Lk, generator=gen, device="cuda").mul_(2).exp_()
        # a cache that has been through evictions: positions are those of kept tokens, slots in no order
        s["pos"] = (torch.rand(B, Hkv, Lk, generator=gen, device="cuda").argsort(-1) * 1.0).to(torch.int32) + (s["seen"] - Lk)[:, None, None]
        s["weight_out"], s["pos_out"] = torch.empty_like(s["weight"]), torch.empty_like(s["pos"])
        s["cache_len_out"] = torch.empty_like(s["cache_len"])
    return s


def run(state):
    s = state
    if own:
        return _run_own(s)
    return {"tree": _plain_tree, "weight": _plain_weight, "append": _plain_append, "evict": _plain_evict}[s["op"]](s)


def _run_own(s):
    from bwd_flashattention_fwd_gb300 import gbattn

    if "ws" not in s:  # kept with the state, as a serving program keeps it
        make = {"tree": lambda: gbattn.tree_workspace(s["q"], s["k"]), "weight": lambda: gbattn.key_weight_workspace(s["q"], s["k"]),
                "append": lambda: None, "evict": lambda: gbattn.evict_workspace(s["k"])}
        s["ws"] = make[s["op"]]()
    if s["op"] == "tree":
        gbattn.attn_fwd_tree(s["q"], s["k"], s["v"], s["k_new"], s["v_new"], s["cache_len"], s["o"], s["lse"], s["ws"], s["scale"],
                             tree_mask=s["mask"], tree_len=s["tree_len"])
        return {"o": s["o"], "lse": s["lse"]}
    if s["op"] == "weight":
        gbattn.attn_key_weight(s["q"], s["k"], s["lse"], s["weight"], s["weight_out"], s["ws"], s["scale"], causal=s["prompt"], limit=s["limit"])
        return {"weight": s["weight_out"]}
    if s["op"] == "append":
        gbattn.attn_cache_append(s["k_new"], s["v_new"], s["k"], s["v"], s["cache_len"], s["accept_len"], s["cache_len_out"], path=s["path"],
                                 pos=s["pos"], seen=s["seen"], seen_out=s["seen_out"], limit=s["limit"])
        return {"k": s["k"], "v": s["v"], "pos": s["pos"], "len": s["cache_len_out"], "seen": s["seen_out"], "limit": s["limit"]}
    gbattn.attn_cache_evict(s["k"], s["v"], s["weight"], s["pos"], s["cache_len"], s["seen"], s["weight_out"], s["pos_out"], s["cache_len_out"],
                            s["ws"], s["keep"], s["recent"])
    return {"k": s["k"], "v": s["v"], "weight": s["weight_out"], "pos": s["pos_out"], "len": s["cache_len_out"]}


def _plain_tree(s):
    B, Hq, Hkv, T, Lk, D = s["B"], s["Hq"], s["Hkv"], s["T"], s["Lk"], s["D"]
    dev = s["q"].device
    q = s["q"].float().view(B, Hkv, -1, D)
    keys = torch.cat([s["k"], s["k_new"]], 2).float()
    vals = torch.cat([s["v"], s["v_new"]], 2).float()
    t = torch.arange(T, device=dev)
    among = (t[None, :] <= t[:, None])[None].expand(B, T, T) if s["mask"] is None else s["mask"] != 0
    among = among & (t[None, None, :] < s["tree_len"][:, None, None])
    context = (torch.arange(Lk, device=dev)[None, :] < s["cache_len"][:, None])[:, None].expand(B, T, Lk)
    see = torch.cat([context, among], 2) & (t[None, :] < s["tree_len"][:, None])[:, :, None]
    sc = (q @ keys.transpose(-1, -2)).view(B, Hq, T, Lk + T) * (s["scale"] * LOG2E)
    sc = sc.masked_fill(~see[:, None], float("-inf"))
    top = sc.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp2(sc - top)
    tot = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, -1, Lk + T) @ vals).view(B, Hq, T, D) / torch.where(tot > 0, tot, torch.ones_like(tot))
    lse = torch.where(tot > 0, top + torch.log2(tot), torch.full_like(tot, float("inf")))
    return {"o": o.to(s["q"].dtype), "lse": lse[..., 0].contiguous()}


def _plain_weight(s):
    B, Hq, Hkv, T, Lk, D = s["B"], s["Hq"], s["Hkv"], s["T"], s["Lk"], s["D"]
    dev = s["q"].device
    sc = (s["q"].float().view(B, Hkv, -1, D) @ s["k"].float().transpose(-1, -2)).view(B, Hq, T, Lk)
    p = torch.exp2(sc * (s["scale"] * LOG2E) - s["lse"][..., None])
    lim = (torch.arange(T, device=dev) + (Lk - T + 1)).expand(B, T) if s["limit"] is None else s["limit"]
    see = torch.arange(Lk, device=dev)[None, None, :] < lim[:, :, None]
    p = torch.where(see[:, None], p, torch.zeros((), device=dev))
    return {"weight": s["weight"] + p.view(B, Hkv, -1, Lk).sum(2)}


def _plain_append(s):
    B, Hkv, T, Lk, D = s["B"], s["Hkv"], s["T"], s["Lk"], s["D"]
    dev = s["k"].device
    i = torch.arange(T, device=dev)
    n, length = s["accept_len"].long(), s["cache_len"].long()
    src = i.expand(B, T) if s["path"] is None else s["path"].long()
    # the draft that lands in each cache slot, -1 where none does
    depth = torch.arange(Lk, device=dev)[None, :] - length[:, None]
    lands = (depth >= 0) & (depth < n[:, None])
    row = torch.gather(src, 1, depth.clamp(0, T - 1))
    at = row[:, None, :, None].expand(B, Hkv, Lk, D)
    put = lands[:, None, :, None]
    k = torch.where(put, torch.gather(s["k_new"], 2, at), s["k"])
    v = torch.where(put, torch.gather(s["v_new"], 2, at), s["v"])
    pos = torch.where(lands[:, None], (s["seen"][:, None].long() + depth)[:, None].int(), s["pos"])
    hit = (src[:, :, None] == i[None, None, :]) & (i[None, :, None] < n[:, None, None]) if s["path"] is not None else None
    if hit is None:
        limit = torch.where(i[None] < n[:, None], length[:, None] + i[None] + 1, torch.zeros((), dtype=torch.long, device=dev))
    else:
        limit = torch.where(hit, length[:, None, None] + i[None, :, None] + 1, torch.zeros((), dtype=torch.long, device=dev)).amax(1)
    return {"k": k, "v": v, "pos": pos, "len": (length + n).int(), "seen": (s["seen"].long() + n).int(), "limit": limit.int()}


def _plain_evict(s):
    B, Hkv, Lk, D, keep = s["B"], s["Hkv"], s["Lk"], s["D"], s["keep"]
    dev = s["k"].device
    slot = torch.arange(Lk, device=dev)[None, None]
    length = s["cache_len"].long()[:, None, None]
    live = (slot < length).expand(B, Hkv, Lk)
    rank = live.long() + (live & (s["pos"] >= (s["seen"] - s["recent"])[:, None, None])).long()
    # heaviest first, lowest slot first among equals; then the recent ones before all
    by = torch.sort(s["weight"], dim=-1, descending=True, stable=True).indices
    by = torch.gather(by, -1, torch.sort(torch.gather(rank, -1, by), dim=-1, descending=True, stable=True).indices)
    kept = torch.zeros(B, Hkv, Lk, dtype=torch.bool, device=dev).scatter_(-1, by[..., :keep], True) & live
    hole = live & ~kept & (slot < keep)
    mover = kept & (slot >= keep)
    spot = torch.zeros(B, Hkv, Lk + 1, dtype=torch.long, device=dev)
    spot.scatter_(-1, torch.where(mover, mover.long().cumsum(-1) - 1, Lk), slot.expand(B, Hkv, Lk))
    src = torch.where(hole, torch.gather(spot, -1, (hole.long().cumsum(-1) - 1).clamp(min=0)), slot)[..., :keep]
    at = src[..., None].expand(B, Hkv, keep, D)
    s["k"][:, :, :keep] = torch.gather(s["k"], 2, at)
    s["v"][:, :, :keep] = torch.gather(s["v"], 2, at)
    new = length.clamp(max=keep)
    weight = torch.zeros_like(s["weight"])
    weight[..., :keep] = torch.where(slot[..., :keep] < new, torch.gather(s["weight"], -1, src), weight[..., :keep])
    pos = torch.full_like(s["pos"], -1)
    pos[..., :keep] = torch.where(slot[..., :keep] < new, torch.gather(s["pos"], -1, src), pos[..., :keep])
    return {"k": s["k"], "v": s["v"], "weight": weight, "pos": pos, "len": new[:, 0, 0].int()}


def work(case):
    c = case
    B, Hkv, Lk, D = c["B"], c["Hkv"], c["Lk"], c["D"]
    if c["op"] == "tree":
        T, Hq = c["T"], c["Hq"]
        n = Lk * (9 / 16 if c["ragged"] else 1)  # mean tokens in the cache
        t = T * (3 / 4 if c["ragged"] else 1)
        return {"bytes": B * Hkv * (n + t) * D * 4 + B * Hq * T * (D * 4 + 4), "flops": 4.0 * D * B * Hq * t * (n + t / 2)}
    if c["op"] == "weight":
        T, Hq = c["T"], c["Hq"]
        pairs = T * (Lk - T) + T * (T + 1) / 2 if c["prompt"] else (T / 2) * Lk
        return {"bytes": B * Hkv * Lk * (D * 2 + 8) + B * Hq * T * (D * 2 + 4), "flops": 2.0 * D * B * Hq * pairs}
    if c["op"] == "append":
        n = c["T"] / 2 if c["tree"] else c["T"]
        return {"bytes": B * Hkv * n * (D * 8 + 4) + B * c["T"] * 8, "flops": 0.0}
    n = Lk * (9 / 16 if c["ragged"] else 1)
    moves = c["keep"] * max(0.0, n - c["keep"]) / n
    return {"bytes": B * Hkv * (n * 8 + Lk * 8 + moves * D * 8), "flops": 0.0}


# ---------------------------------------------------------------------------
# The operators from their definitions, in 64 bits.
# ---------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_tree, "weight": _exact_weight, "append": _exact_append, "evict": _exact_evict}[s["op"]](s)


def _exact_tree(s):
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, math.inf, dtype=torch.float64, device="cuda")
    G, T = s["Hq"] // s["Hkv"], s["T"]
    for b in range(s["B"]):
        n, m = int(s["cache_len"][b]), int(s["tree_len"][b])
        among = torch.ones(T, T, device="cuda").tril() if s["mask"] is None else s["mask"][b]
        bar = torch.zeros(m, n + m, dtype=torch.float64, device="cuda")
        bar[:, n:][among[:m, :m] == 0] = -math.inf
        for h in range(s["Hkv"]):
            kk = torch.cat([s["k"][b, h, :n], s["k_new"][b, h, :m]]).double()
            vv = torch.cat([s["v"][b, h, :n], s["v_new"][b, h, :m]]).double()
            z = s["q"][b, h * G:(h + 1) * G, :m].double() @ kk.T * s["scale"] + bar
            o[b, h * G:(h + 1) * G, :m] = torch.softmax(z, -1) @ vv
            lse[b, h * G:(h + 1) * G, :m] = torch.logsumexp(z, -1) / math.log(2.0)
    return {"o": o, "lse": lse}


def _exact_weight(s):
    G, T, Lk = s["Hq"] // s["Hkv"], s["T"], s["Lk"]
    out = s["weight"].double()
    j = torch.arange(Lk, device="cuda")
    for b in range(s["B"]):
        lim = torch.arange(Lk - T + 1, Lk + 1, device="cuda") if s["limit"] is None else s["limit"][b]
        for hq in range(s["Hq"]):
            z = s["q"][b, hq].double() @ s["k"][b, hq // G].double().T * s["scale"]
            w = torch.exp(z - (s["lse"][b, hq].double() * math.log(2.0))[:, None])
            out[b, hq // G] += (w * (j[None, :] < lim[:, None])).sum(0)
    return {"weight": out}


def _exact_append(s):
    k, v, pos = s["k"].double(), s["v"].double(), s["pos"].clone()
    length, n = s["cache_len"].tolist(), s["accept_len"].tolist()
    limit = torch.zeros_like(s["limit"])
    for b in range(s["B"]):
        rows = list(range(n[b])) if s["path"] is None else s["path"][b, : n[b]].tolist()
        k[b, :, length[b]:length[b] + n[b]] = s["k_new"][b][:, rows].double()
        v[b, :, length[b]:length[b] + n[b]] = s["v_new"][b][:, rows].double()
        first = int(s["seen"][b])
        pos[b, :, length[b]:length[b] + n[b]] = torch.arange(first, first + n[b], device="cuda", dtype=torch.int32)
        limit[b, rows] = torch.arange(length[b] + 1, length[b] + n[b] + 1, device="cuda", dtype=torch.int32)
    return {"k": k, "v": v, "pos": pos, "len": s["cache_len"] + s["accept_len"], "seen": s["seen"] + s["accept_len"], "limit": limit}


def _exact_evict(s):
    B, Hkv, Lk, keep, recent = s["B"], s["Hkv"], s["Lk"], s["keep"], s["recent"]
    k, v = s["k"].double(), s["v"].double()
    w, p = s["weight"].double().cpu().numpy(), s["pos"].cpu().numpy()
    weight, pos = np.zeros_like(w), np.full_like(p, -1)
    length, seen = s["cache_len"].tolist(), s["seen"].tolist()
    for b in range(B):
        n = length[b]
        for h in range(Hkv):
            if n <= keep:
                weight[b, h, :n], pos[b, h, :n] = w[b, h, :n], p[b, h, :n]
                continue
            late = p[b, h, :n] >= seen[b] - recent
            best = np.lexsort((np.arange(n), -w[b, h, :n], ~late))[:keep]
            stay = np.sort(best)
            free = np.setdiff1d(np.arange(keep), stay)
            move = stay[stay >= keep]
            src = np.arange(keep)
            src[free] = move
            weight[b, h, :keep], pos[b, h, :keep] = w[b, h, src], p[b, h, src]
            to, fr = torch.from_numpy(free).cuda(), torch.from_numpy(move).cuda()
            k[b, h, to], v[b, h, to] = k[b, h, fr], v[b, h, fr]
    return {"k": k, "v": v, "weight": torch.from_numpy(weight), "pos": torch.from_numpy(pos), "len": torch.tensor([min(n, keep) for n in length], dtype=torch.int32)}
