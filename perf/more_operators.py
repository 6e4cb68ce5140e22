"""Workloads of the operators around the attention calls: norm and rotation of
queries and keys (forward and backward), a paged key/value cache (writing it,
in 16 bits or quantised to 8, reading it back, attention of new tokens over
it), and the verification of drafted tokens.

`own` chooses between the plain form (elementary torch operations in 32 bits,
in 64 for angles and sampling) and this library's calls; both take what
prepare() made."""

import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
LOG2E = 1.4426950408889634
E_MIN, E_MAX = -64, 120  # exponents of a quantised row


def _rope(name, B, L, Hq, Hkv, D, rot, axes=1, dtype="bf16", norm=True, interleaved=False, packed=True, bwd=False):
    return {"name": name, "op": "rope", "B": B, "L": L, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot, "axes": axes, "dtype": dtype,
            "norm": norm, "interleaved": interleaved, "packed": packed, "bwd": bwd}


def _write(name, B, Hkv, T, cap, D, page, q8, dtype="bf16"):
    return {"name": name, "op": "write", "B": B, "Hkv": Hkv, "T": T, "cap": cap, "D": D, "page": page, "q8": q8, "dtype": dtype}


def _read(name, B, Hkv, cap, D, page, q8, dtype="bf16", ragged=False):
    return {"name": name, "op": "read", "B": B, "Hkv": Hkv, "cap": cap, "D": D, "page": page, "q8": q8, "dtype": dtype, "ragged": ragged}


def _paged(name, B, Hq, Hkv, T, cap, D, page, q8, dtype="bf16", ragged=False):
    return {"name": name, "op": "paged", "B": B, "Hq": Hq, "Hkv": Hkv, "T": T, "cap": cap, "D": D, "page": page, "q8": q8,
            "dtype": dtype, "ragged": ragged}


def _verify(name, B, T, V, ragged=False, greedy=False):
    return {"name": name, "op": "verify", "B": B, "T": T, "V": V, "ragged": ragged, "greedy": greedy}


def listed():
    return [
        # one decode step of 16 sequences: the new tokens' queries and keys out of a packed projection (latency)
        _rope("rope_b16_l1", 16, 1, 32, 8, 128, 128),
        # a video prompt of 8192 tokens: positions with time, height and width
        _rope("rope_video_l8192", 1, 8192, 32, 8, 128, 128, axes=3),
        # the benchmark's training step: gradients through norm and rotation
        _rope("rope_bwd_l8192", 1, 8192, 32, 8, 128, 128, bwd=True),
        # a decode step's keys and values quantised into the pages (latency)
        _write("write8_b16_t1", 16, 8, 1, 2048, 128, 16, True),
        # two prompts go into the pages, quantised
        _write("write8_b2_l2048", 2, 8, 2048, 2304, 128, 64, True),
        # a short cached prefix in 16 bits is read back (latency)
        _read("read_b1_k1000", 1, 8, 1000, 128, 16, False),
        # quantised prefixes of unequal lengths are read back before the rest of their prompts is processed
        _read("read8_b4_k8192_ragged", 4, 8, 8192, 128, 64, True, ragged=True),
        # one interactive user: a new token over a short context (latency)
        _paged("paged_b1_k1000", 1, 32, 8, 1, 1000, 128, 16, False),
        # a serving batch of unequal contexts over a quantised cache
        _paged("paged8_b16_k8192_ragged", 16, 32, 8, 1, 8192, 128, 64, True, ragged=True),
        # two long contexts, head dimension 256
        _paged("paged_b2_k131072_d256", 2, 16, 2, 1, 131072, 256, 128, False, dtype="fp16"),
        # one user's four drafts over a small vocabulary (latency)
        _verify("verify_b1_t4_v32768", 1, 4, 32768),
        # 64 sequences' eight drafts over the vocabulary of the loss benchmark
        _verify("verify_b64_t8_v151936", 64, 8, 151936, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "write", "read", "paged", "paged", "verify"])
    D = rng.choice([64, 96, 128, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 8])
    B = _log(rng, 1, 16)
    page = rng.choice([8, 16, 32, 64, 128, 256])
    q8 = rng.random() < 0.5
    if op == "rope":
        bwd = rng.random() < 0.5
        L = _log(rng, 1, max(1, 41_900_000 // (B * Hkv * (G + 1) * D)))
        rot = rng.choice([D, D, D // 2 if D % 32 == 0 else D])
        c = _rope("", B, min(L, 16384), Hkv * G, Hkv, D, rot, rng.choice([1, 1, 2, 3]), dtype, rng.random() < 0.7, rng.random() < 0.3,
                  rng.random() < 0.6, bwd)
    elif op == "write":
        T = _log(rng, 1, min(4096, 33_000_000 // (8 * B * Hkv * D)))
        c = _write("", B, Hkv, T, T + _log(rng, 16, 1024), D, page, q8, dtype)
    elif op == "read":
        c = _read("", B, Hkv, _log(rng, 16, min(65536, 33_000_000 // (B * Hkv * D))), D, page, q8, dtype, rng.random() < 0.5)
    elif op == "paged":
        T = rng.choice([1, 1, 1, 2, 3, 4])
        cap = _log(rng, 64, min(131072, 500_000_000 // (4 * D * B * Hkv)))
        c = _paged("", B, Hkv * G, Hkv, T, cap, D, page, q8, dtype, rng.random() < 0.6)
    else:
        T = rng.randint(1, 8)
        c = _verify("", _log(rng, 1, 64), T, _log(rng, 1000, 151936), rng.random() < 0.5, rng.random() < 0.3)
    c.pop("name")
    return c


def _pages(gen, cpu, c, s):
    """A pool with random pages given to each sequence, filled with keys and values."""
    B, Hkv, D, page = c["B"], c["Hkv"], c["D"], c["page"]
    most = -(-c["cap"] // page)
    n = B * most + 3
    s["table"] = torch.randperm(n, generator=cpu)[: B * most].view(B, most).to(torch.int32).cuda()
    for name in ("k", "v"):
        rows = torch.randn(n, Hkv, page, D, generator=gen, device="cuda", dtype=_DT[c["dtype"]])
        s[name + "_exp"] = None
        if c["q8"]:
            rows, s[name + "_exp"] = _quantise(rows)
        s[name + "_pages"] = rows


def _lens(cpu, c, most, least=1):
    """Tokens of each sequence: all the room, or spread between an eighth of it and all of it."""
    if not c["ragged"]:
        return torch.full((c["B"],), most, dtype=torch.int32)
    return torch.randint(max(least, most // 8), most + 1, (c["B"],), generator=cpu).to(torch.int32)


def prepare(case, seed):
    c = case
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B = c["B"]
    s = dict(c)
    if c["op"] == "verify":
        T, V = c["T"], c["V"]
        logits = torch.randn(B, T + 1, V, generator=gen, device="cuda") * 2
        s["target"] = torch.softmax(logits, -1)
        # the draft model's distribution is near the target's
        draft = torch.softmax(logits[:, :T] + torch.randn(B, T, V, generator=gen, device="cuda") * 0.6, -1)
        s["tokens"] = torch.multinomial(draft.view(B * T, V), 1, generator=gen).view(B, T).to(torch.int32)
        if c["greedy"]:
            draft, s["tokens"] = None, logits[:, :T].argmax(-1).to(torch.int32)
        s["draft"] = draft
        s["u"] = torch.rand(B, T, generator=gen, device="cuda")
        s["r"] = torch.rand(B, generator=gen, device="cuda")
        s["draft_len"] = (torch.randint(T // 2, T + 1, (B,), generator=cpu).to(torch.int32) if c["ragged"] else torch.full((B,), T, dtype=torch.int32)).cuda()
        s["accept_len"] = torch.empty(B, dtype=torch.int32, device="cuda")
        s["token"] = torch.empty(B, dtype=torch.int32, device="cuda")
        return s
    dt, Hkv, D = _DT[c["dtype"]], c["Hkv"], c["D"]

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dt)

    if c["op"] == "rope":
        L, Hq, half = c["L"], c["Hq"], c["rot"] // 2

        def rows():  # queries and keys: views of a packed projection [B, L, heads, D], or arrays of their own
            if c["packed"]:
                x = rand(B, L, Hq + 2 * Hkv, D).transpose(1, 2)
                return x[:, :Hq], x[:, Hq:Hq + Hkv]
            return rand(B, Hq, L, D), rand(B, Hkv, L, D)

        s["q"], s["k"] = rows()
        s["freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
        first = torch.randint(0, 32768, (1, B, 1), generator=cpu)
        if c["axes"] == 1:  # a running position
            s["pos"] = (first + torch.arange(L)).to(torch.int32).cuda()
            s["axis"] = None
        else:  # frames of a width x height grid; the pairs are shared out among the axes
            w = max(1, int(math.sqrt(L / 4)))
            i = torch.arange(L)
            grid = torch.stack([i // (w * w), i // w % w, i % w][: c["axes"]])[:, None]
            s["pos"] = (first + grid).to(torch.int32).cuda()
            s["axis"] = (torch.arange(half) * c["axes"] // half).to(torch.uint8).cuda()
        s["qw"] = s["kw"] = None
        if c["norm"]:
            s["qw"], s["kw"] = 1 + 0.2 * rand(D), 1 + 0.2 * rand(D)
        s["eps"] = 1e-6
        if c["bwd"]:
            s["dq_out"], s["dk_out"] = rand(B, Hq, L, D), rand(B, Hkv, L, D)
            s["dq"], s["dk"] = rows()
            s["dqw"] = torch.empty(D, device="cuda") if c["norm"] else None
            s["dkw"] = torch.empty(D, device="cuda") if c["norm"] else None
        else:
            s["q_out"], s["k_out"] = torch.empty(B, Hq, L, D, device="cuda", dtype=dt), torch.empty(B, Hkv, L, D, device="cuda", dtype=dt)
        return s
    _pages(gen, cpu, c, s)
    if c["op"] == "write":
        T = c["T"]
        s["k_new"], s["v_new"] = rand(B, Hkv, T, D), rand(B, Hkv, T, D)
        s["cache_len"] = torch.randint(0, c["cap"] - T + 1, (B,), generator=cpu).to(torch.int32).cuda()
        s["cache_len_out"] = torch.empty_like(s["cache_len"])
    elif c["op"] == "read":
        s["cache_len"] = _lens(cpu, c, c["cap"]).cuda()
        s["k"], s["v"] = rand(B, Hkv, c["cap"], D), rand(B, Hkv, c["cap"], D)
    else:
        T = c["T"]
        s["scale"] = float(np.float32(1.0 / math.sqrt(D)))
        s["q"] = rand(B, c["Hq"], T, D)
        s["cache_len"] = _lens(cpu, c, c["cap"], T).cuda()
        s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty(B, c["Hq"], T, device="cuda")
    return s


def run(state):
    s = state
    if own:
        return _run_own(s)
    if s["op"] == "rope":
        return _plain_rope_bwd(s) if s["bwd"] else _plain_rope(s)
    return {"write": _plain_write, "read": _plain_read, "paged": _plain_paged, "verify": _plain_verify}[s["op"]](s)


def _run_own(s):
    from bwd_flashattention_fwd_gb300 import gbattn

    if s["op"] == "rope":
        how = {"axis": s["axis"], "eps": s["eps"], "interleaved": s["interleaved"]}
        if not s["bwd"]:
            gbattn.attn_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["pos"], s["freq"], s["qw"], s["kw"], **how)
            return {"q": s["q_out"], "k": s["k_out"]}
        if "ws" not in s:  # kept with the state, as a training program keeps it
            s["ws"] = gbattn.qk_norm_rope_workspace(s["q"], s["k"])
        gbattn.attn_qk_norm_rope_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], s["pos"], s["freq"], s["dq"], s["dk"], s["qw"], s["kw"],
                                     s["dqw"], s["dkw"], s["ws"], **how)
        return {"dq": s["dq"], "dk": s["dk"], "dqw": s["dqw"], "dkw": s["dkw"]}
    if s["op"] == "write":
        gbattn.attn_paged_write(s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["table"], s["cache_len"], s["cache_len_out"],
                                k_exp=s["k_exp"], v_exp=s["v_exp"])
        return {"k": s["k_pages"], "v": s["v_pages"], "ke": s["k_exp"], "ve": s["v_exp"], "len": s["cache_len_out"]}
    if s["op"] == "read":
        gbattn.attn_paged_read(s["k_pages"], s["v_pages"], s["table"], s["cache_len"], s["k"], s["v"], k_exp=s["k_exp"], v_exp=s["v_exp"])
        return {"k": s["k"], "v": s["v"]}
    if s["op"] == "paged":
        if "ws" not in s:  # kept with the state, as a serving program keeps it
            s["ws"] = gbattn.paged_workspace(s["q"], s["k_pages"], s["table"])
        gbattn.attn_fwd_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["cache_len"], s["o"], s["lse"], s["ws"], s["scale"],
                              k_exp=s["k_exp"], v_exp=s["v_exp"])
        return {"o": s["o"], "lse": s["lse"]}
    gbattn.attn_draft_verify(s["target"], s["draft"], s["tokens"], s["u"], s["r"], s["accept_len"], s["token"], draft_len=s["draft_len"])
    return {"accept_len": s["accept_len"], "token": s["token"]}


# ---------------------------------------------------------------------------
# Plain forms.
# ---------------------------------------------------------------------------


def _turns(s):
    """cos and sin [B, 1, L, rot / 2] of every token's angles, from 64 bits."""
    pos = s["pos"].double()
    at = pos[0][..., None] if s["axis"] is None else pos[s["axis"].long()].permute(1, 2, 0)
    a = at * s["freq"].double()
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _rotate(x, cos, sin, rot, interleaved):
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_rope(s):
    cos, sin = _turns(s)
    out = {}
    for name, w in (("q", s["qw"]), ("k", s["kw"])):
        x = s[name].float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * w.float()
        s[name + "_out"].copy_(_rotate(x, cos, sin, s["rot"], s["interleaved"]))
        out[name] = s[name + "_out"]
    return out


def _plain_rope_bwd(s):
    cos, sin = _turns(s)
    out = {}
    for name, w, dw in (("q", s["qw"], s["dqw"]), ("k", s["kw"], s["dkw"])):
        g = _rotate(s["d" + name + "_out"].float(), cos, -sin, s["rot"], s["interleaved"])
        if w is not None:
            x = s[name].float()
            r = torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
            n = x * r
            dw.copy_((g * n).sum((0, 1, 2)))
            g = g * w.float()
            g = r * (g - n * (g * n).mean(-1, keepdim=True))
        s["d" + name].copy_(g)
        out["d" + name] = s["d" + name]
    return {**out, "dqw": s["dqw"], "dkw": s["dkw"]}


def _quantise(x):
    """Rows as e4m3 codes and one exponent e each: the least with max |x| <= 448 * 2^e, kept within E_MIN .. E_MAX."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0, e - 9 + (m > 0.875), torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn), e.to(torch.int8)


def _place(s):
    """Page and row of every new token [B, T]."""
    at = s["cache_len"].long()[:, None] + torch.arange(s["T"], device="cuda")
    return torch.gather(s["table"].long(), 1, at // s["page"]), at % s["page"]


def _plain_write(s):
    page, row = _place(s)
    for name in ("k", "v"):
        new, pool = s[name + "_new"], s[name + "_pages"]
        if s["q8"]:
            new, e = _quantise(new)
            s[name + "_exp"][page, :, row] = e.transpose(1, 2)
            new, pool = new.view(torch.uint8), pool.view(torch.uint8)
        pool[page, :, row] = new.transpose(1, 2)
    s["cache_len_out"].copy_(s["cache_len"] + s["T"])
    return {"k": s["k_pages"], "v": s["v_pages"], "ke": s["k_exp"], "ve": s["v_exp"], "len": s["cache_len_out"]}


def _gather(s, name):
    """Keys or values of all sequences [B, Hkv, most * page, D] in 32 bits."""
    table, pool, e = s["table"].long(), s[name + "_pages"], s[name + "_exp"]
    if e is None:
        x = pool[table].float()
    else:
        x = torch.ldexp(pool.view(torch.uint8)[table].view(torch.float8_e4m3fn).float(), e[table].int()[..., None])
    return x.transpose(1, 2).reshape(s["B"], s["Hkv"], -1, s["D"])


def _plain_read(s):
    live = (torch.arange(s["cap"], device="cuda") < s["cache_len"][:, None])[:, None, :, None]
    for name in ("k", "v"):
        s[name].copy_(torch.where(live, _gather(s, name)[:, :, : s["cap"]].to(s[name].dtype), s[name]))
    return {"k": s["k"], "v": s["v"]}


def _plain_paged(s):
    B, Hq, Hkv, T, D = s["B"], s["Hq"], s["Hkv"], s["T"], s["D"]
    k, v = _gather(s, "k"), _gather(s, "v")
    n = k.shape[2]
    last = s["cache_len"][:, None] - T + torch.arange(T, device="cuda")  # the last key that each row sees
    see = torch.arange(n, device="cuda") <= last[..., None]
    sc = (s["q"].float().view(B, Hkv, -1, D) @ k.transpose(-1, -2)).view(B, Hq, T, n) * (s["scale"] * LOG2E)
    sc = sc.masked_fill(~see[:, None], float("-inf"))
    top = sc.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp2(sc - top)
    tot = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, -1, n) @ v).view(B, Hq, T, D) / torch.where(tot > 0, tot, torch.ones_like(tot))
    lse = torch.where(tot > 0, top + torch.log2(tot), torch.full_like(tot, float("inf")))
    return {"o": o.to(s["q"].dtype), "lse": lse[..., 0].contiguous()}


def _plain_verify(s):
    B, T, V = s["B"], s["T"], s["V"]
    x, i = s["tokens"].long(), torch.arange(T, device="cuda")
    p = torch.gather(s["target"][:, :T], 2, x[..., None])[..., 0].double()
    q = torch.ones_like(p) if s["draft"] is None else torch.gather(s["draft"], 2, x[..., None])[..., 0].double()
    good = (s["u"].double() * q < p) & (i < s["draft_len"][:, None])
    n = good.long().cumprod(-1).sum(-1)
    b = torch.arange(B, device="cuda")
    rejected = n < s["draft_len"]
    row = s["target"][b, n].double()
    at = n.clamp(max=T - 1)
    if s["draft"] is None:
        less = torch.zeros_like(row).scatter_(1, x[b, at][:, None], float("inf"))
    else:
        less = s["draft"][b, at].double()
    left = torch.where(rejected[:, None], (row - less).clamp(min=0), row)
    left = torch.where(left.sum(-1, keepdim=True) > 0, left, row)
    upto = left.cumsum(-1)
    token = (upto <= s["r"].double()[:, None] * upto[:, -1:]).sum(-1).clamp(max=V - 1)
    s["accept_len"].copy_(n)
    s["token"].copy_(token)
    return {"accept_len": s["accept_len"], "token": s["token"]}


def work(case):
    c = case
    B = c["B"]
    if c["op"] == "verify":  # a row of the target and one of the draft for each sequence
        return {"bytes": B * (c["V"] * (4.0 if c["greedy"] else 8.0) + c["T"] * 16 + 12), "flops": 3.0 * B * c["V"]}
    Hkv, D = c["Hkv"], c["D"]
    if c["op"] == "rope":
        rows = B * c["L"] * (c["Hq"] + Hkv)
        passes = (3 if c["norm"] else 2) if c["bwd"] else 2
        return {"bytes": rows * D * 2.0 * passes + c["axes"] * B * c["L"] * 4, "flops": rows * D * (20.0 if c["bwd"] else 10.0)}
    held = D + 1 if c["q8"] else 2 * D
    if c["op"] == "write":
        return {"bytes": 2.0 * B * Hkv * c["T"] * (2 * D + held), "flops": 2.0 * B * Hkv * c["T"] * D}
    n = B * c["cap"] * (9 / 16 if c["ragged"] else 1)
    if c["op"] == "read":
        return {"bytes": 2.0 * n * Hkv * (2 * D + held), "flops": 2.0 * n * Hkv * D}
    return {"bytes": 2.0 * n * Hkv * held + B * c["Hq"] * c["T"] * (4 * D + 4), "flops": 4.0 * D * c["Hq"] * c["T"] * n}


# ---------------------------------------------------------------------------
# The operators from their definitions, in 64 bits.
# ---------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "write": _exact_write, "read": _exact_read, "paged": _exact_paged, "verify": _exact_verify}[s["op"]](s)


def _exact_rope(s):
    """Pairs as complex numbers: y = x e^{ia}; the gradient of the rotation is the conjugate's product."""
    axis = [0] * (s["rot"] // 2) if s["axis"] is None else s["axis"].tolist()
    angle = torch.stack([s["pos"][a].double() * float(f) for a, f in zip(axis, s["freq"].tolist())], -1)
    unit = torch.polar(torch.ones_like(angle), angle)[:, None]
    half, rot = s["rot"] // 2, s["rot"]
    d = torch.arange(half, device="cuda")
    one, two = (2 * d, 2 * d + 1) if s["interleaved"] else (d, d + half)

    def turn(x, by):
        z = torch.complex(x[..., one], x[..., two]) * by
        y = x.clone()
        y[..., one], y[..., two] = z.real, z.imag
        return y

    out = {}
    for name, w in (("q", s["qw"]), ("k", s["kw"])):
        x = s[name].double()
        rms = torch.sqrt((x * x).sum(-1, keepdim=True) / s["D"] + s["eps"])
        if not s["bwd"]:
            out[name] = turn(x / rms * w.double() if w is not None else x, unit)
            continue
        g = turn(s["d" + name + "_out"].double(), unit.conj())
        if w is None:
            out["d" + name], out["d" + name + "w"] = g, None
            continue
        out["d" + name + "w"] = (g * x / rms).sum((0, 1, 2))
        g = g * w.double()
        out["d" + name] = g / rms - x * (g * x).sum(-1, keepdim=True) / (s["D"] * rms ** 3)
    return out


def _e4m3(y):
    """|y| <= 448 rounded to the nearest value with four significant bits, spaced 2^-9 at least, ties to the even one."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def _exact_write(s):
    out = {"len": s["cache_len"] + s["T"], "ke": None, "ve": None}
    for name in ("k", "v"):
        pool = s[name + "_pages"].double()
        e = None if s[name + "_exp"] is None else s[name + "_exp"].clone()
        for b in range(s["B"]):
            n = int(s["cache_len"][b])
            at = torch.arange(n, n + s["T"], device="cuda")
            page, row = s["table"][b].long()[at // s["page"]], at % s["page"]
            x = s[name + "_new"][b].double()
            if e is not None:
                top = x.abs().amax(-1)
                k = torch.ceil(torch.log2(top / 448)).clamp(E_MIN, E_MAX)
                k = torch.where(top <= 448 * torch.exp2(k - 1), k - 1, k)
                k = torch.where(top > 448 * torch.exp2(k), k + 1, k).clamp(E_MIN, E_MAX)
                x = _e4m3(x / torch.exp2(k)[..., None])
                e[page, :, row] = k.transpose(0, 1).to(torch.int8)
            pool[page, :, row] = x.transpose(0, 1)
        out[name] = pool
        if e is not None:
            out[name + "e"] = e
    return out


def _exact_read(s):
    out = {}
    for name in ("k", "v"):
        x = s[name].double()
        for b in range(s["B"]):
            n = int(s["cache_len"][b])
            x[b, :, :n] = _exact_rows(s, name, b, n)
        out[name] = x
    return out


def _exact_rows(s, name, b, n):
    """Keys or values [Hkv, n, D] of sequence b."""
    at = torch.arange(n, device="cuda")
    page, row = s["table"][b].long()[at // s["page"]], at % s["page"]
    x = s[name + "_pages"]
    if s[name + "_exp"] is None:
        return x[page, :, row].double().transpose(0, 1)
    x = x.view(torch.uint8)[page, :, row].view(torch.float8_e4m3fn).double()
    return (x * torch.exp2(s[name + "_exp"][page, :, row].double())[..., None]).transpose(0, 1)


def _exact_paged(s):
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, math.inf, dtype=torch.float64, device="cuda")
    G, T = s["Hq"] // s["Hkv"], s["T"]
    for b in range(s["B"]):
        n = int(s["cache_len"][b])
        k, v = _exact_rows(s, "k", b, n), _exact_rows(s, "v", b, n)
        for t in range(T):
            m = n - T + 1 + t
            for h in range(s["Hkv"]):
                z = s["q"][b, h * G:(h + 1) * G, t].double() @ k[h, :m].T * s["scale"]
                o[b, h * G:(h + 1) * G, t] = torch.softmax(z, -1) @ v[h, :m]
                lse[b, h * G:(h + 1) * G, t] = torch.logsumexp(z, -1) / math.log(2.0)
    return {"o": o, "lse": lse}


def _exact_verify(s):
    accept, token = torch.zeros_like(s["accept_len"]), torch.zeros_like(s["token"])
    tokens, u, r, most = s["tokens"].tolist(), s["u"].tolist(), s["r"].tolist(), s["draft_len"].tolist()
    for b in range(s["B"]):
        n = 0
        while n < most[b]:
            x = tokens[b][n]
            q = 1.0 if s["draft"] is None else float(s["draft"][b, n, x])
            if not u[b][n] * q < float(s["target"][b, n, x]):
                break
            n += 1
        w = s["target"][b, n].double().cpu().numpy()
        if n < most[b]:
            left = w.copy()
            if s["draft"] is None:
                left[tokens[b][n]] = 0.0
            else:
                left = np.maximum(w - s["draft"][b, n].double().cpu().numpy(), 0.0)
            w = left if left.sum() > 0 else w
        upto = np.cumsum(w)
        accept[b], token[b] = n, int(np.searchsorted(upto, r[b] * upto[-1], side="right"))
    return {"accept_len": accept, "token": token}
