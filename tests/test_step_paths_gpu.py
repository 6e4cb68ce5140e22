"""GPU parity of the calls around attention on the paths that only larger
inputs reach, and at values that only some rows see: equal pieces of the paged
attention with both joins and several blocks of rows, exponents of quantised
values at both ends of their range, several tables of sines in a CTA of the
rotation, elements that are not turned, probabilities that are none, streams.

Tolerances as in test_step_ops_gpu.py, but for what a test says itself.
Launch shapes are those of a GPU with 152 SMs (the launcher's rules are in
sizes, so another count moves a case to another path, not to another result)."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle.step as S
import test_step_ops_gpu as ops
from bwd_flashattention_fwd_gb300 import gbattn
from bwd_flashattention_fwd_gb300.inputs import to_f64
from test_step_ops_gpu import BF, F8, HF, U, X, i32, make_pool, ok, pool64, rand, run_paged, within

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_flashattention_fwd_gb300 import build

    build.build()
    gbattn.load_library()


def roomy(gen, B, page, lens, room, order="random"):
    """A table with `room` tokens for each sequence whose pages past the lengths are holes, and the pool's size."""
    need = [-(-max(n, 0) // page) for n in lens]
    total = sum(need)
    pages = torch.randperm(total, generator=gen) if order == "random" else torch.arange(total)
    table, at = torch.full((B, room // page), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = pages[at:at + n].to(torch.int32)
        at += n
    return table, total + 1


def lengths(kind, B, top):
    if kind == "ragged":  # from nothing to `top`
        return [(i * 97 + 31) * top // 1009 % (top + 1) for i in range(B)]
    if kind == "short":  # long ones with runs of short and empty ones between them: pieces that hold whole heads
        return [top if i % 7 == 0 else (0, 1, 5, 70)[i % 4] for i in range(B)]
    return [top - 13 * i for i in range(B)]


# --- the paged attention's pieces ---------------------------------------------


PIECES = [
    # B, Hq, Hkv, T, D, page, top, lengths, dtype: with room for 40 times top, so pieces; the join's warps a row and the blocks of rows
    (16, 16, 4, 1, 64, 16, 400, "ragged", BF),    # 4 rows; 1 warp
    (16, 16, 4, 1, 128, 16, 400, "ragged", HF),   # 4 rows; 1 warp
    (16, 12, 4, 4, 96, 8, 300, "ragged", BF),     # 12 rows; 1 warp
    (16, 16, 4, 3, 128, 32, 300, "ragged", BF),   # 12 rows; 1 warp
    (16, 32, 4, 4, 128, 16, 300, "ragged", BF),   # 32 rows; 1 warp
    (16, 32, 4, 4, 64, 16, 300, "ragged", HF),    # 32 rows; 1 warp
    (48, 16, 8, 1, 128, 16, 500, "short", BF),    # several heads in a piece
    (48, 8, 8, 1, 64, 64, 500, "short", HF),
    (40, 24, 8, 4, 96, 16, 300, "short", BF),     # the same with 12 rows
    (30, 20, 10, 1, 256, 32, 300, "short", BF),
    (3, 32, 4, 5, 64, 16, 700, "near", BF),       # 40 rows in 2 blocks; 1 warp
    (2, 16, 2, 16, 128, 16, 500, "near", BF),     # 128 rows in 4 blocks; 1 warp
    (2, 12, 2, 11, 96, 16, 500, "near", HF),      # 66 rows in 3 blocks; 8 warps from here on
    (5, 16, 2, 3, 256, 32, 300, "near", BF),      # 24 rows in 2 blocks of 16
    (2, 16, 2, 8, 256, 8, 300, "near", HF),       # 64 rows in 4 blocks of 16
    (2, 8, 2, 1, 256, 64, 2500, "near", HF),      # few heads
    (1, 32, 1, 1, 128, 16, 2500, "near", BF),     # one head of 32 rows
    (1, 10, 1, 1, 64, 16, 3000, "near", BF),
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("case", PIECES)
def test_pieces(case, q8):
    B, Hq, Hkv, T, D, page, top, kind, dt = case
    gen = torch.Generator().manual_seed(41)
    lens = lengths(kind, B, top)
    table, n_pages = roomy(gen, B, page, lens, 40 * top // page * page)
    pool = make_pool(gen, n_pages, Hkv, page, D, dt, q8)
    ops.stale(pool, table, page, lens)
    q, scale = rand(gen, (B, Hq, T, D), dt), float(np.float32(1 / np.sqrt(D)))
    got = run_paged(q, pool, table.cuda(), i32(lens), scale)
    again = run_paged(q, pool, table.cuda(), i32(lens), scale)
    ok()
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    ops.check_paged(q, pool, table[:, :-(-max(lens) // page)], page, lens, scale, got)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_room_within_each_elements_bound(D, q8):
    """The same tokens in a small table (a cluster per head) and in a large one (pieces and a join): both within their
    elements' bounds."""
    gen = torch.Generator().manual_seed(42)
    B, Hq, Hkv, page, lens = 2, 8, 2, 16, [300, 7]
    table, n_pages = roomy(gen, B, page, lens, 304)
    wide = torch.full((B, 20000), -1, dtype=torch.int32)
    wide[:, :19] = table
    pool, q = make_pool(gen, n_pages, Hkv, page, D, BF, q8), rand(gen, (B, Hq, 1, D), BF)
    for t in (table, wide):
        got = run_paged(q, pool, t.cuda(), i32(lens), 0.09)
        ok()
        ops.check_paged(q, pool, table, page, lens, 0.09, got)


def test_cached_prefix_within_each_elements_bound():
    """One new token over pages, and by attn_fwd_ex over the same pages read back: both within the elements' bounds of the
    same definition (attn_fwd_ex rounds P to bf16, over quantised pages attn_fwd_paged to fp16)."""
    gen = torch.Generator().manual_seed(43)
    B, Hq, Hkv, D, page, per_seq, n = 2, 8, 2, 128, 16, 12, 180
    pool = make_pool(gen, B * per_seq, Hkv, page, D, BF, True)
    table = torch.randperm(B * per_seq, generator=gen).view(B, per_seq).to(torch.int32)
    q = rand(gen, (B, Hq, 1, D), BF)
    o, lse = run_paged(q, pool, table.cuda(), i32([n, n]), 0.09)
    k, v = (torch.zeros(B, Hkv, per_seq * page, D, dtype=BF, device="cuda")[:, :, :n] for _ in range(2))
    gbattn.attn_paged_read(pool[0], pool[1], table.cuda(), i32([n, n]), k, v, k_exp=pool[2], v_exp=pool[3])
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    gbattn.attn_fwd_ex(q, k, v, o2, lse2, 0.09, True)
    ok()
    ops.check_paged(q, pool, table, page, [n, n], 0.09, (o, lse))
    ref, lref, mag = S.paged_attention(to_f64(q), *(pool64(t) for t in pool[:2]), *(t.cpu().numpy() for t in pool[2:]), table.numpy(), page, [n, n], 0.09)
    # test_parity_gpu.py's roundings for one row: P's 2^-8, and O's
    within(to_f64(o2), ref, (2.0 ** -8 + 2.0 ** -12) * mag + U[BF] * np.abs(ref), "O of attn_fwd_ex")
    within(to_f64(lse2), lref, 1e-4, "lse of attn_fwd_ex")


@pytest.mark.parametrize("q8", [False, True])
def test_two_streams_over_pieces(q8):
    """Two calls at once that both need their workspaces, with different queries: the same bits as alone."""
    gen = torch.Generator().manual_seed(44)
    B, Hq, Hkv, D, page = 12, 16, 4, 128, 16
    lens = [2000 - 150 * i for i in range(B)]
    table, n_pages = roomy(gen, B, page, lens, 20000)
    pool, table = make_pool(gen, n_pages, Hkv, page, D, BF, q8), table.cuda()
    q = [rand(gen, (B, Hq, 1, D), BF) for _ in range(2)]
    ws = [gbattn.paged_workspace(q[0], pool[0], table) for _ in range(2)]
    want = [run_paged(x, pool, table, i32(lens), 0.1, w) for x, w in zip(q, ws)]
    ok()
    assert not torch.equal(want[0][0], want[1][0])
    streams, n = [torch.cuda.Stream() for _ in range(2)], i32(lens)
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(run_paged(q[i], pool, table, n, 0.1, ws[i]))
    ok()
    for runs, w in zip(got, want):
        for a in runs:
            assert torch.equal(a[0], w[0]) and torch.equal(a[1], w[1])


# --- exponents of quantised values at both ends of their range ------------------


def check_wide(q, pool, table, page, lens, scale, got):
    """As check_paged, with one more term: a score s carries its value's exponent through three sums (s + e, less the
    row's reference, less e), each rounded to 2^-24 of at most E = 2 (max |e| + max |s| log2e + 32): a probability is off by a
    factor within 1 +- 3 ln2 E x more.  What P's type rounds to nothing is 2^-40 of the row's largest product of probability and
    scale, 448 2^e of which some element has half (a row of zeros: 2^-55)."""
    k, v, ke, ve = pool
    D, dt, n = q.shape[-1], q.dtype, max(lens)
    e = [t.cpu().numpy() for t in (ke, ve)]
    ref, lref, mag = S.paged_attention(to_f64(q), pool64(k), pool64(v), *e, table.numpy(), page, lens, scale)
    used = np.unique(table.numpy())
    used = used[used >= 0]
    kk = pool64(k)[used] * 2.0 ** e[0][used][..., None].astype(float)
    s = scale * np.sqrt((to_f64(q) ** 2).sum(-1).max()) * np.sqrt((kk ** 2).sum(-1).max())
    d = (D + 16) * X * s + 3 * np.log(2) * X * 2 * (np.abs(e[1][used].astype(int)).max() + 1.45 * s + 32)
    o, lse = to_f64(got[0]), to_f64(got[1])
    tol = (2.0 ** -11 + 4 * d + n * X + 2.0 ** -20) * mag + U[dt] * np.abs(ref) + 2.0 ** -38 * n * (2 * mag.max(-1, keepdims=True) + 2.0 ** -55)
    within(o, ref, tol, "O")
    inf = np.isposinf(lref)
    assert np.array_equal(inf, np.isposinf(lse)) and (o[inf] == 0).all()
    within(lse[~inf], lref[~inf], 1.45 * (2 * d + n * X + 2.0 ** -21) + 2 * X * np.abs(lref[~inf]), "lse")


# which tokens (of n) hold large values, the others being zero or tiny: in one tile, by warps' tiles, by clusters' and pieces' parts
SPLITS = {
    "alternate": lambda j, n: j % 2 == 0,
    "one": lambda j, n: j == n // 3,
    "tiles": lambda j, n: j // 16 % 2 == 1,
    "steps": lambda j, n: j // 128 % 2 == 1,
    "first half": lambda j, n: j < n // 2,
    "last half": lambda j, n: j >= n // 2,
}


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("high", [40, 60, 92, 119])
@pytest.mark.parametrize("split", list(SPLITS))
def test_exponents_far_apart(split, high, D):
    """Rows of V that are zero (exponent -64) or tiny beside rows with exponents up to `high`: every key keeps its weight in
    the sum of the softmax, whatever its value's exponent."""
    gen = torch.Generator().manual_seed(45)
    n, page, G = 600, 16, {64: 12, 128: 20, 256: 8}[D]
    rng = np.random.default_rng(46)
    large = SPLITS[split](np.arange(n), n)
    for room, low in ((608, -64), (608, -30), (40000, -64)):  # a cluster per head; pieces and a join
        table, n_pages = roomy(gen, 1, page, [n], room, order="sorted")
        pool = make_pool(gen, n_pages, 1, page, D, BF, True)
        k, v, ke, ve = pool
        e = np.full(n_pages * page, low)
        e[:n][large] = high - rng.integers(0, 3, large.sum())
        ve.copy_(torch.from_numpy(e).to(torch.int8).view(n_pages, 1, page))
        if low == -64:  # zero rows
            v.view(torch.uint8).masked_fill_((ve == -64)[..., None], 0)
        q = rand(gen, (1, G, 1, D), BF, 0.5)
        q[0, 0] = 0  # equal scores
        got = run_paged(q, pool, table.cuda(), i32([n]), 0.1)
        ok()
        check_wide(q, pool, table[:, :38], page, [n], 0.1, got)


@pytest.mark.parametrize("D", [64, 128])
def test_exponents_of_every_size(D):
    """Sequences whose values' exponents run through the whole range, with scores that favour the small ones."""
    gen = torch.Generator().manual_seed(47)
    page = 16
    for room, lens in ((512, [500, 400, 1]), (40000, [500, 400, 1]), (40000, lengths("ragged", 40, 300))):  # a cluster; 8 and 1 warps in the join
        table, n_pages = roomy(gen, len(lens), page, lens, room, order="sorted")
        pool = make_pool(gen, n_pages, 2, page, D, BF, True, std=0.3)
        k, v, ke, ve = pool
        ve.copy_(torch.randint(-64, 120, ve.shape, generator=gen).to(torch.int8))
        # (the product with q below is the exponent's share of the score: -0.7 of it)
        first = (-ve.float() / 16).cpu().numpy()
        c, _ = S.quantise(np.repeat(first[..., None].astype(np.float64), D, -1))
        k64 = pool64(k) * 2.0 ** ke.cpu().numpy()[..., None].astype(float)
        k64[..., 0] = first
        c, e = S.quantise(k64)
        k.copy_(torch.from_numpy(c).float().to(F8)), ke.copy_(torch.from_numpy(e).to(torch.int8))
        q = rand(gen, (len(lens), 4, 1, D), BF, 0.3)
        q[..., 0] = 80
        got = run_paged(q, pool, table.cuda(), i32(lens), 0.1)
        ok()
        check_wide(q, pool, table[:, :32], page, lens, 0.1, got)


# --- the rotation: long prompts, elements that are not turned --------------------


LONG = [
    # B, L, Hq, Hkv, D, rot, axes, dtype, norm, interleaved, packed
    (1, 7400, 1, 1, 256, 256, 2, BF, True, False, False),    # two tables of sines in a CTA
    (2, 11000, 2, 1, 256, 64, 1, HF, False, True, True),     # three CTAs after one another, two tables in each
    (1, 14700, 2, 1, 128, 128, 1, BF, True, False, True),    # three CTAs after one another
    (1, 44000, 1, 1, 128, 128, 1, BF, True, False, False),   # both
    (1, 15001, 1, 2, 96, 48, 3, BF, True, True, True),
]


@pytest.mark.parametrize("case", LONG)
def test_rope_long(case):
    c = ops.rope_case(51, *case)
    got = ops.run_rope(c)
    ok()
    ops.check_rope(c, got)


LONG_BWD = [
    (1, 5000, 1, 1, 256, 256, 2, BF, True, False, False),    # two tables of sines in a CTA
    (1, 9900, 2, 1, 128, 128, 1, BF, True, False, True),
    (1, 15001, 1, 2, 96, 48, 3, HF, True, True, True),
    (2, 10000, 1, 1, 64, 64, 1, BF, True, False, True),
    (1, 12000, 1, 1, 256, 64, 1, BF, False, True, False),    # three tables
]


@pytest.mark.parametrize("case", LONG_BWD)
def test_rope_backward_long(case):
    c = ops.rope_case(52, *case)
    got = ops.run_rope_bwd(c)
    ok()
    ops.check_rope_bwd(c, got)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 16), (64, 48), (96, 32), (96, 80), (128, 64), (256, 16), (256, 192)])
def test_rope_unturned_elements_are_their_own(D, rot, interleaved, value):
    """One element that is not turned is infinite or no number: every other element of the row is as without it, and it
    comes out as it went in (no norm; forward, and the gradient)."""
    gen = torch.Generator().manual_seed(53)
    L = D - rot  # token t has it at element rot + t
    pos = torch.arange(L, dtype=torch.int32, device="cuda")[None] * 7
    freq = torch.rand(rot // 2, generator=gen).cuda()
    clean = [rand(gen, (1, h, L, D), BF) for h in (3, 2)]
    dirty = [x.clone() for x in clean]
    at = torch.arange(L, device="cuda")
    for x, y in zip(clean, dirty):
        x[:, :, at, rot + at] = 0
        y[:, :, at, rot + at] = value
    mark = torch.zeros(L, D, dtype=torch.bool, device="cuda")
    mark[at, rot + at] = True

    def forward(x):
        out = [torch.empty_like(t) for t in x]
        gbattn.attn_qk_norm_rope(*x, *out, pos, freq, interleaved=interleaved)
        return out

    def backward(x):
        out = [torch.empty_like(t) for t in x]
        gbattn.attn_qk_norm_rope_bwd(*clean, *x, pos, freq, *out, None, None, None, None, gbattn.qk_norm_rope_workspace(*x), interleaved=interleaved)
        return out

    for f in (forward, backward):
        want, got = f(clean), f(dirty)
        ok()
        for w, g, x in zip(want, got, dirty):
            assert torch.equal(torch.where(mark, torch.zeros_like(g), g), w)
            assert torch.equal(g[..., rot:].view(torch.int16), x[..., rot:].view(torch.int16)) or value != value
            if value != value:
                assert g[:, :, at, rot + at].isnan().all()


@pytest.mark.parametrize("layout", ["one KV head", "side by side", "heads outermost"])
def test_rope_backward_into_any_packed_gradient(layout):
    """One array for the gradients of q, k (and v, left as it was), in other orders than heads one after the other: the same
    bits as into arrays of their own."""
    B, L, Hq, Hkv, D = 2, 45, 4, 1 if layout == "one KV head" else 4, 64
    c = ops.rope_case(54, B, L, Hq, Hkv, D, D, 1, BF, True, False, False)
    want = ops.run_rope_bwd(c)
    if layout == "one KV head":
        packed = torch.full((B, L, Hq + 2, D), 7.0, dtype=BF, device="cuda")
        dq, dk, rest = packed[:, :, :Hq].transpose(1, 2), packed[:, :, Hq].unsqueeze(1), packed[:, :, Hq + 1]
    elif layout == "side by side":
        packed = torch.full((B, L, Hq, 3, D), 7.0, dtype=BF, device="cuda")
        dq, dk, rest = (packed[:, :, :, i].transpose(1, 2) for i in range(3))
    else:
        packed = torch.full((B, Hq, 2, L, D), 7.0, dtype=BF, device="cuda")
        dq, dk, rest = packed[:, :, 0], packed[:, :, 1], None
    gbattn.attn_qk_norm_rope_bwd(c["q"], c["k"], want[0], want[1], c["pos"], c["freq"], dq, dk, c["qw"], c["kw"], want[4].clone(), want[5].clone(),
                                 gbattn.qk_norm_rope_workspace(c["q"], c["k"]), eps=c["eps"])
    ok()
    assert torch.equal(dq, want[2]) and torch.equal(dk, want[3]) and (rest is None or bool((rest == 7).all()))


# --- verification -----------------------------------------------------------------


@pytest.mark.parametrize("V", [70, 72, 5003, 5004])
def test_verify_draft_that_is_no_probability(V):
    """NaN, negative, infinite and large entries of the draft: NaN and what is negative count as 0, what is above 1 as 1."""
    nan, inf = float("nan"), float("inf")
    p = torch.zeros(10, 2, V)
    q = torch.zeros(10, 1, V)
    p[:, 0, 0], p[:, 0, 1], p[:, 0, V - 1] = 0.25, 0.25, 0.5
    p[:, 1, 2] = 1
    q[:, 0, 1], q[:, 0, V - 1] = 0.9, 0.1
    q[0, 0, 0] = q[1, 0, 0] = nan
    q[2, 0, 0] = -3.0
    q[3, 0, 0] = -inf
    q[4, 0, 0] = inf
    q[5, 0, 0] = 7.0
    q[6, 0] = nan          # at the token as well: rejected, and p is left
    q[7, 0, V - 1] = nan
    p[8, 0, 0] = nan       # both
    q[8, 0, 0] = nan
    p[9, 0, 0], q[9, 0, 0] = 2.5, 1.5
    tokens = torch.ones(10, 1, dtype=torch.int32)
    u, r = torch.full((10, 1), 0.9), torch.full((10,), 0.1)
    r[1] = 0.9
    a, t = ops.verify(*(x.cuda() for x in (p, q, tokens, u, r)))
    assert a.tolist() == [0] * 10
    assert t.tolist() == [0, V - 1, 0, 0, V - 1, V - 1, 0, 0, V - 1, V - 1]


@pytest.mark.parametrize("V", [(1 << 19) - 4, 1 << 19, (1 << 19) + 8, 1 << 20, (1 << 20) + 3])
def test_verify_sums_past_64_bits(V):
    """Rows whose entries add up to 2^19 and more (no probabilities, then): sums stop at 2^64 - 1 multiples of 2^-45, so the
    token is still the one that the definition gives."""
    most, one = 2 ** 64 - 1, 2 ** 45
    p = torch.ones(4, 2, V, device="cuda")
    r = torch.tensor([0.0, 0.25, 0.5, 1 - 2.0 ** -24])
    total = min(V * one, most)
    want = [(int(float(x) * 2.0 ** 64) * total >> 64) // one for x in r]  # the least x with (x + 1) one > limit
    for draft, skip in ((None, None), (torch.zeros(4, 1, V, device="cuda"), None)):
        accept, token = i32([-9] * 4), i32([-9] * 4)
        # draft_len 0: the token is drawn from the whole row
        gbattn.attn_draft_verify(p, draft, i32([[5]] * 4), torch.full((4, 1), 0.5, device="cuda"), r.cuda(), accept, token, draft_len=i32([0] * 4))
        ok()
        assert accept.tolist() == [0] * 4 and token.tolist() == want
    # a rejected deterministic draft (u q < p does not hold): its token has no weight
    accept, token = i32([-9] * 4), i32([-9] * 4)
    gbattn.attn_draft_verify(p, None, i32([[5]] * 4), torch.full((4, 1), 1.0, device="cuda"), r.cuda(), accept, token)
    ok()
    total = min((V - 1) * one, most)
    least = [(int(float(x) * 2.0 ** 64) * total >> 64) // one for x in r]
    assert accept.tolist() == [0] * 4 and token.tolist() == [x if x < 5 else x + 1 for x in least]


# --- streams ------------------------------------------------------------------------


def stream_calls():
    """Six calls as (inputs whose values matter, outputs, the call)."""
    gen = torch.Generator().manual_seed(61)
    c = ops.rope_case(62, 2, 40, 4, 2, 64, 64, 1, BF, True, False, True)
    q, k = c["q"].contiguous(), c["k"].contiguous()
    qo, ko, dq, dk = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q), torch.empty_like(k)
    gq, gk = rand(gen, tuple(q.shape), BF), rand(gen, tuple(k.shape), BF)
    dqw, dkw, ws = torch.empty(64, device="cuda"), torch.empty(64, device="cuda"), gbattn.qk_norm_rope_workspace(q, k)
    tail = (c["pos"], c["freq"])
    yield "rope", (q, k), (qo, ko), lambda **s: gbattn.attn_qk_norm_rope(q, k, qo, ko, *tail, c["qw"], c["kw"], **s)
    yield "rope_bwd", (gq, gk), (dq, dk, dqw, dkw), lambda **s: gbattn.attn_qk_norm_rope_bwd(q, k, gq, gk, *tail, dq, dk, c["qw"], c["kw"], dqw, dkw,
                                                                                            ws, **s)
    pk, pv, _, _ = make_pool(gen, 40, 2, 16, 64, BF, False)
    table, n = torch.randperm(40, generator=gen).view(2, 20).to(torch.int32).cuda(), i32([300, 200])
    kn, vn, kp, vp, after = rand(gen, (2, 2, 5, 64), BF), rand(gen, (2, 2, 5, 64), BF), torch.zeros_like(pk), torch.zeros_like(pv), i32([0, 0])
    yield "write", (kn, vn), (kp, vp, after), lambda **s: gbattn.attn_paged_write(kn, vn, kp, vp, table, n, after, **s)
    kr, vr = torch.zeros(2, 2, 320, 64, dtype=BF, device="cuda"), torch.zeros(2, 2, 320, 64, dtype=BF, device="cuda")
    yield "read", (pk, pv), (kr, vr), lambda **s: gbattn.attn_paged_read(pk, pv, table, n, kr, vr, **s)
    x = rand(gen, (2, 8, 1, 64), BF)
    o, lse, ws2 = torch.empty_like(x), torch.empty(2, 8, 1, device="cuda"), gbattn.paged_workspace(x, pk, table)
    yield "paged", (x,), (o, lse), lambda **s: gbattn.attn_fwd_paged(x, pk, pv, table, n, o, lse, ws2, 0.3, **s)
    target, draft = (torch.softmax(torch.randn(2, t, 500, generator=gen), -1).cuda() for t in (4, 3))
    tokens, u, r, acc, tok = i32([[1, 2, 3]] * 2), torch.rand(2, 3, generator=gen).cuda(), torch.rand(2, generator=gen).cuda(), i32([0, 0]), i32([0, 0])
    yield "verify", (target, u), (acc, tok), lambda **s: gbattn.attn_draft_verify(target, draft, tokens, u, r, acc, tok, **s)


def test_calls_run_in_their_streams_order():
    """Each call's inputs hold wrong values until a copy on its stream, behind long products, puts the right ones there: a
    call that ran on another stream would read the wrong ones.  With a stream given, another one is current."""
    st, other = torch.cuda.Stream(), torch.cuda.Stream()
    for name, inputs, outputs, call in stream_calls():
        call()
        ok()
        want, right = [t.clone() for t in outputs], [t.clone() for t in inputs]
        wrong = [torch.zeros_like(t) if t.dtype != torch.float32 else torch.ones_like(t) for t in inputs]
        for t, w in zip(inputs, wrong):
            t.copy_(w)
        call()
        ok()
        assert not all(torch.equal(a, b) for a, b in zip(outputs, want)), name  # (what reading the wrong ones would give)
        for how in (st, st.cuda_stream, None):
            for t, w in zip(inputs, wrong):
                t.copy_(w)
            for t in outputs:
                t.zero_()
            torch.cuda.synchronize()
            with torch.cuda.stream(st):
                big = torch.randn(3000, 3000, device="cuda")
                for _ in range(20):
                    big = big @ big * 1e-4
                for t, w in zip(inputs, right):
                    t.copy_(w)
                if how is None:
                    call()
            if how is not None:
                with torch.cuda.stream(other):
                    call(stream=how)
            torch.cuda.synchronize()
            for a, b in zip(outputs, want):
                assert torch.equal(a, b), (name, how)
    ok()


@pytest.mark.skipif(os.environ.get("GBATTN_DEBUG") == "1", reason="this is the child")
def test_no_index_check_fires_on_these_paths():
    """The pieces, the long prompts and the extreme exponents in the debug build, whose kernels check their indices."""
    from bwd_flashattention_fwd_gb300 import build

    build.build(debug=True)
    run = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-k", "pieces or long or every_size or unturned or verify",
                          os.path.abspath(__file__)], cwd=ROOT, env=dict(os.environ, GBATTN_DEBUG="1"), capture_output=True, text=True, timeout=900)
    assert run.returncode == 0, run.stdout[-3000:] + run.stderr[-1000:]
