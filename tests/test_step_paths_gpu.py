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
    page, lens = 16, [500, 400, 1]
    for room in (512, 40000):
        table, n_pages = roomy(gen, 3, page, lens, room, order="sorted")
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
        q = rand(gen, (3, 4, 1, D), BF, 0.3)
        q[..., 0] = 80
        got = run_paged(q, pool, table.cuda(), i32(lens), 0.1)
        ok()
        check_wide(q, pool, table[:, :32], page, lens, 0.1, got)


# --- the rotation: elements that are not turned --------------------


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
