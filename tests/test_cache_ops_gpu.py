"""GPU parity of the cache calls (attn_fwd_tree, attn_cache_append,
attn_key_weight, attn_cache_evict) against the fp64 oracle.

Tolerances.  u = eps/2 of the 16-bit type (bf16 2^-8, fp16 2^-11), x = 2^-24.
A score s = scale * sum_d q_d k_d is summed in fp32: |ds| <= (D + 8) x S with
S = max scale * sum |q_d k_d|; scaling by log2 e and subtracting the row's
reference adds 3 x |s|, so a probability is off by a factor within
1 +- (d + 2^-21), d = (D + 16) x S (exp2 in hardware: 2^-22).
O: P is rounded to 16 bits (u of each p, in fp16 at least 2^-25 of the row's
largest), the sum of P is not, and O is rounded at the end:
  |dO| <= (u + 4 d + n x + 2^-20) A + u |O| + [fp16] 2^-25 sum |v|,
  A = sum p |v| / sum p, n the number of keys.
lse: |dl| <= 1.45 (2 d + n x + 2^-21) + 2 x |lse|.
Weights: every term is off by a factor within 1 +- (2 d + 2 x |lse| + 2^-21),
the sum of r terms by (r + 2) x."""

import math

import numpy as np
import pytest
import torch

import oracle.cache as C
from bwd_flashattention_fwd_gb300 import gbattn
from bwd_flashattention_fwd_gb300.inputs import to_f64

pytestmark = pytest.mark.gpu

X = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_flashattention_fwd_gb300 import build

    build.build()
    gbattn.load_library()


def ok():
    torch.cuda.synchronize()
    assert gbattn.attn_last_device_status() == gbattn.ATTN_OK


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rand(gen, shape, dt, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(dt).cuda()


def cache(gen, B, H, Lk, D, dt, pitch=0, stale=None, lens=None):
    """A cache [B,H,Lk,D] (the first rows of a longer buffer with pitch), rows from lens[b] on filled with `stale`."""
    t = torch.randn((B, H, pitch or Lk, D), generator=gen).to(dt)
    if stale is not None:
        for b in range(B):
            t[b, :, max(0, min(lens[b], Lk)):] = stale
    return t.cuda()[:, :, :Lk]


def score_bound(scale, q, *keys):
    """S: the largest scale * sum_d |q_d k_d| (an upper bound: the largest row norms)."""
    qn = np.sqrt(np.nanmax((to_f64(q) ** 2).sum(-1)))
    kn = max(np.sqrt(np.nanmax(np.nan_to_num((to_f64(k) ** 2).sum(-1), posinf=0.0))) for k in keys)
    return scale * qn * kn


def run_tree(q, k, v, kn, vn, lens, tl, mask, scale, ws=None):
    B, Hq, T, _ = q.shape
    o = torch.full_like(q, float("nan"))
    lse = torch.full((B, Hq, T), float("nan"), device="cuda")
    ws = gbattn.tree_workspace(q, k).fill_(0xFF) if ws is None else ws
    gbattn.attn_fwd_tree(q, k, v, kn, vn, lens, o, lse, ws, scale, tree_mask=mask, tree_len=tl)
    return o, lse


def check_tree(q, k, v, kn, vn, lens, tl, mask, scale, got):
    o, lse = to_f64(got[0]), to_f64(got[1])
    args = [None if t is None else t.cpu().numpy() for t in (lens, tl, mask)]
    ref, lref, mag = C.tree_forward(to_f64(q), to_f64(k), to_f64(v), to_f64(kn), to_f64(vn), *args, scale)
    D, dt, n = q.shape[-1], q.dtype, k.shape[2] + q.shape[2]
    live_k = [k[b, :, :max(0, int(lens[b]))] for b in range(q.shape[0]) if int(lens[b]) > 0]
    real = [kn[b, :, : (kn.shape[2] if tl is None else max(0, min(int(tl[b]), kn.shape[2])))] for b in range(q.shape[0])]
    keys = [t for t in live_k + real if t.numel()] or [torch.zeros(1, D, dtype=dt)]
    d = (D + 16) * X * score_bound(scale, torch.nan_to_num(q, nan=0.0), *keys)
    vmax = max([float(t.abs().float().nan_to_num(0.0).max()) for t in (v, vn)])
    tol = (U[dt] + 4 * d + n * X + 2.0 ** -20) * mag + U[dt] * np.abs(ref)
    if dt == torch.float16:
        tol = tol + 2.0 ** -25 * n * vmax + 2.0 ** -25
    assert np.isfinite(o).all()
    err = np.abs(o - ref)
    assert (err <= tol).all(), f"O off by {err.max():.3g}, {int((err > tol).sum())} of {err.size} outside"
    inf = np.isposinf(lref)
    assert np.array_equal(inf, np.isposinf(lse)) and (o[inf] == 0).all()
    lerr = np.abs(lse[~inf] - lref[~inf])
    ltol = 1.45 * (2 * d + n * X + 2.0 ** -21) + 2 * X * np.abs(lref[~inf])
    assert (lerr <= ltol).all(), f"lse off by {lerr.max():.3g} (tolerance {ltol.min():.3g})"


def tree_mask(rng, B, T):
    mask = np.zeros((B, T, T), dtype=np.uint8)
    for b in range(B):
        for t in range(T):
            p = rng.integers(-1, t) if t else -1
            if p >= 0:
                mask[b, t] = mask[b, p]
            mask[b, t, t] = 255 if t % 2 else 1
    return mask


BF, HF = torch.bfloat16, torch.float16
TREES = [
    # B, Hq, Hkv, T, Lk, D, dtype, context lengths, draft counts, mask
    (1, 1, 1, 1, 1, 64, BF, [1], None, None),
    (1, 1, 1, 1, 5, 64, BF, [0], None, None),
    (2, 4, 2, 1, 300, 128, BF, [300, 17], None, None),
    (1, 8, 1, 3, 129, 96, HF, [129], None, "tree"),
    (3, 8, 2, 7, 200, 64, HF, [0, 63, 200], [7, 1, 0], "tree"),
    (2, 12, 4, 8, 1000, 128, BF, [1000, 449], None, "tree"),
    (1, 32, 8, 8, 1000, 128, BF, [1000], None, "tree"),
    (2, 6, 2, 11, 513, 128, BF, [512, 511], [11, 10], None),
    (1, 10, 2, 13, 700, 256, BF, [640], None, "tree"),
    (2, 8, 1, 16, 257, 256, HF, [64, 257], [16, 3], "tree"),
    (2, 4, 1, 32, 190, 128, BF, [190, 64], None, "tree"),
    (1, 4, 1, 33, 90, 96, BF, [77], None, "tree"),
    (1, 8, 2, 61, 450, 128, BF, [450], [50], "tree"),
    (2, 4, 1, 64, 321, 64, BF, [320, 1], None, "tree"),
    (1, 4, 1, 65, 130, 128, HF, [130], None, "tree"),
    (1, 8, 1, 70, 100, 256, BF, [100], [65], None),
    (1, 3, 1, 130, 40, 64, BF, [33], [129], "tree"),
    (1, 2, 1, 200, 64, 128, BF, [64], None, None),
    (4, 2, 2, 2, 4097, 128, BF, [4097, 1, 4096, 2050], None, None),
    (1, 2, 1, 1, 9000, 96, BF, [8999], None, None),
    (40, 2, 1, 3, 150, 64, BF, [(37 * i) % 151 for i in range(40)], [i % 4 for i in range(40)], "tree"),
    (1000, 1, 1, 1, 70, 64, HF, [(7 * i) % 71 for i in range(1000)], None, None),
    (1, 40, 1, 1000, 60, 64, BF, [50], [990], None),  # more blocks of rows than SMs
    (1, 1, 1, 1024, 10, 128, BF, [10], None, "tree"),
    (2, 4, 1, 20, 333, 64, BF, [333, 128], [20, 7], "tree"),
    (1, 2, 1, 60, 200, 96, HF, [129], None, "tree"),
    (2, 2, 1, 30, 500, 64, BF, [500, 127], [30, 29], "tree"),
    (1, 3, 1, 21, 450, 96, BF, [450], [20], None),
    (1, 1, 1, 100, 260, 64, BF, [256], [97], "tree"),
    (1, 1, 1, 128, 300, 96, BF, [299], None, "tree"),
]


@pytest.mark.parametrize("case", TREES, ids=lambda c: f"b{c[0]}_h{c[1]}x{c[2]}_t{c[3]}_k{c[4]}_d{c[5]}")
@pytest.mark.parametrize("stale", [None, float("nan"), float("inf")], ids=["dirty", "nan", "inf"])
def test_tree(case, stale):
    B, Hq, Hkv, T, Lk, D, dt, lens, tl, kind = case
    gen = torch.Generator().manual_seed(B * 1000 + T * 10 + D)
    q = rand(gen, (B, Hq, T, D), dt)
    k, v = (cache(gen, B, Hkv, Lk, D, dt, pitch=Lk + 3, stale=stale, lens=lens) for _ in range(2))
    kn, vn = rand(gen, (B, Hkv, T, D), dt), rand(gen, (B, Hkv, T, D), dt)
    if stale is not None and tl is not None:  # padding drafts hold anything
        for b in range(B):
            q[b, :, tl[b]:], kn[b, :, tl[b]:], vn[b, :, tl[b]:] = stale, stale, stale
    mask = None if kind is None else torch.from_numpy(tree_mask(np.random.default_rng(T), B, T)).cuda()
    scale = float(np.float32(1 / math.sqrt(D)))
    args = (q, k, v, kn, vn, i32(lens), None if tl is None else i32(tl), mask, scale)
    got = run_tree(*args)
    ok()
    check_tree(*args, got)
    again = run_tree(*args)
    ok()
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


# Small caches (whole KV heads, several of them per CTA, empty ones between)
# and short contexts in large ones (divided into single stages).
TREES_WHOLE_OR_DIVIDED = [
    (64, 16, 8, 2, 200, 128, BF, [(53 * i) % 201 for i in range(64)], [i % 3 for i in range(64)], "tree"),
    (20, 8, 8, 5, 380, 256, HF, [(91 * i) % 381 for i in range(20)], [(i + 1) % 6 for i in range(20)], None),
    (40, 16, 2, 128, 70, 64, BF, [(19 * i) % 71 for i in range(40)], [(41 * i) % 129 for i in range(40)], "tree"),
    (30, 12, 6, 31, 300, 96, HF, [(77 * i) % 301 for i in range(30)], None, "tree"),
    (19, 8, 8, 1, 512, 128, BF, [512] * 18 + [0], [1] * 17 + [0, 1], None),
    (6, 16, 4, 7, 4000, 128, BF, [0, 1, 64, 65, 130, 200], [7, 0, 1, 7, 3, 5], "tree"),
    (6, 16, 4, 50, 3900, 64, HF, [0, 1, 64, 65, 130, 200], [50, 0, 1, 33, 3, 5], "tree"),
    (3, 8, 2, 9, 2500, 256, BF, [5, 0, 129], None, "tree"),
    (5, 4, 4, 20, 5000, 96, BF, [128, 5000, 0, 3, 129], [20, 1, 0, 17, 20], "tree"),
]


@pytest.mark.parametrize("case", TREES_WHOLE_OR_DIVIDED, ids=lambda c: f"b{c[0]}_h{c[1]}x{c[2]}_t{c[3]}_k{c[4]}_d{c[5]}")
@pytest.mark.parametrize("stale", [None, float("nan")], ids=["dirty", "nan"])
def test_tree_whole_or_divided_heads(case, stale):
    test_tree(case, stale)


@pytest.mark.parametrize("D,G,T", [(128, 2, 3), (64, 1, 17), (96, 3, 21), (128, 4, 61), (256, 1, 67), (64, 4, 131)])
def test_tree_mask_at_any_byte(D, G, T):
    """A mask that begins at any byte of its buffer, whose neighbours are not zero."""
    gen = torch.Generator().manual_seed(T)
    B, Hkv, Lk = 2, 2, 40
    q = rand(gen, (B, G * Hkv, T, D), BF)
    kn, vn = rand(gen, (B, Hkv, T, D), BF), rand(gen, (B, Hkv, T, D), BF)
    k, v = cache(gen, B, Hkv, Lk, D, BF), cache(gen, B, Hkv, Lk, D, BF)
    bits = np.random.default_rng(T).random((B, T, T)) < 0.4
    host = torch.from_numpy(bits.astype(np.uint8) * np.array([1, 2, 16, 128, 255], np.uint8)[np.arange(T) % 5])
    for offset in range(4):
        buf = torch.full((offset + host.numel() + 5,), 255, dtype=torch.uint8, device="cuda")
        mask = buf[offset:offset + host.numel()].view(B, T, T)
        mask.copy_(host)
        args = (q, k, v, kn, vn, i32([Lk, 0]), i32([T, T - 1]), mask, 0.1)
        got = run_tree(*args)
        ok()
        check_tree(*args, got)


def test_tree_rows_without_keys_and_lengths_out_of_range():
    gen = torch.Generator().manual_seed(5)
    B, Hq, Hkv, T, Lk, D = 4, 4, 2, 6, 150, 128
    q, kn, vn = rand(gen, (B, Hq, T, D), BF), rand(gen, (B, Hkv, T, D), BF), rand(gen, (B, Hkv, T, D), BF)
    k, v = cache(gen, B, Hkv, Lk, D, BF), cache(gen, B, Hkv, Lk, D, BF)
    mask = torch.from_numpy((np.random.default_rng(3).random((B, T, T)) < 0.3).astype(np.uint8)).cuda()
    mask[0, 2] = 0
    lens, tl = i32([0, -7, 10 ** 6, 3]), i32([6, 99, 4, -1])
    args = (q, k, v, kn, vn, lens, tl, mask, 0.08)
    got = run_tree(*args)
    ok()
    check_tree(q, k, v, kn, vn, i32([0, 0, Lk, 3]), i32([6, 6, 4, 0]), mask, 0.08, got)
    assert torch.isposinf(got[1][0, :, 2]).all() and torch.isposinf(got[1][3]).all()


def test_tree_rising_and_large_scores():
    """Scores that keep rising along the cache (the running maximum moves in
    every tile), and scores far beyond the exponent's range."""
    gen = torch.Generator().manual_seed(6)
    B, Hq, Hkv, T, Lk, D = 1, 4, 1, 8, 1500, 128
    q, kn, vn = rand(gen, (B, Hq, T, D), BF), rand(gen, (B, Hkv, T, D), BF), rand(gen, (B, Hkv, T, D), BF)
    k, v = cache(gen, B, Hkv, Lk, D, BF), cache(gen, B, Hkv, Lk, D, BF)
    k = (k.float() * torch.linspace(0.1, 12.0, Lk, device="cuda")[:, None]).to(BF)
    k = torch.cat([k, torch.zeros_like(k[:, :, :1])], 2)[:, :, :Lk]
    for scale in (0.088, 3.0):
        args = (q, k, v, kn, vn, i32([Lk]), None, None, scale)
        got = run_tree(*args)
        ok()
        check_tree(*args, got)


def test_tree_long_cache_offsets_past_32_bits():
    """A cache whose last head starts past 2^32 elements of the buffer."""
    D, Lk, pitch, Hkv = 64, 200, (1 << 25) + 64, 3
    gen = torch.Generator().manual_seed(7)
    q, kn, vn = rand(gen, (1, 6, 2, D), BF), rand(gen, (1, Hkv, 2, D), BF), rand(gen, (1, Hkv, 2, D), BF)
    bufs = [torch.empty((1, Hkv, pitch, D), dtype=BF, device="cuda") for _ in range(2)]
    small = [cache(gen, 1, Hkv, Lk, D, BF).contiguous() for _ in range(2)]
    for a, s in zip(bufs, small):
        a[:, :, :Lk].copy_(s)
    k, v = bufs[0][:, :, :Lk], bufs[1][:, :, :Lk]
    got = run_tree(q, k, v, kn, vn, i32([Lk]), None, None, 0.125)
    same = run_tree(q, *small, kn, vn, i32([Lk]), None, None, 0.125)
    ok()
    assert torch.equal(got[0], same[0]) and torch.equal(got[1], same[1])
    check_tree(q, *small, kn, vn, i32([Lk]), None, None, 0.125, got)


WEIGHTS = [
    # B, Hq, Hkv, Lq, Lk, D, dtype, causal / dense / limit
    (1, 1, 1, 1, 1, 64, BF, "causal"),
    (1, 2, 1, 1, 300, 128, BF, "limit"),
    (2, 8, 2, 8, 1000, 128, BF, "limit"),
    (2, 6, 2, 5, 257, 96, HF, "limit"),
    (1, 8, 1, 16, 513, 256, BF, "limit"),
    (2, 4, 1, 33, 300, 128, HF, "limit"),
    (1, 8, 1, 40, 700, 64, BF, "limit"),
    (1, 6, 2, 100, 383, 128, BF, "limit"),
    (1, 2, 1, 700, 900, 256, BF, "limit"),
    (2, 4, 2, 128, 128, 128, BF, "causal"),
    (1, 4, 1, 300, 517, 64, HF, "causal"),
    (2, 4, 4, 257, 300, 96, BF, "causal"),
    (1, 8, 2, 777, 1030, 128, BF, "causal"),
    (1, 4, 2, 520, 520, 256, HF, "causal"),
    (1, 4, 2, 200, 130, 128, BF, "dense"),
    (3, 3, 1, 7, 65, 96, BF, "dense"),
    (1, 16, 2, 1024, 1500, 128, BF, "limit"),
    (2, 6, 2, 20, 300, 128, BF, "causal"),
    (1, 4, 1, 40, 513, 96, HF, "causal"),
    (40, 2, 1, 2, 300, 64, BF, "limit"),
    (40, 4, 1, 40, 300, 64, BF, "limit"),
    (2, 8, 1, 30, 400, 256, BF, "causal"),
    (1, 4, 4, 1500, 1500, 128, BF, "dense"),
]


def row_limits(rng, B, Lq, Lk):
    lim = rng.integers(0, Lk + 1, (B, Lq)).astype(np.int32)
    lim[rng.random((B, Lq)) < 0.3] = 0
    lim[0, 0] = Lk
    return lim


def weight_lse(q, k, scale, kind, lim):
    """The rows' true base-2 log-sum-exps over the keys they see (+inf for none)."""
    B, Hq, Lq, _ = q.shape
    Lk = k.shape[2]
    x = scale * C.LOG2E * np.einsum("bhid,bhjd->bhij", to_f64(q), np.repeat(to_f64(k), Hq // k.shape[1], 1))
    if kind == "causal":
        lim = np.broadcast_to(np.arange(Lq) + Lk - Lq + 1, (B, Lq))
    elif kind == "dense":
        lim = np.full((B, Lq), Lk)
    x = np.where(np.arange(Lk)[None, None, None] < np.asarray(lim)[:, None, :, None], x, -np.inf)
    top = x.max(-1)
    with np.errstate(invalid="ignore", divide="ignore"):
        lse = top + np.log2(np.exp2(x - np.where(np.isfinite(top), top, 0.0)[..., None]).sum(-1))
    return np.where(np.isfinite(top), lse, np.inf)


def check_weight(q, k, lse, w0, got, scale, kind, lim):
    want = C.key_weight(to_f64(q), to_f64(k), to_f64(lse), scale, kind == "causal", lim)
    D, rows = q.shape[-1], q.shape[2] * q.shape[1] // k.shape[1]
    d = (D + 16) * X * score_bound(scale, q, k)
    lmax = float(lse[torch.isfinite(lse)].abs().max()) if torch.isfinite(lse).any() else 0.0
    base = 0.0 if w0 is None else to_f64(w0)
    tol = (2 * d + 2 * X * lmax + 2.0 ** -21 + (rows + 2) * X) * want + 2 * X * np.abs(base + want) + 1e-37
    err = np.abs(to_f64(got) - (base + want))
    assert (err <= tol).all(), f"off by {(err / (np.abs(base + want) + 1e-30)).max():.3g} relative, {int((err > tol).sum())} of {err.size}"


@pytest.mark.parametrize("case", WEIGHTS, ids=lambda c: f"b{c[0]}_h{c[1]}x{c[2]}_q{c[3]}_k{c[4]}_d{c[5]}_{c[7]}")
def test_key_weight(case):
    B, Hq, Hkv, Lq, Lk, D, dt, kind = case
    gen = torch.Generator().manual_seed(Lq * 7 + Lk)
    q, k = rand(gen, (B, Hq, Lq, D), dt), cache(gen, B, Hkv, Lk, D, dt, pitch=Lk + 5)
    scale = float(np.float32(1 / math.sqrt(D)))
    lim = row_limits(np.random.default_rng(Lq), B, Lq, Lk) if kind == "limit" else None
    lse = torch.from_numpy(weight_lse(q, k, scale, kind, lim)).float().cuda()
    limit = None if lim is None else torch.from_numpy(lim).cuda()
    w0 = torch.rand((B, Hkv, Lk), generator=gen).cuda()
    ws = gbattn.key_weight_workspace(q, k).fill_(0xFF)
    for start in (None, w0):
        out = torch.full((B, Hkv, Lk), float("nan"), device="cuda")
        gbattn.attn_key_weight(q, k, lse, start, out, ws, scale, causal=kind == "causal", limit=limit)
        ok()
        check_weight(q, k, lse, start, out, scale, kind, lim)
    inplace = w0.clone()
    gbattn.attn_key_weight(q, k, lse, inplace, inplace, ws, scale, causal=kind == "causal", limit=limit)
    ok()
    assert torch.equal(inplace, out)  # in place, and the same bits again


def test_key_weight_rows_that_count_for_nothing():
    """Rows with lse = +inf, limits out of range, non-finite padding rows and
    keys behind every limit."""
    gen = torch.Generator().manual_seed(11)
    B, Hq, Hkv, Lq, Lk, D = 2, 4, 2, 6, 200, 128
    q, k = rand(gen, (B, Hq, Lq, D), BF), cache(gen, B, Hkv, Lk, D, BF).contiguous()
    lim = np.array([[50, 0, -3, 150, 10 ** 6, 20], [0, 0, 0, 0, 0, 0]], dtype=np.int32)
    q[0, :, 1], q[0, :, 2], q[1] = float("nan"), float("inf"), float("nan")
    lim[0, 4] = 150
    k[:, :, 150:] = float("nan")
    qc = torch.nan_to_num(q, nan=0.0, posinf=0.0, neginf=0.0)
    kc = torch.nan_to_num(k, nan=0.0)
    lse = torch.from_numpy(weight_lse(qc, kc, 0.08, "limit", np.clip(lim, 0, Lk))).float().cuda()
    lse[0, :, 5] = float("inf")
    lse[1] = float("nan")
    w0 = torch.rand((B, Hkv, Lk), generator=gen).cuda()
    out = torch.empty_like(w0)
    gbattn.attn_key_weight(q, k, lse, w0, out, gbattn.key_weight_workspace(q, k), 0.08, limit=torch.from_numpy(lim).cuda())
    ok()
    lse2 = torch.nan_to_num(lse, nan=0.0, posinf=float("inf"))
    check_weight(qc, kc, lse2, w0, out, 0.08, "limit", np.clip(lim, 0, Lk))
    assert torch.equal(out[1], w0[1]) and torch.equal(out[0, :, 150:], w0[0, :, 150:])
    lim[0, 4] = 10 ** 6  # past the end: sees every key
    lse3 = torch.from_numpy(weight_lse(qc, kc, 0.08, "limit", np.clip(lim, 0, Lk))).float().cuda()
    gbattn.attn_key_weight(qc, kc, lse3, w0, out, gbattn.key_weight_workspace(q, k), 0.08, limit=torch.from_numpy(lim).cuda())
    ok()
    check_weight(qc, kc, lse3, w0, out, 0.08, "limit", np.clip(lim, 0, Lk))


APPENDS = [
    # B, Hkv, T, Lk, D, lengths, accepted, path
    (1, 1, 1, 4, 64, [3], None, None),
    (2, 2, 8, 40, 128, [0, 30], [3, 8], "random"),
    (3, 2, 5, 20, 96, [20, 18, 0], [5, 5, 0], "random"),
    (2, 1, 300, 700, 256, [100, 650], None, None),
    (2, 2, 4, 9, 64, [-5, 99], [9, -1], "random"),
    (4, 1, 6, 30, 128, [1, 2, 3, 4], [6, 6, 6, 6], "bad"),
    (1, 2, 1024, 2000, 64, [7], [1000], "random"),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"b{c[0]}_t{c[2]}_k{c[3]}_d{c[4]}_{c[7]}")
def test_append(case):
    B, Hkv, T, Lk, D, lens, acc, kind = case
    gen = torch.Generator().manual_seed(T + Lk)
    rng = np.random.default_rng(T)
    k, v = (cache(gen, B, Hkv, Lk, D, BF, pitch=Lk + 2) for _ in range(2))
    kn, vn = rand(gen, (B, Hkv, T, D), BF), rand(gen, (B, Hkv, T, D), BF)
    path = None if kind is None else rng.integers(0, T, (B, T)).astype(np.int32)
    if kind == "bad":
        path[0, 2], path[1, 0], path[2, 5], path[3] = -1, T, 10 ** 9, 3
    seen, pos = np.arange(B) * 100 + 50, rng.integers(0, 99, (B, Hkv, Lk))
    want = C.append(to_f64(kn), to_f64(vn), to_f64(k), to_f64(v), lens, acc, path, seen, pos)
    kb, vb = k._base.clone(), v._base.clone()
    posd, out, so = i32(pos), i32([0] * B), i32([0] * B)
    limit = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
    gbattn.attn_cache_append(kn, vn, k, v, i32(lens), None if acc is None else i32(acc), out,
                             path=None if path is None else torch.from_numpy(path).cuda(), pos=posd, seen=i32(seen),
                             seen_out=so, limit=limit)
    ok()
    for got, ref in zip((k, v, posd, out, so, limit), want):
        assert np.array_equal(to_f64(got), np.asarray(ref, dtype=np.float64))
    assert torch.equal(k._base[:, :, Lk:], kb[:, :, Lk:]) and torch.equal(v._base[:, :, Lk:], vb[:, :, Lk:])


EVICTS = [
    # B, Hkv, Lk, D, lengths, keep, recent, weights
    (1, 1, 1, 64, [1], 1, 0, "random"),
    (1, 1, 2, 64, [2], 1, 1, "random"),
    (2, 2, 100, 128, [100, 60], 50, 10, "random"),
    (2, 2, 100, 128, [50, 0], 50, 10, "random"),
    (1, 2, 300, 96, [300], 299, 299, "random"),
    (1, 2, 300, 256, [300], 1, 0, "random"),
    (2, 1, 1500, 128, [1500, 1499], 700, 100, "ties"),
    (1, 1, 2100, 64, [2100], 1024, 0, "equal"),
    (1, 2, 500, 64, [500], 100, 7, "odd values"),
    (2, 1, 64, 64, [-3, 10 ** 6], 20, 5, "random"),
    (1, 3, 9000, 128, [9000], 8192, 512, "random"),
    (1, 1, 20000, 64, [19999], 2500, 128, "heavy"),
    (1, 1, 700, 64, [700], 300, 300, "all recent"),
    (1, 2, 32768, 64, [32768], 16384, 500, "heavy"),
    (2, 1, 32769, 64, [32769, 17000], 16390, 77, "ties"),
    (1, 1, 50001, 64, [50000], 4000, 100, "heavy"),
    (1, 1, 33000, 64, [33000], 100, 0, "equal"),
    (1, 1, 400000, 64, [399990], 200000, 1000, "ties"),
]


@pytest.mark.parametrize("case", EVICTS, ids=lambda c: f"b{c[0]}_k{c[2]}_d{c[3]}_keep{c[5]}_recent{c[6]}_{c[7].replace(' ', '_')}")
def test_evict(case):
    B, Hkv, Lk, D, lens, keep, recent, kind = case
    gen = torch.Generator().manual_seed(Lk + keep)
    rng = np.random.default_rng(Lk)
    k, v = (cache(gen, B, Hkv, Lk, D, BF, pitch=Lk + 1) for _ in range(2))
    w = rng.random((B, Hkv, Lk)).astype(np.float32)
    if kind == "ties":
        w = np.floor(w * 4).astype(np.float32)
    elif kind == "equal":
        w[:] = 1.5
    elif kind == "heavy":
        w = np.exp(8 * rng.standard_normal(w.shape)).astype(np.float32)
    elif kind == "odd values":
        w = rng.choice(np.array([0.0, -0.0, 1.0, -1.0, np.inf, -np.inf, np.nan, 1e-42, -1e-42, 3e38], dtype=np.float32), w.shape)
    seen = np.array([1000 + Lk] * B)
    pos = np.stack([[rng.permutation(Lk) + 1000 for _ in range(Hkv)] for _ in range(B)])
    if kind == "all recent":
        pos[:] = 1000 + Lk - 1
    want = C.evict(to_f64(k), to_f64(v), w, pos, lens, seen, keep, recent)
    kb, vb = k._base.clone(), v._base.clone()
    wo, po = torch.full((B, Hkv, Lk), 7.0, device="cuda"), torch.full((B, Hkv, Lk), 7, dtype=torch.int32, device="cuda")
    out = i32([0] * B)
    ws = gbattn.evict_workspace(k).fill_(0xFF)
    for _ in range(2):  # the inputs are as they were, so the call repeats
        gbattn.attn_cache_evict(k, v, torch.from_numpy(w).cuda(), i32(pos), i32(lens), i32(seen), wo, po, out, ws, keep, recent)
        ok()
        for got, ref in zip((k, v, wo, po, out), want):
            assert np.array_equal(to_f64(got), np.asarray(ref, dtype=np.float64), equal_nan=True)
    assert torch.equal(k._base[:, :, Lk:], kb[:, :, Lk:]) and torch.equal(v._base[:, :, Lk:], vb[:, :, Lk:])


class Serving:
    """A cache and its bookkeeping, driven by the calls; `model` keeps the same state in 64 bits on the host."""

    def __init__(self, B, Hq, Hkv, T, Lk, D, seed):
        self.B, self.Hq, self.Hkv, self.T, self.Lk, self.D = B, Hq, Hkv, T, Lk, D
        self.gen = torch.Generator().manual_seed(seed)
        self.rng = np.random.default_rng(seed)
        self.scale = float(np.float32(1 / math.sqrt(D)))
        z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.k, self.v = (torch.full((B, Hkv, Lk, D), float("nan"), dtype=BF, device="cuda") for _ in range(2))
        self.pos, self.pos2 = z(B, Hkv, Lk) - 1, z(B, Hkv, Lk)
        self.w, self.w2 = torch.zeros(B, Hkv, Lk, device="cuda"), torch.zeros(B, Hkv, Lk, device="cuda")
        self.len, self.len2, self.seen, self.seen2 = z(B), z(B), z(B), z(B)
        self.limit = z(B, T)

    def step(self, keep, recent):
        B, T = self.B, self.T
        q = rand(self.gen, (B, self.Hq, T, self.D), BF)
        kn, vn = (rand(self.gen, (B, self.Hkv, T, self.D), BF) for _ in range(2))
        mask = torch.from_numpy(tree_mask(self.rng, B, T)).cuda()
        o, lse = run_tree(q, self.k, self.v, kn, vn, self.len, None, mask, self.scale)
        ok()
        check_tree(q, self.k, self.v, kn, vn, self.len, None, mask, self.scale, (o, lse))
        # accept the path to one draft: its ancestors in order
        path, acc = np.zeros((B, T), dtype=np.int32), np.zeros(B, dtype=np.int32)
        for b in range(B):
            up = np.flatnonzero(mask[b, self.rng.integers(0, T)].cpu().numpy())
            path[b, : len(up)], acc[b] = up, len(up)
        ref = C.append(to_f64(kn), to_f64(vn), to_f64(self.k), to_f64(self.v), self.len.cpu().numpy(), acc, path,
                       self.seen.cpu().numpy(), self.pos.cpu().numpy())
        gbattn.attn_cache_append(kn, vn, self.k, self.v, self.len, i32(acc), self.len2, path=torch.from_numpy(path).cuda(),
                                 pos=self.pos, seen=self.seen, seen_out=self.seen2, limit=self.limit)
        ok()
        for got, want in zip((self.k, self.v, self.pos, self.len2, self.seen2, self.limit), ref):
            assert np.array_equal(to_f64(got), np.asarray(want, dtype=np.float64), equal_nan=True)
        # the accepted rows' lse is the one over the cache as it is now
        lim = self.limit.cpu().numpy()
        kz = torch.nan_to_num(self.k, nan=0.0)
        true = weight_lse(q, kz, self.scale, "limit", lim)
        on = np.broadcast_to(lim[:, None] > 0, true.shape)
        assert np.abs(to_f64(lse) - true)[on].max() < 1e-4
        before = self.w.clone()
        gbattn.attn_key_weight(q, self.k, lse, self.w, self.w, gbattn.key_weight_workspace(q, self.k), self.scale, limit=self.limit)
        ok()
        check_weight(q, kz, lse, before, self.w, self.scale, "limit", lim)
        assert abs(float((self.w - before).sum()) - self.Hq * acc.sum()) < 1e-3 * self.Hq * acc.sum()
        self.len, self.len2, self.seen, self.seen2 = self.len2, self.len, self.seen2, self.seen
        ref = C.evict(to_f64(self.k), to_f64(self.v), self.w.cpu().numpy(), self.pos.cpu().numpy(), self.len.cpu().numpy(),
                      self.seen.cpu().numpy(), keep, recent)
        gbattn.attn_cache_evict(self.k, self.v, self.w, self.pos, self.len, self.seen, self.w2, self.pos2, self.len2,
                                gbattn.evict_workspace(self.k), keep, recent)
        ok()
        for got, want in zip((self.k, self.v, self.w2, self.pos2, self.len2), ref):
            assert np.array_equal(to_f64(got), np.asarray(want, dtype=np.float64), equal_nan=True)
        self.w, self.w2, self.pos, self.pos2, self.len, self.len2 = self.w2, self.w, self.pos2, self.pos, self.len2, self.len


@pytest.mark.parametrize("D,T,keep", [(128, 8, 14), (64, 5, 10), (96, 17, 20), (256, 9, 12)])
def test_serving_run(D, T, keep):
    """Draft, verify, append, weigh, evict, from an empty cache on."""
    s = Serving(2, 8, 2, T, keep + T, D, seed=D)
    for _ in range(12):
        s.step(keep, recent=8)
    assert (s.len == keep).any() and (s.seen > s.len).any()
    assert (s.pos.max(-1).values == (s.seen - 1)[:, None]).all()  # the newest token is always kept


def test_calls_in_a_graph_on_another_stream_and_two_at_once():
    gen = torch.Generator().manual_seed(21)
    B, Hq, Hkv, T, Lk, D = 2, 8, 2, 8, 900, 128
    lens, keep = i32([700, 850]), 600
    made = []
    for _ in range(2):
        q, kn, vn = (rand(gen, (B, h, T, D), BF) for h in (Hq, Hkv, Hkv))
        k, v = cache(gen, B, Hkv, Lk, D, BF).contiguous(), cache(gen, B, Hkv, Lk, D, BF).contiguous()
        made.append((q, k, v, kn, vn))

    def chain(data, stream, hold):
        q, k, v, kn, vn = data
        o, lse, k, v = torch.empty_like(q), torch.empty((B, Hq, T), device="cuda"), hold["k"], hold["v"]
        gbattn.attn_fwd_tree(q, k, v, kn, vn, lens, o, lse, hold["ws"][0], 0.09, stream=stream)
        gbattn.attn_cache_append(kn, vn, k, v, lens, None, hold["len"], pos=hold["pos"], seen=lens, seen_out=hold["seen"],
                                 limit=hold["limit"], stream=stream)
        gbattn.attn_key_weight(q, k, lse, None, hold["w"], hold["ws"][1], 0.09, limit=hold["limit"], stream=stream)
        gbattn.attn_cache_evict(k, v, hold["w"], hold["pos"], hold["len"], hold["seen"], hold["w2"], hold["pos2"], hold["len2"],
                                hold["ws"][2], keep, 30, stream=stream)
        hold["o"], hold["lse"] = o, lse

    def holder(data):
        q, k, v = data[:3]
        z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        return {"k": k.clone(), "v": v.clone(), "len": z(B), "len2": z(B), "seen": z(B), "limit": z(B, T),
                "pos": torch.arange(Lk, dtype=torch.int32, device="cuda").repeat(B, Hkv, 1), "pos2": z(B, Hkv, Lk),
                "w": torch.zeros(B, Hkv, Lk, device="cuda"), "w2": torch.zeros(B, Hkv, Lk, device="cuda"),
                "ws": (gbattn.tree_workspace(q, k), gbattn.key_weight_workspace(q, k), gbattn.evict_workspace(k))}

    names = ("o", "lse", "k", "v", "w", "w2", "pos2", "len2", "seen", "limit")
    plain = []
    for data in made:
        h = holder(data)
        chain(data, None, h)
        ok()
        plain.append([h[n].clone() for n in names])
    # two chains at once on two streams
    streams = [torch.cuda.Stream() for _ in made]
    hs = [holder(d) for d in made]
    torch.cuda.synchronize()
    for s, d, h in zip(streams, made, hs):
        with torch.cuda.stream(s):
            chain(d, s, h)
    ok()
    for h, want in zip(hs, plain):
        assert all(torch.equal(h[n], w) for n, w in zip(names, want))
    # captured, replayed, with the cache put back in between
    h = holder(made[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain(made[0], None, h)
    for _ in range(3):
        h["k"].copy_(made[0][1])
        h["v"].copy_(made[0][2])
        h["pos"].copy_(torch.arange(Lk, dtype=torch.int32, device="cuda").repeat(B, Hkv, 1))
        g.replay()
        ok()
        assert all(torch.equal(h[n], w) for n, w in zip(names, plain[0]))


def test_binding_refuses_wrong_tensors():
    """Each wrong dtype, shape or layout raises, and names its tensor or type."""
    gen = torch.Generator().manual_seed(1)
    B, Hq, Hkv, T, Lk, D = 2, 4, 2, 3, 40, 64
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    f = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    q, k, kn = rand(gen, (B, Hq, T, D), BF), rand(gen, (B, Hkv, Lk, D), BF), rand(gen, (B, Hkv, T, D), BF)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    tree = dict(q=q, k=k, v=k.clone(), k_new=kn, v_new=kn.clone(), cache_len=z(B), o=torch.empty_like(q), lse=f(B, Hq, T),
                workspace=ws, scale=0.1, tree_mask=torch.ones(B, T, T, dtype=torch.uint8, device="cuda"), tree_len=z(B))
    weight = dict(q=q, k=k, lse=f(B, Hq, T), weight=f(B, Hkv, Lk), weight_out=f(B, Hkv, Lk), workspace=ws, scale=0.1,
                  limit=z(B, T))
    append = dict(k_new=kn, v_new=kn.clone(), k=k, v=k.clone(), cache_len=z(B), accept_len=z(B), cache_len_out=z(B),
                  path=z(B, T), pos=z(B, Hkv, Lk), seen=z(B), seen_out=z(B), limit=z(B, T))
    evict = dict(k=k, v=k.clone(), weight=f(B, Hkv, Lk), pos=z(B, Hkv, Lk), cache_len=z(B), seen=z(B),
                 weight_out=f(B, Hkv, Lk), pos_out=z(B, Hkv, Lk), cache_len_out=z(B), workspace=ws, keep=10, recent=2)
    for call, good in ((gbattn.attn_fwd_tree, tree), (gbattn.attn_key_weight, weight), (gbattn.attn_cache_append, append),
                       (gbattn.attn_cache_evict, evict)):
        assert call(**good) == gbattn.ATTN_OK
        for name, t in good.items():
            if not isinstance(t, torch.Tensor):
                continue
            with pytest.raises((TypeError, ValueError)):
                call(**dict(good, **{name: t.to(torch.float64)}))
            with pytest.raises(ValueError):
                call(**dict(good, **{name: t.cpu()}))
            if name != "workspace":
                with pytest.raises(ValueError):
                    call(**dict(good, **{name: t[..., :-1].contiguous()}))
                if t.dim() > 1:
                    with pytest.raises(ValueError):  # right shape, other strides
                        call(**dict(good, **{name: t.transpose(0, 1).contiguous().transpose(0, 1)}))
    ok()
