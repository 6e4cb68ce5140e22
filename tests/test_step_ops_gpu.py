"""GPU parity of the calls around attention (attn_qk_norm_rope and its
gradient, the paged cache, attn_draft_verify) against the fp64 oracle.

Tolerances.  u = eps/2 of the 16-bit type (bf16 2^-8, fp16 2^-11, its smallest
step 2^-25), x = 2^-24.
Rotation: the angle is off by 2^-32 of a turn and the rounding of a half-turn's
fraction to 24 bits (pi 2^-25), sincospi by 2 ulp (2^-23): sine and cosine by
less than 2^-21.  The norm sums D squares (D x), rsqrt is within 2 ulp, three
products follow: a factor within 1 +- N, N = (D + 16) x.
  |dy| <= u |y| + (N + 2^-21 + 3 x) (|n_a| + |n_b|)
Backward: g is off by e_g = (2^-21 + 3 x) (|dy_a| + |dy_b|), and
  |d dx| <= u |dx| + r (|w| e_g + |x| r^2 mean(|w x| e_g)
                        + 2 N (|g w| + |x| r^2 mean |g w x|)),
  |d dw| <= sum (e_g |x| r) + (rows + D + 32) x sum |g x r|.
Attention: scores as in test_cache_ops_gpu.py: a probability is off by a factor
within 1 +- (d + 2^-21), d = (D + 16) x S, S = scale max |q| max |k|.  P is
rounded by u_p: bf16 2^-8, fp16 and over quantised pages (fp16 products) 2^-11
and below 2^-40 of the row's largest (times its value's scale) to nothing:
  |dO| <= (u_p + 4 d + n x + 2^-20) A + u |O| + 2^-38 n max |v|.
lse: |dl| <= 1.45 (2 d + n x + 2^-21) + 2 x |lse|.
The paged cache's rows, codes, exponents and lengths, accepted lengths and
tokens are equal."""

import numpy as np
import pytest
import torch

import oracle.step as S
from bwd_flashattention_fwd_gb300 import gbattn
from bwd_flashattention_fwd_gb300.inputs import to_f64

pytestmark = pytest.mark.gpu

X = 2.0 ** -24
BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
U = {BF: 2.0 ** -8, HF: 2.0 ** -11}


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


def within(got, want, tol, what):
    err = np.abs(got - want)
    assert (err <= tol).all(), f"{what} off by {np.nanmax(err):.3g}, {int((~(err <= tol)).sum())} of {err.size} outside"


# --- norm and rotation -------------------------------------------------------

ROPES = [
    # B, L, Hq, Hkv, D, rot, axes, dtype, norm, interleaved, packed
    (1, 1, 1, 1, 64, 64, 1, BF, True, False, False),
    (1, 1, 32, 8, 128, 128, 1, BF, True, False, True),
    (16, 1, 8, 2, 128, 128, 1, BF, True, True, True),
    (2, 37, 3, 1, 96, 96, 3, HF, True, False, True),
    (2, 37, 3, 1, 96, 32, 3, HF, False, True, False),
    (1, 65, 5, 5, 64, 16, 2, BF, True, False, False),
    (3, 11, 4, 2, 256, 256, 1, BF, True, False, True),
    (1, 40, 16, 2, 256, 64, 8, HF, True, True, True),
    (1, 130, 6, 2, 128, 64, 2, BF, False, False, True),
    (1, 700, 12, 4, 128, 128, 3, BF, True, False, True),
    (1, 700, 9, 3, 64, 64, 1, HF, True, True, False),
    (1, 3000, 3, 1, 96, 48, 1, BF, True, False, True),
]


def rope_case(seed, B, L, Hq, Hkv, D, rot, axes, dt, norm, inter, packed):
    gen = torch.Generator().manual_seed(seed)

    def rows():
        if packed:
            x = rand(gen, (B, L, Hq + 2 * Hkv, D), dt, 1.7).transpose(1, 2)
            return x[:, :Hq], x[:, Hq:Hq + Hkv]
        return rand(gen, (B, Hq, L, D), dt, 1.7), rand(gen, (B, Hkv, L, D), dt, 1.7)

    q, k = rows()
    top = 1 << 20  # far positions: an angle in 32 bits would be off by whole radians' fractions
    pos = torch.randint(-50 if B == 1 else 0, top, (axes, B, L), generator=gen).to(torch.int32).cuda()
    freq = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))).float().cuda()
    axis = None if axes == 1 else torch.randint(0, axes + 1, (rot // 2,), generator=gen).to(torch.uint8).cuda()
    qw, kw = (rand(gen, (D,), dt), rand(gen, (D,), dt)) if norm else (None, None)
    return dict(q=q, k=k, pos=pos, freq=freq, axis=axis, qw=qw, kw=kw, rows=rows, eps=1e-5, inter=inter, gen=gen, dt=dt, rot=rot, D=D)


def run_rope(c, q_out=None, k_out=None):
    q_out = torch.full(c["q"].shape, float("nan"), dtype=c["dt"], device="cuda") if q_out is None else q_out
    k_out = torch.full(c["k"].shape, float("nan"), dtype=c["dt"], device="cuda") if k_out is None else k_out
    gbattn.attn_qk_norm_rope(c["q"], c["k"], q_out, k_out, c["pos"], c["freq"], c["qw"], c["kw"], axis=c["axis"], eps=c["eps"],
                             interleaved=c["inter"])
    return q_out, k_out


def f64(t):
    return None if t is None else to_f64(t)


def rope_angles(c):
    return S.angles(c["pos"].cpu().numpy(), c["freq"].cpu().numpy(), None if c["axis"] is None else c["axis"].cpu().numpy())


def check_rope(c, got, names=("q", "k")):
    ang, D, dt = rope_angles(c), c["D"], c["dt"]
    N = (D + 16) * X
    for name, y in zip(names, got):
        w = f64(c[name + "w"])
        want, n = S.norm_rope(to_f64(c[name]), w, c["eps"], ang, c["inter"])
        tol = U[dt] * np.abs(want) + (N + 2.0 ** -21 + 3 * X) * S.pair_mag(n, c["rot"], c["inter"]) + (2.0 ** -25 if dt == HF else 0)
        within(to_f64(y), want, tol, name)


@pytest.mark.parametrize("case", ROPES)
def test_rope(case):
    c = rope_case(1, *case)
    got = run_rope(c)
    ok()
    check_rope(c, got)


def run_rope_bwd(c, ws=None):
    dt = c["dt"]
    dq_out, dk_out = (rand(c["gen"], tuple(c[n].shape), dt) for n in ("q", "k"))
    dq, dk = c["rows"]()
    dq.fill_(float("nan")), dk.fill_(float("nan"))
    dqw, dkw = (torch.full((c["D"],), float("nan"), device="cuda") if c["qw"] is not None else None for _ in range(2))
    ws = gbattn.qk_norm_rope_workspace(c["q"], c["k"]).fill_(0xFF) if ws is None else ws
    gbattn.attn_qk_norm_rope_bwd(c["q"], c["k"], dq_out, dk_out, c["pos"], c["freq"], dq, dk, c["qw"], c["kw"], dqw, dkw, ws, axis=c["axis"],
                                 eps=c["eps"], interleaved=c["inter"])
    return dq_out, dk_out, dq, dk, dqw, dkw


def check_rope_bwd(c, got):
    dq_out, dk_out, dq, dk, dqw, dkw = got
    ang, D, dt = rope_angles(c), c["D"], c["dt"]
    N = (D + 16) * X
    for name, dy, dx, dw in (("q", dq_out, dq, dqw), ("k", dk_out, dk, dkw)):
        x, w, dy = to_f64(c[name]), f64(c[name + "w"]), to_f64(dy)
        want, wantw = S.norm_rope_bwd(x, w, c["eps"], dy, ang, c["inter"])
        eg = (2.0 ** -21 + 3 * X) * S.pair_mag(dy, c["rot"], c["inter"])
        tol = U[dt] * np.abs(want) + (2.0 ** -25 if dt == HF else 0)
        if w is None:
            within(to_f64(dx), want, tol + eg, "d" + name)
            continue
        g = S.rotate(dy, -ang, c["inter"])
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + c["eps"])
        t = np.abs(g * w)
        tol = tol + r * (np.abs(w) * eg + np.abs(x) * r * r * (np.abs(w * x) * eg).mean(-1, keepdims=True)
                         + 2 * N * (t + np.abs(x) * r * r * (t * np.abs(x)).mean(-1, keepdims=True)))
        within(to_f64(dx), want, tol, "d" + name)
        rows = x.size // D
        tolw = (eg * np.abs(x) * r).sum((0, 1, 2)) + (rows + D + 32) * X * np.abs(g * x * r).sum((0, 1, 2))
        within(to_f64(dw), wantw, tolw, f"d{name}_weight")


@pytest.mark.parametrize("case", ROPES)
def test_rope_backward(case):
    c = rope_case(2, *case)
    got = run_rope_bwd(c)
    ok()
    check_rope_bwd(c, got)


def test_rope_backward_is_the_difference_quotient():
    """The kernels' gradients against difference quotients of the function in 64 bits (good to 1e-8; fp16 outputs)."""
    c = rope_case(3, 1, 5, 2, 1, 64, 64, 1, HF, True, False, False)
    dq_out, dk_out, dq, dk, dqw, dkw = run_rope_bwd(c)
    ok()
    ang, h = rope_angles(c), 1e-5
    for name, dy, dx, dw in (("q", dq_out, dq, dqw), ("k", dk_out, dk, dkw)):
        x, w, dy = to_f64(c[name]), to_f64(c[name + "w"]), to_f64(dy)

        def loss(x, w):
            return (S.norm_rope(x, w, c["eps"], ang, c["inter"])[0] * dy).sum()

        got, gotw = to_f64(dx), to_f64(dw)
        for i in [(0, 0, 0, 0), (0, 0, 2, 33), (0, 0, 4, 63)]:
            d = np.zeros_like(x)
            d[i] = h
            num = (loss(x + d, w) - loss(x - d, w)) / (2 * h)
            assert abs(num - got[i]) <= 2.0 ** -11 * abs(num) + 1e-4
        for i in (0, 31, 63):
            d = np.zeros_like(w)
            d[i] = h
            num = (loss(x, w + d) - loss(x, w - d)) / (2 * h)
            assert abs(num - gotw[i]) <= 1e-4 * max(1.0, abs(num))


def test_rope_same_bits_and_packed_gradient_leaves_v():
    c = rope_case(4, 2, 300, 6, 2, 128, 128, 2, BF, True, False, True)
    g = c["gen"].get_state()
    a = run_rope_bwd(c)
    c["gen"].set_state(g)
    b = run_rope_bwd(c)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    # one packed gradient: the heads of v are left as they were
    packed = torch.full((2, 300, 10, 128), 7.0, dtype=BF, device="cuda").transpose(1, 2)
    ws = gbattn.qk_norm_rope_workspace(c["q"], c["k"])
    gbattn.attn_qk_norm_rope_bwd(c["q"], c["k"], a[0], a[1], c["pos"], c["freq"], packed[:, :6], packed[:, 6:8], c["qw"], c["kw"], a[4].clone(),
                                 a[5].clone(), ws, axis=c["axis"], eps=c["eps"])
    ok()
    assert torch.equal(packed[:, :6], a[2]) and torch.equal(packed[:, 6:8], a[3]) and bool((packed[:, 8:] == 7).all())


@pytest.mark.parametrize("norm", [False, True])
def test_rope_in_place(norm):
    c = rope_case(5, 2, 90, 4, 2, 96, 96, 1, BF, norm, False, False)
    want = run_rope(c)
    q, k = c["q"].clone(), c["k"].clone()
    c["q"], c["k"] = q, k
    run_rope(c, q, k)
    ok()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_rope_strides_of_other_orders():
    """Rows found through strides: heads or tokens skipped, sequences outermost or innermost."""
    c = rope_case(6, 2, 33, 4, 2, 64, 64, 1, BF, True, False, False)
    want = run_rope(c)
    big = torch.zeros(33, 3, 2, 9, 64, dtype=BF, device="cuda")  # [L, ., B, heads, D]
    q = big[:, 1, :, 0:8:2].permute(1, 2, 0, 3)
    k = big[:, 2, :, 5:7].permute(1, 2, 0, 3)
    q.copy_(c["q"]), k.copy_(c["k"])
    c["q"], c["k"] = q, k
    got = run_rope(c)
    ok()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_one_position_per_sequence_and_axis_edge(interleaved):
    """The extreme positions of int32, zero and negative frequencies."""
    c = rope_case(7, 1, 6, 2, 1, 64, 32, 1, BF, False, interleaved, False)
    c["pos"] = i32([[[0, 1, -1, 2 ** 31 - 1, -(2 ** 31), 12345678]]])
    c["freq"][1], c["freq"][2], c["freq"][3] = 0.0, -0.3, 3.0
    c["freq"][4:] *= 1e-3
    # F is off by up to 2^-54 of freq / 2 pi turns (its rounding to 64 bits 2^-63): 2^31 positions on, 2^-21 radians at freq 3
    got = run_rope(c)
    ok()
    ang = rope_angles(c)
    for name, y in zip("qk", got):
        want, n = S.norm_rope(to_f64(c[name]), None, 0, ang, interleaved)
        # the oracle's own angle in 64 bits: 2^31 * 3 radians are spaced 2^-20
        tol = U[BF] * np.abs(want) + 2.0 ** -18 * S.pair_mag(n, 32, interleaved)
        within(to_f64(y), want, tol, name)


# --- the paged cache ---------------------------------------------------------


def make_pool(gen, n_pages, H, page, D, dt, q8, std=1.0, spread=0):
    """Pages with values in every row, as (k, v, k_exp, v_exp) on the GPU; spread: rows' scales vary by 2^+-spread."""
    out = []
    for _ in range(2):
        x = torch.randn(n_pages, H, page, D, generator=gen) * std
        if spread:
            x = x * 2.0 ** torch.randint(-spread, spread + 1, (n_pages, H, page, 1), generator=gen).float()
        if q8:
            c, e = S.quantise(x.to(dt).double().numpy())
            out.append((torch.from_numpy(c).float().to(F8).cuda(), torch.from_numpy(e).to(torch.int8).cuda()))
        else:
            out.append((x.to(dt).cuda(), None))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def pool64(t):
    return t.float().double().cpu().numpy()


WRITES = [
    # B, Hkv, T, D, page, per_seq, dtype, q8, cache_len, new_len
    (1, 1, 1, 64, 8, 1, BF, True, [0], None),
    (2, 2, 1, 128, 16, 4, BF, True, [0, 63], None),
    (2, 2, 1, 128, 16, 4, BF, False, [64, 15], None),  # no room in the first
    (3, 2, 5, 96, 8, 6, HF, True, [0, 6, 46], [5, 3, 9]),
    (3, 2, 5, 96, 8, 6, HF, False, [-4, 6, 999], [0, -1, 5]),
    (1, 8, 300, 128, 64, 5, BF, True, [17], None),
    (2, 3, 70, 256, 32, 3, BF, True, [3, 1], [70, 41]),
    (2, 3, 70, 256, 32, 3, HF, False, [3, 1], [70, 41]),
    (1, 1, 200, 64, 128, 2, HF, True, [55], None),
]


@pytest.mark.parametrize("case", WRITES)
def test_paged_write(case):
    B, H, T, D, page, per_seq, dt, q8, lens, new = case
    gen = torch.Generator().manual_seed(11)
    n_pages = B * per_seq + 2
    k, v, ke, ve = make_pool(gen, n_pages, H, page, D, dt, q8)
    table = torch.randperm(n_pages, generator=gen)[: B * per_seq].view(B, per_seq).to(torch.int32)
    if per_seq > 2:  # holes
        table[0, 1], table[-1, 2] = -1, n_pages
    kn, vn = rand(gen, (B, H, T, D), dt), rand(gen, (B, H, T, D), dt, 30.0)
    kn[0, 0, 0] = 0
    vn[-1, -1, -1, :3] = torch.tensor([float("inf"), float("nan"), -2.0])
    want = [pool64(k), pool64(v)] + [t.cpu().numpy().astype(np.int64) if q8 else None for t in (ke, ve)]
    room, out_len = per_seq * page, []
    for b in range(B):
        at = min(max(lens[b], 0), room)
        n = min(T if new is None else min(max(new[b], 0), T), room - at)
        out_len.append(at + n)
        for i in range(n):
            where = S.place(table.numpy(), page, n_pages, b, at + i)
            if where is None:
                continue
            for p, e, x in ((0, 2, kn), (1, 3, vn)):
                row = to_f64(x[b, :, i])
                if q8:
                    row, want[e][where[0], :, where[1]] = S.quantise(row)
                want[p][where[0], :, where[1]] = row
    length = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    gbattn.attn_paged_write(kn, vn, k, v, table.cuda(), i32(lens), length, new_len=None if new is None else i32(new), k_exp=ke, v_exp=ve)
    ok()
    assert length.tolist() == out_len
    for got, ref in zip((k, v), want):
        assert np.array_equal(pool64(got), ref, equal_nan=True)
    if q8:
        assert np.array_equal(ke.cpu().numpy(), want[2]) and np.array_equal(ve.cpu().numpy(), want[3])


@pytest.mark.parametrize("dt", [BF, HF])
def test_paged_write_every_value(dt):
    """All finite 16-bit values as a row's largest, and rows of the codes' borders: exponents at their limits, ties, subnormal codes."""
    bits = torch.arange(1 << 16, dtype=torch.int32)
    top = bits.to(torch.int16).view(dt)
    top = top[torch.isfinite(top.float())]
    n = top.numel() // 64 * 64
    x = top[:n].view(-1, 1).repeat(1, 64)
    scale = torch.tensor([1.0, 0.5, 0.97, 0.031, 2.0 ** -9, 2.0 ** -17, 2.0 ** -18, 1.5 * 2.0 ** -18])
    x = (x.float() * scale.repeat(8)).to(dt)
    x[:, 0] = top[:n]
    x = x.view(1, 1, n, 64).cuda()
    pages = n // 64
    k, v = torch.zeros(pages, 1, 64, 64, dtype=torch.uint8, device="cuda").view(F8), torch.zeros(pages, 1, 64, 64, dtype=torch.uint8, device="cuda").view(F8)
    ke, ve = torch.zeros(pages, 1, 64, dtype=torch.int8, device="cuda"), torch.zeros(pages, 1, 64, dtype=torch.int8, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    gbattn.attn_paged_write(x, x, k, v, table, i32([0]), i32([0]), k_exp=ke, v_exp=ve)
    ok()
    c, e = S.quantise(to_f64(x[0, 0]))
    assert np.array_equal(ke.cpu().numpy().reshape(-1), e)
    assert np.array_equal(pool64(k).reshape(n, 64), c)
    # and back: every code times its exponent, in the type (past its largest value: that)
    ko, vo = torch.zeros_like(x), torch.zeros_like(x)
    gbattn.attn_paged_read(k, v, table, i32([n]), ko, vo, k_exp=ke, v_exp=ve)
    ok()
    big = torch.finfo(dt).max
    want = torch.from_numpy(np.clip(c * 2.0 ** e[:, None].astype(float), -big, big)).to(dt)
    assert torch.equal(ko[0, 0].cpu(), want) and torch.equal(vo, ko)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("case", [(1, 1, 64, 8, 3, 24, [24], BF), (2, 2, 128, 16, 7, 100, [100, 33], BF), (3, 2, 96, 8, 5, 39, [0, 40, -1], HF),
                                  (2, 1, 256, 64, 3, 150, [150, 1], HF), (1, 8, 128, 32, 40, 1280, [1111], BF)])
def test_paged_read(case, q8):
    B, H, D, page, per_seq, Lk, lens, dt = case
    gen = torch.Generator().manual_seed(12)
    n_pages = B * per_seq
    k, v, ke, ve = make_pool(gen, n_pages, H, page, D, dt, q8, spread=6)
    table = torch.randperm(n_pages, generator=gen).view(B, per_seq).to(torch.int32)
    if per_seq > 3:
        table[-1, 1], table[0, 3] = -5, n_pages + 3
    ko, vo = (torch.full((B, H, Lk + 13, D), 9.0, dtype=dt, device="cuda") for _ in range(2))  # slices of a longer cache
    gbattn.attn_paged_read(k, v, table.cuda(), i32(lens), ko[:, :, :Lk], vo[:, :, :Lk], k_exp=ke, v_exp=ve)
    ok()
    for got, pool, e in ((ko, k, ke), (vo, v, ve)):
        want = torch.full_like(got, 9.0).cpu()
        for b in range(B):
            n = min(max(lens[b], 0), Lk)
            x, there = S.tokens_of(pool64(pool), None if e is None else e.cpu().numpy(), table.numpy(), page, b, n)
            want[b][:, :n][:, there] = torch.from_numpy(x[:, there]).to(dt)
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("q8", [False, True])
def test_pages_on_16_bytes(q8):
    """Arrays that start on 16 bytes, not on 32: the same bits as aligned ones."""
    gen = torch.Generator().manual_seed(25)
    B, H, T, D, page, per_seq = 2, 3, 40, 96, 16, 4

    def shifted(t):
        n = t.numel() * t.element_size()
        buf = torch.empty(n + 64, dtype=torch.uint8, device="cuda")
        out = buf[16: 16 + n].view(t.dtype).view(t.shape)
        assert out.data_ptr() % 32 == 16
        return out.copy_(t) if t.dtype != F8 else out.view(torch.uint8).copy_(t.view(torch.uint8)).view(F8)

    pool = make_pool(gen, 8, H, page, D, HF, q8)
    kn, vn = rand(gen, (B, H, T, D), HF), rand(gen, (B, H, T, D), HF)
    table, lens = torch.randperm(8, generator=gen).view(B, per_seq).to(torch.int32).cuda(), i32([3, 17])
    results = []
    for move in (lambda t: t.clone(), shifted):
        k, v = move(pool[0]), move(pool[1])
        ke, ve = (None, None) if not q8 else (pool[2].clone(), pool[3].clone())
        out = i32([0, 0])
        gbattn.attn_paged_write(move(kn), move(vn), k, v, table, lens, out, k_exp=ke, v_exp=ve)
        ko, vo = move(torch.zeros(B, H, 60, D, dtype=HF, device="cuda")), move(torch.zeros(B, H, 60, D, dtype=HF, device="cuda"))
        gbattn.attn_paged_read(k, v, table, out, ko, vo, k_exp=ke, v_exp=ve)
        q = move(rand(torch.Generator().manual_seed(1), (B, 6, 1, D), HF))
        o = run_paged(q, (k, v, ke, ve), table, out, 0.1)
        ok()
        results.append([out, pool64(k), pool64(v), ko.clone(), vo.clone(), *o])
    for x, y in zip(*results):
        assert np.array_equal(x, y) if isinstance(x, np.ndarray) else torch.equal(x, y)


PAGED = [
    # B, Hq, Hkv, T, D, page, per_seq, dtype, lengths
    (1, 1, 1, 1, 64, 8, 1, BF, [1]),
    (1, 4, 1, 1, 64, 8, 2, BF, [0]),
    (2, 8, 2, 1, 128, 16, 20, BF, [300, 17]),
    (1, 32, 8, 1, 128, 16, 63, BF, [1000]),
    (3, 6, 2, 1, 96, 8, 33, HF, [257, 0, 64]),
    (2, 16, 2, 1, 256, 32, 20, HF, [640, 511]),
    (2, 9, 1, 1, 128, 64, 8, BF, [512, 449]),       # nine rows
    (1, 8, 2, 4, 128, 16, 30, BF, [470]),           # a chain of four
    (3, 4, 2, 5, 64, 16, 12, HF, [190, 3, 5]),      # chains longer than what is cached
    (2, 4, 1, 8, 256, 8, 20, BF, [155, 7]),
    (1, 4, 1, 32, 128, 16, 9, HF, [140]),           # 128 rows, several blocks of them
    (1, 6, 1, 11, 96, 32, 4, BF, [128]),            # 66 rows
    (2, 3, 1, 33, 256, 128, 2, HF, [256, 40]),      # 99 rows in blocks of 16
    (5, 4, 4, 1, 64, 256, 3, BF, [768, 1, 255, 256, 700]),
    (4, 2, 2, 2, 128, 4096, 1, BF, [4096, 1, 4095, 2050]),
    (1, 2, 1, 1, 96, 64, 150, BF, [9599]),
    (40, 2, 1, 3, 64, 8, 19, BF, [(37 * i) % 153 for i in range(40)]),
    (1000, 1, 1, 1, 64, 8, 9, HF, [(7 * i) % 73 for i in range(1000)]),
]


def run_paged(q, pool, table, lens, scale, ws=None):
    k, v, ke, ve = pool
    o, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:3], float("nan"), device="cuda")
    ws = gbattn.paged_workspace(q, k, table).fill_(0xFF) if ws is None else ws
    gbattn.attn_fwd_paged(q, k, v, table, lens, o, lse, ws, scale, k_exp=ke, v_exp=ve)
    return o, lse


def check_paged(q, pool, table, page, lens, scale, got):
    k, v, ke, ve = pool
    D, dt, n = q.shape[-1], q.dtype, table.shape[1] * page
    k64, v64 = np.nan_to_num(pool64(k), nan=0.0, posinf=0.0, neginf=0.0), np.nan_to_num(pool64(v), nan=0.0, posinf=0.0, neginf=0.0)
    e = [None if t is None else t.cpu().numpy() for t in (ke, ve)]
    ref, lref, mag = S.paged_attention(to_f64(q), k64, v64, *e, table.cpu().numpy(), page, lens, scale)
    o, lse = to_f64(got[0]), to_f64(got[1])
    kk = k64 if e[0] is None else k64 * 2.0 ** e[0][..., None].astype(float)
    vv = v64 if e[1] is None else v64 * 2.0 ** e[1][..., None].astype(float)
    used = np.unique(table.cpu().numpy())
    used = used[(used >= 0) & (used < k.shape[0])]
    d = (D + 16) * X * scale * np.sqrt((to_f64(q) ** 2).sum(-1).max()) * np.sqrt((kk[used] ** 2).sum(-1).max())
    up = 2.0 ** -8 if dt == BF and ke is None else 2.0 ** -11
    tol = (up + 4 * d + n * X + 2.0 ** -20) * mag + U[dt] * np.abs(ref) + 2.0 ** -38 * n * np.abs(vv[used]).max() + (2.0 ** -25 if dt == HF else 0)
    within(o, ref, tol, "O")
    inf = np.isposinf(lref)
    assert np.array_equal(inf, np.isposinf(lse)) and (o[inf] == 0).all()
    within(lse[~inf], lref[~inf], 1.45 * (2 * d + n * X + 2.0 ** -21) + 2 * X * np.abs(lref[~inf]), "lse")


def stale(pool, table, page, lens, exponent=120):
    """Rows that hold no token filled with what must not matter: NaN and infinities (NaN codes, extreme exponents)."""
    k, v, ke, ve = pool
    live = torch.zeros(k.shape[0], page, dtype=torch.bool)
    for b in range(len(lens)):
        for j in range(max(0, min(lens[b], table.shape[1] * page))):
            p = int(table[b, j // page])
            if 0 <= p < k.shape[0]:
                live[p, j % page] = True
    dead = (~live).cuda()[:, None, :, None].expand(k.shape)
    if ke is None:
        k.masked_fill_(dead, float("inf")), v.masked_fill_(dead, float("nan"))
    else:
        for t, e in ((k, ke), (v, ve)):
            t.view(torch.uint8).masked_fill_(dead, 0x7F)
            e.masked_fill_(dead[..., 0], exponent)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("case", PAGED)
def test_paged_attention(case, q8):
    B, Hq, Hkv, T, D, page, per_seq, dt, lens = case
    gen = torch.Generator().manual_seed(13)
    n_pages = B * per_seq + 1
    pool = make_pool(gen, n_pages, Hkv, page, D, dt, q8)
    table = torch.randperm(n_pages, generator=gen)[: B * per_seq].view(B, per_seq).to(torch.int32)
    stale(pool, table, page, lens)
    q, scale = rand(gen, (B, Hq, T, D), dt), float(np.float32(1 / np.sqrt(D)))
    got = run_paged(q, pool, table.cuda(), i32(lens), scale)
    ok()
    check_paged(q, pool, table, page, lens, scale, got)


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("exponent", [-128, -127, 127])
def test_paged_attention_any_exponent_in_unused_rows(D, exponent):
    """Rows behind the last token, in the same four whose exponents are fetched together: any byte may stand there."""
    gen = torch.Generator().manual_seed(26)
    B, Hq, Hkv, page, per_seq = 4, 4, 2, 16, 3
    pool = make_pool(gen, B * per_seq, Hkv, page, D, BF, True)
    table = torch.randperm(B * per_seq, generator=gen).view(B, per_seq).to(torch.int32)
    lens = [1, 18, 35, 45]
    stale(pool, table, page, lens, exponent)
    q = rand(gen, (B, Hq, 1, D), BF)
    got = run_paged(q, pool, table.cuda(), i32(lens), 0.1)
    ok()
    check_paged(q, pool, table, page, lens, 0.1, got)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("rise", [0.01, 0.05, 0.056, 0.12, 0.9, 3.0])
def test_paged_attention_rising_scores(rise, dt, q8):
    """Scores that rise (and fall, for every other query head) by a little from key to key: the largest is always new."""
    gen = torch.Generator().manual_seed(27)
    D, Hkv, G, page, n = 128, 1, 8, 16, 500
    pool = make_pool(gen, 32, Hkv, page, D, dt, q8)
    table = torch.randperm(32, generator=gen).view(1, 32).to(torch.int32)
    k = pool[0]
    j = torch.empty(32, page)
    j[table[0].long()] = torch.arange(32 * page, dtype=torch.float32).view(32, page)
    full = torch.zeros(32, Hkv, page, D)
    full[:, 0, :, 0], full[:, 0, :, 1] = torch.floor(j / 16), j / 16 % 1  # exact as codes but for wholes above 16
    k.copy_(full.to(k.dtype))
    if q8:
        pool[2].zero_()
    q = torch.zeros(1, G, 1, D)
    for g in range(G):
        q[0, g, 0, :2] = (g + 1) * (1 if g % 2 == 0 else -1)
    q = q.to(dt).cuda()
    got = run_paged(q, pool, table.cuda(), i32([n]), 16 * rise)
    ok()
    check_paged(q, pool, table, page, [n], 16 * rise, got)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("log2_scale", [0, 8, 14, 17, 18, 19, 20, 21, 22, 23, 24, 26, 30, 60])
def test_paged_attention_large_scores(log2_scale, dt, q8):
    """Scores of any size: values of one average to one, |dO| <= u_p + n x + 2^-20 + u, whatever the weights are."""
    gen = torch.Generator().manual_seed(29)
    D, Hkv, G, page, n = 64, 2, 4, 16, 1600
    pool = make_pool(gen, 100, Hkv, page, D, dt, q8)
    if q8:
        pool[1].copy_(torch.ones(pool[1].shape).to(F8))
        pool[3].zero_()
    else:
        pool[1].fill_(1)
    table = torch.randperm(100, generator=gen).view(1, 100).to(torch.int32)
    q = rand(gen, (1, G * Hkv, 1, D), dt)
    o, lse = run_paged(q, pool, table.cuda(), i32([n]), 2.0 ** log2_scale)
    ok()
    up = 2.0 ** -8 if dt == BF and not q8 else 2.0 ** -11
    within(to_f64(o), np.ones(o.shape), up + n * X + 2.0 ** -20 + U[dt], "O")
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [40, 3000, 11000])
def test_paged_attention_nan_query(D, q8, n):
    """A row of Q with a NaN has a NaN result and a NaN lse, not those of a row that sees no key; its neighbours' stand."""
    gen = torch.Generator().manual_seed(28)
    page, per_seq = 16, 700
    pool = make_pool(gen, 2 * per_seq, 2, page, D, BF, q8)
    table = torch.randperm(2 * per_seq, generator=gen).view(2, per_seq).to(torch.int32)
    q = rand(gen, (2, 4, 1, D), BF)
    ref = run_paged(q, pool, table.cuda(), i32([n, 17]), 0.1)
    bad = q.clone()
    bad[0, 1, 0, 3] = float("nan")
    o, lse = run_paged(bad, pool, table.cuda(), i32([n, 17]), 0.1)
    ok()
    assert o[0, 1].isnan().all() and lse[0, 1].isnan().all()
    keep = torch.ones(2, 4, dtype=torch.bool)
    keep[0, 1] = False
    assert torch.equal(o[keep.cuda()], ref[0][keep.cuda()]) and torch.equal(lse[keep.cuda()], ref[1][keep.cuda()])


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_paged_attention_holes_and_lengths_out_of_range(D, q8):
    gen = torch.Generator().manual_seed(14)
    B, Hq, Hkv, T, page, per_seq = 4, 6, 2, 2, 8, 30
    n_pages = B * per_seq
    pool = make_pool(gen, n_pages, Hkv, page, D, BF, q8)
    table = torch.randperm(n_pages, generator=gen).view(B, per_seq).to(torch.int32)
    table[0, ::2], table[1, 3:9], table[2, :] = -1, n_pages, -(2 ** 31)  # every other page, a run, all of them
    lens = [200, 240, 100, 10 ** 6]
    stale(pool, table, page, lens)
    q = rand(gen, (B, Hq, T, D), BF)
    got = run_paged(q, pool, table.cuda(), i32(lens), 0.1)
    ok()
    check_paged(q, pool, table, page, lens, 0.1, got)
    got = run_paged(q, pool, table.cuda(), i32([-3, 0, 1, 2]), 0.1)
    ok()
    check_paged(q, pool, table, page, [0, 0, 1, 2], 0.1, got)


@pytest.mark.parametrize("dt", [BF, HF])
def test_paged_attention_rows_of_unequal_scales(dt):
    """Quantised rows whose exponents differ widely, among them heavy keys with tiny values and light keys with large ones."""
    gen = torch.Generator().manual_seed(15)
    B, Hq, Hkv, D, page, per_seq = 2, 8, 2, 128, 16, 40
    pool = make_pool(gen, B * per_seq, Hkv, page, D, dt, True, std=0.5, spread=7)
    table = torch.arange(B * per_seq).view(B, per_seq).to(torch.int32)
    q = rand(gen, (B, Hq, 1, D), dt, 0.2)
    q[0, 0], q[1, 3] = 0, q[1, 3] * 2.0 ** -12
    lens = [640, 333]
    got = run_paged(q, pool, table.cuda(), i32(lens), 0.05)
    ok()
    check_paged(q, pool, table, page, lens, 0.05, got)


def test_paged_attention_many_light_keys_fp16():
    """Keys of 2^-30 of the row's largest probability, with values 2^8 times its: together they count."""
    D, page, per_seq = 64, 64, 512
    n = page * per_seq
    gen = torch.Generator().manual_seed(16)
    for q8 in (False, True):
        k = torch.zeros(per_seq, 1, page, D)
        k[..., 0] = -30 * np.log(2.0) / 8
        k[0, 0, 0, 0] = 0
        v = torch.full((per_seq, 1, page, D), 256.0) * (1 + 0.25 * torch.randint(0, 4, (per_seq, 1, page, D), generator=gen))
        v[0, 0, 0] = 0
        if q8:
            parts = [S.quantise(t.to(HF).double().numpy()) for t in (k, v)]
            pool = tuple(torch.from_numpy(c).float().to(F8).cuda() for c, _ in parts) + tuple(torch.from_numpy(e).to(torch.int8).cuda() for _, e in parts)
        else:
            pool = (k.to(HF).cuda(), v.to(HF).cuda(), None, None)
        table = torch.arange(per_seq).view(1, per_seq).to(torch.int32)
        q = torch.zeros(1, 1, 1, D, dtype=HF, device="cuda")
        q[..., 0] = 8
        got = run_paged(q, pool, table.cuda(), i32([n]), 1.0)
        ok()
        # keys' scores are exact to fp16 roundings of k (8 bits over codes): taken from the pool as it is
        check_paged(q, pool, table, page, [n], 1.0, got)


@pytest.mark.parametrize("q8", [False, True])
def test_paged_attention_non_finite(q8):
    """A NaN key reaches the rows that see it, a NaN value every row of its sequence, neither another sequence."""
    gen = torch.Generator().manual_seed(17)
    B, Hq, Hkv, T, D, page, per_seq = 2, 2, 1, 2, 64, 8, 4
    pool = make_pool(gen, B * per_seq, Hkv, page, D, BF, q8)
    table = torch.arange(B * per_seq).view(B, per_seq).to(torch.int32)
    q = rand(gen, (B, Hq, T, D), BF)
    k = pool[0]
    if q8:
        k.view(torch.uint8)[3, 0, 5, 7] = 0x7F  # token 29 of sequence 0: the last of 30, seen by its second row only
    else:
        k[3, 0, 5, 7] = float("nan")
    o, lse = run_paged(q, pool, table.cuda(), i32([30, 32]), 0.1)
    ok()
    bad = torch.isnan(o.float()).any(-1)
    assert bad[0, :, 1].all() and not bad[0, :, 0].any() and not bad[1].any()


@pytest.mark.parametrize("q8", [False, True])
def test_paged_attention_past_32_bits(q8):
    """A pool of more than 2^32 bytes and 2^31 elements: tokens in its last pages."""
    H, page, D = 8, 64, 128
    n_pages = (1 << 32) // (H * page * D * (1 if q8 else 2)) + 5
    gen = torch.Generator().manual_seed(18)
    dtype = torch.uint8 if q8 else BF
    k, v = (torch.empty(n_pages, H, page, D, dtype=dtype, device="cuda") for _ in range(2))
    small = make_pool(gen, 3, H, page, D, BF, q8)
    table = torch.tensor([[n_pages - 1, 0, n_pages - 3]], dtype=torch.int32)
    kn, vn = rand(gen, (1, H, 150, D), BF), rand(gen, (1, H, 150, D), BF)
    ke = ve = None
    if q8:
        k, v = k.view(F8), v.view(F8)
        ke, ve = (torch.zeros(n_pages, H, page, dtype=torch.int8, device="cuda") for _ in range(2))
    length = i32([0])
    gbattn.attn_paged_write(kn, vn, k, v, table.cuda(), i32([0]), length, k_exp=ke, v_exp=ve)
    gbattn.attn_paged_write(kn, vn, small[0], small[1], i32([[0, 1, 2]]), i32([0]), length, k_exp=small[2], v_exp=small[3])
    q = rand(gen, (1, 32, 1, D), BF)
    a = run_paged(q, (k, v, ke, ve), table.cuda(), length, 0.1)
    b = run_paged(q, small, i32([[0, 1, 2]]), length, 0.1)
    ko, vo, ks, vs = (torch.zeros(1, H, 150, D, dtype=BF, device="cuda") for _ in range(4))
    gbattn.attn_paged_read(k, v, table.cuda(), length, ko, vo, k_exp=ke, v_exp=ve)
    gbattn.attn_paged_read(small[0], small[1], i32([[0, 1, 2]]), length, ks, vs, k_exp=small[2], v_exp=small[3])
    ok()
    assert length.tolist() == [150]
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(ko, ks) and torch.equal(vo, vs)
    if not q8:
        assert torch.equal(ko, kn) and torch.equal(vo, vn)


# --- verification ------------------------------------------------------------


def verify(target, draft, tokens, u, r, dl=None):
    B = tokens.shape[0]
    accept, token = torch.full((B,), -9, dtype=torch.int32, device="cuda"), torch.full((B,), -9, dtype=torch.int32, device="cuda")
    gbattn.attn_draft_verify(target, draft, tokens, u, r, accept, token, draft_len=dl)
    ok()
    n, t = S.verify(target.cpu().numpy(), None if draft is None else draft.cpu().numpy(), tokens.cpu().numpy(), u.cpu().numpy(), r.cpu().numpy(),
                    None if dl is None else dl.cpu().numpy())
    assert accept.tolist() == n.tolist()
    assert token.tolist() == t.tolist()
    return accept, token


@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (1, 1, 2), (2, 3, 33), (3, 8, 1000), (5, 4, 4097), (2, 5, 32768), (1, 40, 130), (130, 2, 65), (1, 3, 151936)])
def test_verify(B, T, V, greedy):
    gen = torch.Generator().manual_seed(19 + V)
    logits = torch.randn(B, T + 1, V, generator=gen) * 2
    target = torch.softmax(logits, -1)
    draft = torch.softmax(logits[:, :T] + 0.5 * torch.randn(B, T, V, generator=gen), -1)
    tokens = torch.multinomial(draft.view(B * T, V), 1, generator=gen).view(B, T).to(torch.int32)
    if greedy:
        tokens = logits[:, :T].argmax(-1).to(torch.int32)
    u, r = torch.rand(B, T, generator=gen), torch.rand(B, generator=gen)
    dl = torch.randint(0, T + 1, (B,), generator=gen).to(torch.int32)
    args = [t.cuda() for t in (target, draft, tokens, u, r, dl)]
    verify(args[0], None if greedy else args[1], *args[2:5])
    verify(args[0], None if greedy else args[1], *args[2:])


def test_verify_edges():
    """Nothing left of the residual, empty rows, tokens and lengths out of range, r at its ends, NaN and negative entries."""
    V = 70
    p = torch.zeros(12, 2, V)
    q = torch.zeros(12, 1, V)
    p[:, 0, 3], p[:, 0, 69], p[:, 1, 5] = 0.25, 0.75, 1.0
    q[:, 0, 3], q[:, 0, 69] = 0.5, 0.75
    tokens = torch.full((12, 1), 3, dtype=torch.int32)
    u = torch.full((12, 1), 0.75)  # 0.75 * 0.5 >= 0.25: rejected, and nothing is left: p_0 itself
    r = torch.tensor([0.0, 0.2, 0.25, 0.26, 1 - 2.0 ** -24, 0.5, 0.5, 0.5, 0.5, 0.5, 1e-30, 0.9])
    u[5] = 0.49999  # accepted
    u[6] = 0.5      # 0.5 * 0.5 < 0.25 does not hold
    tokens[7], tokens[8] = -1, V
    p[9, 0] = 0     # an empty row: rejected (0.75 * 0.5 < 0 does not hold), token -1
    p[10, 0, 0], p[10, 0, 1] = float("nan"), -1.0
    q[11, 0, 69] = 0.25
    dl = torch.tensor([1] * 11 + [5], dtype=torch.int32)
    a, t = verify(*(x.cuda() for x in (p, q, tokens, u, r, dl)))
    assert a.tolist() == [0, 0, 0, 0, 0, 1, 0, 0, 0, 0, 0, 0]
    assert t.tolist() == [3, 3, 69, 69, 69, 5, 69, 69, 69, -1, 3, 69]
    # no drafts at all: the token comes from target_0
    a, t = verify(*(x.cuda() for x in (p, q, tokens, u, r, torch.zeros(12, dtype=torch.int32))))
    assert a.tolist() == [0] * 12


def test_verify_flat_vocabulary_borders():
    """Equal probabilities: every border is a multiple of 1 / V, and r on it takes the next token."""
    V = 4096
    p = torch.full((64, 2, V), 1.0 / V)
    r = torch.arange(64) / 64.0
    a, t = verify(p.cuda(), None, torch.zeros(64, 1, dtype=torch.int32).cuda(), torch.zeros(64, 1).cuda(), r.cuda())
    assert a.tolist() == [1] * 64 and t.tolist() == [64 * i for i in range(64)]


# --- together ----------------------------------------------------------------


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("captured", [False, True])
def test_serving_run(q8, captured):
    """Steps of a loop as a program runs it: norm and rotation, the new keys and values into the pages, attention over
    them, verification of the drafts, the next length; eager, or one captured step replayed (positions and lengths
    live on the device).  Checked against the oracle at every step."""
    gen = torch.Generator().manual_seed(20)
    B, Hq, Hkv, T, D, page, per_seq, V, dt, scale = 3, 8, 2, 3, 128, 16, 8, 501, BF, 0.09
    n_pages = B * per_seq + 2
    pool = make_pool(gen, n_pages, Hkv, page, D, dt, q8)
    table = torch.randperm(n_pages, generator=gen)[: B * per_seq].view(B, per_seq).to(torch.int32)
    k, v, ke, ve = pool
    table_d = table.cuda()
    freq = (10000.0 ** (-torch.arange(D // 2) / (D // 2))).float().cuda()
    qw, kw = rand(gen, (D,), dt), rand(gen, (D,), dt)
    qkv = torch.empty(B, T, Hq + 2 * Hkv, D, dtype=dt, device="cuda")
    q_in, k_in, v_in = qkv.transpose(1, 2).split([Hq, Hkv, Hkv], 1)
    q, kn, vn = (torch.empty(B, h, T, D, dtype=dt, device="cuda") for h in (Hq, Hkv, Hkv))
    pos = torch.empty(B, T, dtype=torch.int32, device="cuda")
    length, after = i32([5, 40, 0]), i32([0, 0, 0])
    o, lse = torch.empty_like(q), torch.empty(B, Hq, T, device="cuda")
    ws = gbattn.paged_workspace(q, k, table_d)
    target, draft = torch.empty(B, T + 1, V, device="cuda"), torch.empty(B, T, V, device="cuda")
    tokens, u, r = i32([[0] * T] * B), torch.empty(B, T, device="cuda"), torch.empty(B, device="cuda")
    accept, token = i32([0] * B), i32([0] * B)
    steps = torch.arange(T, dtype=torch.int32, device="cuda")

    def step():
        torch.add(length[:, None], steps, out=pos)
        gbattn.attn_qk_norm_rope(q_in, k_in, q, kn, pos, freq, qw, kw)
        vn.copy_(v_in)
        gbattn.attn_paged_write(kn, vn, k, v, table_d, length, after, k_exp=ke, v_exp=ve)
        gbattn.attn_fwd_paged(q, k, v, table_d, after, o, lse, ws, scale, k_exp=ke, v_exp=ve)
        gbattn.attn_draft_verify(target, draft, tokens, u, r, accept, token)

    graph = None
    if captured:
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    lens = length.tolist()
    for _ in range(5):
        qkv.copy_(torch.randn(qkv.shape, generator=gen))
        logits = torch.randn(B, T + 1, V, generator=gen)
        target.copy_(torch.softmax(logits, -1))
        draft.copy_(torch.softmax(logits[:, :T] + 0.3 * torch.randn(B, T, V, generator=gen), -1))
        tokens.copy_(torch.randint(0, V, (B, T), generator=gen))
        u.copy_(torch.rand(B, T, generator=gen) * 0.5), r.copy_(torch.rand(B, generator=gen))
        graph.replay() if captured else step()
        ok()
        c = dict(q=q_in, k=k_in, qw=qw, kw=kw, pos=pos[None], freq=freq, axis=None, eps=1e-6, inter=False, dt=dt, rot=D, D=D)
        check_rope(c, (q, kn))
        room = per_seq * page
        want_len = [min(n + T, room) for n in lens]
        assert after.tolist() == want_len
        for b in range(B):
            for pl, e, new in ((k, ke, kn), (v, ve, vn)):
                vals, _ = S.tokens_of(pool64(pl), None if e is None else e.cpu().numpy(), table.numpy(), page, b, want_len[b])
                row = to_f64(new[b, :, : want_len[b] - lens[b]])
                if q8:
                    cc, ee = S.quantise(row)
                    row = cc * 2.0 ** ee[..., None].astype(float)
                assert np.array_equal(vals[:, lens[b]:], row)
        check_paged(q, pool, table, page, want_len, scale, (o, lse))
        n, t = S.verify(target.cpu().numpy(), draft.cpu().numpy(), tokens.cpu().numpy(), u.cpu().numpy(), r.cpu().numpy())
        assert accept.tolist() == n.tolist() and token.tolist() == t.tolist()
        lens = [min(a + int(b), room) for a, b in zip(lens, n)]
        length.copy_(i32(lens))


def test_training_run():
    """Norm and rotation in front of the attention of the training path, and its gradients through both (fp64 end to end)."""
    import oracle.attention as A

    gen = torch.Generator().manual_seed(21)
    B, L, Hq, Hkv, D, dt, scale = 1, 70, 4, 2, 64, BF, 0.125
    qkv = rand(gen, (B, L, Hq + 2 * Hkv, D), dt).transpose(1, 2)
    q_in, k_in, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:].contiguous()
    qw, kw = rand(gen, (D,), dt), rand(gen, (D,), dt)
    pos, freq = torch.arange(L, dtype=torch.int32, device="cuda")[None], (10000.0 ** (-torch.arange(D // 2) / (D // 2))).float().cuda()
    q, k = torch.empty(B, Hq, L, D, dtype=dt, device="cuda"), torch.empty(B, Hkv, L, D, dtype=dt, device="cuda")
    gbattn.attn_qk_norm_rope(q_in, k_in, q, k, pos, freq, qw, kw)
    o, lse = gbattn.forward(q, k, v, scale)
    do = rand(gen, (B, Hq, L, D), dt)
    dq_out, dk_out, dv = gbattn.backward(q, k, v, o, do, lse, gbattn.delta(o, do), scale)
    dqkv = torch.empty(B, L, Hq + 2 * Hkv, D, dtype=dt, device="cuda").transpose(1, 2)
    dqw, dkw = torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    gbattn.attn_qk_norm_rope_bwd(q_in, k_in, dq_out, dk_out, pos, freq, dqkv[:, :Hq], dqkv[:, Hq:Hq + Hkv], qw, kw, dqw, dkw,
                                 gbattn.qk_norm_rope_workspace(q_in, k_in))
    ok()
    ang = S.angles(pos.cpu().numpy()[None], freq.cpu().numpy(), None)
    q64, _ = S.norm_rope(to_f64(q_in), to_f64(qw), 1e-6, ang, False)
    k64, _ = S.norm_rope(to_f64(k_in), to_f64(kw), 1e-6, ang, False)
    o64, _, _ = A.forward(q64, k64, to_f64(v), scale, True)
    gq, gk, _ = A.backward(q64, k64, to_f64(v), o64, to_f64(do), scale, True)
    for name, x, w, g, dx, dw in (("q", q_in, qw, gq, dqkv[:, :Hq], dqw), ("k", k_in, kw, gk, dqkv[:, Hq:Hq + Hkv], dkw)):
        want, wantw = S.norm_rope_bwd(to_f64(x), to_f64(w), 1e-6, g, ang, False)
        # bf16 q, k, P, dS and gradients: each element within a few of their steps of the row's size
        assert np.linalg.norm(to_f64(dx) - want) <= 8 * 2.0 ** -8 * np.linalg.norm(want), name
        assert np.linalg.norm(to_f64(dw) - wantw) <= 8 * 2.0 ** -8 * np.linalg.norm(wantw), name


def test_prompt_over_a_cached_prefix():
    """Pages read back give attn_fwd_ex the same keys that attn_fwd_paged reads: one new token by both."""
    gen = torch.Generator().manual_seed(22)
    B, Hq, Hkv, D, page, per_seq, n = 2, 8, 2, 128, 16, 12, 180
    pool = make_pool(gen, B * per_seq, Hkv, page, D, BF, True)
    table = torch.randperm(B * per_seq, generator=gen).view(B, per_seq).to(torch.int32).cuda()
    q = rand(gen, (B, Hq, 1, D), BF)
    o, lse = run_paged(q, pool, table, i32([n, n]), 0.09)
    buf = [torch.zeros(B, Hkv, per_seq * page, D, dtype=BF, device="cuda") for _ in range(2)]
    k, v = (t[:, :, :n] for t in buf)
    gbattn.attn_paged_read(pool[0], pool[1], table, i32([n, n]), k, v, k_exp=pool[2], v_exp=pool[3])
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    gbattn.attn_fwd_ex(q, k, v, o2, lse2, 0.09, True)
    ok()
    # reading back is exact here, so both are within their own bounds of one value: P's and O's roundings, bf16
    mag = float(v.float().abs().max())
    assert float((o.float() - o2.float()).abs().max()) <= (2.0 ** -8 + 2.0 ** -11 + 2 * 2.0 ** -8) * mag
    assert float((lse - lse2).abs().max()) <= 1e-4


def test_two_streams_and_shared_pages():
    """The same pages read by two calls on two streams at once, each with its workspace; same bits as alone."""
    gen = torch.Generator().manual_seed(23)
    pool = make_pool(gen, 200, 4, 16, 128, BF, True)
    table = torch.randint(0, 200, (6, 50), generator=gen).to(torch.int32).cuda()  # sequences share pages
    q = [rand(gen, (6, 16, 1, 128), BF) for _ in range(2)]
    lens = i32([800, 1, 799, 400, 17, 650])
    ws = [gbattn.paged_workspace(q[0], pool[0], table) for _ in range(2)]
    want = [run_paged(x, pool, table, lens, 0.1, ws[0]) for x in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [None, None]
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = run_paged(q[i], pool, table, lens, 0.1, ws[i])
        ok()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_streams_given_and_current():
    """A stream as an object, as a handle and as the current one: the same results, in that stream's order."""
    gen = torch.Generator().manual_seed(24)
    c = rope_case(8, 2, 40, 4, 2, 64, 64, 1, BF, True, False, True)
    want = run_rope(c)
    ok()
    st = torch.cuda.Stream()
    for how in (st, st.cuda_stream, "current"):
        got = [torch.full_like(t, float("nan")) for t in want]
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            big = torch.randn(3000, 3000, device="cuda")
            for _ in range(20):
                big = big @ big * 1e-4
            c["q"].mul_(1), c["k"].mul_(1)  # on st, behind the products
            gbattn.attn_qk_norm_rope(c["q"], c["k"], *got, c["pos"], c["freq"], c["qw"], c["kw"], eps=c["eps"],
                                     **({} if how == "current" else {"stream": how}))
        st.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ok()


def test_binding_refuses_shapes_and_types():
    z = torch.zeros
    q, k = z(2, 4, 3, 64, dtype=BF, device="cuda"), z(2, 2, 3, 64, dtype=BF, device="cuda")
    pos, freq = z(2, 3, dtype=torch.int32, device="cuda"), z(32, device="cuda")
    with pytest.raises(ValueError):
        gbattn.attn_qk_norm_rope(q, k, q, k, pos[:1], freq)
    with pytest.raises(ValueError):
        gbattn.attn_qk_norm_rope(q, k, q[:, :, :2], k, pos, freq)
    with pytest.raises(TypeError):
        gbattn.attn_qk_norm_rope(q, k.half(), q, k, pos, freq)
    with pytest.raises(ValueError):  # rows that are not contiguous
        gbattn.attn_qk_norm_rope(q.transpose(2, 3).contiguous().transpose(2, 3), k, q.clone(), k.clone(), pos, freq)
    pages, table, n = z(5, 2, 8, 64, dtype=BF, device="cuda"), z(2, 2, dtype=torch.int32, device="cuda"), z(2, dtype=torch.int32, device="cuda")
    e = z(5, 2, 8, dtype=torch.int8, device="cuda")
    o, lse, ws = torch.empty_like(q), z(2, 4, 3, device="cuda"), z(1 << 20, dtype=torch.uint8, device="cuda")
    with pytest.raises(TypeError):  # exponents go with 8-bit pages
        gbattn.attn_fwd_paged(q, pages, pages.clone(), table, n, o, lse, ws, 0.1, k_exp=e, v_exp=e.clone())
    with pytest.raises((TypeError, ValueError)):
        gbattn.attn_fwd_paged(q, pages.view(torch.uint8)[..., :64].contiguous().view(F8), pages, table, n, o, lse, ws, 0.1)
    with pytest.raises(ValueError):
        gbattn.attn_fwd_paged(q, pages, pages.clone(), table[:1], n, o, lse, ws, 0.1)
    with pytest.raises(gbattn.AttnError):  # workspace too small
        gbattn.attn_fwd_paged(q, pages, pages.clone(), table, n, o, lse, ws[:100], 0.1)
    with pytest.raises(ValueError):
        gbattn.attn_paged_write(k, k[:, :1], pages, pages.clone(), table, n, n.clone())
    with pytest.raises(ValueError):
        gbattn.attn_paged_read(pages, pages.clone(), table, n, k, k.clone()[:, :, :2])
    with pytest.raises(ValueError):  # an expanded target
        gbattn.attn_paged_read(pages, pages.clone(), table, n, k[:1].expand(2, 2, 3, 64), k[:1].clone().expand(2, 2, 3, 64))
    t = z(2, 4, 100, device="cuda")
    with pytest.raises(ValueError):
        gbattn.attn_draft_verify(t, t, pos, z(2, 3, device="cuda"), z(2, device="cuda"), n, n.clone())
