"""The calls around attention, without a GPU: the oracle against independent
forms, and every refusal on the host before any device memory is touched."""

import ctypes
import math

import numpy as np
import pytest
import torch

import oracle.step as S
from bwd_flashattention_fwd_gb300 import build, gbattn

INV, UNS = gbattn.ATTN_ERR_INVALID_ARG, gbattn.ATTN_ERR_UNSUPPORTED
A = [0x100000000 * (i + 1) for i in range(16)]  # addresses 4 GB apart that are never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gbattn.load_library()


# --- the oracle --------------------------------------------------------------


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("weights", [False, True])
def test_oracle_rope_gradient_is_the_difference_quotient(interleaved, weights):
    rng = np.random.default_rng(3)
    B, H, L, D, rot, eps = 1, 2, 3, 8, 6, 1e-5
    x, dy = rng.normal(size=(B, H, L, D)), rng.normal(size=(B, H, L, D))
    w = rng.normal(size=D) if weights else None
    ang = S.angles(rng.integers(0, 50, (2, B, L)), rng.uniform(0.01, 1, rot // 2), [0, 1, 7])
    dx, dw = S.norm_rope_bwd(x, w, eps, dy, ang, interleaved)

    def loss(x, w):
        return (S.norm_rope(x, w, eps, ang, interleaved)[0] * dy).sum()

    h = 1e-6
    for i in [(0, 0, 0, 0), (0, 1, 2, 5), (0, 1, 1, 7)]:
        d = np.zeros_like(x)
        d[i] = h
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * h) - dx[i]) < 1e-7
    for i in range(D if weights else 0):
        d = np.zeros(D)
        d[i] = h
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * h) - dw[i]) < 1e-7


def test_oracle_quantise_is_the_type():
    """Codes are values of float8_e4m3fn, the nearest ones (torch's own cast), and the exponent is the least."""
    rng = np.random.default_rng(5)
    x = rng.normal(size=(300, 64)) * 2.0 ** rng.integers(-30, 30, (300, 1))
    x[:50] = np.round(x[:50] * 8) / 8
    c, e = S.quantise(x)
    want = torch.from_numpy(x / 2.0 ** e[:, None].astype(float)).float().to(torch.float8_e4m3fn).double().numpy()
    exact32 = torch.from_numpy(x / 2.0 ** e[:, None].astype(float)).float().double().numpy() == x / 2.0 ** e[:, None].astype(float)
    assert np.array_equal(c[exact32], want[exact32])
    top = np.abs(x).max(-1)
    assert (top <= 448 * 2.0 ** e).all() and ((top > 448 * 2.0 ** (e - 1.0)) | (e == S.EXP_MIN)).all()
    assert (np.abs(c * 2.0 ** e[:, None].astype(float) - x) <= np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** (e[:, None] - 10.0))).all()
    c, e = S.quantise(np.array([[0.0, 0.0], [np.inf, 448.0], [448.1, np.nan]]))
    assert list(e) == [-64, 0, 1] and np.isnan(c[1, 0]) and c[1, 1] == 448 and c[2, 0] == 224 and np.isnan(c[2, 1])


def test_oracle_verify_keeps_the_targets_distribution():
    """Accepted drafts and residual draws together follow the target: over a grid of u and r, token shares are target's."""
    p, q = np.array([0.5, 0.2, 0.2, 0.1]), np.array([0.25, 0.25, 0.4, 0.1])
    share = np.zeros(4)
    n = 64
    for x in range(4):
        for i in range(n):
            for j in range(n):
                a, t = S.verify(np.array([[p, p]]), np.array([[q]]), np.array([[x]]), np.array([[(i + 0.5) / n]]),
                                np.array([(j + 0.5) / n]))
                share[x if a[0] else t[0]] += q[x] / n / n
    assert np.abs(share - p).max() < 2.0 / n


# --- refusals ----------------------------------------------------------------


KEEP = []  # the stride arrays whose addresses the calls get


def st(*s):
    KEEP.append((ctypes.c_int64 * 3)(*s))
    return ctypes.addressof(KEEP[-1])


def rope(lib, B=2, Hq=8, Hkv=2, L=16, D=128, rot=128, axes=1, eps=1e-6, inter=0, dtype=1, **over):
    a = dict(zip(("q", "k", "qw", "kw", "pos", "freq", "axis", "q_out", "k_out"), A))
    a["qs"], a["ks"] = st(Hq * L * D, L * D, D), st(Hkv * L * D, L * D, D)
    a.update({k: v or 0 for k, v in over.items()})  # (None: a null pointer)
    return lib.attn_qk_norm_rope(a["q"], a["k"], a["qw"], a["kw"], a["pos"], a["freq"], a["axis"], a["q_out"], a["k_out"], a["qs"],
                                 a["ks"], B, Hq, Hkv, L, D, rot, axes, ctypes.c_float(eps), inter, dtype, 0)


def rope_bwd(lib, B=2, Hq=8, Hkv=2, L=16, D=128, rot=128, axes=1, eps=1e-6, inter=0, dtype=1, nbytes=1 << 20, **over):
    a = dict(zip(("q", "k", "qw", "kw", "pos", "freq", "axis", "dq_out", "dk_out", "dq", "dk", "dqw", "dkw", "ws"), A))
    a["qs"], a["ks"] = st(Hq * L * D, L * D, D), st(Hkv * L * D, L * D, D)
    a["dqs"], a["dks"] = a["qs"], a["ks"]
    a.update({k: v or 0 for k, v in over.items()})  # (None: a null pointer)
    return lib.attn_qk_norm_rope_bwd(a["q"], a["k"], a["qw"], a["kw"], a["pos"], a["freq"], a["axis"], a["dq_out"], a["dk_out"], a["dq"],
                                     a["dk"], a["dqw"], a["dkw"], a["ws"], nbytes, a["qs"], a["ks"], a["dqs"], a["dks"], B, Hq, Hkv, L, D,
                                     rot, axes, ctypes.c_float(eps), inter, dtype, 0)


@pytest.mark.parametrize("call", [rope, rope_bwd])
def test_rope_rejects(lib, call):
    for name in ("q", "k", "pos", "freq", "qs", "ks"):
        assert call(lib, **{name: None}) == INV, name
    for name in ("q", "k", "qw", "kw"):
        assert call(lib, **{name: A[0] + 8}) == INV, name
    assert call(lib, pos=A[4] + 2) == INV and call(lib, freq=A[5] + 1) == INV
    assert call(lib, qw=None) == INV and call(lib, kw=None) == INV  # both or neither
    for kw in (dict(B=0), dict(Hq=0), dict(Hkv=0), dict(L=0), dict(rot=0), dict(rot=136), dict(axes=0), dict(eps=-1.0), dict(eps=math.nan),
               dict(eps=math.inf), dict(inter=2), dict(dtype=5)):
        assert call(lib, **kw) == INV, kw
    for kw in (dict(D=80, rot=16), dict(rot=24), dict(rot=8), dict(axes=9), dict(B=1 << 16, L=1 << 16), dict(B=1, L=1 << 24), dict(Hq=70000)):
        assert call(lib, **kw) == UNS, kw
    for name in ("qs", "ks"):
        assert call(lib, **{name: st(16384, 2048, 124)}) == INV  # rows not 16 bytes apart
        assert call(lib, **{name: st(16384, -2048, 128)}) == INV
        assert call(lib, **{name: st(1 << 41, 2048, 128)}) == UNS and call(lib, **{name: st(1 << 40, 1 << 31, 128)}) == UNS


def test_rope_refuses_shared_storage(lib):
    assert rope(lib, q_out=A[8]) == INV  # q_out over k_out
    assert rope(lib, q_out=A[1]) == INV and rope(lib, k_out=A[0]) == INV  # over the other input
    assert rope(lib, q_out=A[0] + 256) == INV  # shifted against q
    assert rope(lib, q_out=A[0], qs=st(8 * 16 * 128, 128, 8 * 128)) == INV  # in place, but q is in another order
    assert rope(lib, q_out=A[2]) == INV and rope(lib, q_out=A[4]) == INV  # weights, positions
    # gradients: over inputs, outputs, the workspace
    for name, at in (("dq", A[0]), ("dq", A[7]), ("dk", A[7]), ("dk", A[9]), ("dqw", A[12]), ("dqw", A[2]), ("dq", A[13]), ("dkw", A[13]),
                     ("dq", A[4])):
        assert rope_bwd(lib, **{name: at}) == INV, name
    assert rope_bwd(lib, dqw=None) == INV and rope_bwd(lib, qw=None, kw=None) == INV  # gradients and weights go together
    assert rope_bwd(lib, ws=None) == INV and rope_bwd(lib, nbytes=100) == INV and rope_bwd(lib, ws=A[13] + 4) == INV
    # rows of a gradient that share elements
    for s in (st(0, 2048, 128), st(16384, 0, 128), st(16384, 2048, 0), st(16384, 2048, 64), st(2048, 2048, 128)):
        assert rope_bwd(lib, dqs=s) == INV
    # packed gradients [B, L, Hq + 2 Hkv, D] may interleave, but not overlap: dk starts at head 7 of q's 8
    packed = st(16 * 12 * 128, 128, 12 * 128)
    for head in (7, 0, 11):
        assert rope_bwd(lib, dqs=packed, dks=packed, dk=A[9] + 2 * head * 128) == INV, head
    assert rope_bwd(lib, dqs=packed, dks=packed, dk=A[9] + 2 * 8 * 128 + 16) == INV
    need = lib.attn_qk_norm_rope_workspace_bytes
    assert need(128) > 0 and need(100) == 0


def write(lib, B=2, Hkv=2, T=4, n_pages=10, page=16, per_seq=5, D=128, dtype=1, **over):
    a = dict(zip(("k_new", "v_new", "k", "v", "ke", "ve", "table", "len", "new", "out"), A))
    a.update({k: v or 0 for k, v in over.items()})  # (None: a null pointer)
    return lib.attn_paged_write(a["k_new"], a["v_new"], a["k"], a["v"], a["ke"], a["ve"], a["table"], a["len"], a["new"], a["out"], B, Hkv,
                                T, n_pages, page, per_seq, D, dtype, 0)


def read(lib, B=2, Hkv=2, Lk=70, n_pages=10, page=16, per_seq=5, D=128, dtype=1, pitch=0, **over):
    a = dict(zip(("k", "v", "ke", "ve", "table", "len", "ko", "vo"), A))
    a.update({k: v or 0 for k, v in over.items()})  # (None: a null pointer)
    return lib.attn_paged_read(a["k"], a["v"], a["ke"], a["ve"], a["table"], a["len"], a["ko"], a["vo"], pitch, B, Hkv, Lk, n_pages, page,
                               per_seq, D, dtype, 0)


def paged(lib, B=2, Hq=8, Hkv=2, T=1, n_pages=10, page=16, per_seq=5, D=128, scale=0.1, dtype=1, nbytes=1 << 26, **over):
    a = dict(zip(("q", "k", "v", "ke", "ve", "table", "len", "o", "lse", "ws"), A))
    a.update({k: v or 0 for k, v in over.items()})  # (None: a null pointer)
    return lib.attn_fwd_paged(a["q"], a["k"], a["v"], a["ke"], a["ve"], a["table"], a["len"], a["o"], a["lse"], a["ws"], nbytes, B, Hq, Hkv,
                              T, n_pages, page, per_seq, D, ctypes.c_float(scale), dtype, 0)


@pytest.mark.parametrize("call", [write, read, paged])
def test_paged_cache_rejects(lib, call):
    for name in ("k", "v", "table", "len"):
        assert call(lib, **{name: None}) == INV, name
        assert call(lib, **{name: A[0] + 2}) == INV, name
    assert call(lib, ke=None) == INV and call(lib, ve=None) == INV and call(lib, ke=A[4] + 2) == INV
    for kw in (dict(B=0), dict(Hkv=0), dict(n_pages=0), dict(page=0), dict(per_seq=0), dict(dtype=4)):
        assert call(lib, **kw) == INV, kw
    for kw in (dict(D=72), dict(page=4), dict(page=24), dict(page=8192), dict(B=1025), dict(per_seq=(1 << 26) + 1)):
        assert call(lib, **kw) == UNS, kw


def test_paged_write_rejects(lib):
    for name in ("k_new", "v_new", "out"):
        assert write(lib, **{name: None}) == INV
    assert write(lib, k_new=A[0] + 8) == INV and write(lib, new=A[8] + 1) == INV and write(lib, T=0) == INV
    for name, at in (("out", A[7]), ("out", A[8]), ("out", A[6]), ("k", A[0]), ("v", A[2]), ("ke", A[5]), ("k", A[6])):
        assert write(lib, **{name: at}) == INV, name


def test_paged_read_rejects(lib):
    for name in ("ko", "vo"):
        assert read(lib, **{name: None}) == INV and read(lib, **{name: A[6] + 8}) == INV
    assert read(lib, Lk=0) == INV and read(lib, pitch=69) == INV and read(lib, pitch=-1) == INV
    assert read(lib, pitch=1 << 40) == UNS and read(lib, Lk=(1 << 30) + 1) == UNS
    for name, at in (("ko", A[7]), ("ko", A[0]), ("vo", A[1]), ("vo", A[3]), ("ko", A[5])):
        assert read(lib, **{name: at}) == INV, name


def test_paged_attention_rejects(lib):
    for name in ("q", "o", "lse", "ws"):
        assert paged(lib, **{name: None}) == INV and paged(lib, **{name: A[9] + 8}) == INV
    need = lib.attn_paged_workspace_bytes(2, 8, 2, 1, 16, 5, 128)
    assert need > 0 and paged(lib, nbytes=need - 1) == INV
    for kw in (dict(Hq=0), dict(Hq=9), dict(T=0), dict(scale=0.0), dict(scale=math.nan), dict(scale=math.inf)):
        assert paged(lib, **kw) == INV, kw
    for kw in (dict(T=33), dict(Hq=258), dict(Hkv=1, T=17), dict(Hkv=512, Hq=512 * 128, B=1024), dict(per_seq=1 << 26, B=1024)):
        assert paged(lib, **kw) == UNS, kw
    for name, at in (("o", A[0]), ("o", A[8]), ("o", A[9]), ("lse", A[6]), ("ws", A[1]), ("lse", A[9]), ("o", A[3])):
        assert paged(lib, **{name: at}) == INV, name
    ws = lib.attn_paged_workspace_bytes
    assert ws(2, 8, 3, 1, 16, 5, 128) == 0 and ws(2, 8, 2, 33, 16, 5, 128) == 0 and ws(2, 8, 2, 1, 16, 5, 90) == 0 and ws(2, 8, 2, 1, 16, 0, 128) == 0


def verify(lib, B=2, T=3, V=100, **over):
    a = dict(zip(("target", "draft", "tokens", "u", "r", "len", "accept", "token"), A))
    a.update({k: v or 0 for k, v in over.items()})  # (None: a null pointer)
    return lib.attn_draft_verify(a["target"], a["draft"], a["tokens"], a["u"], a["r"], a["len"], a["accept"], a["token"], B, T, V, 0)


def test_verify_rejects(lib):
    for name in ("target", "tokens", "u", "r", "accept", "token"):
        assert verify(lib, **{name: None}) == INV and verify(lib, **{name: A[0] + 2}) == INV, name
    assert verify(lib, draft=A[1] + 4) == INV and verify(lib, len=A[5] + 1) == INV
    for kw in (dict(B=0), dict(T=0), dict(V=0)):
        assert verify(lib, **kw) == INV, kw
    for kw in (dict(T=1025), dict(B=65536), dict(V=(1 << 30) + 1)):
        assert verify(lib, **kw) == UNS, kw
    for name, at in (("accept", A[7]), ("accept", A[2]), ("token", A[0]), ("token", A[5]), ("accept", A[1]), ("token", A[4])):
        assert verify(lib, **{name: at}) == INV, name


def test_fast_path_refuses_what_it_cannot_take(lib):
    """The compiled binding answers -1 (and leaves no error behind) for host tensors, other objects and wrong counts."""
    from bwd_flashattention_fwd_gb300 import _binding

    x = torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16)
    for name, n in (("qk_norm_rope", 12), ("qk_norm_rope_bwd", 17), ("paged_write", 11), ("paged_read", 9), ("fwd_paged", 12),
                    ("draft_verify", 9)):
        f = getattr(_binding, name)
        for args in ((x,) * n, (None,) * n, ("x",) * n, (x,) * (n - 1), (x,) * (n + 1), ()):
            assert f(*args) == -1, name
    with pytest.raises(KeyError):
        _binding.init({"attn_paged_read": 1})
    gbattn._lib, keep = None, gbattn._lib
    assert gbattn.load_library() is not None  # (the addresses are set again)
    gbattn._lib = keep


def test_binding_rejects_host_tensors():
    q = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    pages = torch.zeros(4, 2, 8, 64, dtype=torch.bfloat16)
    f, i = torch.zeros(32), torch.zeros(1, 8, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gbattn.attn_qk_norm_rope(q, q, q, q, i, f)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gbattn.attn_qk_norm_rope_bwd(q, q, q, q, i, f, q, q, None, None, None, None, f)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gbattn.attn_paged_write(q, q, pages, pages, i, i[0], i[0])
    with pytest.raises(ValueError, match="CUDA tensor"):
        gbattn.attn_paged_read(pages, pages, i, i[0], q, q)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gbattn.attn_fwd_paged(q, pages, pages, i, i[0], q, f, f, 0.1)
    with pytest.raises(ValueError, match="CUDA tensor"):
        gbattn.attn_draft_verify(f.view(1, 2, 16), None, i[:, :1], f, f, i, i)


# --- gradients that share an array ---------------------------------------------


def rows_of(at, B, H, L, D, s):
    """Every element (in units of 8) of rows [B, H, L, D] at strides s from address `at`."""
    i = np.arange(B)[:, None, None, None] * s[0] + np.arange(H)[None, :, None, None] * s[1] + np.arange(L)[None, None, :, None] * s[2]
    return set(((at - A[9]) // 16 + (i + np.arange(0, D, 8)) // 8).reshape(-1).tolist())


@pytest.mark.skipif(torch.cuda.is_available(), reason="an accepted call would run on these addresses")
def test_rope_takes_any_packed_gradient(lib):
    """Layouts of one packed gradient that the header allows: one KV head under any stride, q and k of each head side by
    side, sizes of one whose strides say nothing.  (Without a GPU an accepted call ends at the device.)"""
    D, L = 64, 16
    at = A[9]
    ok = lambda **kw: rope_bwd(lib, D=D, rot=D, L=L, **kw) not in (INV, UNS)
    # [B, L, Hq + 2, D], one KV head taken by an index and unsqueezed
    packed = (L * 10 * D, D, 10 * D)
    assert ok(Hkv=1, dqs=st(*packed), dks=st(packed[0], L * 10 * D, 10 * D), dk=at + 2 * 8 * D)
    assert ok(Hkv=1, dqs=st(*packed), dks=st(packed[0], 0, 10 * D), dk=at + 2 * 9 * D)
    assert ok(Hq=1, Hkv=1, dqs=st(L * 3 * D, 8, 3 * D), dks=st(L * 3 * D, 1 << 20, 3 * D), dk=at + 2 * D)
    # [B, L, H, 3, D]: q, k and v of a head side by side
    side = (L * 4 * 3 * D, 3 * D, 4 * 3 * D)
    assert ok(Hq=4, Hkv=4, dqs=st(*side), dks=st(*side), dk=at + 2 * D)
    assert ok(Hq=4, Hkv=4, dqs=st(*side), dks=st(*side), dk=at + 2 * 2 * D, dq=at)
    # one sequence, one token
    assert ok(B=1, dqs=st(7, D, 12 * D), dks=st(1 << 30, D, 12 * D), dk=at + 2 * 8 * D)
    assert rope_bwd(lib, D=D, rot=D, L=1, dqs=st(12 * D, D, 1), dks=st(12 * D, D, 5), dk=at + 2 * 8 * D) not in (INV, UNS)
    # heads outermost, tokens of both beside one another
    assert ok(Hq=4, Hkv=2, dqs=st(2 * D * L, 4 * D * L, 2 * D), dks=st(2 * D * L, 4 * D * L, 2 * D), dk=at + 2 * D)
    # and the same where they do meet
    for kw in (dict(Hkv=1, dqs=st(*packed), dks=st(packed[0], L * 10 * D, 10 * D), dk=at + 2 * 7 * D),
               dict(Hq=4, Hkv=4, dqs=st(*side), dks=st(*side), dk=at + 2 * 3 * D), dict(Hq=4, Hkv=4, dqs=st(*side), dks=st(*side), dk=at + D),
               dict(Hq=4, Hkv=2, dqs=st(2 * D * L, 4 * D * L, 2 * D), dks=st(2 * D * L, 4 * D * L, 2 * D), dk=at + 2 * 4 * D * L)):
        assert rope_bwd(lib, **dict(dict(D=D, rot=D, L=L), **kw)) == INV


@pytest.mark.skipif(torch.cuda.is_available(), reason="an accepted call would run on these addresses")
def test_rope_overlap_of_gradients_is_exact(lib):
    """Random layouts of two gradients with common strides, whole rows apart: refused exactly where an element belongs to both."""
    rng = np.random.default_rng(9)
    D, seen = 64, {True: 0, False: 0}
    for _ in range(4000):
        B, L, Hq, Hkv = (int(rng.integers(1, 4)) for _ in range(4))
        sizes, s, span = {0: B, 1: max(Hq, Hkv), 2: L}, [0, 0, 0], D
        for i in rng.permutation(3):  # each stride past what the smaller ones span
            s[i] = span + 8 * int(rng.integers(0, 30))
            span += (sizes[i] - 1) * s[i]
        at = A[9] + 2 * D * int(rng.integers(-span // D, span // D + 1))
        meet = bool(rows_of(A[9], B, Hq, L, D, s) & rows_of(at, B, Hkv, L, D, s))
        got = rope_bwd(lib, B=B, Hq=Hq, Hkv=Hkv, L=L, D=D, rot=D, dqs=st(*s), dks=st(*s), dk=at)
        assert (got == INV) == meet, (B, Hq, Hkv, L, s, at - A[9], meet)
        seen[meet] += 1
    assert min(seen.values()) > 500


def test_paged_workspace_is_0_for_what_the_call_refuses(lib):
    """A size that attn_fwd_paged refuses has no workspace (and one that it takes has)."""
    for kw in (dict(page=4), dict(page=24), dict(page=8192), dict(page=7), dict(B=1025), dict(B=1000, Hkv=66, Hq=66), dict(per_seq=(1 << 26) + 1)):
        a = dict(dict(B=2, Hq=8, Hkv=2, T=1, page=16, per_seq=5, D=128), **kw)
        assert paged(lib, **kw) == UNS, kw
        assert lib.attn_paged_workspace_bytes(a["B"], a["Hq"], a["Hkv"], a["T"], a["page"], a["per_seq"], a["D"]) == 0, kw
    for kw in (dict(page=8), dict(page=4096), dict(B=1024), dict(B=1000, Hkv=65, Hq=65), dict(per_seq=1 << 26)):
        a = dict(dict(B=2, Hq=8, Hkv=2, T=1, page=16, per_seq=5, D=128), **kw)
        assert lib.attn_paged_workspace_bytes(a["B"], a["Hq"], a["Hkv"], a["T"], a["page"], a["per_seq"], a["D"]) > 0, kw


# --- the compiled fast path of the binding --------------------------------------

WITHOUT = r"""
import ctypes, sys, types
import torch
import bwd_flashattention_fwd_gb300 as package
from bwd_flashattention_fwd_gb300 import gbattn

name = "bwd_flashattention_fwd_gb300._binding"
x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
for module in (None, types.SimpleNamespace(), types.SimpleNamespace(built_for="Python 3.1, torch 0.1")):
    sys.modules[name] = module
    if module is not None:
        package._binding = module
    lib = gbattn.load_library()
    # every other call works without it
    assert lib.attn_fwd(0, 0, 0, 0, 0, 1, 1, 1, 1, 1, 64, ctypes.c_float(1.0), 0, 1, 0) == gbattn.ATTN_ERR_INVALID_ARG
    assert gbattn.status_string(gbattn.ATTN_OK) and gbattn.attn_paged_workspace_bytes(1, 1, 1, 1, 16, 1, 64) > 0
    for call in (lambda: gbattn.attn_qk_norm_rope(x, x, x, x, x, x), lambda: gbattn.attn_paged_read(x, x, x, x, x, x)):
        try:
            call()
        except RuntimeError as e:
            assert "build" in str(e) and "torch " + torch.__version__ in str(e), e
        else:
            raise SystemExit("no error")
print("older calls work")
"""


def test_library_works_without_the_fast_path(lib):
    """No extension module, one of another source, one built for another Python and torch: the calls that need it say so,
    the others run."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", WITHOUT], cwd=root, env=dict(os.environ, PYTHONPATH=root), capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "older calls work" in run.stdout, run.stdout + run.stderr


def test_extension_module_is_built_for_this_python_and_torch(lib, tmp_path, monkeypatch):
    """A change of Python or torch makes the extension module stale, and nothing else; the debug build brings it as well."""
    import sysconfig

    from bwd_flashattention_fwd_gb300 import _binding

    assert _binding.built_for == build.built_for() and torch.__version__ in build.built_for()
    assert build.BINDING.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert build._stale() == (False, False)
    ran = []

    def run(cmd):
        ran.append(cmd)
        (tmp_path / cmd[cmd.index("-o") + 1].rsplit("/", 1)[-1]).write_text("")
        return ""

    monkeypatch.setattr(build, "_run", run)
    for name in ("BINDING", "BINDING_STAMP"):
        path = tmp_path / getattr(build, name).rsplit("/", 1)[-1]
        path.write_text(build._read(build.BINDING_STAMP) if name == "BINDING_STAMP" else "")
        monkeypatch.setattr(build, name, str(path))
    assert build._stale() == (False, False)
    build.build()
    assert ran == []
    monkeypatch.setattr(build, "built_for", lambda: "Python 3.99, torch 9.9")
    assert build._stale() == (False, True)
    build.build()
    assert len(ran) == 1 and any(a.endswith("binding.cpp") for a in ran[0])
    assert '-DGBATTN_BUILT_FOR="Python 3.99, torch 9.9"' in ran[0] and build._stale() == (False, False)
    (tmp_path / "libgbattn_debug.so").write_text("")  # (a debug library that is there, without the module)
    monkeypatch.setattr(build, "DEBUG_LIB", str(tmp_path / "libgbattn_debug.so"))
    (tmp_path / build.BINDING.rsplit("/", 1)[-1]).unlink()
    assert build._stale(debug=True) == (False, True)
    build.build(debug=True)
    assert len(ran) == 2 and build._stale(debug=True) == (False, False)


def test_libraries_are_built_where_the_extension_module_cannot_be(lib, tmp_path, monkeypatch):
    """No compiler or headers for the extension module: the build says so, after it has linked the libraries."""
    def run(cmd):
        if any(a.endswith("binding.cpp") for a in cmd):
            raise RuntimeError("no Python.h")
        (tmp_path / cmd[cmd.index("-o") + 1].rsplit("/", 1)[-1]).write_text("")
        return ""

    monkeypatch.setattr(build, "_run", run)
    for name in ("LIB", "CHECKS_LIB", "BINDING", "BINDING_STAMP"):
        monkeypatch.setattr(build, name, str(tmp_path / getattr(build, name).rsplit("/", 1)[-1]))
    with pytest.raises(RuntimeError, match="no Python.h"):
        build.build()
    assert (tmp_path / "libgbattn.so").exists() and (tmp_path / "libgbattn_checks.so").exists()
    assert build._stale() == (False, True)
