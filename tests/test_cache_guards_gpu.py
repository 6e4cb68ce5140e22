"""The cache calls where their inputs are at the edge of what they take: keys
whose probabilities are far below the row's largest, rows and keys that hold
anything in the key-weight kernel for many rows, arrays that are neighbours
in one buffer, layouts that are refused.  Bounds as in test_cache_ops_gpu.py,
whose helpers are used."""

import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import test_cache_ops_gpu as ops
from bwd_flashattention_fwd_gb300 import gbattn
from bwd_flashattention_fwd_gb300.inputs import to_f64

pytestmark = pytest.mark.gpu

BF, HF, X, U = ops.BF, ops.HF, ops.X, ops.U


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_flashattention_fwd_gb300 import build

    build.build()
    gbattn.load_library()


@pytest.mark.parametrize("dt", [HF, BF], ids=["fp16", "bf16"])
@pytest.mark.parametrize("B,G,T,Lk,D", [(1, 4, 8, 4096, 128), (2, 2, 16, 700, 64), (1, 3, 20, 3000, 96), (1, 1, 48, 2000, 64),
                                        (1, 4, 25, 2500, 128), (1, 4, 61, 1500, 128), (1, 8, 1, 20000, 256), (9, 1, 3, 200, 96)])
def test_tree_light_keys_are_not_lost(dt, B, G, T, Lk, D):
    """Every 16th key has score 0 and value 0, the others score -26 (log2
    units) and value 1024: all of O is what the light keys add,
      O = 1024 * light * 2^-26 / (heavy + light * 2^-26).
    Their probabilities, 2^-26 of the row's largest, are below half of fp16's
    least number, 2^-25.  The kernel's P is scaled by 2^7 in fp16, so that each
    is off by at most 2^-25 / 2^7 = 2^-32 of the largest:
      |dO| <= (u + 4 d + n x + 2^-20) O + u O + [fp16] (2^-32 * 1024 * light / heavy + 2^-25),
    the last term half a step of fp16 at O.  d = (D + 16) x S, S = 26."""
    Hkv = 2
    q, kn = torch.zeros(B, G * Hkv, T, D, dtype=dt, device="cuda"), torch.zeros(B, Hkv, T, D, dtype=dt, device="cuda")
    k, v = torch.zeros(B, Hkv, Lk, D, dtype=dt, device="cuda"), torch.zeros(B, Hkv, Lk, D, dtype=dt, device="cuda")
    vn = torch.zeros_like(kn)
    q[..., 3] = 1.0
    light = torch.arange(Lk, device="cuda") % 16 != 0
    k[:, :, light, 3], v[:, :, light] = -26.0, 1024.0
    scale = float(np.float32(math.log(2.0)))
    mask = torch.eye(T, dtype=torch.uint8, device="cuda").repeat(B, 1, 1)  # each draft sees itself: one more heavy key
    o, lse = ops.run_tree(q, k, v, kn, vn, ops.i32([Lk] * B), None, mask, scale)
    ops.ok()
    n_light = int(light.sum())
    heavy = Lk - n_light + 1
    p = math.exp(-26.0 * scale)
    ref = 1024.0 * n_light * p / (heavy + n_light * p)
    d, n = (D + 16) * X * 26.0, Lk + T
    tol = (U[dt] + 4 * d + n * X + 2.0 ** -20) * ref + U[dt] * ref
    if dt == HF:
        tol += 2.0 ** -32 * 1024 * n_light / heavy + 2.0 ** -25
    err = np.abs(to_f64(o) - ref).max()
    assert err <= tol, f"O off by {err:.3g} of {ref:.3g} (tolerance {tol:.3g})"
    lref = math.log2(heavy + n_light * p)
    assert np.abs(to_f64(lse) - lref).max() <= 1.45 * (2 * d + n * X + 2.0 ** -21) + 2 * X * lref


ROWS_OF_ALL_KINDS = [
    # B, Hkv, G, Lq, Lk, D: G * Lq > 128 rows, several key tiles of 256
    (4, 2, 4, 100, 900, 128),   # every step a CTA of its own: all key tiles are joined
    (4, 8, 2, 200, 1000, 128),  # three steps a CTA, four row tiles: ranges end inside key tiles
    (4, 2, 3, 70, 700, 256),    # steps of 64 rows
    (4, 3, 1, 300, 520, 64),
    (4, 2, 2, 97, 800, 96),
    (4, 2, 2, 24, 600, 128),    # the kernel for few rows
]


@pytest.mark.parametrize("B,Hkv,G,Lq,Lk,D", ROWS_OF_ALL_KINDS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=["nan", "inf"])
def test_key_weight_rows_that_count_for_nothing_many_rows(B, Hkv, G, Lq, Lk, D, bad):
    """Rejected rows (limit 0, negative, or lse = +inf) hold anything, in q and
    in lse, keys behind every limit too; limits past the end see every key."""
    gen = torch.Generator().manual_seed(Lq + D)
    rng = np.random.default_rng(Lq)
    Hq = G * Hkv
    q, k = ops.rand(gen, (B, Hq, Lq, D), BF), ops.cache(gen, B, Hkv, Lk, D, BF, pitch=Lk + 3)
    end = [Lk - 150, Lk, Lk - 1, 300]  # keys that exist, per sequence
    lim = np.stack([rng.integers(1, end[b] + 1, Lq) for b in range(B)]).astype(np.int32)
    kind = rng.integers(0, 6, (B, Lq))
    lim[kind == 0], lim[kind == 1] = 0, -7
    lim[1][kind[1] == 2] = 10 ** 9
    lim[2] = 0  # a sequence of which nothing is accepted
    kind[2] = 0
    lim[3] = np.sort(np.clip(lim[3], 0, None))  # ascending limits: whole row tiles see nothing of late key tiles
    kind[3] = np.where(lim[3] == 0, 0, 5)
    for b in range(B):
        k[b, :, end[b]:] = bad
    none = torch.from_numpy((kind == 0) | (kind == 1)).cuda()[:, None].expand(B, Hq, Lq)
    away = torch.from_numpy(kind == 3).cuda()[:, None].expand(B, Hq, Lq)  # lse = +inf
    qc, kc = q.clone(), torch.nan_to_num(k, nan=0.0, posinf=0.0)
    scale = float(np.float32(1 / math.sqrt(D)))
    seen = np.clip(lim, 0, Lk)
    true = ops.weight_lse(qc, kc, scale, "limit", seen)
    lse = torch.from_numpy(true).float().cuda()
    clean = lse.clone()
    q[none], q[away] = bad, bad
    lse[none], clean[none] = torch.where(torch.rand(int(none.sum()), generator=gen).cuda() < 0.5, bad, -bad), 0.0
    lse[away], clean[away] = float("inf"), float("inf")
    w0 = torch.rand((B, Hkv, Lk), generator=gen).cuda()
    ws = gbattn.key_weight_workspace(q, k).fill_(0xFF)
    out = []
    for _ in range(2):
        out.append(torch.full_like(w0, float("nan")))
        gbattn.attn_key_weight(q, k, lse, w0, out[-1], ws, scale, limit=torch.from_numpy(lim).cuda())
        ops.ok()
    assert torch.equal(out[0], out[1])
    ops.check_weight(qc, kc, clean, w0, out[0], scale, "limit", seen)
    for b in range(B):
        assert torch.equal(out[0][b, :, end[b]:], w0[b, :, end[b]:])
    assert torch.equal(out[0][2], w0[2])


@pytest.mark.parametrize("G,Lq,D", [(1, 3, 128), (2, 70, 128), (4, 40, 256)])
def test_key_weight_many_sequences(G, Lq, D):
    B, Hkv, Lk = 130, 1, 300
    gen = torch.Generator().manual_seed(Lq)
    q, k = ops.rand(gen, (B, G, Lq, D), BF), ops.cache(gen, B, Hkv, Lk, D, BF)
    lim = ops.row_limits(np.random.default_rng(Lq), B, Lq, Lk)
    lim[5:60:3] = 0
    scale = float(np.float32(1 / math.sqrt(D)))
    lse = torch.from_numpy(ops.weight_lse(q, k, scale, "limit", lim)).float().cuda()
    out = torch.full((B, Hkv, Lk), float("nan"), device="cuda")
    gbattn.attn_key_weight(q, k, lse, None, out, gbattn.key_weight_workspace(q, k), scale, limit=torch.from_numpy(lim).cuda())
    ops.ok()
    ops.check_weight(q, k, lse, None, out, scale, "limit", lim)


def test_arrays_side_by_side_in_one_buffer():
    """Neighbours that do not overlap are taken, and nothing is written next to an output."""
    B, Hkv, T, Lk, D = 8, 2, 4, 64, 64
    gen = torch.Generator().manual_seed(3)
    k, v = ops.cache(gen, B, Hkv, Lk, D, BF).contiguous(), ops.cache(gen, B, Hkv, Lk, D, BF).contiguous()
    kn, vn = ops.rand(gen, (B, Hkv, T, D), BF), ops.rand(gen, (B, Hkv, T, D), BF)
    ints = torch.arange(6 * B, dtype=torch.int32, device="cuda")
    lens, lens_out, seen, seen_out, acc, last = ints.view(6, B)
    lens.copy_(ops.i32([10 + b for b in range(B)])), acc.fill_(3)
    before = ints.clone()
    gbattn.attn_cache_append(kn, vn, k, v, lens, acc, lens_out, seen=seen, seen_out=seen_out)
    ops.ok()
    assert torch.equal(lens_out, before[:B] + 3) and torch.equal(seen_out, before[2 * B:3 * B] + 3)
    assert torch.equal(lens, before[:B]) and torch.equal(seen, before[2 * B:3 * B]) and torch.equal(ints[4 * B:], before[4 * B:])
    w = torch.rand(2, B, Hkv, Lk, generator=gen).cuda()
    pos = torch.arange(2 * B * Hkv * Lk, dtype=torch.int32, device="cuda").view(2, B, Hkv, Lk) % Lk
    w0, p0 = w[0].clone(), pos[0].clone()
    gbattn.attn_cache_evict(k, v, w[0], pos[0], lens_out, seen, w[1], pos[1], last, gbattn.evict_workspace(k), 12, 0)
    ops.ok()
    assert torch.equal(w[0], w0) and torch.equal(pos[0], p0) and torch.equal(last, torch.clamp(lens_out, max=12))


def test_binding_refuses_expanded_caches_and_pitches_past_the_tensors():
    B, Hq, Hkv, T, Lk, D = 2, 4, 2, 3, 40, 64
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    f = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    gen = torch.Generator().manual_seed(1)
    q, kn = ops.rand(gen, (B, Hq, T, D), BF), ops.rand(gen, (B, Hkv, T, D), BF)
    k = ops.rand(gen, (B, Hkv, Lk, D), BF)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")

    def calls(k, **kw):
        return (lambda: gbattn.attn_fwd_tree(q, k, k, kn, kn, z(B), torch.empty_like(q), f(B, Hq, T), ws, 0.1, **kw),
                lambda: gbattn.attn_key_weight(q, k, f(B, Hq, T), None, f(B, Hkv, Lk), ws, 0.1, limit=z(B, T), **kw),
                lambda: gbattn.attn_cache_append(kn, kn, k, k, z(B), None, z(B), **kw),
                lambda: gbattn.attn_cache_evict(k, k, f(B, Hkv, Lk), z(B, Hkv, Lk), z(B), z(B), f(B, Hkv, Lk),
                                                z(B, Hkv, Lk), z(B), ws, 10, 2, **kw))

    for call in calls(k[:1, :1].expand(B, Hkv, Lk, D)):
        with pytest.raises(ValueError, match="not a slice"):
            call()
    for call in calls(k, kv_pitch=Lk + 1):
        with pytest.raises(ValueError, match="kv_pitch"):
            call()
    for call in calls(k, kv_pitch=Lk - 1):
        with pytest.raises(gbattn.AttnError):
            call()
    for call in calls(k, kv_pitch=Lk):
        assert call() == gbattn.ATTN_OK
    ops.ok()


FIRST_CALL = r"""
import torch
from bwd_flashattention_fwd_gb300 import gbattn

B, H, T, Lk, D = 1, 2, 3, 300, 64
h = lambda n: torch.ones(B, H, n, D, dtype=torch.bfloat16, device="cuda")
z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
f = lambda *s: torch.zeros(s, device="cuda")
q, k, v, n, o, lens, ws = h(T), h(Lk), h(Lk), h(T), h(T), z(B), torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
lens += Lk - T
calls = (lambda: gbattn.attn_fwd_tree(q, k, v, n, n, lens, o, lse, ws, 0.1),
         lambda: gbattn.attn_cache_append(n, n, k, v, lens, None, out),
         lambda: gbattn.attn_key_weight(q, k, lse, None, w, ws, 0.1),
         lambda: gbattn.attn_cache_evict(k, v, w, pos, lens, lens, w2, pos2, out, ws, 100, 10))
lse, w, w2, pos, pos2, out = f(B, H, T), f(B, H, Lk), f(B, H, Lk), z(B, H, Lk), z(B, H, Lk), z(B)
torch.cuda.synchronize()
for call in calls:
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o.zero_()
        try:
            call()
            raise SystemExit("a first call inside a capture was not refused")
        except gbattn.AttnError as e:
            assert e.status == gbattn.ATTN_ERR_INVALID_ARG, e
    g.replay()  # the capture is whole
    torch.cuda.synchronize()
calls[0]()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):  # the other kernels' first calls, captured
    for call in calls:
        call()
g.replay()
torch.cuda.synchronize()
assert gbattn.attn_last_device_status() == gbattn.ATTN_OK
assert (o == 1).all() and out.tolist() == [100]
print("first calls refused, later ones captured")
"""


def test_first_call_inside_a_capture_is_refused():
    """In a process of its own: no call has set the library up yet."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, env=dict(os.environ, PYTHONPATH=root),
                         capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "later ones captured" in run.stdout, run.stdout[-2000:] + run.stderr[-2000:]


@pytest.mark.skipif(os.environ.get("GBATTN_DEBUG") == "1", reason="this is the child")
def test_no_index_check_fires_here():
    """This file's cases in the debug build, whose kernels check their indices."""
    from bwd_flashattention_fwd_gb300 import build

    build.build(debug=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", os.path.abspath(__file__)], cwd=root,
                         env=dict(os.environ, GBATTN_DEBUG="1"), capture_output=True, text=True, timeout=600)
    assert run.returncode == 0, run.stdout[-3000:] + run.stderr[-1000:]
