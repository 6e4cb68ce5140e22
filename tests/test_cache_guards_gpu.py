"""The cache calls where their inputs are at the edge of what they take: keys
whose probabilities are far below the row's largest.  Bounds as in
test_cache_ops_gpu.py, whose helpers are used."""

import math

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
