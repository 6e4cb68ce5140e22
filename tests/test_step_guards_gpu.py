"""The calls around attention where a slip would not show in their results:
the library's first call inside a stream capture, memory beside the outputs,
padded batches, and every access checked against its array (debug build)."""

import os
import subprocess
import sys

import pytest
import torch

from bwd_flashattention_fwd_gb300 import gbattn

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_flashattention_fwd_gb300 import build

    build.build()
    gbattn.load_library()


FIRST_CALL = r"""
import torch
from bwd_flashattention_fwd_gb300 import gbattn

B, H, T, D = 2, 2, 3, 64
h = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device="cuda")
z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
f = lambda *s: torch.zeros(s, device="cuda")
x, y, pages, pos, freq, dw = h(B, H, T, D), h(B, H, T, D), h(4, H, 16, D), z(B, T), f(32), f(D)
table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
lens, out, lse, ws = z(B) + 5, z(B), f(B, H, T), torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
w, p, acc, tok = h(D), f(B, T + 1, 100) + 0.01, z(B), z(B)
dx, dx2, dw2, v = h(B, H, T, D), h(B, H, T, D), f(D), pages.clone()
y2, y3, k_out, v_out = h(B, H, T, D), h(B, H, T, D), h(B, H, 20, D), h(B, H, 20, D)
calls = (lambda: gbattn.attn_qk_norm_rope(x, y, dx, dx2, pos, freq, w, w),
         lambda: gbattn.attn_qk_norm_rope_bwd(x, y, y2, y3, pos, freq, dx, dx2, w, w, dw, dw2, ws),
         lambda: gbattn.attn_paged_write(x, y, pages, v, table, lens, out),
         lambda: gbattn.attn_paged_read(pages, v, table, lens, k_out, v_out),
         lambda: gbattn.attn_fwd_paged(x, pages, v, table, lens, y, lse, ws, 0.1),
         lambda: gbattn.attn_draft_verify(p, None, z2, lse2, r, acc, tok))
z2, lse2, r = z(B, T), f(B, T) + 0.5, f(B) + 0.5
torch.cuda.synchronize()
for call in calls:
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out.zero_()
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
assert (y == 1).all() and out.tolist() == [8, 8] and acc.tolist() == [0, 0]
print("first calls refused, later ones captured")
"""


def test_first_call_inside_a_capture_is_refused():
    """In a process of its own: no call has set the library up yet."""
    run = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=ROOT, env=dict(os.environ, PYTHONPATH=ROOT), capture_output=True, text=True,
                         timeout=300)
    assert run.returncode == 0 and "later ones captured" in run.stdout, run.stdout[-2000:] + run.stderr[-2000:]


def guarded(shape, dtype, fill):
    """A tensor in the middle of a buffer, and the two guards beside it."""
    n = torch.Size(shape).numel() * torch.empty((), dtype=dtype).element_size()
    buf = torch.full((n + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
    t = buf[4096: 4096 + n].view(dtype).view(shape)
    return t.fill_(fill), (buf[:4096], buf[4096 + n:])


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("q8", [False, True])
def test_memory_beside_the_outputs(D, q8):
    """Odd sizes, every output between guards: they stay as they were."""
    gen = torch.Generator().manual_seed(31)
    guards = []

    def out(*shape, dtype=BF, fill=0):
        t, g = guarded(shape, dtype, fill)
        guards.extend(g)
        return t

    def rand(*shape):
        return torch.randn(shape, generator=gen).to(BF).cuda()

    B, Hq, Hkv, T, page, per_seq = 3, 6, 2, 5, 8, 5
    q, k, do, dk = rand(B, Hq, T, D), rand(B, Hkv, T, D), rand(B, Hq, T, D), rand(B, Hkv, T, D)
    pos, freq, w = torch.arange(T, dtype=torch.int32, device="cuda").expand(B, T).contiguous(), torch.rand(8, generator=gen).cuda(), rand(D)
    qo, ko = out(B, Hq, T, D), out(B, Hkv, T, D)
    gbattn.attn_qk_norm_rope(q, k, qo, ko, pos, freq, w, w)
    need = gbattn.attn_qk_norm_rope_workspace_bytes(D)
    gbattn.attn_qk_norm_rope_bwd(q, k, do, dk, pos, freq, out(B, Hq, T, D), out(B, Hkv, T, D), w, w, out(D, dtype=torch.float32),
                                 out(D, dtype=torch.float32), out(need, dtype=torch.uint8))
    held = torch.float8_e4m3fn if q8 else BF
    n = B * per_seq
    if q8:
        kp, vp = out(n, Hkv, page, D, dtype=torch.uint8).view(held), out(n, Hkv, page, D, dtype=torch.uint8).view(held)
        ke, ve = out(n, Hkv, page, dtype=torch.int8), out(n, Hkv, page, dtype=torch.int8)
    else:
        kp, vp, ke, ve = out(n, Hkv, page, D), out(n, Hkv, page, D), None, None
    table = torch.randperm(n, generator=gen).view(B, per_seq).to(torch.int32).cuda()
    lens, after = torch.tensor([0, 38, 17], dtype=torch.int32, device="cuda"), out(B, dtype=torch.int32)
    for _ in range(3):
        gbattn.attn_paged_write(ko, k, kp, vp, table, lens, after, k_exp=ke, v_exp=ve)
    assert after.tolist() == [5, 40, 22]
    gbattn.attn_paged_read(kp, vp, table, after, out(B, Hkv, 39, D), out(B, Hkv, 39, D), k_exp=ke, v_exp=ve)
    ws = out(gbattn.attn_paged_workspace_bytes(B, Hq, Hkv, T, page, per_seq, D), dtype=torch.uint8)
    gbattn.attn_fwd_paged(qo, kp, vp, table, after, out(B, Hq, T, D), out(B, Hq, T, dtype=torch.float32), ws, 0.1, k_exp=ke, v_exp=ve)
    # a table with room that no sequence fills: equal pieces and a join, few of them with work
    wide = torch.full((B, 4096), -1, dtype=torch.int32, device="cuda")
    wide[:, :per_seq] = table
    ws = out(gbattn.attn_paged_workspace_bytes(B, Hq, Hkv, T, page, 4096, D), dtype=torch.uint8)
    gbattn.attn_fwd_paged(qo, kp, vp, wide, after, out(B, Hq, T, D), out(B, Hq, T, dtype=torch.float32), ws, 0.1, k_exp=ke, v_exp=ve)
    V = 333
    target = torch.softmax(torch.randn(B, T + 1, V, generator=gen), -1).cuda()
    gbattn.attn_draft_verify(target, target[:, :T].contiguous(), torch.zeros(B, T, dtype=torch.int32, device="cuda"), torch.rand(B, T).cuda(),
                             torch.rand(B).cuda(), out(B, dtype=torch.int32), out(B, dtype=torch.int32))
    torch.cuda.synchronize()
    assert gbattn.attn_last_device_status() == gbattn.ATTN_OK
    assert all(bool((g == 0x5A).all()) for g in guards)


@pytest.mark.parametrize("q8", [False, True])
def test_room_does_not_change_the_result(q8):
    """The same tokens in a small table (a cluster per head) and in a large one (pieces and a join): the same to rounding."""
    gen = torch.Generator().manual_seed(32)
    B, Hq, Hkv, D, page, n = 2, 8, 2, 128, 16, 300
    per_seq = -(-n // page)
    if q8:
        import oracle.step as S

        (kc, ke), (vc, ve) = (S.quantise(torch.randn(B * per_seq, Hkv, page, D, generator=gen).double().numpy()) for _ in range(2))
        kp, vp = (torch.from_numpy(c).float().to(torch.float8_e4m3fn).cuda() for c in (kc, vc))
        ke, ve = (torch.from_numpy(e).to(torch.int8).cuda() for e in (ke, ve))
    else:
        kp, vp = (torch.randn(B * per_seq, Hkv, page, D, generator=gen).to(BF).cuda() for _ in range(2))
        ke = ve = None
    table = torch.randperm(B * per_seq, generator=gen).view(B, per_seq).to(torch.int32).cuda()
    wide = torch.zeros(B, 20000, dtype=torch.int32, device="cuda")
    wide[:, :per_seq] = table
    q = torch.randn(B, Hq, 1, D, generator=gen).to(BF).cuda()
    lens = torch.tensor([n, 7], dtype=torch.int32, device="cuda")
    got = []
    for t in (table, wide):
        o, lse = torch.empty_like(q), torch.empty(B, Hq, 1, device="cuda")
        gbattn.attn_fwd_paged(q, kp, vp, t, lens, o, lse, gbattn.paged_workspace(q, kp, t), 0.09, k_exp=ke, v_exp=ve)
        got.append((o.float(), lse))
    torch.cuda.synchronize()
    assert gbattn.attn_last_device_status() == gbattn.ATTN_OK
    # P's rounding and O's, each by a path of its own: 2 (2^-8 + 2^-8) of the largest value; the sums' order: 2^-18 of lse's few units
    assert float((got[0][0] - got[1][0]).abs().max()) <= 4 * 2.0 ** -8 * 5.5
    assert float((got[0][1] - got[1][1]).abs().max()) <= 2.0 ** -16


@pytest.mark.skipif(os.environ.get("GBATTN_DEBUG") == "1", reason="this is the child")
def test_no_index_check_fires():
    """These cases and the parity tests in the debug build, whose kernels check their indices."""
    from bwd_flashattention_fwd_gb300 import build

    build.build(debug=True)
    run = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-k", "not 32_bits and not capture", os.path.abspath(__file__),
                          os.path.join(ROOT, "tests", "test_step_ops_gpu.py")],
                         cwd=ROOT, env=dict(os.environ, GBATTN_DEBUG="1"), capture_output=True, text=True, timeout=900)
    assert run.returncode == 0, run.stdout[-3000:] + run.stderr[-1000:]
