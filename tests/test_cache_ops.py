"""The cache calls' refusals (no GPU): every bad argument is an error on the
host, before any device memory is touched."""

import ctypes
import math

import pytest
import torch

from bwd_flashattention_fwd_gb300 import build, gbattn

INV, UNS = gbattn.ATTN_ERR_INVALID_ARG, gbattn.ATTN_ERR_UNSUPPORTED
FAKE = 0x10000  # a 16-byte aligned address that is never dereferenced
FAKE2 = 0x20000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gbattn.load_library()


def tree(lib, ptrs=None, mask=None, tree_len=None, nbytes=1 << 40, pitch=0, B=2, Hq=8, Hkv=2, T=8, Lk=100, D=128,
         scale=0.1, dtype=1, ws=FAKE):
    q, k, v, kn, vn, cl, o, lse = ptrs or [FAKE] * 6 + [FAKE2, FAKE]
    return lib.attn_fwd_tree(q, k, v, kn, vn, mask, cl, tree_len, o, lse, ws, nbytes, pitch, B, Hq, Hkv, T, Lk, D,
                             ctypes.c_float(scale), dtype, None)


def test_tree_rejects(lib):
    for i in range(8):
        ptrs = [FAKE] * 6 + [FAKE2, FAKE]
        ptrs[i] = None
        assert tree(lib, ptrs) == INV
        ptrs[i] = FAKE + (2 if i == 5 else 8)
        assert tree(lib, ptrs) == INV
    assert tree(lib, [FAKE] * 8) == INV  # o over q
    assert tree(lib, ws=None) == INV and tree(lib, ws=FAKE + 8) == INV
    assert tree(lib, tree_len=FAKE + 1) == INV
    need = lib.attn_tree_workspace_bytes(2, 8, 2, 8, 100, 128)
    assert need > 0 and tree(lib, nbytes=need - 1) == INV
    for kw in (dict(B=0), dict(Hq=0), dict(Hkv=0), dict(T=0), dict(Lk=0), dict(Hq=7), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(dtype=3), dict(pitch=-1),
               dict(pitch=99)):
        assert tree(lib, **kw) == INV, kw
    for kw in (dict(D=80), dict(D=512), dict(T=1025), dict(B=1025), dict(pitch=1 << 40), dict(Hkv=40000, Hq=40000),
               dict(T=1024, Hq=128), dict(Lk=(1 << 30) + 1), dict(Lk=1 << 30, B=1024)):
        assert tree(lib, **kw) == UNS, kw
    ws = lib.attn_tree_workspace_bytes
    assert ws(0, 8, 2, 8, 100, 128) == 0 and ws(2, 8, 3, 8, 100, 128) == 0 and ws(2, 8, 2, 1025, 100, 128) == 0
    assert ws(2, 8, 2, 8, 100, 100) == 0 and ws(2, 8, 2, 8, 0, 128) == 0


def weight(lib, ptrs=None, limit=None, win=None, nbytes=1 << 40, pitch=0, B=2, Hq=8, Hkv=2, Lq=8, Lk=100, D=128,
           scale=0.1, causal=0, dtype=1, ws=FAKE):
    q, k, lse, wout = ptrs or [FAKE] * 4
    return lib.attn_key_weight(q, k, lse, limit, win, wout, ws, nbytes, pitch, B, Hq, Hkv, Lq, Lk, D,
                               ctypes.c_float(scale), causal, dtype, None)


def test_key_weight_rejects(lib):
    for i in range(4):
        ptrs = [FAKE] * 4
        ptrs[i] = None
        assert weight(lib, ptrs) == INV
        ptrs[i] = FAKE + 8
        assert weight(lib, ptrs) == INV
    assert weight(lib, ws=None) == INV and weight(lib, win=FAKE + 4) == INV and weight(lib, limit=FAKE + 2) == INV
    need = lib.attn_key_weight_workspace_bytes(2, 8, 2, 8, 100, 128)
    assert need > 0 and weight(lib, nbytes=need - 1) == INV
    for kw in (dict(B=0), dict(Hq=0), dict(Lq=0), dict(Lk=0), dict(Hq=9), dict(scale=math.nan), dict(causal=2),
               dict(causal=1, Lq=101), dict(causal=1, limit=FAKE), dict(dtype=-1), dict(pitch=50)):
        assert weight(lib, **kw) == INV, kw
    for kw in (dict(D=72), dict(limit=FAKE, Lq=1025), dict(limit=FAKE, B=1025), dict(pitch=1 << 40),
               dict(Lk=(1 << 30) + 1), dict(Lq=(1 << 28) + 1), dict(Lq=1 << 22, Lk=1 << 24, B=16)):
        assert weight(lib, **kw) == UNS, kw
    ws = lib.attn_key_weight_workspace_bytes
    assert ws(2, 8, 2, 8, 100, 90) == 0 and ws(2, 7, 2, 8, 100, 128) == 0 and ws(2, 8, 2, 0, 100, 128) == 0


def append(lib, req=None, path=None, acc=None, seen=None, pos=None, seen_out=None, limit=None, pitch=0, B=2, Hkv=2,
           T=8, Lk=100, D=128, dtype=1):
    kn, vn, cl, k, v, clo = req or [FAKE, FAKE, FAKE, FAKE, FAKE, FAKE2]
    return lib.attn_cache_append(kn, vn, path, acc, cl, seen, k, v, pos, clo, seen_out, limit, pitch, B, Hkv, T, Lk, D,
                                 dtype, None)


def test_append_rejects(lib):
    good = [FAKE, FAKE, FAKE, FAKE, FAKE, FAKE2]
    for i in range(6):
        bad = list(good)
        bad[i] = None
        assert append(lib, bad) == INV
        bad[i] = FAKE2 + 2
        assert append(lib, bad) == INV
    assert append(lib, [FAKE, FAKE, FAKE, FAKE, FAKE, FAKE]) == INV  # new lengths over the old ones
    assert append(lib, pos=FAKE) == INV and append(lib, seen_out=FAKE) == INV  # need `seen`
    assert append(lib, seen=FAKE, seen_out=FAKE) == INV
    for name in ("path", "acc", "limit"):
        assert append(lib, **{name: FAKE + 1}) == INV
    for kw in (dict(B=0), dict(Hkv=0), dict(T=0), dict(Lk=0), dict(pitch=7), dict(dtype=9)):
        assert append(lib, **kw) == INV, kw
    assert append(lib, D=100) == UNS and append(lib, B=70000) == UNS
    assert append(lib, path=FAKE, T=1025, Lk=4000) == UNS


def evict(lib, ptrs=None, nbytes=1 << 40, ws=FAKE, pitch=0, B=2, Hkv=2, Lk=100, D=128, keep=50, recent=10, dtype=1):
    k, v, w, p, cl, seen, wo, po, clo = ptrs or [FAKE] * 6 + [FAKE2] * 3
    return lib.attn_cache_evict(k, v, w, p, cl, seen, wo, po, clo, ws, nbytes, pitch, B, Hkv, Lk, D, keep, recent,
                                dtype, None)


def test_evict_rejects(lib):
    good = [FAKE] * 6 + [FAKE2] * 3
    for i in range(9):
        bad = list(good)
        bad[i] = None
        assert evict(lib, bad) == INV
        bad[i] = FAKE2 + 2
        assert evict(lib, bad) == INV
    for i in (6, 7, 8):  # outputs over their inputs
        bad = list(good)
        bad[i] = FAKE
        assert evict(lib, bad) == INV
    need = lib.attn_cache_evict_workspace_bytes(2, 2, 100)
    assert need > 0 and evict(lib, nbytes=need - 1) == INV and evict(lib, ws=None) == INV
    for kw in (dict(keep=0), dict(keep=101), dict(recent=-1), dict(recent=51), dict(B=0), dict(Lk=0, keep=1),
               dict(pitch=60), dict(dtype=4)):
        assert evict(lib, **kw) == INV, kw
    assert evict(lib, D=48) == UNS and evict(lib, Lk=(1 << 20) + 1) == UNS
    ws = lib.attn_cache_evict_workspace_bytes
    assert ws(0, 1, 1) == 0 and ws(1, 1, (1 << 20) + 1) == 0 and ws(1, 1, 1) > 0


def test_binding_rejects_shapes_and_host_tensors():
    q = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    u = torch.zeros(64, dtype=torch.uint8)
    f = torch.zeros(1, 2, 3)
    for call in (lambda: gbattn.attn_fwd_tree(q, q, q, q, q, i, q, f, u, 0.1),
                 lambda: gbattn.attn_key_weight(q, q, f, None, f, u, 0.1),
                 lambda: gbattn.attn_cache_append(q, q, q, q, i, None, i),
                 lambda: gbattn.attn_cache_evict(q, q, f, i, i, i, f, i, i, u, 1, 0)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
