"""Thin Python binding of libgbattn.so (declared in include/gbattn.h).

Argument marshalling only: torch tensors supply device pointers, shapes and
the stream; every step of the computation runs in the library's CUDA kernels.
There is no fallback: if the library is missing or a call fails, an exception
is raised.
"""

from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgbattn.so")
# the debug build: the same kernels with index checks (GBATTN_DEBUG_CHECKS)
DEBUG_LIB_PATH = os.path.join(_HERE, "libgbattn_debug.so")

ATTN_OK = 0
ATTN_ERR_INVALID_ARG = 1
ATTN_ERR_UNSUPPORTED = 2
ATTN_ERR_CUDA = 3
ATTN_ERR_TIMEOUT = 4
ATTN_ERR_DEVICE_CHECK = 5
ATTN_DTYPE_FP16 = 0
ATTN_DTYPE_BF16 = 1

EXPORTED = ("attn_fwd", "attn_bwd_delta", "attn_bwd", "attn_bwd_dq", "attn_bwd_dkv", "attn_bwd_noalloc",
            "attn_fwd_masked", "attn_bwd_masked", "attn_fwd_ex", "attn_bwd_ex", "attn_decode_workspace_bytes",
            "attn_fwd_decode", "attn_bwd_decode", "attn_last_device_status", "attn_wait_probe", "attn_status_string",
            "lce_workspace_bytes", "lce_fwd", "lce_bwd", "attn_tree_workspace_bytes", "attn_fwd_tree",
            "attn_cache_append", "attn_key_weight_workspace_bytes", "attn_key_weight",
            "attn_cache_evict_workspace_bytes", "attn_cache_evict")

_lib = None


class AttnError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call} failed: {status_string(status)} ({status})")


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libgbattn.so once and declare its C signatures.  With
    GBATTN_DEBUG=1 in the environment the process uses the debug build
    (libgbattn_debug.so) instead."""
    global _lib
    if _lib is not None:
        return _lib
    if path is None:
        path = DEBUG_LIB_PATH if os.environ.get("GBATTN_DEBUG") == "1" else LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is not built; run bwd_flashattention_fwd_gb300.build.build() (or __graft_entry__.build())"
        )
    lib = ctypes.CDLL(path)
    vp, ci, cf = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.attn_fwd.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, cf, ci, ci, vp]
    lib.attn_fwd.restype = ci
    lib.attn_bwd_delta.argtypes = [vp, vp, vp, ci, ci, ci, ci, ci, vp]
    lib.attn_bwd_delta.restype = ci
    lib.attn_bwd.argtypes = [vp] * 10 + [ci, ci, ci, ci, ci, ci, cf, ci, ci, vp]
    lib.attn_bwd.restype = ci
    lib.attn_bwd_dq.argtypes = [vp] * 7 + [ci, ci, ci, ci, ci, ci, cf, ci, ci, vp]
    lib.attn_bwd_dq.restype = ci
    lib.attn_bwd_dkv.argtypes = [vp] * 8 + [ci, ci, ci, ci, ci, ci, cf, ci, ci, vp]
    lib.attn_bwd_dkv.restype = ci
    lib.attn_bwd_noalloc.argtypes = [vp] * 9 + [ci, ci, ci, ci, ci, ci, cf, ci, ci, vp]
    lib.attn_bwd_noalloc.restype = ci
    lib.attn_fwd_masked.argtypes = [vp] * 6 + [ci, ci, ci, ci, ci, ci, cf, ci, ci, vp]
    lib.attn_fwd_masked.restype = ci
    lib.attn_bwd_masked.argtypes = [vp] * 11 + [ci, ci, ci, ci, ci, ci, cf, ci, ci, vp]
    lib.attn_bwd_masked.restype = ci
    i64 = ctypes.c_int64
    lib.attn_fwd_ex.argtypes = [vp] * 6 + [i64, ci, ci, ci, ci, ci, ci, cf, ci, ci, vp]
    lib.attn_fwd_ex.restype = ci
    lib.attn_bwd_ex.argtypes = [vp] * 8 + [i64] + [vp] * 3 + [ci, ci, ci, ci, ci, ci, cf, ci, ci, vp]
    lib.attn_bwd_ex.restype = ci
    sz = ctypes.c_size_t
    lib.attn_decode_workspace_bytes.argtypes = [ci] * 6
    lib.attn_decode_workspace_bytes.restype = sz
    lib.attn_fwd_decode.argtypes = [vp] * 6 + [sz, ci, ci, ci, ci, ci, ci, cf, ci, ci, vp]
    lib.attn_fwd_decode.restype = ci
    lib.attn_bwd_decode.argtypes = [vp] * 11 + [sz, ci, ci, ci, ci, ci, ci, cf, ci, ci, vp]
    lib.attn_bwd_decode.restype = ci
    lib.lce_workspace_bytes.argtypes = [ci, ci, ci]
    lib.lce_workspace_bytes.restype = sz
    lib.lce_fwd.argtypes = [vp] * 6 + [sz, ci, ci, ci, ci, vp]
    lib.lce_fwd.restype = ci
    lib.lce_bwd.argtypes = [vp] * 8 + [sz, ci, ci, ci, ci, vp]
    lib.lce_bwd.restype = ci
    lib.attn_tree_workspace_bytes.argtypes = [ci] * 6
    lib.attn_tree_workspace_bytes.restype = sz
    lib.attn_fwd_tree.argtypes = [vp] * 11 + [sz, i64] + [ci] * 6 + [cf, ci, vp]
    lib.attn_fwd_tree.restype = ci
    lib.attn_cache_append.argtypes = [vp] * 12 + [i64] + [ci] * 6 + [vp]
    lib.attn_cache_append.restype = ci
    lib.attn_key_weight_workspace_bytes.argtypes = [ci] * 6
    lib.attn_key_weight_workspace_bytes.restype = sz
    lib.attn_key_weight.argtypes = [vp] * 7 + [sz, i64] + [ci] * 6 + [cf, ci, ci, vp]
    lib.attn_key_weight.restype = ci
    lib.attn_cache_evict_workspace_bytes.argtypes = [ci] * 3
    lib.attn_cache_evict_workspace_bytes.restype = sz
    lib.attn_cache_evict.argtypes = [vp] * 10 + [sz, i64] + [ci] * 7 + [vp]
    lib.attn_cache_evict.restype = ci
    lib.attn_last_device_status.argtypes = [vp]
    lib.attn_last_device_status.restype = ci
    lib.attn_wait_probe.argtypes = [vp]
    lib.attn_wait_probe.restype = ci
    lib.attn_status_string.argtypes = [ci]
    lib.attn_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().attn_status_string(int(status)).decode()


_F32, _U8, _I32, _BF16, _F16 = torch.float32, torch.uint8, torch.int32, torch.bfloat16, torch.float16


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype is _BF16:
        return ATTN_DTYPE_BF16
    if t.dtype is _F16:
        return ATTN_DTYPE_FP16
    raise TypeError(f"unsupported dtype {t.dtype}; expected bfloat16 or float16")


# torch.cuda.current_device() without its check that CUDA is initialised (a CUDA tensor exists by then)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
# the handle of a device's current stream, without a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _stream_handle(stream) -> int:
    if stream is None:
        return _raw_stream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _require(call: str, dense=(), sliced=(), f32=(), u8=(), i32=()):
    """Reject tensors the C ABI cannot take before any pointer crosses it.
    dense: 16-bit tensors that must be contiguous (one dtype for all of them
    and for `sliced`); sliced: 16-bit tensors whose layout the caller has
    checked separately (k / v slices of a cache); f32 / u8 / i32: contiguous
    float32 / uint8 / int32 tensors.  Every tensor must be on the current CUDA
    device.  None entries are skipped."""
    half = None
    dev = None
    for ts, want, contig in ((dense, None, True), (sliced, None, False), (f32, _F32, True), (u8, _U8, True),
                             (i32, _I32, True)):
        for t in ts:
            if t is None:
                continue
            d = t.get_device() if isinstance(t, torch.Tensor) else -1
            if d != dev:
                if d < 0 or not t.is_cuda:
                    raise ValueError(f"{call}: every tensor must be a CUDA tensor; got {getattr(t, 'device', type(t))}")
                dev = torch.cuda.current_device()
                if d != dev:
                    raise ValueError(
                        f"{call}: every tensor must be on the current CUDA device (cuda:{dev}); got {t.device}")
            if contig and not t.is_contiguous():
                raise ValueError(f"{call}: tensor of shape {tuple(t.shape)} strides {t.stride()} is not contiguous")
            dt = t.dtype
            if want is not None:
                if dt is not want:
                    raise TypeError(f"{call}: expected {want}, got {dt}")
            elif dt is not half:
                if half is not None or (dt is not _BF16 and dt is not _F16):
                    raise TypeError(f"{call}: 16-bit tensors must all be bfloat16 or all float16; got {dt}")
                half = dt


def _check(status: int, call: str, check: bool) -> int:
    if check and status != ATTN_OK:
        raise AttnError(status, call)
    return status


def attn_fwd(q, k, v, o, lse, scale: float, causal: bool, stream=None, check: bool = True) -> int:
    """O and base-2 LSE of causal/non-causal GQA attention (writes o, lse)."""
    _require("attn_fwd", dense=(q, k, v, o), f32=(lse,))
    B, Hq, Lq, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    st = load_library().attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Lq, Lk, D,
                                 float(scale), int(bool(causal)), _dtype_code(q), _stream_handle(stream))
    return _check(st, "attn_fwd", check)


def attn_bwd_delta(o, dO, delta, stream=None, check: bool = True) -> int:
    """delta = rowsum(dO * O) in float32 (writes delta)."""
    _require("attn_bwd_delta", dense=(o, dO), f32=(delta,))
    B, Hq, Lq, D = o.shape
    st = load_library().attn_bwd_delta(_ptr(o), _ptr(dO), _ptr(delta), B, Hq, Lq, D, _dtype_code(o),
                                       _stream_handle(stream))
    return _check(st, "attn_bwd_delta", check)


def attn_bwd(q, k, v, o, dO, lse, delta, dq, dk, dv, scale: float, causal: bool, stream=None,
             check: bool = True) -> int:
    """dQ, dK, dV of the attention (writes dq, dk, dv)."""
    _require("attn_bwd", dense=(q, k, v, o, dO, dq, dk, dv), f32=(lse, delta))
    B, Hq, Lq, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    st = load_library().attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(delta),
                                 _ptr(dq), _ptr(dk), _ptr(dv), B, Hq, Hkv, Lq, Lk, D, float(scale),
                                 int(bool(causal)), _dtype_code(q), _stream_handle(stream))
    return _check(st, "attn_bwd", check)


def attn_bwd_dq(q, k, v, dO, lse, delta, dq, scale: float, causal: bool, stream=None, check: bool = True) -> int:
    """dQ only (the query-row-owning half of attn_bwd)."""
    _require("attn_bwd_dq", dense=(q, k, v, dO, dq), f32=(lse, delta))
    B, Hq, Lq, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    st = load_library().attn_bwd_dq(_ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(lse), _ptr(delta), _ptr(dq), B, Hq,
                                    Hkv, Lq, Lk, D, float(scale), int(bool(causal)), _dtype_code(q),
                                    _stream_handle(stream))
    return _check(st, "attn_bwd_dq", check)


def attn_bwd_dkv(q, k, v, dO, lse, delta, dk, dv, scale: float, causal: bool, stream=None,
                 check: bool = True) -> int:
    """dK and dV only (the key-row-owning half of attn_bwd)."""
    _require("attn_bwd_dkv", dense=(q, k, v, dO, dk, dv), f32=(lse, delta))
    B, Hq, Lq, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    st = load_library().attn_bwd_dkv(_ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(lse), _ptr(delta), _ptr(dk),
                                     _ptr(dv), B, Hq, Hkv, Lq, Lk, D, float(scale), int(bool(causal)),
                                     _dtype_code(q), _stream_handle(stream))
    return _check(st, "attn_bwd_dkv", check)


def attn_bwd_noalloc(q, k, v, o, dO, lse, dq, dk, dv, scale: float, causal: bool, stream=None,
                     check: bool = True) -> int:
    """attn_bwd for callers that cannot allocate device memory: delta and the
    status word live in the library's fixed scratch array (B*Hq*Lq <= 2**20)."""
    _require("attn_bwd_noalloc", dense=(q, k, v, o, dO, dq, dk, dv), f32=(lse,))
    B, Hq, Lq, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    st = load_library().attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(dq),
                                         _ptr(dk), _ptr(dv), B, Hq, Hkv, Lq, Lk, D, float(scale),
                                         int(bool(causal)), _dtype_code(q), _stream_handle(stream))
    return _check(st, "attn_bwd_noalloc", check)


def attn_fwd_masked(q, k, v, o, lse, block_mask, scale: float, causal: bool, stream=None,
                    check: bool = True) -> int:
    """attn_fwd with a uint8 block mask [ceil(Lq/128), ceil(Lk/128)] on the device."""
    _require("attn_fwd_masked", dense=(q, k, v, o), f32=(lse,), u8=(block_mask,))
    B, Hq, Lq, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    st = load_library().attn_fwd_masked(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(block_mask), B, Hq,
                                        Hkv, Lq, Lk, D, float(scale), int(bool(causal)), _dtype_code(q),
                                        _stream_handle(stream))
    return _check(st, "attn_fwd_masked", check)


def attn_bwd_masked(q, k, v, o, dO, lse, delta, block_mask, dq, dk, dv, scale: float, causal: bool, stream=None,
                    check: bool = True) -> int:
    """attn_bwd with the block mask of attn_fwd_masked."""
    _require("attn_bwd_masked", dense=(q, k, v, o, dO, dq, dk, dv), f32=(lse, delta), u8=(block_mask,))
    B, Hq, Lq, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    st = load_library().attn_bwd_masked(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(delta),
                                        _ptr(block_mask), _ptr(dq), _ptr(dk), _ptr(dv), B, Hq, Hkv, Lq, Lk, D,
                                        float(scale), int(bool(causal)), _dtype_code(q), _stream_handle(stream))
    return _check(st, "attn_bwd_masked", check)


def kv_row_pitch(k, v) -> int:
    """Row pitch of k and v for attn_fwd_ex / attn_bwd_ex: 0 when both are
    contiguous, else the capacity P of a [B, Hkv, P, D] buffer they are the
    first Lk rows of (cache[:, :, :Lk, :]).  Any other layout is rejected,
    expanded heads (stride 0) and heads that overlap among them: the calls
    count on P >= Lk rows of storage per head, and 0 means "contiguous" to them."""
    if k.is_contiguous() and v.is_contiguous():
        return 0
    B, Hkv, Lk, D = k.shape
    st = k.stride()
    if (st[3] != 1 or st[2] != D or st[1] % D or st[1] < Lk * D or st[0] != Hkv * st[1]
            or tuple(v.stride()) != tuple(st)):
        raise ValueError(f"k/v strides {tuple(k.stride())}, {tuple(v.stride())} are not a slice of a "
                         f"[B, Hkv, capacity, D] cache")
    return st[1] // D


def attn_fwd_ex(q, k, v, o, lse, scale: float, causal: bool, block_mask=None, kv_pitch=None, stream=None,
                check: bool = True) -> int:
    """attn_fwd with an optional block mask and k / v sliced from a longer
    cache (kv_pitch None: taken from the tensors' strides)."""
    _require("attn_fwd_ex", dense=(q, o), sliced=(k, v), f32=(lse,), u8=(block_mask,))
    B, Hq, Lq, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    pitch = kv_row_pitch(k, v) if kv_pitch is None else int(kv_pitch)
    st = load_library().attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(block_mask), pitch, B, Hq,
                                    Hkv, Lq, Lk, D, float(scale), int(bool(causal)), _dtype_code(q),
                                    _stream_handle(stream))
    return _check(st, "attn_fwd_ex", check)


def attn_bwd_ex(q, k, v, o, dO, lse, delta, dq, dk, dv, scale: float, causal: bool, block_mask=None, kv_pitch=None,
                stream=None, check: bool = True) -> int:
    """attn_bwd with the options of attn_fwd_ex (dk, dv contiguous)."""
    _require("attn_bwd_ex", dense=(q, o, dO, dq, dk, dv), sliced=(k, v), f32=(lse, delta), u8=(block_mask,))
    B, Hq, Lq, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    pitch = kv_row_pitch(k, v) if kv_pitch is None else int(kv_pitch)
    st = load_library().attn_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(delta),
                                    _ptr(block_mask), pitch, _ptr(dq), _ptr(dk), _ptr(dv), B, Hq, Hkv, Lq, Lk, D,
                                    float(scale), int(bool(causal)), _dtype_code(q), _stream_handle(stream))
    return _check(st, "attn_bwd_ex", check)


def attn_decode_workspace_bytes(B: int, Hq: int, Hkv: int, Lq: int, Lk: int, D: int) -> int:
    """Bytes of device workspace attn_fwd_decode / attn_bwd_decode need (0: shape not served)."""
    return int(load_library().attn_decode_workspace_bytes(B, Hq, Hkv, Lq, Lk, D))


def decode_workspace(q, k) -> torch.Tensor:
    """A workspace tensor (uint8, on q's device) for the decode calls on q, k."""
    B, Hq, Lq, D = q.shape
    n = attn_decode_workspace_bytes(B, Hq, k.shape[1], Lq, k.shape[2], D)
    if n == 0:
        raise AttnError(ATTN_ERR_UNSUPPORTED, "attn_decode_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def attn_fwd_decode(q, k, v, o, lse, workspace, scale: float, causal: bool, stream=None, check: bool = True) -> int:
    """attn_fwd for short query lengths (G * Lq <= 128), key range split over CTAs."""
    _require("attn_fwd_decode", dense=(q, k, v, o), f32=(lse,), u8=(workspace,))
    B, Hq, Lq, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    st = load_library().attn_fwd_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), B, Hq, Hkv, Lq, Lk, D,
                                        float(scale), int(bool(causal)), _dtype_code(q), _stream_handle(stream))
    return _check(st, "attn_fwd_decode", check)


def attn_bwd_decode(q, k, v, o, dO, lse, delta, dq, dk, dv, workspace, scale: float, causal: bool, stream=None,
                    check: bool = True) -> int:
    """attn_bwd for short query lengths (G * Lq <= 128)."""
    _require("attn_bwd_decode", dense=(q, k, v, o, dO, dq, dk, dv), f32=(lse, delta), u8=(workspace,))
    B, Hq, Lq, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    st = load_library().attn_bwd_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(delta),
                                        _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), B, Hq, Hkv, Lq, Lk, D,
                                        float(scale), int(bool(causal)), _dtype_code(q), _stream_handle(stream))
    return _check(st, "attn_bwd_decode", check)


def lce_workspace_bytes(N: int, Dm: int, V: int) -> int:
    """Bytes of device workspace lce_fwd / lce_bwd need (0: shape rejected)."""
    return int(load_library().lce_workspace_bytes(N, Dm, V))


def lce_workspace(hidden, weight) -> torch.Tensor:
    N, Dm = hidden.shape
    n = lce_workspace_bytes(N, Dm, weight.shape[0])
    if n == 0:
        raise AttnError(ATTN_ERR_UNSUPPORTED, "lce_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=hidden.device)


def lce_fwd(hidden, weight, targets, loss, lse, workspace, stream=None, check: bool = True) -> int:
    """Per-row linear cross-entropy loss and natural-log lse (writes loss, lse)."""
    _require("lce_fwd", dense=(hidden, weight), f32=(loss, lse), u8=(workspace,), i32=(targets,))
    N, Dm = hidden.shape
    st = load_library().lce_fwd(_ptr(hidden), _ptr(weight), _ptr(targets), _ptr(loss), _ptr(lse), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), N, Dm, weight.shape[0],
                                _dtype_code(hidden), _stream_handle(stream))
    return _check(st, "lce_fwd", check)


def lce_bwd(hidden, weight, targets, lse, dloss, dhidden, dweight, workspace, stream=None, check: bool = True) -> int:
    """dhidden and dweight of sum_i dloss[i] * loss[i] (writes both)."""
    _require("lce_bwd", dense=(hidden, weight, dhidden, dweight), f32=(lse, dloss), u8=(workspace,),
             i32=(targets,))
    N, Dm = hidden.shape
    st = load_library().lce_bwd(_ptr(hidden), _ptr(weight), _ptr(targets), _ptr(lse), _ptr(dloss), _ptr(dhidden),
                                _ptr(dweight), _ptr(workspace), workspace.numel() * workspace.element_size(), N, Dm,
                                weight.shape[0], _dtype_code(hidden), _stream_handle(stream))
    return _check(st, "lce_bwd", check)


# The serving calls below run every few tens of microseconds, so what their
# checks cost counts: each tests all of its tensors in one expression (the
# same conditions as _require and _shapes, which are called only when it does
# not hold, to name what is wrong and raise).


def _plain(t, dtype, dev: int, shape) -> bool:
    return t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and t.shape == shape


def _shapes(call: str, *named) -> None:
    """Reject (tensor or None, wanted shape, name) triples whose shapes differ from what the call reads."""
    for t, want, name in named:
        if t is not None and t.shape != want:
            raise ValueError(f"{call}: {name} has shape {tuple(t.shape)}; expected {tuple(want)}")


def _cache_pitch(call: str, k, v, p: int) -> int:
    """A serving call's explicit kv_pitch p, where it is the layout that the
    strides of k and v say.  A larger one would reach past the tensors; one
    below Lk is the C ABI's to refuse."""
    own, Lk = kv_row_pitch(k, v), k.shape[2]
    if k.shape[0] * k.shape[1] > 1 and (p or Lk) != (own or Lk) and not (own == 0 and p < Lk):
        raise ValueError(f"{call}: kv_pitch {p} is not the layout of k and v ({own or Lk} rows between heads)")
    return p


def attn_tree_workspace_bytes(B: int, Hq: int, Hkv: int, T: int, Lk: int, D: int) -> int:
    """Bytes of device workspace attn_fwd_tree needs (0: shape not served)."""
    return int(load_library().attn_tree_workspace_bytes(B, Hq, Hkv, T, Lk, D))


def _workspace(n: int, call: str, device) -> torch.Tensor:
    if n == 0:
        raise AttnError(ATTN_ERR_UNSUPPORTED, call)
    return torch.empty(n, dtype=torch.uint8, device=device)


def tree_workspace(q, k) -> torch.Tensor:
    """A workspace tensor for attn_fwd_tree on drafts q [B,Hq,T,D] over a cache k [B,Hkv,Lk,D]."""
    B, Hq, T, D = q.shape
    return _workspace(attn_tree_workspace_bytes(B, Hq, k.shape[1], T, k.shape[2], D), "attn_tree_workspace_bytes",
                      q.device)


def attn_fwd_tree(q, k, v, k_new, v_new, cache_len, o, lse, workspace, scale: float, tree_mask=None, tree_len=None,
                  kv_pitch=None, stream=None, check: bool = True) -> int:
    """Attention of drafted tokens over a cache and each other (writes o, lse):
    cache_len [B] int32 context lengths, tree_len [B] int32 draft counts (None:
    all T), tree_mask uint8 [B,T,T] (None: a chain).  k and v may be slices of
    a longer cache, as for attn_fwd_ex."""
    B, Hq, T, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    dt, dev, lens, new = q.dtype, q.get_device(), (B,), (B, Hkv, T, D)
    if not (dev >= 0 and dev == _current_device() and (dt is _BF16 or dt is _F16)
            and dt is k.dtype is v.dtype is k_new.dtype is v_new.dtype is o.dtype
            and lse.dtype is _F32 and cache_len.dtype is _I32 and workspace.dtype is _U8
            and dev == k.get_device() == v.get_device() == k_new.get_device() == v_new.get_device() == o.get_device()
            == lse.get_device() == cache_len.get_device() == workspace.get_device()
            and q.is_contiguous() and k_new.is_contiguous() and v_new.is_contiguous() and o.is_contiguous()
            and lse.is_contiguous() and cache_len.is_contiguous() and workspace.is_contiguous()
            and (k.shape, v.shape, k_new.shape, v_new.shape, o.shape, lse.shape, cache_len.shape)
            == ((B, Hkv, Lk, D), k.shape, new, new, q.shape, (B, Hq, T), lens)
            and (tree_len is None or _plain(tree_len, _I32, dev, lens))
            and (tree_mask is None or _plain(tree_mask, _U8, dev, (B, T, T)))):
        _require("attn_fwd_tree", dense=(q, k_new, v_new, o), sliced=(k, v), f32=(lse,), u8=(tree_mask, workspace),
                 i32=(cache_len, tree_len))
        _shapes("attn_fwd_tree", (k, (B, Hkv, Lk, D), "k"), (v, (B, Hkv, Lk, D), "v"), (k_new, new, "k_new"),
                (v_new, new, "v_new"), (o, q.shape, "o"), (lse, (B, Hq, T), "lse"), (cache_len, lens, "cache_len"),
                (tree_len, lens, "tree_len"), (tree_mask, (B, T, T), "tree_mask"))
    pitch = kv_row_pitch(k, v) if kv_pitch is None else _cache_pitch("attn_fwd_tree", k, v, int(kv_pitch))
    st = load_library().attn_fwd_tree(q.data_ptr(), k.data_ptr(), v.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
                                      _ptr(tree_mask), cache_len.data_ptr(), _ptr(tree_len), o.data_ptr(),
                                      lse.data_ptr(), workspace.data_ptr(), workspace.numel(), pitch, B, Hq, Hkv, T,
                                      Lk, D, float(scale), ATTN_DTYPE_BF16 if dt is _BF16 else ATTN_DTYPE_FP16,
                                      _raw_stream(dev) if stream is None else _stream_handle(stream))
    return _check(st, "attn_fwd_tree", check)


def attn_cache_append(k_new, v_new, k, v, cache_len, accept_len, cache_len_out, path=None, pos=None, seen=None,
                      seen_out=None, limit=None, kv_pitch=None, stream=None, check: bool = True) -> int:
    """Accepted drafts into the cache (writes k, v, cache_len_out and, where
    given, pos, seen_out, limit): rows path[b][:accept_len[b]] of k_new / v_new
    (None: all T rows; the first ones) become cache rows cache_len[b] on."""
    B, Hkv, T, D = k_new.shape
    Lk = k.shape[2]
    dt, dev, lens = k_new.dtype, k_new.get_device(), (B,)
    if not (dev >= 0 and dev == _current_device() and (dt is _BF16 or dt is _F16)
            and dt is v_new.dtype is k.dtype is v.dtype and cache_len.dtype is _I32 and cache_len_out.dtype is _I32
            and dev == v_new.get_device() == k.get_device() == v.get_device() == cache_len.get_device()
            == cache_len_out.get_device()
            and k_new.is_contiguous() and v_new.is_contiguous() and cache_len.is_contiguous()
            and cache_len_out.is_contiguous()
            and (v_new.shape, k.shape, v.shape, cache_len.shape, cache_len_out.shape)
            == (k_new.shape, (B, Hkv, Lk, D), k.shape, lens, lens)
            and (accept_len is None or _plain(accept_len, _I32, dev, lens))
            and (path is None or _plain(path, _I32, dev, (B, T)))
            and (pos is None or _plain(pos, _I32, dev, (B, Hkv, Lk)))
            and (seen is None or _plain(seen, _I32, dev, lens))
            and (seen_out is None or _plain(seen_out, _I32, dev, lens))
            and (limit is None or _plain(limit, _I32, dev, (B, T)))):
        _require("attn_cache_append", dense=(k_new, v_new), sliced=(k, v),
                 i32=(cache_len, accept_len, cache_len_out, path, pos, seen, seen_out, limit))
        _shapes("attn_cache_append", (k, (B, Hkv, Lk, D), "k"), (v, (B, Hkv, Lk, D), "v"),
                (v_new, k_new.shape, "v_new"), (cache_len, lens, "cache_len"), (accept_len, lens, "accept_len"),
                (cache_len_out, lens, "cache_len_out"), (path, (B, T), "path"), (pos, (B, Hkv, Lk), "pos"),
                (seen, lens, "seen"), (seen_out, lens, "seen_out"), (limit, (B, T), "limit"))
    pitch = kv_row_pitch(k, v) if kv_pitch is None else _cache_pitch("attn_cache_append", k, v, int(kv_pitch))
    st = load_library().attn_cache_append(k_new.data_ptr(), v_new.data_ptr(), _ptr(path), _ptr(accept_len),
                                          cache_len.data_ptr(), _ptr(seen), k.data_ptr(), v.data_ptr(), _ptr(pos),
                                          cache_len_out.data_ptr(), _ptr(seen_out), _ptr(limit), pitch, B, Hkv, T, Lk,
                                          D, ATTN_DTYPE_BF16 if dt is _BF16 else ATTN_DTYPE_FP16,
                                          _raw_stream(dev) if stream is None else _stream_handle(stream))
    return _check(st, "attn_cache_append", check)


def attn_key_weight_workspace_bytes(B: int, Hq: int, Hkv: int, Lq: int, Lk: int, D: int) -> int:
    """Bytes of device workspace attn_key_weight needs (0: shape not served)."""
    return int(load_library().attn_key_weight_workspace_bytes(B, Hq, Hkv, Lq, Lk, D))


def key_weight_workspace(q, k) -> torch.Tensor:
    """A workspace tensor for attn_key_weight on q [B,Hq,Lq,D] and k [B,Hkv,Lk,D]."""
    B, Hq, Lq, D = q.shape
    return _workspace(attn_key_weight_workspace_bytes(B, Hq, k.shape[1], Lq, k.shape[2], D),
                      "attn_key_weight_workspace_bytes", q.device)


def attn_key_weight(q, k, lse, weight, weight_out, workspace, scale: float, causal: bool = False, limit=None,
                    kv_pitch=None, stream=None, check: bool = True) -> int:
    """weight_out = weight (None: zeros) + the attention weight each key of k
    got from q's rows, whose base-2 log-sum-exps are lse; limit int32 [B,Lq]:
    how many keys each row sees (0: the row adds nothing)."""
    B, Hq, Lq, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    dt, dev, slots = q.dtype, q.get_device(), (B, Hkv, Lk)
    if not (dev >= 0 and dev == _current_device() and (dt is _BF16 or dt is _F16) and k.dtype is dt
            and lse.dtype is _F32 and weight_out.dtype is _F32 and workspace.dtype is _U8
            and dev == k.get_device() == lse.get_device() == weight_out.get_device() == workspace.get_device()
            and q.is_contiguous() and lse.is_contiguous() and weight_out.is_contiguous() and workspace.is_contiguous()
            and (k.shape, lse.shape, weight_out.shape) == ((B, Hkv, Lk, D), (B, Hq, Lq), slots)
            and (weight is None or _plain(weight, _F32, dev, slots))
            and (limit is None or _plain(limit, _I32, dev, (B, Lq)))):
        _require("attn_key_weight", dense=(q,), sliced=(k,), f32=(lse, weight, weight_out), u8=(workspace,),
                 i32=(limit,))
        _shapes("attn_key_weight", (k, (B, Hkv, Lk, D), "k"), (lse, (B, Hq, Lq), "lse"), (weight, slots, "weight"),
                (weight_out, slots, "weight_out"), (limit, (B, Lq), "limit"))
    pitch = kv_row_pitch(k, k) if kv_pitch is None else _cache_pitch("attn_key_weight", k, k, int(kv_pitch))
    st = load_library().attn_key_weight(q.data_ptr(), k.data_ptr(), lse.data_ptr(), _ptr(limit), _ptr(weight),
                                        weight_out.data_ptr(), workspace.data_ptr(), workspace.numel(), pitch, B, Hq,
                                        Hkv, Lq, Lk, D, float(scale), int(bool(causal)),
                                        ATTN_DTYPE_BF16 if dt is _BF16 else ATTN_DTYPE_FP16,
                                        _raw_stream(dev) if stream is None else _stream_handle(stream))
    return _check(st, "attn_key_weight", check)


def attn_cache_evict_workspace_bytes(B: int, Hkv: int, Lk: int) -> int:
    """Bytes of device workspace attn_cache_evict needs (0: shape not served)."""
    return int(load_library().attn_cache_evict_workspace_bytes(B, Hkv, Lk))


def evict_workspace(k) -> torch.Tensor:
    """A workspace tensor for attn_cache_evict on a cache k [B,Hkv,Lk,D]."""
    return _workspace(attn_cache_evict_workspace_bytes(*k.shape[:3]), "attn_cache_evict_workspace_bytes", k.device)


def attn_cache_evict(k, v, weight, pos, cache_len, seen, weight_out, pos_out, cache_len_out, workspace, keep: int,
                     recent: int, kv_pitch=None, stream=None, check: bool = True) -> int:
    """Keep, in every KV head, the `recent` newest tokens and the heaviest
    others, `keep` in all (changes k and v in place, writes weight_out,
    pos_out, cache_len_out)."""
    B, Hkv, Lk, D = k.shape
    dt, dev, lens, slots = k.dtype, k.get_device(), (B,), (B, Hkv, Lk)
    if not (dev >= 0 and dev == _current_device() and (dt is _BF16 or dt is _F16) and v.dtype is dt
            and weight.dtype is weight_out.dtype is _F32 and workspace.dtype is _U8
            and pos.dtype is cache_len.dtype is seen.dtype is pos_out.dtype is cache_len_out.dtype is _I32
            and dev == v.get_device() == weight.get_device() == pos.get_device() == cache_len.get_device()
            == seen.get_device() == weight_out.get_device() == pos_out.get_device() == cache_len_out.get_device()
            == workspace.get_device()
            and weight.is_contiguous() and pos.is_contiguous() and cache_len.is_contiguous() and seen.is_contiguous()
            and weight_out.is_contiguous() and pos_out.is_contiguous() and cache_len_out.is_contiguous()
            and workspace.is_contiguous()
            and (v.shape, weight.shape, pos.shape, weight_out.shape, pos_out.shape, cache_len.shape, seen.shape,
                 cache_len_out.shape) == (k.shape, slots, slots, slots, slots, lens, lens, lens)):
        _require("attn_cache_evict", sliced=(k, v), f32=(weight, weight_out), u8=(workspace,),
                 i32=(pos, cache_len, seen, pos_out, cache_len_out))
        _shapes("attn_cache_evict", (v, k.shape, "v"), (weight, slots, "weight"), (pos, slots, "pos"),
                (weight_out, slots, "weight_out"), (pos_out, slots, "pos_out"), (cache_len, lens, "cache_len"),
                (seen, lens, "seen"), (cache_len_out, lens, "cache_len_out"))
    pitch = kv_row_pitch(k, v) if kv_pitch is None else _cache_pitch("attn_cache_evict", k, v, int(kv_pitch))
    st = load_library().attn_cache_evict(k.data_ptr(), v.data_ptr(), weight.data_ptr(), pos.data_ptr(),
                                         cache_len.data_ptr(), seen.data_ptr(), weight_out.data_ptr(),
                                         pos_out.data_ptr(), cache_len_out.data_ptr(), workspace.data_ptr(),
                                         workspace.numel(), pitch, B, Hkv, Lk, D, int(keep), int(recent),
                                         ATTN_DTYPE_BF16 if dt is _BF16 else ATTN_DTYPE_FP16,
                                         _raw_stream(dev) if stream is None else _stream_handle(stream))
    return _check(st, "attn_cache_evict", check)


def attn_last_device_status(stream=None) -> int:
    return load_library().attn_last_device_status(_stream_handle(stream))


def attn_wait_probe(stream=None, check: bool = True) -> int:
    """Launch the failure-reporting check: one wait that can only run out
    (after GBATTN_WAIT_LIMIT_NS); the next attn_last_device_status reports
    ATTN_ERR_TIMEOUT."""
    return _check(load_library().attn_wait_probe(_stream_handle(stream)), "attn_wait_probe", check)


def attn_status_string(status: int) -> str:
    return status_string(status)


# ---------------------------------------------------------------------------
# Conveniences that allocate the outputs with torch and call the ABI.
# ---------------------------------------------------------------------------


def forward(q, k, v, scale: float, causal: bool = True, stream=None):
    B, Hq, Lq, D = q.shape
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device)
    attn_fwd(q, k, v, o, lse, scale, causal, stream)
    return o, lse


def delta(o, dO, stream=None):
    B, Hq, Lq, _ = o.shape
    d = torch.empty((B, Hq, Lq), dtype=torch.float32, device=o.device)
    attn_bwd_delta(o, dO, d, stream)
    return d


def backward(q, k, v, o, dO, lse, dlt, scale: float, causal: bool = True, stream=None):
    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dv = torch.empty_like(v)
    attn_bwd(q, k, v, o, dO, lse, dlt, dq, dk, dv, scale, causal, stream)
    return dq, dk, dv
