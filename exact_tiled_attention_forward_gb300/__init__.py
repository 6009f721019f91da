"""Exact tiled attention forward (FlashAttention forward) for GB300 / sm_103a.

The compute path is the C-ABI library ``libfa`` (``include/fa.h``): hand-written
CUDA kernels built for sm_103a by ``build.py``. This module is a thin binding
with the same entry-point names; it only marshals arguments (device pointers,
sizes, the current CUDA stream). There is no fallback: if ``libfa.so`` is
missing or fails to load, every call raises.

    import exact_tiled_attention_forward_gb300 as fa
    o, lse = fa.fa_forward(q, k, v, causal=False)          # torch CUDA tensors

Tensors: q ``[B, H_q, N_q, d]``, k/v ``[B, H_kv, N_k, d]`` BF16 (or FP16, through
``fa_forward_fp16``) contiguous; returns o ``[B, H_q, N_q, d]`` of the same type
and lse ``[B, H_q, N_q]`` FP32.

A paged K/V cache, 16-bit or E4M3, is written by ``fa_cache_append``, attended over by
``fa_extend_paged`` and read back by ``fa_cache_read`` (``include/fa_serving.h``);
``fa_forward_window`` and ``fa_backward_window`` are causal attention under a sliding
window with sinks (``include/fa_window.h``).
"""
from __future__ import annotations

import ctypes
import math
import os
import re

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libfa.so")
LIB_SINGLE_GPU_PATH = os.path.join(_PKG, "_build", "libfa_single_gpu.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "fa.h")
HEADER_SINGLE_GPU = os.path.join(os.path.dirname(_PKG), "include", "fa_single_gpu.h")
HEADER_SERVING = os.path.join(os.path.dirname(_PKG), "include", "fa_serving.h")
HEADER_WINDOW = os.path.join(os.path.dirname(_PKG), "include", "fa_window.h")

FA_OK = 0
FA_ERR_INVALID_ARG = -1
FA_ERR_UNSUPPORTED = -2
FA_ERR_CUDA = -3
FA_ERR_NO_MEMORY = -4
FA_ERR_TIMEOUT = -5
FA_ERR_TOO_LARGE = -6
FA_ERR_BOUNDS = -7

FA_DTYPE_BF16 = 0
FA_DTYPE_FP16 = 1

FA_CACHE_16BIT = 0
FA_CACHE_E4M3 = 1

_lib = None
_lib_single = None


class FaError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        msg = lib().fa_status_string(status).decode()
        if status == FA_ERR_CUDA:
            msg += f" (cudaError {lib().fa_get_last_cuda_error()})"
        super().__init__(f"{what}: {msg}" if what else msg)


_c_int, _c_float, _c_size, _vp = ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_void_p
_c_ll = ctypes.c_longlong

_SIGNATURES = {
    "fa_forward": (_c_int, [_vp, _vp, _vp, _vp, _vp] + [_c_int] * 7 + [_c_float, _vp]),
    "fa_forward_fp16": (_c_int, [_vp, _vp, _vp, _vp, _vp] + [_c_int] * 7 + [_c_float, _vp]),
    "fa_forward_fp8": (_c_int, [_vp, _vp, _vp, _vp, _vp] + [_c_int] * 7 + [_c_float] * 4 + [_vp]),
    "fa_forward_host": (_c_int, [_c_int] + [ctypes.POINTER(_vp)] * 5 + [_c_int] * 7 +
                        [_c_float, _c_int, _vp]),
    "fa_forward_host_packed": (_c_int, [_c_int] + [ctypes.POINTER(_vp)] * 2 + [_c_int] * 7 +
                               [_c_float, _c_int, _vp]),
    "fa_forward_noalloc": (_c_int, [_vp, _vp, _vp, _vp, _vp] + [_c_int] * 7 + [_c_float, _vp]),
    "fa_backward": (_c_int, [_vp] * 9 + [_c_int] * 7 + [_c_float, _c_int, _vp]),
    "fa_decode_paged": (_c_int, [_vp] * 7 + [_c_int] * 8 + [_c_float, _c_int, _vp]),
    "fa_forward_window": (_c_int, [_vp] * 5 + [_c_int] * 8 + [_c_float, _c_int, _vp]),
    "fa_backward_window": (_c_int, [_vp] * 9 + [_c_int] * 8 + [_c_float, _c_int, _vp]),
    "fa_cache_append": (_c_int, [_vp] * 9 + [_c_int] * 6 + [_c_ll] * 2 + [_c_int] * 2 + [_vp]),
    "fa_cache_read": (_c_int, [_vp] * 9 + [_c_int] * 8 + [_vp]),
    "fa_extend_paged": (_c_int, [_vp] * 10 + [_c_int] * 8 + [_c_ll] + [_c_int] * 2 + [_c_float] + [_c_int] * 2 +
                        [_vp]),
    "fa_naive_forward": (_c_int, [_vp, _vp, _vp, _vp, _vp] + [_c_int] * 7 +
                         [_c_float, _vp, _c_size, _vp]),
    "fa_naive_workspace_bytes": (_c_size, [_c_int] * 4),
    "fa_forward_plan": (_c_int, [_c_int] * 7 + [ctypes.POINTER(ctypes.c_longlong),
                                                ctypes.POINTER(_c_int), ctypes.POINTER(_c_size)]),
    "fa_selftest_wait_timeout": (_c_int, [ctypes.c_ulonglong, _vp]),
    "fa_selftest_bounds": (_c_int, [_vp]),
    "fa_debug_build": (_c_int, []),
    "fa_status_string": (ctypes.c_char_p, [_c_int]),
    "fa_get_last_cuda_error": (_c_int, []),
    "fa_device_status": (_c_int, [_c_int]),
    "fa_version": (_c_int, []),
}


def lib() -> ctypes.CDLL:
    """Load libfa.so (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libfa.so not found at {LIB_PATH}: build it first "
                              "(python -m exact_tiled_attention_forward_gb300.build)")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


def lib_single_gpu() -> ctypes.CDLL:
    """Load libfa_single_gpu.so (once): libfa plus the cluster-multicast forward
    of ``include/fa_single_gpu.h``. Only for a process that uses one GPU."""
    global _lib_single
    if _lib_single is None:
        if not os.path.exists(LIB_SINGLE_GPU_PATH):
            raise ImportError(f"libfa_single_gpu.so not found at {LIB_SINGLE_GPU_PATH}: build it first "
                              "(python -m exact_tiled_attention_forward_gb300.build)")
        l = ctypes.CDLL(LIB_SINGLE_GPU_PATH)
        sigs = dict(_SIGNATURES)
        sigs["fa_forward_cluster_multicast"] = _SIGNATURES["fa_forward"]
        for name, (res, args) in sigs.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib_single = l
    return _lib_single


def header_functions(header: str = HEADER) -> list[str]:
    """Names of the functions a header (default ``include/fa.h``) declares."""
    text = open(header).read()
    return sorted(set(re.findall(r"^\s*(?:int|size_t|const char\*)\s+(fa_\w+)\s*\(", text, re.M)))


def _check(status: int, what: str):
    if status != FA_OK:
        raise FaError(status, what)


def _stream_ptr(stream):
    """Raw handle of `stream` (a torch stream or an int), or of the current
    stream of the current device when None."""
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # ~10x cheaper than current_stream()
        if raw is not None:
            return raw(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _empty(shape, dtype, device, stream):
    """Memory that a call on `stream` (see _stream_ptr) writes. On another stream than the
    current one it belongs to that stream, whose earlier work is all that may still use it,
    and when it is dropped it stays untouched until the current stream, which will read
    it, has passed that point too."""
    import torch
    if stream is None or device.type != "cuda":   # (libfa refuses what is not on the device)
        return torch.empty(shape, dtype=dtype, device=device)
    handle = _stream_ptr(stream)
    here = torch.cuda.current_stream(device)
    if handle == here.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(here)
    return t


def _dims(q, k):
    B, H_q, N_q, d = q.shape
    Bk, H_kv, N_k, dk = k.shape
    if Bk != B or dk != d:
        raise ValueError("q and k/v disagree on batch or head dim")
    return B, H_q, H_kv, N_q, N_k, d


def _ptr(t):
    """Device address of a tensor as an int (0 for None or an empty tensor); the
    c_void_p argtypes take ints directly."""
    return t.data_ptr() if t is not None and t.numel() > 0 else 0


def _check_dtypes(dtype, q, k, v, out, lse):
    """All of q, k, v, out in `dtype`, lse FP32 (or None): libfa reads raw memory."""
    import torch
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        if t is not None and t.dtype != dtype:
            raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if lse is not None and lse.dtype != torch.float32:
        raise TypeError(f"lse is {lse.dtype}, expected torch.float32")


def fa_forward(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None,
               return_lse: bool = True, stream=None):
    """Fused forward on the current CUDA stream. Returns ``(o, lse)``.
    BF16 tensors; FP16 tensors are passed on to ``fa_forward_fp16``."""
    import torch
    if q.dtype == torch.float16:
        return fa_forward_fp16(q, k, v, causal=causal, scale=scale, out=out, lse=lse,
                               return_lse=return_lse, stream=stream)
    _check_dtypes(torch.bfloat16, q, k, v, out, lse)
    B, H_q, H_kv, N_q, N_k, d = _dims(q, k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _empty((B, H_q, N_q, d), torch.bfloat16, q.device, stream)
    if lse is None and return_lse:
        lse = _empty((B, H_q, N_q), torch.float32, q.device, stream)
    st = lib().fa_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H_q, H_kv, N_q, N_k,
                          d, int(bool(causal)), float(scale), _stream_ptr(stream))
    _check(st, "fa_forward")
    return out, lse


def fa_forward_fp16(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None,
                    return_lse: bool = True, stream=None):
    """Fused forward on FP16 q, k, v (FP16 o, FP32 lse). Returns ``(o, lse)``."""
    import torch
    _check_dtypes(torch.float16, q, k, v, out, lse)
    B, H_q, H_kv, N_q, N_k, d = _dims(q, k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _empty((B, H_q, N_q, d), torch.float16, q.device, stream)
    if lse is None and return_lse:
        lse = _empty((B, H_q, N_q), torch.float32, q.device, stream)
    st = lib().fa_forward_fp16(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H_q, H_kv, N_q,
                               N_k, d, int(bool(causal)), float(scale), _stream_ptr(stream))
    _check(st, "fa_forward_fp16")
    return out, lse


def fa_forward_fp8(q, k, v, descale, causal: bool = False, scale: float | None = None, out=None, lse=None,
                   return_lse: bool = True, stream=None):
    """Fused forward on FP8 E4M3 inputs: q, k, v hold E4M3 codes (torch.uint8 or
    torch.float8_e4m3fn, one byte each) standing for code * factor, with
    ``descale = (factor_q, factor_k, factor_v)``. Returns ``(o, lse)``: o BF16,
    lse FP32. d must be 64 or 128."""
    import torch
    allowed = {torch.uint8, getattr(torch, "float8_e4m3fn", torch.uint8)}
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype not in allowed:
            raise TypeError(f"{name} is {t.dtype}, expected E4M3 codes (torch.uint8 or torch.float8_e4m3fn)")
    if out is not None and out.dtype != torch.bfloat16:
        raise TypeError(f"out is {out.dtype}, expected torch.bfloat16")
    if lse is not None and lse.dtype != torch.float32:
        raise TypeError(f"lse is {lse.dtype}, expected torch.float32")
    B, H_q, H_kv, N_q, N_k, d = _dims(q, k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _empty((B, H_q, N_q, d), torch.bfloat16, q.device, stream)
    if lse is None and return_lse:
        lse = _empty((B, H_q, N_q), torch.float32, q.device, stream)
    dq, dk, dv = (float(x) for x in descale)
    st = lib().fa_forward_fp8(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H_q, H_kv, N_q, N_k,
                              d, int(bool(causal)), float(scale), dq, dk, dv, _stream_ptr(stream))
    _check(st, "fa_forward_fp8")
    return out, lse


def fa_forward_host(qs, ks, vs, outs, lses=None, causal: bool = False, scale: float | None = None,
                    stream=None) -> None:
    """n requests whose tensors are in host memory (lists of CPU tensors of one
    shape and type, BF16 or FP16; page-locked memory lets the copies overlap the
    kernels). Results land in ``outs`` (and ``lses`` when given) once ``stream``
    has been synchronised; see ``include/fa.h``."""
    import torch
    n = len(qs)
    if not (len(ks) == len(vs) == len(outs) == n) or (lses is not None and len(lses) != n):
        raise ValueError("qs, ks, vs, outs (and lses) must have one entry per request")
    if n == 0:
        return
    dtype = qs[0].dtype
    if dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"q is {dtype}, expected torch.bfloat16 or torch.float16")
    B, H_q, H_kv, N_q, N_k, d = _dims(qs[0], ks[0])
    for i in range(n):
        _check_dtypes(dtype, qs[i], ks[i], vs[i], outs[i], None if lses is None else lses[i])
        group = [qs[i], ks[i], vs[i], outs[i]] + ([] if lses is None or lses[i] is None else [lses[i]])
        for t in group:
            if t.device.type != "cpu" or not t.is_contiguous():
                raise ValueError("fa_forward_host takes contiguous CPU tensors")
        if (qs[i].shape != qs[0].shape or ks[i].shape != ks[0].shape or vs[i].shape != ks[0].shape
                or tuple(outs[i].shape) != (B, H_q, N_q, d)
                or (lses is not None and lses[i] is not None and tuple(lses[i].shape) != (B, H_q, N_q))):
            raise ValueError(f"request {i} does not have the shape of request 0")
    if scale is None:
        scale = 1.0 / math.sqrt(d)

    def arr(ts):
        return (_vp * n)(*[t.data_ptr() if t is not None else 0 for t in ts])

    st = lib().fa_forward_host(n, arr(qs), arr(ks), arr(vs), arr(outs),
                               None if lses is None else arr(lses), B, H_q, H_kv, N_q, N_k, d,
                               int(bool(causal)), float(scale),
                               FA_DTYPE_FP16 if dtype == torch.float16 else FA_DTYPE_BF16,
                               _stream_ptr(stream))
    _check(st, "fa_forward_host")


def fa_forward_host_packed(qkvs, outs, shape, causal: bool = False, scale: float | None = None,
                           dtype=None, stream=None) -> None:
    """``fa_forward_host`` with each request packed in two contiguous CPU
    buffers: ``qkvs[i]`` holds Q, K, V back to back and ``outs[i]`` receives O
    then LSE (FP32). ``shape`` = (B, H_q, H_kv, N_q, N_k, d); ``dtype``
    torch.bfloat16 (default) or torch.float16 names the element type."""
    import torch
    dtype = torch.bfloat16 if dtype is None else dtype
    if dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"dtype is {dtype}, expected torch.bfloat16 or torch.float16")
    B, H_q, H_kv, N_q, N_k, d = (int(x) for x in shape)
    n = len(qkvs)
    if len(outs) != n:
        raise ValueError("qkvs and outs must have one entry per request")
    if n == 0:
        return
    in_bytes = (B * H_q * N_q + 2 * B * H_kv * N_k) * d * 2
    out_bytes = B * H_q * N_q * (d * 2 + 4)
    for t, need in [(t, in_bytes) for t in qkvs] + [(t, out_bytes) for t in outs]:
        if t.device.type != "cpu" or not t.is_contiguous():
            raise ValueError("fa_forward_host_packed takes contiguous CPU buffers")
        if t.numel() * t.element_size() < need:
            raise ValueError(f"a buffer holds {t.numel() * t.element_size()} bytes, needs {need}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    ptrs = lambda ts: (_vp * n)(*[t.data_ptr() for t in ts])
    st = lib().fa_forward_host_packed(n, ptrs(qkvs), ptrs(outs), B, H_q, H_kv, N_q, N_k, d,
                                      int(bool(causal)), float(scale),
                                      FA_DTYPE_FP16 if dtype == torch.float16 else FA_DTYPE_BF16,
                                      _stream_ptr(stream))
    _check(st, "fa_forward_host_packed")


def _check_layout(what, **tensors):
    """Each named tensor (name -> (tensor, expected shape)) is a contiguous CUDA
    tensor of that shape: libfa derives every size from the shapes of q and k."""
    for t, shape in tensors.values():   # the usual case: nothing to say
        if t is not None and (t.shape != shape or not t.is_contiguous() or not t.is_cuda):
            break
    else:
        return
    given = [(name, t, shape) for name, (t, shape) in tensors.items() if t is not None]
    for name, t, shape in given:
        if tuple(t.shape) != tuple(shape):
            raise ValueError(f"{what}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    for name, t, _ in given:
        if not t.is_contiguous():
            raise ValueError(f"{what}: {name} must be contiguous")
    for name, t, _ in given:
        if t.numel() > 0 and t.device.type != "cuda":
            raise ValueError(f"{what}: {name} must be a CUDA tensor")


def _int32(what, name, x):
    """An argument that the library takes in 32 bits (ctypes would cut a larger one down)."""
    x = int(x)
    if not -1 << 31 <= x < 1 << 31:
        raise ValueError(f"{what}: {name} = {x} does not fit in 32 bits")
    return x


def _backward(what, q, k, v, o, lse, do, mask, scale, dq, dk, dv, stream):
    """The call behind fa_backward and fa_backward_window (``mask``: their integers)."""
    import torch
    dtype = q.dtype
    if dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"q is {dtype}, expected torch.bfloat16 or torch.float16")
    for name, t in (("k", k), ("v", v), ("o", o), ("do", do), ("dq", dq), ("dk", dk), ("dv", dv)):
        if t is not None and t.dtype != dtype:
            raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if lse is None or lse.dtype != torch.float32:
        raise TypeError("lse (FP32, from the forward) is required")
    B, H_q, H_kv, N_q, N_k, d = _dims(q, k)
    qs, ks = (B, H_q, N_q, d), (B, H_kv, N_k, d)
    _check_layout(what, q=(q, qs), k=(k, ks), v=(v, ks), o=(o, qs), lse=(lse, (B, H_q, N_q)),
                  do=(do, qs), dq=(dq, qs), dk=(dk, ks), dv=(dv, ks))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = _empty(qs, dtype, q.device, stream) if dq is None else dq
    dk = _empty(ks, dtype, q.device, stream) if dk is None else dk
    dv = _empty(ks, dtype, q.device, stream) if dv is None else dv
    st = getattr(lib(), what)(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk),
                              _ptr(dv), B, H_q, H_kv, N_q, N_k, d, *mask, float(scale),
                              FA_DTYPE_FP16 if dtype == torch.float16 else FA_DTYPE_BF16,
                              _stream_ptr(stream))
    _check(st, what)
    return dq, dk, dv


def fa_backward(q, k, v, o, lse, do, causal: bool = False, scale: float | None = None, dq=None,
                dk=None, dv=None, stream=None):
    """Gradients (dq, dk, dv) of the forward given its o and lse and the upstream
    gradient do; BF16 or FP16 tensors (all one type), FP32 lse. Returns (dq, dk, dv)."""
    return _backward("fa_backward", q, k, v, o, lse, do, (int(bool(causal)),), scale, dq, dk, dv, stream)


def fa_forward_window(q, k, v, window: int, sinks: int = 0, scale: float | None = None, out=None, lse=None,
                      return_lse: bool = True, stream=None):
    """Causal forward under a sliding window: row i, at position ``i + N_k - N_q``, sees its
    last ``window`` keys (itself among them) and the first ``sinks``. q ``[B, H_q, N_q, d]``, k
    and v ``[B, H_kv, N_k, d]``, BF16 or FP16, d 64 or 128. Returns ``(o, lse)``. See
    ``include/fa_window.h``."""
    import torch
    what = "fa_forward_window"
    dtype = q.dtype
    if dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"q is {dtype}, expected torch.bfloat16 or torch.float16")
    _check_dtypes(dtype, q, k, v, out, lse)
    B, H_q, H_kv, N_q, N_k, d = _dims(q, k)
    qs, ks = (B, H_q, N_q, d), (B, H_kv, N_k, d)
    _check_layout(what, q=(q, qs), k=(k, ks), v=(v, ks), out=(out, qs), lse=(lse, qs[:3]))
    if out is None:
        out = _empty(q.shape, dtype, q.device, stream)
    if lse is None and return_lse:
        lse = _empty(qs[:3], torch.float32, q.device, stream)
    st = lib().fa_forward_window(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H_q, H_kv, N_q, N_k, d,
                                 _int32(what, "window", window), _int32(what, "sinks", sinks),
                                 1.0 / math.sqrt(d) if scale is None else float(scale),
                                 FA_DTYPE_FP16 if dtype == torch.float16 else FA_DTYPE_BF16, _stream_ptr(stream))
    _check(st, what)
    return out, lse


def fa_backward_window(q, k, v, o, lse, do, window: int, sinks: int = 0, scale: float | None = None, dq=None,
                       dk=None, dv=None, stream=None):
    """Gradients (dq, dk, dv) of ``fa_forward_window`` given its o and lse and the upstream
    gradient do; tensors as ``fa_backward`` takes them. o and lse must be those of exactly
    the keys that this call shows (not of a whole whose piece k and v are)."""
    what = "fa_backward_window"
    mask = _int32(what, "window", window), _int32(what, "sinks", sinks)
    return _backward(what, q, k, v, o, lse, do, mask, scale, dq, dk, dv, stream)


def fa_decode_paged(q, k_cache, v_cache, block_table, seqlens_k, causal: bool = False,
                    scale: float | None = None, out=None, lse=None, return_lse: bool = True, stream=None):
    """Decode over a paged K/V cache. q ``[B, H_q, N_q, d]``; k_cache, v_cache
    ``[num_pages, H_kv, 128, d]`` (BF16 or FP16, q's type); block_table int32
    ``[B, max_pages]``; seqlens_k int32 ``[B]``; all on the device. Returns
    ``(o, lse)`` as ``fa_forward`` does."""
    import torch
    dtype = q.dtype
    if dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"q is {dtype}, expected torch.bfloat16 or torch.float16")
    _check_dtypes(dtype, q, k_cache, v_cache, out, lse)
    for name, t in (("block_table", block_table), ("seqlens_k", seqlens_k)):
        if t.dtype != torch.int32:
            raise TypeError(f"{name} is {t.dtype}, expected torch.int32")
    B, H_q, N_q, d = q.shape
    num_pages, H_kv, page, dk = k_cache.shape
    if page != 128 or dk != d or tuple(v_cache.shape) != tuple(k_cache.shape):
        raise ValueError("k_cache / v_cache must be [num_pages, H_kv, 128, d] with q's d")
    if block_table.dim() != 2 or block_table.shape[0] != B or tuple(seqlens_k.shape) != (B,):
        raise ValueError("block_table must be [B, max_pages] and seqlens_k [B]")
    _check_layout("fa_decode_paged", q=(q, q.shape), k_cache=(k_cache, k_cache.shape),
                  v_cache=(v_cache, k_cache.shape), block_table=(block_table, block_table.shape),
                  seqlens_k=(seqlens_k, (B,)), out=(out, q.shape), lse=(lse, (B, H_q, N_q)))
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _empty(q.shape, dtype, q.device, stream)
    if lse is None and return_lse:
        lse = _empty((B, H_q, N_q), torch.float32, q.device, stream)
    st = lib().fa_decode_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seqlens_k),
                               _ptr(out), _ptr(lse), B, H_q, H_kv, N_q, num_pages, block_table.shape[1], d,
                               int(bool(causal)), float(scale),
                               FA_DTYPE_FP16 if dtype == torch.float16 else FA_DTYPE_BF16, _stream_ptr(stream))
    _check(st, "fa_decode_paged")
    return out, lse


def _cache_refuse(what, dtype, k_cache, v_cache, k_exp, v_exp, block_table, cu_seqlens, seqlens_k, d):
    """Raise for the first thing wrong with a paged cache and its ragged batch."""
    import torch
    if dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"{what}: element type {dtype}, expected torch.bfloat16 or torch.float16")
    cdt, shape = k_cache.dtype, tuple(k_cache.shape)
    if v_cache.dtype != cdt:
        raise TypeError(f"{what}: v_cache is {v_cache.dtype}, k_cache {cdt}")
    fp8 = cdt in (torch.uint8, torch.float8_e4m3fn)
    if not fp8 and cdt != dtype:
        raise TypeError(f"{what}: caches of {cdt}: expected {dtype} or E4M3 codes "
                        "(torch.uint8 or torch.float8_e4m3fn)")
    if not fp8 and (k_exp is not None or v_exp is not None):
        raise TypeError(f"{what}: k_exp / v_exp go with E4M3 caches only")
    if fp8 and (k_exp is None or v_exp is None or k_exp.dtype != torch.uint8 or v_exp.dtype != torch.uint8):
        raise TypeError(f"{what}: an E4M3 cache needs k_exp and v_exp (torch.uint8)")
    if len(shape) != 4 or shape[2] != 128 or shape[3] != d or tuple(v_cache.shape) != shape:
        raise ValueError(f"{what}: k_cache / v_cache must be [num_pages, H_kv, 128, d] with d = {d}")
    if fp8 and (tuple(k_exp.shape) != shape[:3] or tuple(v_exp.shape) != shape[:3]):
        raise ValueError(f"{what}: k_exp / v_exp must be [num_pages, H_kv, 128]")
    B = seqlens_k.shape[0] if seqlens_k.dim() == 1 else -1
    if B < 0 or block_table.dim() != 2 or block_table.shape[0] != B or tuple(cu_seqlens.shape) != (B + 1,):
        raise ValueError(f"{what}: block_table must be [B, max_pages], cu_seqlens [B + 1] and seqlens_k [B]")
    given = (("k_cache", k_cache), ("v_cache", v_cache), ("k_exp", k_exp), ("v_exp", v_exp),
             ("block_table", block_table), ("cu_seqlens", cu_seqlens), ("seqlens_k", seqlens_k))
    for name, t in given[4:]:
        if t.dtype != torch.int32:
            raise TypeError(f"{what}: {name} is {t.dtype}, expected torch.int32")
    for name, t in given:
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{what}: {name} must be contiguous")
    for name, t in given:
        if t is not None and not t.is_cuda and t.numel() > 0:
            raise ValueError(f"{what}: {name} must be a CUDA tensor")


_kinds = None   # (torch.bfloat16, torch.float16, torch.uint8, torch.float8_e4m3fn, torch.int32)


def _cache_format(what, dtype, k_cache, v_cache, k_exp, v_exp, block_table, cu_seqlens, seqlens_k, d):
    """Checks of a paged cache and its ragged batch (``include/fa_serving.h``); returns
    (FA_DTYPE_*, FA_CACHE_*, num_pages, H_kv, B, max_pages). One pass over what must hold
    (a decode step makes two such calls a layer); the message is looked for when it does not."""
    global _kinds
    if _kinds is None:
        import torch
        _kinds = (torch.bfloat16, torch.float16, torch.uint8, torch.float8_e4m3fn, torch.int32)
    bf16, f16, u8, e4m3, i32 = _kinds
    shape, cdt = k_cache.shape, k_cache.dtype
    fmt = FA_CACHE_16BIT if cdt is dtype else FA_CACHE_E4M3
    lens, table = seqlens_k.shape, block_table.shape
    if ((dtype is bf16 or dtype is f16) and v_cache.dtype is cdt and len(shape) == 4 and shape[2] == 128
            and shape[3] == d and v_cache.shape == shape and len(lens) == 1 and len(table) == 2
            and table[0] == lens[0] and cu_seqlens.shape == (lens[0] + 1,)
            and block_table.dtype is i32 and cu_seqlens.dtype is i32 and seqlens_k.dtype is i32
            and k_cache.is_contiguous() and v_cache.is_contiguous() and block_table.is_contiguous()
            and cu_seqlens.is_contiguous() and seqlens_k.is_contiguous()
            and k_cache.is_cuda and v_cache.is_cuda and block_table.is_cuda and cu_seqlens.is_cuda
            and seqlens_k.is_cuda
            and ((k_exp is None and v_exp is None) if cdt is dtype else
                 ((cdt is u8 or cdt is e4m3) and k_exp is not None and v_exp is not None
                  and k_exp.dtype is u8 and v_exp.dtype is u8 and k_exp.shape == shape[:3]
                  and v_exp.shape == shape[:3] and k_exp.is_contiguous() and v_exp.is_contiguous()
                  and k_exp.is_cuda and v_exp.is_cuda))):
        return FA_DTYPE_FP16 if dtype is f16 else FA_DTYPE_BF16, fmt, shape[0], shape[1], lens[0], table[1]
    _cache_refuse(what, dtype, k_cache, v_cache, k_exp, v_exp, block_table, cu_seqlens, seqlens_k, d)
    # only empty tensors off the device are left (B = 0)
    return FA_DTYPE_FP16 if dtype is f16 else FA_DTYPE_BF16, fmt, shape[0], shape[1], lens[0], table[1]


def _token_stride(what, name, t):
    """Elements between the tokens of a ``[T, H, d]`` CUDA tensor whose rows of one
    token are contiguous (a slice of a fused projection, say)."""
    T, H, d = t.shape
    if t.is_contiguous() and t.is_cuda:
        return H * d
    if not t.is_cuda and t.numel() > 0:
        raise ValueError(f"{what}: {name} must be a CUDA tensor")
    st = t.stride()
    if (d > 1 and st[2] != 1) or (H > 1 and st[1] != d):
        raise ValueError(f"{what}: the [H, d] rows of each token of {name} must be contiguous")
    if T <= 1:
        return H * d
    if st[0] < H * d or st[0] % 8 != 0:
        raise ValueError(f"{what}: tokens of {name} are {st[0]} elements apart: at least {H * d}, a multiple of 8")
    return st[0]


def _at(t):
    """Device address of a tensor (0 for None; an empty tensor's is 0 already)."""
    return 0 if t is None else t.data_ptr()


def fa_cache_append(k, v, k_cache, v_cache, block_table, cu_seqlens, seqlens_k, k_exp=None, v_exp=None,
                    stream=None) -> None:
    """Write new tokens' K and V (``[T, H_kv, d]`` BF16 or FP16, tokens packed by
    ``cu_seqlens``; token strides allowed) into a paged cache ``[num_pages, H_kv,
    128, d]``: as they are, or, for E4M3 caches (torch.uint8 or
    torch.float8_e4m3fn) with ``k_exp`` / ``v_exp`` (torch.uint8 ``[num_pages,
    H_kv, 128]``), quantised with one power of two per row. ``seqlens_k`` counts the
    new tokens. See ``include/fa_serving.h``."""
    what = "fa_cache_append"
    if k.dim() != 3 or v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError(f"{what}: k and v must be [T, H_kv, d] of one type")
    T, H_kv, d = k.shape
    elem, fmt, pages, heads, B, width = _cache_format(what, k.dtype, k_cache, v_cache, k_exp, v_exp, block_table,
                                                      cu_seqlens, seqlens_k, d)
    if heads != H_kv:
        raise ValueError(f"{what}: the cache has {heads} KV heads, k has {H_kv}")
    st = lib().fa_cache_append(k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _at(k_exp),
                               _at(v_exp), block_table.data_ptr(), cu_seqlens.data_ptr(), seqlens_k.data_ptr(), B, T,
                               H_kv, pages, width, d, _token_stride(what, "k", k), _token_stride(what, "v", v), elem,
                               fmt, _stream_ptr(stream))
    _check(st, what)


def fa_cache_read(k_cache, v_cache, block_table, cu_seqlens, seqlens_k, num_tokens: int, k_exp=None, v_exp=None,
                  dtype=None, k=None, v=None, stream=None):
    """Read the last ``cu_seqlens[b + 1] - cu_seqlens[b]`` of each sequence's first
    ``seqlens_k[b]`` positions back out of a paged cache, as ``(k, v)``, each
    ``[num_tokens, H_kv, d]`` of ``dtype`` (default: the cache's own type, BF16 for
    E4M3 caches); rows of no sequence are not written. See ``include/fa_serving.h``."""
    import torch
    what = "fa_cache_read"
    if dtype is None:
        dtype = k.dtype if k is not None else k_cache.dtype if k_cache.dtype.itemsize == 2 else torch.bfloat16
    d = k_cache.shape[-1]
    elem, fmt, pages, H_kv, B, width = _cache_format(what, dtype, k_cache, v_cache, k_exp, v_exp, block_table,
                                                     cu_seqlens, seqlens_k, d)
    shape = (int(num_tokens), H_kv, d)
    if k is None:
        k = _empty(shape, dtype, k_cache.device, stream)
    if v is None:
        v = _empty(shape, dtype, k_cache.device, stream)
    for name, t in (("k", k), ("v", v)):
        if t.dtype != dtype:
            raise TypeError(f"{what}: {name} is {t.dtype}, expected {dtype}")
    _check_layout(what, k=(k, shape), v=(v, shape))
    st = lib().fa_cache_read(k_cache.data_ptr(), v_cache.data_ptr(), _at(k_exp), _at(v_exp), block_table.data_ptr(),
                             cu_seqlens.data_ptr(), seqlens_k.data_ptr(), k.data_ptr(), v.data_ptr(), B, shape[0],
                             H_kv, pages, width, d, elem, fmt, _stream_ptr(stream))
    _check(st, what)
    return k, v


def fa_extend_paged(q, k_cache, v_cache, block_table, cu_seqlens, seqlens_k, max_q: int, window: int = 0,
                    sinks: int = 0, scale: float | None = None, k_exp=None, v_exp=None, out=None, lse=None,
                    return_lse: bool = True, stream=None):
    """Attention of the new tokens of a ragged batch over a paged cache that holds them
    already (``fa_cache_append``): chunks of prompts, single tokens, or both. q ``[T, H_q,
    d]`` (tokens packed by ``cu_seqlens``; a token stride is allowed), the cache as
    ``fa_cache_append`` takes it, ``max_q`` the largest number of new tokens of a sequence.
    ``window > 0``: a token sees its last ``window`` keys and the first ``sinks``. Returns
    ``(o, lse)``: ``[T, H_q, d]`` and FP32 ``[T, H_q]``; rows of no sequence, and tokens past
    ``max_q`` of one that has more, are not written (without ``out`` and ``lse`` they hold
    anything). See ``include/fa_serving.h``."""
    import torch
    what = "fa_extend_paged"
    if q.dim() != 3:
        raise ValueError(f"{what}: q must be [T, H_q, d]")
    T, H_q, d = shape = q.shape
    dtype = q.dtype
    elem, fmt, pages, H_kv, B, width = _cache_format(what, dtype, k_cache, v_cache, k_exp, v_exp, block_table,
                                                     cu_seqlens, seqlens_k, d)
    if out is None:
        out = _empty(shape, dtype, q.device, stream)
    else:
        if out.dtype != dtype:
            raise TypeError(f"{what}: out is {out.dtype}, expected {dtype}")
        _check_layout(what, out=(out, shape))
    if lse is not None:
        if lse.dtype != torch.float32:
            raise TypeError(f"{what}: lse is {lse.dtype}, expected torch.float32")
        _check_layout(what, lse=(lse, shape[:2]))
    elif return_lse:
        lse = _empty(shape[:2], torch.float32, q.device, stream)
    st = lib().fa_extend_paged(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _at(k_exp), _at(v_exp),
                               block_table.data_ptr(), cu_seqlens.data_ptr(), seqlens_k.data_ptr(), out.data_ptr(),
                               _at(lse), B, T, _int32(what, "max_q", max_q), H_q, H_kv, pages, width, d,
                               _token_stride(what, "q", q), _int32(what, "window", window),
                               _int32(what, "sinks", sinks), 1.0 / math.sqrt(d) if scale is None else float(scale), elem,
                               fmt, _stream_ptr(stream))
    _check(st, what)
    return out, lse


def fa_forward_noalloc(q, k, v, causal: bool = False, scale: float | None = None, out=None,
                       lse=None, return_lse: bool = True, stream=None):
    """``fa_forward`` that allocates no device memory inside libfa: split
    partials use libfa's fixed 32 MiB device array (see ``include/fa.h``).
    Concurrent calls race on that array; keep them on one stream. Returns ``(o, lse)``."""
    import torch
    _check_dtypes(torch.bfloat16, q, k, v, out, lse)
    B, H_q, H_kv, N_q, N_k, d = _dims(q, k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _empty((B, H_q, N_q, d), torch.bfloat16, q.device, stream)
    if lse is None and return_lse:
        lse = _empty((B, H_q, N_q), torch.float32, q.device, stream)
    st = lib().fa_forward_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H_q, H_kv,
                                  N_q, N_k, d, int(bool(causal)), float(scale), _stream_ptr(stream))
    _check(st, "fa_forward_noalloc")
    return out, lse


def fa_forward_cluster_multicast(q, k, v, causal: bool = False, scale: float | None = None, out=None,
                                 lse=None, return_lse: bool = True, stream=None):
    """``fa_forward`` (BF16) with CTA pairs sharing K/V tile loads by cluster
    multicast, from libfa_single_gpu.so (``include/fa_single_gpu.h``): for a
    process that uses one GPU only. Returns ``(o, lse)``."""
    import torch
    _check_dtypes(torch.bfloat16, q, k, v, out, lse)
    B, H_q, H_kv, N_q, N_k, d = _dims(q, k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _empty((B, H_q, N_q, d), torch.bfloat16, q.device, stream)
    if lse is None and return_lse:
        lse = _empty((B, H_q, N_q), torch.float32, q.device, stream)
    l = lib_single_gpu()
    st = l.fa_forward_cluster_multicast(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H_q, H_kv,
                                        N_q, N_k, d, int(bool(causal)), float(scale), _stream_ptr(stream))
    if st != FA_OK:
        raise FaError(st, "fa_forward_cluster_multicast")
    return out, lse


def fa_forward_plan(B: int, H_q: int, H_kv: int, N_q: int, N_k: int, d: int,
                    causal: bool = False) -> dict:
    """How fa_forward runs this request on the current device: CTAs of its main
    kernel, kernels it launches, workspace bytes it allocates (the scratch that
    fa_forward_noalloc needs)."""
    ctas, launches, ws = ctypes.c_longlong(0), _c_int(0), _c_size(0)
    st = lib().fa_forward_plan(B, H_q, H_kv, N_q, N_k, d, int(bool(causal)), ctypes.byref(ctas),
                               ctypes.byref(launches), ctypes.byref(ws))
    _check(st, "fa_forward_plan")
    return {"ctas": int(ctas.value), "launches": int(launches.value), "workspace_bytes": int(ws.value)}


def fa_naive_workspace_bytes(B: int, H_q: int, N_q: int, N_k: int) -> int:
    return int(lib().fa_naive_workspace_bytes(B, H_q, N_q, N_k))


def fa_naive_forward(q, k, v, causal: bool = False, scale: float | None = None, out=None,
                     lse=None, workspace=None, return_lse: bool = True, stream=None):
    """Unfused three-kernel baseline (BF16). Returns ``(o, lse)``."""
    import torch
    _check_dtypes(torch.bfloat16, q, k, v, out, lse)
    B, H_q, H_kv, N_q, N_k, d = _dims(q, k)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = _empty((B, H_q, N_q, d), torch.bfloat16, q.device, stream)
    if lse is None and return_lse:
        lse = _empty((B, H_q, N_q), torch.float32, q.device, stream)
    nbytes = fa_naive_workspace_bytes(B, H_q, N_q, N_k)
    if workspace is None:
        workspace = _empty(max(nbytes, 16), torch.uint8, q.device, stream)
    st = lib().fa_naive_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H_q, H_kv, N_q,
                                N_k, d, int(bool(causal)), float(scale), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream_ptr(stream))
    _check(st, "fa_naive_forward")
    return out, lse


def fa_device_status(reset: bool = True) -> int:
    """Synchronise and return the device status word (FA_OK or FA_ERR_TIMEOUT)."""
    return int(lib().fa_device_status(int(bool(reset))))


def fa_status_string(status: int) -> str:
    return lib().fa_status_string(status).decode()


def fa_version() -> tuple[int, int]:
    v = int(lib().fa_version())
    return v >> 16, v & 0xFFFF
