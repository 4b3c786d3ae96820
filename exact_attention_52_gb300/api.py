"""Python binding of libattn_sm103a.so (ctypes, and csrc/attn_call.cpp for the streaming
calls): argument marshalling only.

Every function here checks dtypes, shapes and devices, allocates outputs with
PyTorch when the caller did not pass them, and calls the C ABI declared in
``include/attn_sm103a.h`` on the current PyTorch CUDA stream.  All arithmetic
runs in the library's CUDA kernels; there is no fallback path.  If the shared
library is missing, every call raises ``RuntimeError``.
"""

from __future__ import annotations

import ctypes
import fractions
import functools
import math
import os
import struct
import sys
import threading
import warnings

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libattn_sm103a.so")
# The same library built with device-side range checks (see attn_build_flags).
DEBUG_LIB_PATH = os.path.join(_PKG, "libattn_sm103a_debug.so")
CALL_PATH = os.path.join(_PKG, "_attn_call.so")

ATTN_OK = 0
STATUS_NAMES = {0: "ATTN_OK", -1: "ATTN_ERR_INVALID", -2: "ATTN_ERR_UNSUPPORTED",
                -3: "ATTN_ERR_CUDA", -4: "ATTN_ERR_TIMEOUT", -5: "ATTN_ERR_PAGE"}


class Strides(ctypes.Structure):
    """attn_strides_t: element strides (b, h, n) of a [B, heads, N, d] view."""
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("n", ctypes.c_int64)]


# Every symbol the header declares, with (restype, argtypes).
_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_st = Strides
SIGNATURES = {
    "attn_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp]),
    "attn_bwd_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "attn_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp]),
    "attn_bwd_preprocess": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp]),
    "attn_bwd_main": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp]),
    "attn_bwd_dq_convert": (_i, [_vp, _vp, _i, _i, _i, _i, _f, _vp]),
    "attn_bwd_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i,
                              _vp]),
    "attn_fwd_gqa": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp]),
    "attn_bwd_gqa": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f,
                          _i, _vp]),
    "attn_fwd_splitkv_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "attn_fwd_splitkv": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _i, _vp]),
    "attn_fwd_window": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _i, _vp]),
    "attn_bwd_window": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i,
                             _f, _i, _i, _vp]),
    "attn_fwd_strided": (_i, [_vp, _st, _vp, _st, _vp, _st, _vp, _st, _vp, _i, _i, _i, _i, _i, _f,
                              _i, _i, _vp]),
    "attn_bwd_strided": (_i, [_vp, _st, _vp, _st, _vp, _st, _vp, _st, _vp, _st, _vp, _vp, _st, _vp,
                              _st, _vp, _st, _vp, _i, _i, _i, _i, _i, _f, _i, _i, _vp]),
    "attn_fwd_sinks": (_i, [_vp, _st, _vp, _st, _vp, _st, _vp, _st, _vp, _i, _i, _i, _i, _i, _f, _i, _i,
                            _i, _vp]),
    "attn_bwd_sinks_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i]),
    "attn_bwd_sinks": (_i, [_vp, _st, _vp, _st, _vp, _st, _vp, _st, _vp, _st, _vp, _vp, _st, _vp, _st,
                            _vp, _st, _vp, _i, _i, _i, _i, _i, _f, _i, _i, _i, _vp]),
    "attn_fwd_fp8": (_i, [_vp, _vp, _vp, _f, _f, _f, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp]),
    "attn_cache_append": (_i, [_vp, _vp, _st, _vp, _st, _vp, _i, _i, _i, _i, _vp]),
    "attn_fwd_cache_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "attn_fwd_cache": (_i, [_vp, _vp, _st, _vp, _st, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f,
                            _i, _i, _vp]),
    "attn_rope": (_i, [_vp, _vp, _st, _vp, _st, _vp, _st, _vp, _st, _vp, ctypes.c_int64, _i, _i, _i, _i, _i, _vp]),
    "attn_rope_bwd_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "attn_rope_bwd": (_i, [_vp, _vp, _st, _vp, _st, _vp, _st, _vp, _vp, _st, _vp, _st, _vp, _st, _vp, _vp, _vp,
                           ctypes.c_int64, _i, _i, _i, _i, _i, _vp]),
    "attn_cache_append_rope": (_i, [_vp, _vp, _vp, _st, _vp, _st, _vp, _st, _vp, _st, _vp, _i, _i, _i, _i, _i, _vp]),
    "attn_fwd_cache_prefix_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "attn_fwd_cache_prefix": (_i, [_vp, _vp, _vp, _i, _vp, _st, _vp, _st, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp]),
    "attn_check_device_error": (_i, [_vp, ctypes.POINTER(ctypes.c_uint)]),
    "attn_set_wait_limit_ns": (None, [ctypes.c_ulonglong]),
    "attn_set_exp2_offload": (None, [_i]),
    "attn_selftest_wait_timeout": (_i, [_vp]),
    "attn_status_string": (ctypes.c_char_p, [_i]),
    "attn_kernel_smem_bytes": (_i, [_i, _i]),
    "attn_build_flags": (_i, []),
}

_lib = None


class AttnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)}")
        self.status = status


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Open the shared library and declare every C signature (no GPU needed)."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{os.path.basename(path)} is not built; run "
                           "`python -m exact_attention_52_gb300.build` (needs nvcc)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path == LIB_PATH:
        _lib = lib
    return lib


def _check(fn: str, status: int) -> None:
    if status != ATTN_OK:
        raise AttnError(fn, status)


def _c_int(x) -> int:
    """A bound or count as a C int.  ctypes would keep the low 32 bits of a larger one, another
    number; the nearest C int means the same, as no length is above it."""
    return min(max(int(x), -2 ** 31), 2 ** 31 - 1)


def _stream_handle(stream) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _check_qkv(name, t, shape, dtype):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous [B, H, N, d]")


def _checked_workspace(t, need, device):
    """The workspace that a call was given, of ``need`` bytes one after the other, or a new one."""
    import torch
    if t is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    _explain_workspace(device, t, need)
    return t


def fwd(q, k, v, scale: float | None = None, causal: bool = False, o=None, lse=None,
        stream=None):
    """Forward pass on bf16 CUDA tensors [B, H, N, d]; returns (O bf16, LSE fp32 [B, H, N])."""
    import torch
    B, H, N, d = q.shape
    Hk = k.shape[1] if getattr(k, "dim", lambda: 0)() == 4 else H
    _check_qkv("q", q, (B, H, N, d), torch.bfloat16)
    for name, t in (("k", k), ("v", v)):
        _check_qkv(name, t, (B, Hk, N, d), torch.bfloat16)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check_qkv("o", o, (B, H, N, d), torch.bfloat16)
    _check_qkv("lse", lse, (B, H, N), torch.float32)
    lib = load_library()
    if Hk == H:
        _check("attn_fwd", lib.attn_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                        lse.data_ptr(), B, H, N, d, scale, int(bool(causal)),
                                        _stream_handle(stream)))
    else:
        _check("attn_fwd_gqa", lib.attn_fwd_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                                o.data_ptr(), lse.data_ptr(), B, H, Hk, N, d, scale,
                                                int(bool(causal)), _stream_handle(stream)))
    return o, lse


def fwd_splitkv(q, k, v, num_splits: int = 0, scale: float | None = None, causal: bool = False,
                o=None, lse=None, workspace=None, stream=None):
    """Split-KV forward (bf16, Hk = H): returns (O, LSE) like ``fwd``."""
    import torch
    B, H, N, d = q.shape
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_qkv(name, t, (B, H, N, d), torch.bfloat16)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if o is None else o
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    lib = load_library()
    need = int(lib.attn_fwd_splitkv_workspace_bytes(B, H, N, d, _c_int(num_splits)))
    if need == 0:
        raise ValueError("invalid sizes or num_splits")
    workspace = _checked_workspace(workspace, need, q.device)
    _check("attn_fwd_splitkv", lib.attn_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                                    o.data_ptr(), lse.data_ptr(),
                                                    workspace.data_ptr(), B, H, N, d, scale,
                                                    int(bool(causal)), _c_int(num_splits),
                                                    _stream_handle(stream)))
    return o, lse


def fwd_window(q, k, v, window_left: int, window_right: int, scale: float | None = None,
               o=None, lse=None, stream=None):
    """Sliding-window forward: key j visible to query i iff
    i - window_left <= j <= i + window_right (-1: unbounded side)."""
    import torch
    B, H, N, d = q.shape
    Hk = k.shape[1]
    _check_qkv("q", q, (B, H, N, d), torch.bfloat16)
    for name, t in (("k", k), ("v", v)):
        _check_qkv(name, t, (B, Hk, N, d), torch.bfloat16)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if o is None else o
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check("attn_fwd_window", load_library().attn_fwd_window(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, Hk, N, d,
        scale, _c_int(window_left), _c_int(window_right), _stream_handle(stream)))
    return o, lse


def bwd_window(q, k, v, o, dout, lse, window_left: int, window_right: int,
               scale: float | None = None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Sliding-window backward; dK, dV have K's head count."""
    import torch
    B, H, N, d = q.shape
    Hk = k.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for name, t in (("q", q), ("o", o), ("dout", dout), ("dq", dq)):
        _check_qkv(name, t, (B, H, N, d), torch.bfloat16)
    for name, t in (("k", k), ("v", v), ("dk", dk), ("dv", dv)):
        _check_qkv(name, t, (B, Hk, N, d), torch.bfloat16)
    need = bwd_workspace_bytes(B, H, N, d)
    workspace = _checked_workspace(workspace, need, q.device)
    _check("attn_bwd_window", load_library().attn_bwd_window(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(), lse.data_ptr(),
        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), workspace.data_ptr(), B, H, Hk, N, d, scale,
        _c_int(window_left), _c_int(window_right), _stream_handle(stream)))
    return dq, dk, dv


def bwd_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(load_library().attn_bwd_workspace_bytes(B, H, N, d))


def bwd(q, k, v, o, dout, lse, scale: float | None = None, causal: bool = False,
        dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Backward pass; returns (dQ, dK, dV) bf16 [B, H, N, d]."""
    import torch
    B, H, N, d = q.shape
    Hk = k.shape[1] if getattr(k, "dim", lambda: 0)() == 4 else H
    for name, t in (("q", q), ("o", o), ("dout", dout)):
        _check_qkv(name, t, (B, H, N, d), torch.bfloat16)
    for name, t in (("k", k), ("v", v)):
        _check_qkv(name, t, (B, Hk, N, d), torch.bfloat16)
    _check_qkv("lse", lse, (B, H, N), torch.float32)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check_qkv("dq", dq, (B, H, N, d), torch.bfloat16)
    for name, t in (("dk", dk), ("dv", dv)):
        _check_qkv(name, t, (B, Hk, N, d), torch.bfloat16)
    need = bwd_workspace_bytes(B, H, N, d)
    workspace = _checked_workspace(workspace, need, q.device)
    lib = load_library()
    if Hk == H:
        _check("attn_bwd", lib.attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                        dout.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                        dv.data_ptr(), workspace.data_ptr(), B, H, N, d, scale,
                                        int(bool(causal)), _stream_handle(stream)))
    else:
        _check("attn_bwd_gqa", lib.attn_bwd_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                                o.data_ptr(), dout.data_ptr(), lse.data_ptr(),
                                                dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                                workspace.data_ptr(), B, H, Hk, N, d, scale,
                                                int(bool(causal)), _stream_handle(stream)))
    return dq, dk, dv


def fwd_fp8(q8, k8, v8, sq: float, sk: float, sv: float, scale: float | None = None,
            causal: bool = False, o=None, lse=None, stream=None):
    """FP8 forward: uint8 E4M3 codes [B, H, N, d] with per-tensor scales; returns (O bf16, LSE)."""
    import torch
    B, H, N, d = q8.shape
    for name, t in (("q8", q8), ("k8", k8), ("v8", v8)):
        _check_qkv(name, t, (B, H, N, d), torch.uint8)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if o is None:
        o = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=q8.device)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q8.device)
    _check_qkv("o", o, (B, H, N, d), torch.bfloat16)
    _check_qkv("lse", lse, (B, H, N), torch.float32)
    lib = load_library()
    _check("attn_fwd_fp8", lib.attn_fwd_fp8(q8.data_ptr(), k8.data_ptr(), v8.data_ptr(),
                                            float(sq), float(sk), float(sv), o.data_ptr(),
                                            lse.data_ptr(), B, H, N, d, scale,
                                            int(bool(causal)), _stream_handle(stream)))
    return o, lse


def check_device_error(stream=None) -> tuple[int, int]:
    """Synchronise and read/clear the device error word: (status, site)."""
    site = ctypes.c_uint(0)
    rc = load_library().attn_check_device_error(_stream_handle(stream), ctypes.byref(site))
    return int(rc), int(site.value)


def set_wait_limit_ns(ns: int) -> None:
    load_library().attn_set_wait_limit_ns(int(ns))


def set_exp2_offload(on: bool) -> None:
    """FP8 forward: compute one group of exponentials in eight on the FMA pipe."""
    load_library().attn_set_exp2_offload(int(bool(on)))


def selftest_wait_timeout(stream=None) -> None:
    _check("attn_selftest_wait_timeout",
           load_library().attn_selftest_wait_timeout(_stream_handle(stream)))


def bwd_stages(q, k, v, o, dout, lse, dq, dk, dv, workspace, scale: float, causal: bool,
               stream=None, events=None):
    """attn_bwd as its three C-ABI stages; ``events`` (4 CUDA events, optional)
    are recorded before, between and after them on the same stream."""
    B, H, N, d = q.shape
    lib = load_library()
    h = _stream_handle(stream)
    c = int(bool(causal))
    ev = events or [None] * 4
    if ev[0] is not None:
        ev[0].record(stream)
    _check("attn_bwd_preprocess", lib.attn_bwd_preprocess(o.data_ptr(), dout.data_ptr(),
                                                          lse.data_ptr(), workspace.data_ptr(),
                                                          B, H, N, d, h))
    if ev[1] is not None:
        ev[1].record(stream)
    _check("attn_bwd_main", lib.attn_bwd_main(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                              dout.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                              workspace.data_ptr(), B, H, N, d, float(scale), c, h))
    if ev[2] is not None:
        ev[2].record(stream)
    _check("attn_bwd_dq_convert", lib.attn_bwd_dq_convert(dq.data_ptr(), workspace.data_ptr(),
                                                          B, H, N, d, float(scale), h))
    if ev[3] is not None:
        ev[3].record(stream)
    return dq, dk, dv


def _bhnd_strides(t, layout):
    """Strides of a 4-D CUDA tensor seen as [B, heads, N, d]: layout "bhnd" (the
    tensor is [B, heads, N, d]) or "bnhd" (the tensor is [B, N, heads, d])."""
    sb, s1, s2, sd = t.stride()
    if sd != 1:
        raise ValueError("the last (d) dimension must be contiguous")
    if layout == "bhnd":
        return Strides(sb, s1, s2)
    if layout == "bnhd":
        return Strides(sb, s2, s1)
    raise ValueError(f"unknown layout {layout!r}")


def _bhnd_shape(t, layout):
    B, a, b, d = t.shape
    return (B, a, b, d) if layout == "bhnd" else (B, b, a, d)


def fwd_strided(q, k, v, layout: str = "bnhd", scale: float | None = None, window=(-1, -1),
                o=None, lse=None, stream=None):
    """Forward on bf16 tensors of any strides (multiples of 8) with a contiguous last dimension.
    ``layout`` says how the 4 dimensions are ordered ("bnhd": [B, N, H, d] as
    produced by most projections; "bhnd": [B, H, N, d]).  Returns (O in the same
    layout as q, LSE [B, H, N])."""
    import torch
    B, H, N, d = _bhnd_shape(q, layout)
    Hk = _bhnd_shape(k, layout)[1]
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be a bf16 CUDA tensor")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if o is None else o
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    _check("attn_fwd_strided", load_library().attn_fwd_strided(
        q.data_ptr(), _bhnd_strides(q, layout), k.data_ptr(), _bhnd_strides(k, layout),
        v.data_ptr(), _bhnd_strides(v, layout), o.data_ptr(), _bhnd_strides(o, layout),
        lse.data_ptr(), B, H, Hk, N, d, scale, _c_int(window[0]), _c_int(window[1]),
        _stream_handle(stream)))
    return o, lse


def bwd_strided(q, k, v, o, dout, lse, layout: str = "bnhd", scale: float | None = None,
                window=(-1, -1), dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Backward counterpart of ``fwd_strided``; gradients take the layout of
    their inputs (dq like q, dk like k, dv like v)."""
    import torch
    B, H, N, d = _bhnd_shape(q, layout)
    Hk = _bhnd_shape(k, layout)[1]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = bwd_workspace_bytes(B, H, N, d)
    workspace = _checked_workspace(workspace, need, q.device)
    st = lambda t: _bhnd_strides(t, layout)
    _check("attn_bwd_strided", load_library().attn_bwd_strided(
        q.data_ptr(), st(q), k.data_ptr(), st(k), v.data_ptr(), st(v), o.data_ptr(), st(o),
        dout.data_ptr(), st(dout), lse.data_ptr(), dq.data_ptr(), st(dq), dk.data_ptr(), st(dk),
        dv.data_ptr(), st(dv), workspace.data_ptr(), B, H, Hk, N, d, scale, _c_int(window[0]),
        _c_int(window[1]), _stream_handle(stream)))
    return dq, dk, dv


# ---------------------------------------------------------------------------
# Sliding window with sinks; paged 8-bit key/value cache
# ---------------------------------------------------------------------------
# A decode step runs these for single tokens, where the host's share of a call
# counts.  Calls on the current stream are read by csrc/attn_call.cpp, which gives
# back None for arguments that it does not take: then, or where it is not built,
# each function here makes one pass of cheap comparisons, and only when one fails
# do the functions named _explain_* look for the argument to name.  They are handed
# `torch`, and ask torch._C, for the same reason: an import statement or a look
# whether CUDA has been set up costs 0.1 to 0.2 us.
def _call_stream(torch, device_index, stream):
    """Handle of the stream a call runs on (the current one without an argument)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device_index)


def _is_current(torch, dev):
    """Whether ``dev`` is the current device's index (a CPU tensor's is -1)."""
    return dev >= 0 and dev == torch._C._cuda_getDevice()


def _on_stream(stream):
    """Context in which what a call allocates belongs to the stream that the call runs on."""
    import contextlib

    import torch
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


# The compiled half of the binding: (the library that it calls, the module or None).
_calls = None
_CALL_FUNCTIONS = ("attn_cache_append", "attn_fwd_cache_workspace_bytes", "attn_fwd_cache", "attn_fwd_sinks",
                   "attn_bwd_sinks_workspace_bytes", "attn_bwd_sinks", "attn_rope", "attn_rope_bwd_workspace_bytes",
                   "attn_rope_bwd", "attn_cache_append_rope", "attn_fwd_cache_prefix_workspace_bytes",
                   "attn_fwd_cache_prefix")


def _call_tag(torch):
    """PyTorch and Python that csrc/attn_call.cpp is compiled for: it reads their objects directly."""
    return f"torch {torch.__version__}, {sys.implementation.cache_tag}"


def _load_calls(torch, lib):
    """csrc/attn_call.cpp's module, calling ``lib``; None, with a warning, where it does not load
    or was built for another PyTorch or Python: the arguments are then read in Python."""
    try:
        import importlib.util
        spec = importlib.util.spec_from_file_location("_attn_call", CALL_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        if module.built_for != _call_tag(torch):
            raise ImportError(f"it was built for {module.built_for}, this is {_call_tag(torch)}")
        module.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in _CALL_FUNCTIONS))
        return module
    except (ImportError, OSError, AttributeError, TypeError, SystemError) as e:
        warnings.warn(f"{os.path.basename(CALL_PATH)} is not used, calls read their arguments in Python: {e}; "
                      "run `python -m exact_attention_52_gb300.build`", RuntimeWarning, stacklevel=4)
        return None


def _compiled_calls():
    """The compiled half of the binding, calling the loaded library; None where it or a GPU is missing."""
    global _calls
    lib = load_library()
    if _calls is None or _calls[0] is not lib:
        import torch
        module = None
        if os.path.exists(CALL_PATH) and torch.cuda.is_available():
            module = _load_calls(torch, lib)
            torch.cuda.init()
        _calls = lib, module
    return _calls[1]


def _read(torch, stream, layout):
    """The compiled half, for a call that it may read (and (device, stream) of the call), or None."""
    calls = _compiled_calls() if stream is None and layout in ("bhnd", "bnhd") else None
    if calls is None:
        return None, None, None
    dev = torch._C._cuda_getDevice()
    return calls, dev, torch._C._cuda_getCurrentRawStream(dev)


_kept = threading.local()


def _call_workspace(torch, dev, stream, handle, need):
    """Workspace of a call that was given none.  Calls of one thread on one stream run one after
    the other, so they share one that is kept (an allocation took 7 us of a 22 us call).  A call
    that is being captured, whose workspace the graph goes on using, and a call on a stream given
    as an argument get one of their own."""
    if stream is not None or torch._C._cuda_isCurrentStreamCapturing():
        with _on_stream(stream):
            return torch.empty(need, dtype=torch.uint8, device=dev)
    kept = _kept.__dict__
    ws = kept.get((dev, handle))
    if ws is None or ws.nbytes < need:
        ws = kept[(dev, handle)] = torch.empty(need, dtype=torch.uint8, device=dev)
    return ws


def release_workspaces() -> None:
    """Gives back the workspaces that calls of this thread without one have kept (one for each
    stream they ran on, 43 MB for prompts at d = 128); the next call makes its own again."""
    _kept.__dict__.clear()


def _explain_on(device, name, t, dtype, ndim):
    import torch
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype != dtype or t.dim() != ndim:
        raise ValueError(f"{name} must be {dtype} with {ndim} dimensions, got {t.dtype} {tuple(t.shape)}")


def _explain_device(t, name):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    return t.device


def _explain_like(device, name, t, like):
    import torch
    _explain_on(device, name, t, torch.bfloat16, 4)
    if t.shape != like.shape:
        raise ValueError(f"{name} must have shape {tuple(like.shape)}, got {tuple(t.shape)}")
    if t.stride(3) != 1:
        raise ValueError(f"the last (d) dimension of {name} must be contiguous")


def _explain_lse(device, t, shape):
    import torch
    _explain_on(device, "lse", t, torch.float32, 3)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"lse must be a contiguous {shape}")


def _workspace_ok(torch, dev, t, need):
    """Whether ``t`` has ``need`` bytes one after the other on device ``dev`` (an expanded tensor
    counts bytes that it does not have)."""
    return isinstance(t, torch.Tensor) and t.get_device() == dev and t.nbytes >= need and t.is_contiguous()


def _explain_workspace(device, t, need):
    import torch
    if not isinstance(t, torch.Tensor) or t.device != device or t.nbytes < need or not t.is_contiguous():
        raise ValueError(f"workspace needs {need} contiguous bytes on {device}")


def _strides4(t, layout):
    """(b, h, n) strides of a 4-D tensor in ``layout``, or None if d is not contiguous."""
    sb, s1, s2, sd = t.stride()
    if sd != 1:
        return None
    return Strides(sb, s1, s2) if layout == "bhnd" else Strides(sb, s2, s1)


def _like_strides(torch, dev, t, like, layout):
    """``_strides4`` of a bf16 tensor of ``like``'s shape on device ``dev``; None for any other."""
    try:
        if t.dtype is torch.bfloat16 and t.shape == like.shape and t.get_device() == dev:
            return _strides4(t, layout)
    except (AttributeError, ValueError):
        pass
    return None


def _lse_ok(torch, dev, t, shape):
    try:
        return t.dtype is torch.float32 and t.shape == shape and t.get_device() == dev and t.is_contiguous()
    except (AttributeError, ValueError):
        return False


def _layout_shape(t, layout):
    if layout not in ("bhnd", "bnhd"):
        raise ValueError(f"unknown layout {layout!r}")
    try:
        return _bhnd_shape(t, layout)
    except (AttributeError, ValueError):
        raise ValueError(f"a 4-dimensional tensor is expected, got {getattr(t, 'shape', type(t))}") from None


def _explain_qkv(q, k, v, layout):
    import torch
    device = _explain_device(q, "q")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _explain_on(device, name, t, torch.bfloat16, 4)
        if t.stride(3) != 1:
            raise ValueError(f"the last (d) dimension of {name} must be contiguous")
    B, _, N, d = _bhnd_shape(q, layout)
    Bk, _, Nk, dk = _bhnd_shape(k, layout)
    if (Bk, Nk, dk) != (B, N, d) or k.shape != v.shape:
        raise ValueError(f"k and v must have q's batch, length and d, got {tuple(k.shape)} and {tuple(v.shape)}")
    raise ValueError("q, k and v must be bf16 CUDA tensors of one device")


def _sinks_args(q, k, v, layout):
    """Sizes and strides of a whole-sequence call's inputs, checked."""
    import torch
    B, H, N, d = _layout_shape(q, layout)
    Bk, Hk, Nk, dk = _layout_shape(k, layout)
    try:
        dev, bf16 = q.get_device(), torch.bfloat16
        strides = _strides4(q, layout), _strides4(k, layout), _strides4(v, layout)
        ok = (None not in strides and (Bk, Nk, dk) == (B, N, d) and k.shape == v.shape
              and q.dtype is bf16 and k.dtype is bf16 and v.dtype is bf16
              and dev == k.get_device() == v.get_device() and _is_current(torch, dev))
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        _explain_qkv(q, k, v, layout)
    return B, H, Hk, N, d, dev, strides


def fwd_sinks(q, k, v, window_left: int, sinks: int, window_right: int = 0, layout: str = "bhnd",
              scale: float | None = None, o=None, lse=None, stream=None):
    """Sliding-window forward whose first ``sinks`` tokens stay visible: key j visible to query i
    iff j <= i + window_right (-1: no bound) and (window_left is -1, or j >= i - window_left, or
    j < sinks).  bf16 q [B, H, N, d], k and v [B, Hk, N, d] (``layout`` "bhnd") or [B, N, heads, d]
    ("bnhd"), any strides (multiples of 8) with a contiguous last dimension.  Returns (O like q, LSE [B, H, N])."""
    import torch
    calls, dev, handle = _read(torch, stream, layout)
    if calls is not None:
        done = calls.fwd_sinks(q, k, v, window_left, sinks, window_right, layout == "bnhd", scale, o, lse, dev, handle)
        if done.__class__ is tuple:
            return done
        if done is not None:
            _check("attn_fwd_sinks", done)
    B, H, Hk, N, d, dev, (qs, ks, vs) = _sinks_args(q, k, v, layout)
    device = q.device
    if o is None or lse is None:
        with _on_stream(stream):
            if o is None:
                o = torch.empty_like(q)
            if lse is None:
                lse = torch.empty((B, H, N), dtype=torch.float32, device=device)
    os_ = _like_strides(torch, dev, o, q, layout)
    if os_ is None or not _lse_ok(torch, dev, lse, (B, H, N)):
        _explain_like(device, "o", o, q)
        _explain_lse(device, lse, (B, H, N))
        raise ValueError(f"o and lse must be tensors on {device}")
    _check("attn_fwd_sinks", load_library().attn_fwd_sinks(
        q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, o.data_ptr(), os_, lse.data_ptr(),
        B, H, Hk, N, d, 1.0 / math.sqrt(d) if scale is None else float(scale), _c_int(window_left),
        _c_int(window_right), _c_int(sinks), _call_stream(torch, dev, stream)))
    return o, lse


@functools.lru_cache(maxsize=256)
def bwd_sinks_workspace_bytes(B: int, H: int, Hk: int, N: int, d: int, sinks: int) -> int:
    return int(load_library().attn_bwd_sinks_workspace_bytes(*map(_c_int, (B, H, Hk, N, d, sinks))))


def bwd_sinks(q, k, v, o, dout, lse, window_left: int, sinks: int, window_right: int = 0,
              layout: str = "bhnd", scale: float | None = None, dq=None, dk=None, dv=None,
              workspace=None, stream=None):
    """Backward of ``fwd_sinks``: (dQ, dK, dV), each in the layout of its input; dK and dV are
    summed over the query heads that share them.  ``workspace``: ``bwd_sinks_workspace_bytes``
    bytes, one for each call that may overlap."""
    import torch
    calls, dev, handle = _read(torch, stream, layout)
    if calls is not None:
        done = calls.bwd_sinks(q, k, v, o, dout, lse, window_left, sinks, window_right, layout == "bnhd", scale, dq, dk,
                               dv, workspace, dev, handle)
        if done.__class__ is tuple:
            return done
        if done is not None:
            _check("attn_bwd_sinks", done)
    B, H, Hk, N, d, dev, (qs, ks, vs) = _sinks_args(q, k, v, layout)
    device = q.device
    need = bwd_sinks_workspace_bytes(B, H, Hk, N, d, _c_int(sinks))
    if need == 0:
        raise ValueError(f"invalid sizes: B {B}, H {H}, Hk {Hk}, N {N}, d {d}, sinks {sinks}")
    if dq is None or dk is None or dv is None or workspace is None:
        with _on_stream(stream):
            if dq is None:
                dq = torch.empty_like(q)
            if dk is None:
                dk = torch.empty_like(k)
            if dv is None:
                dv = torch.empty_like(v)
            if workspace is None:
                workspace = torch.empty(need, dtype=torch.uint8, device=device)
    os_, dos = _like_strides(torch, dev, o, q, layout), _like_strides(torch, dev, dout, q, layout)
    dqs, dks, dvs = (_like_strides(torch, dev, dq, q, layout), _like_strides(torch, dev, dk, k, layout),
                     _like_strides(torch, dev, dv, v, layout))
    if (None in (os_, dos, dqs, dks, dvs) or not _lse_ok(torch, dev, lse, (B, H, N))
            or not _workspace_ok(torch, dev, workspace, need)):
        for name, t, like in (("o", o, q), ("dout", dout, q), ("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
            _explain_like(device, name, t, like)
        _explain_lse(device, lse, (B, H, N))
        _explain_workspace(device, workspace, need)
        raise ValueError(f"the gradients, o, dout, lse and workspace must be tensors on {device}")
    _check("attn_bwd_sinks", load_library().attn_bwd_sinks(
        q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, o.data_ptr(), os_, dout.data_ptr(),
        dos, lse.data_ptr(), dq.data_ptr(), dqs, dk.data_ptr(), dks, dv.data_ptr(), dvs, workspace.data_ptr(), B, H,
        Hk, N, d,
        1.0 / math.sqrt(d) if scale is None else float(scale), _c_int(window_left), _c_int(window_right), _c_int(sinks),
        _call_stream(torch, dev, stream)))
    return dq, dk, dv


# attn_cache_t, packed (native alignment): pages, strides, scales, table, its stride, lengths, sizes
_CACHE = struct.Struct("@PPqqqqqqPPPqPiii")


def _explain_lens(device, name, t, B):
    import torch
    _explain_on(device, name, t, torch.int32, 1)
    if t.shape[0] != B or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{B}]")


def _explain_cache(device, B, Hk, d, k_pages, v_pages, k_scale, v_scale, page_table, seq_lens, new_lens, new_name):
    import torch
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        _explain_on(device, name, t, torch.uint8, 4)
        if t.stride(3) != 1:
            raise ValueError(f"the last (d) dimension of {name} must be contiguous")
    P, heads, page, dim = k_pages.shape
    if v_pages.shape != k_pages.shape or heads != Hk or dim != d:
        raise ValueError(f"k_pages and v_pages must be [pages, {Hk}, page_size, {d}], got "
                         f"{tuple(k_pages.shape)} and {tuple(v_pages.shape)}")
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        _explain_on(device, name, t, torch.float32, 2)
        if t.shape != (P, Hk) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [{P}, {Hk}]")
    _explain_on(device, "page_table", page_table, torch.int32, 2)
    if page_table.shape[0] != B or page_table.shape[1] < 1 or 1 not in (page_table.shape[1], page_table.stride(1)):
        raise ValueError(f"page_table must be [{B}, pages] with contiguous rows")
    _explain_lens(device, "seq_lens", seq_lens, B)
    if new_lens is not None:
        _explain_lens(device, new_name, new_lens, B)
    raise ValueError(f"the cache's tensors must all be on {device}, the current device")


def _cache_arg(torch, dev, device, B, Hk, d, k_pages, v_pages, k_scale, v_scale, page_table, seq_lens, new_lens, new_name):
    """attn_cache_t of a call, its tensors checked."""
    try:
        P, heads, page, dim = shape = k_pages.shape
        i32, u8, f32 = torch.int32, torch.uint8, torch.float32
        ka, kb, kc, kd = k_pages.stride()
        va, vb, vc, vd = v_pages.stride()
        tb, t1 = page_table.stride()
        rows, cols = page_table.shape
        ok = (heads == Hk and dim == d and v_pages.shape == shape and kd == 1 and vd == 1
              and k_pages.dtype is u8 and v_pages.dtype is u8 and k_scale.dtype is f32 and v_scale.dtype is f32
              and page_table.dtype is i32 and seq_lens.dtype is i32
              and dev == k_pages.get_device() == v_pages.get_device() == k_scale.get_device()
              == v_scale.get_device() == page_table.get_device() == seq_lens.get_device()
              and k_scale.shape == (P, Hk) and v_scale.shape == (P, Hk) and k_scale.is_contiguous()
              and v_scale.is_contiguous() and rows == B and cols >= 1 and 1 in (cols, t1)
              and seq_lens.shape == (B,) and seq_lens.is_contiguous()
              and (new_lens is None or (new_lens.dtype is i32 and new_lens.get_device() == dev
                                        and new_lens.shape == (B,) and new_lens.is_contiguous())))
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        _explain_cache(device, B, Hk, d, k_pages, v_pages, k_scale, v_scale, page_table, seq_lens, new_lens, new_name)
    return _CACHE.pack(k_pages.data_ptr(), v_pages.data_ptr(), ka, kb, kc, va, vb, vc, k_scale.data_ptr(),
                       v_scale.data_ptr(), page_table.data_ptr(), tb, seq_lens.data_ptr(), P, page, cols)


def cache_append(k, v, k_pages, v_pages, k_scale, v_scale, page_table, seq_lens, new_lens=None,
                 layout: str = "bhnd", stream=None):
    """Write new tokens into a paged 8-bit cache, in place.

    k, v: bf16 [B, Hk, T, d] (``layout`` "bhnd") or [B, T, Hk, d] ("bnhd"), any strides
    (multiples of 8) with a contiguous last dimension.  k_pages, v_pages: uint8 E4M3 codes
    [pages, Hk, page_size, d], any strides (multiples of 16) with a contiguous last dimension;
    k_scale, v_scale: fp32 [pages, Hk].
    page_table: int32 [B, max_pages]; seq_lens: int32 [B], tokens of each sequence after the
    call; new_lens: int32 [B], how many of the T tokens are new (default: all): token t goes to
    position seq_lens - new_lens + t.  A page's scale is a power of two that covers its largest
    value and grows with it, the codes that are there being rounded again: a page that is written to
    belongs to one sequence."""
    import torch
    calls, dev, handle = _read(torch, stream, layout)
    if calls is not None:
        done = calls.cache_append(k, v, k_pages, v_pages, k_scale, v_scale, page_table, seq_lens, new_lens,
                                  layout == "bnhd", dev, handle)
        if done is not None:
            return _check("attn_cache_append", done)
    B, Hk, T, d = _layout_shape(k, layout)
    try:
        dev, bf16 = k.get_device(), torch.bfloat16
        ks, vs = _strides4(k, layout), _strides4(v, layout)
        ok = (ks is not None and vs is not None and k.shape == v.shape and k.dtype is bf16 and v.dtype is bf16
              and dev == v.get_device() and _is_current(torch, dev))
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        _explain_device(k, "k")
        _explain_like(k.device, "k", k, k)
        _explain_like(k.device, "v", v, k)
        raise ValueError("k and v must be bf16 CUDA tensors of one device")
    cache = _cache_arg(torch, dev, k.device, B, Hk, d, k_pages, v_pages, k_scale, v_scale, page_table, seq_lens,
                       new_lens, "new_lens")
    _check("attn_cache_append", load_library().attn_cache_append(
        cache, k.data_ptr(), ks, v.data_ptr(), vs, None if new_lens is None else new_lens.data_ptr(),
        B, Hk, T, d, _call_stream(torch, dev, stream)))


@functools.lru_cache(maxsize=256)
def fwd_cache_workspace_bytes(B: int, H: int, Hk: int, T: int, d: int) -> int:
    return int(load_library().attn_fwd_cache_workspace_bytes(*map(_c_int, (B, H, Hk, T, d))))


def fwd_cache(q, k_pages, v_pages, k_scale, v_scale, page_table, seq_lens, q_lens=None,
              layout: str = "bhnd", scale: float | None = None, window_left: int = -1, sinks: int = 0,
              o=None, lse=None, workspace=None, stream=None):
    """Attention of T new queries per sequence over a paged 8-bit cache (see ``cache_append``),
    their own tokens included; returns (O bf16 like q, LSE fp32 [B, H, T]).

    q: bf16 [B, H, T, d] or, with ``layout`` "bnhd", [B, T, H, d]; H a multiple of the cache's
    heads.  Query t of q_lens[b] (default T) sits at position p = seq_lens[b] - q_lens[b] + t and
    sees key j iff j <= p and (window_left is -1, or j >= p - window_left, or j < sinks).  Rows
    behind q_lens[b] are left as they were; a row that sees nothing gives 0 and LSE +inf.
    Pages that hold no key a query sees are not read.  Decode (T * H / Hk up to 64) and prompts
    run different kernels, each with its own split of the keys over the device.
    ``workspace``: ``fwd_cache_workspace_bytes`` bytes, one for each call that may overlap; without
    one, the calls of a thread on its current stream share a kept one (``release_workspaces``)."""
    import torch
    calls, dev, handle = _read(torch, stream, layout)
    if calls is not None:
        ws = workspace
        if ws is None and not torch._C._cuda_isCurrentStreamCapturing():
            ws = _kept.__dict__.get((dev, handle))
        if ws is not None:
            done = calls.fwd_cache(q, k_pages, v_pages, k_scale, v_scale, page_table, seq_lens, q_lens, layout == "bnhd",
                                   scale, window_left, sinks, o, lse, ws, dev, handle)
            if done.__class__ is tuple:
                return done
            if done is not None:
                _check("attn_fwd_cache", done)
    B, H, T, d = _layout_shape(q, layout)
    try:
        dev, qs, Hk = q.get_device(), _strides4(q, layout), k_pages.shape[1]
        ok = qs is not None and q.dtype is torch.bfloat16 and _is_current(torch, dev)
    except (AttributeError, IndexError):
        ok = False
    if not ok:
        _explain_device(q, "q")
        _explain_like(q.device, "q", q, q)
        raise ValueError("k_pages must be a tensor [pages, Hk, page_size, d]")
    device = q.device
    cache = _cache_arg(torch, dev, device, B, Hk, d, k_pages, v_pages, k_scale, v_scale, page_table, seq_lens,
                       q_lens, "q_lens")
    need = fwd_cache_workspace_bytes(B, H, Hk, T, d)
    if need == 0:
        raise ValueError(f"invalid sizes: B {B}, H {H}, Hk {Hk}, T {T}, d {d}")
    handle = _call_stream(torch, dev, stream)
    if o is None or lse is None:
        with _on_stream(stream):
            if o is None:
                o = torch.empty_like(q)
            if lse is None:
                lse = torch.empty((B, H, T), dtype=torch.float32, device=device)
    if workspace is None:
        workspace = _call_workspace(torch, dev, stream, handle, need)
    try:
        os_ = _strides4(o, layout)
        ok = (os_ is not None and o.dtype is torch.bfloat16 and o.shape == q.shape and lse.shape == (B, H, T)
              and lse.dtype is torch.float32 and lse.is_contiguous()
              and dev == o.get_device() == lse.get_device() and _workspace_ok(torch, dev, workspace, need))
    except (AttributeError, ValueError):
        ok = False
    if not ok:
        _explain_like(device, "o", o, q)
        _explain_lse(device, lse, (B, H, T))
        _explain_workspace(device, workspace, need)
        raise ValueError("o, lse and workspace must be tensors of the current device")
    _check("attn_fwd_cache", load_library().attn_fwd_cache(
        cache, q.data_ptr(), qs, o.data_ptr(), os_, lse.data_ptr(), workspace.data_ptr(),
        None if q_lens is None else q_lens.data_ptr(), B, H, Hk, T, d,
        1.0 / math.sqrt(d) if scale is None else float(scale), _c_int(window_left), _c_int(sinks), handle))
    return o, lse


# ---------------------------------------------------------------------------
# Rotary positions and norms of heads, by themselves and in the cache's write
# ---------------------------------------------------------------------------
_TWO_PI = 2 * fractions.Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
# attn_rope_t, packed (native alignment): table, weights, their type, rot, interleaved, factor, eps
_ROPE = struct.Struct("@PPPiiiff")


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original_len: int | None = None, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """Angles per position, in radians, of the rot / 2 pairs of a head, and what the rotated elements
    are multiplied by: theta_i = base^(-2 i / rot) and 1, or scaled for a context ``factor`` times
    as long as the trained one:

    "linear"  theta_i / factor: positions are squeezed into the trained range;
    "ntk"     the base times factor^(rot / (rot - 2)): the slowest pair is stretched by the factor, the
              fastest not at all;
    "yarn"    (Peng et al., 2023) pairs that turn more than beta_fast times within original_len tokens
              stay, those that turn less than beta_slow times are stretched by the factor, those between
              in proportion to their turns, as the paper's formula has it; elements are multiplied by
              0.1 ln(factor) + 1.  Published models are often run with another ramp, over the pair's
              index between two bounds rounded to whole pairs: the pairs between differ.  For such a
              model give its own numbers to ``rope_table`` (frequencies, magnitude)."""
    if not isinstance(rot, int) or rot < 2 or rot % 2:
        raise ValueError(f"rot must be an even number of elements, got {rot!r}")
    if not (math.isfinite(base) and base > 0):
        raise ValueError(f"base must be finite and above 0, got {base!r}")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling is not None and not (math.isfinite(factor) and factor > 0):
        raise ValueError(f"factor must be finite and above 0, got {factor!r}")
    if scaling == "ntk":
        if rot < 4:
            raise ValueError("ntk scaling needs two pairs at least")
        base = base * factor ** (rot / (rot - 2))
    theta = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [t / factor for t in theta], 1.0
    if scaling == "yarn":
        if original_len is None or original_len < 1 or not beta_fast > beta_slow:
            raise ValueError("yarn scaling needs original_len, and beta_fast above beta_slow")
        turns = [original_len * t / (2.0 * math.pi) for t in theta]
        keep = [min(1.0, max(0.0, (x - beta_slow) / (beta_fast - beta_slow))) for x in turns]
        return [t * (k + (1.0 - k) / factor) for t, k in zip(theta, keep)], 0.1 * math.log(factor) + 1.0
    return theta, 1.0


class RopeTable:
    """Rotary frequencies as the kernels take them, laid out once for a model (``rope_table``):
    ``turns``, int64 [rot / 2] on the device, in units of 2^-64 turns a position."""
    __slots__ = ("turns", "rot", "interleaved", "magnitude")

    def __init__(self, turns, interleaved: bool, magnitude: float):
        self.turns = turns
        self.rot = 2 * turns.shape[0]
        self.interleaved = bool(interleaved)
        self.magnitude = float(magnitude)


def _turns(theta: float) -> int:
    """theta radians in units of 2^-64 turns, modulo a turn, as a signed number."""
    t = round(fractions.Fraction(theta) / _TWO_PI * 2 ** 64) % 2 ** 64
    return t - 2 ** 64 if t >= 2 ** 63 else t


def rope_table(rot: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
               original_len: int | None = None, beta_fast: float = 32.0, beta_slow: float = 1.0,
               interleaved: bool = False, frequencies=None, magnitude: float | None = None, device="cuda"):
    """The table that ``rope`` and ``cache_append_rope`` take, for the first ``rot`` elements of a head
    (a multiple of 16): the frequencies of ``rope_frequencies``, or ``frequencies``, rot / 2 numbers
    in radians a position.  ``interleaved``: pairs are elements (2i, 2i + 1), otherwise
    (i, i + rot / 2).  ``magnitude`` multiplies the rotated elements (default: what the scaling
    asks for)."""
    import torch
    if not isinstance(rot, int) or rot < 16 or rot % 16:
        raise ValueError(f"rot must be a multiple of 16, got {rot!r}")
    if frequencies is None:
        theta, m = rope_frequencies(rot, base, scaling, factor, original_len, beta_fast, beta_slow)
    else:
        theta, m = [float(t) for t in frequencies], 1.0
        if len(theta) != rot // 2 or not all(map(math.isfinite, theta)):
            raise ValueError(f"frequencies must be {rot // 2} finite numbers")
    m = m if magnitude is None else float(magnitude)
    if not math.isfinite(m):
        raise ValueError(f"magnitude must be finite, got {m!r}")
    return RopeTable(torch.tensor([_turns(t) for t in theta], dtype=torch.int64, device=device), interleaved, m)


def _explain_rope(device, d, table, q_weight, k_weight):
    import torch
    if not isinstance(table, RopeTable):
        raise ValueError("table must be a RopeTable (rope_table)")
    _explain_on(device, "the table's turns", table.turns, torch.int64, 1)
    if not table.turns.is_contiguous() or table.rot != 2 * table.turns.shape[0] or table.rot > d:
        raise ValueError(f"the table must be of at most {d} elements of a head, got {table.rot}")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is None:
            continue
        if not isinstance(w, torch.Tensor) or w.device != device or w.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"{name} must be a fp32 or bf16 tensor on {device}")
        if w.shape != (d,) or not w.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [{d}], got {tuple(w.shape)}")
    if q_weight is not None and k_weight is not None and q_weight.dtype != k_weight.dtype:
        raise ValueError("q_weight and k_weight must be of one type")


def _rope_arg(torch, device, d, table, q_weight, k_weight, eps):
    """attn_rope_t of a call, its tensors checked."""
    _explain_rope(device, d, table, q_weight, k_weight)
    w = q_weight if q_weight is not None else k_weight
    return _ROPE.pack(table.turns.data_ptr(), 0 if q_weight is None else q_weight.data_ptr(),
                      0 if k_weight is None else k_weight.data_ptr(), int(w is not None and w.dtype is torch.bfloat16),
                      table.rot, int(table.interleaved), table.magnitude, float(eps))


def _rope_positions(device, positions, B, N):
    """Address and stride of a call's positions."""
    import torch
    if positions is None:
        return None, 0
    if not isinstance(positions, torch.Tensor) or positions.device != device or positions.dtype != torch.int32:
        raise ValueError(f"positions must be an int32 tensor on {device}")
    if positions.shape not in ((N,), (B, N)) or 1 not in (N, positions.stride(-1)):
        raise ValueError(f"positions must be [{N}] or [{B}, {N}] with contiguous rows, got {tuple(positions.shape)}")
    return positions.data_ptr(), positions.stride(0) if positions.dim() == 2 and B > 1 else 0


def _rope_heads(device, name, t, layout, like=None):
    """(shape, strides) of a bf16 tensor of heads, checked; ``like``: of its shape."""
    import torch
    _explain_on(device, name, t, torch.bfloat16, 4)
    st = _strides4(t, layout)
    if st is None:
        raise ValueError(f"the last (d) dimension of {name} must be contiguous")
    if like is not None and t.shape != like.shape:
        raise ValueError(f"{name} must have shape {tuple(like.shape)}, got {tuple(t.shape)}")
    return _bhnd_shape(t, layout), st


_NO_STRIDES = Strides(0, 0, 0)


def _rope_qk(q, k, layout, names=("q", "k")):
    """Device, sizes and strides of the queries and keys (which may be None) of a call."""
    if layout not in ("bhnd", "bnhd"):
        raise ValueError(f"unknown layout {layout!r}")
    device = _explain_device(q, names[0])
    (B, H, N, d), qs = _rope_heads(device, names[0], q, layout)
    if k is None:
        return device, B, H, 0, N, d, qs, _NO_STRIDES
    (Bk, Hk, Nk, dk), ks = _rope_heads(device, names[1], k, layout)
    if (Bk, Nk, dk) != (B, N, d):
        raise ValueError(f"{names[1]} must have {names[0]}'s batch, length and d, got {tuple(k.shape)}")
    return device, B, H, Hk, N, d, qs, ks


def _ptr(t):
    return None if t is None else t.data_ptr()


def rope(q, k, table, positions=None, q_weight=None, k_weight=None, eps: float = 1e-6, layout: str = "bhnd",
         q_out=None, k_out=None, stream=None):
    """Rotary positions on the heads of q and k (which may be None), each head normed first where its
    weight is given; returns (q_out, k_out).

    q [B, H, N, d] and k [B, Hk, N, d] (``layout`` "bhnd") or [B, N, heads, d] ("bnhd"), bf16, any
    strides (multiples of 8) with a contiguous last dimension; an output may be its input.
    table: ``rope_table``.  positions: int32 [B, N] or [N] (default: token n at n).  With a weight
    ([d], fp32 or bf16) a head x becomes x / sqrt(mean(x^2) + eps) * weight before its first
    ``table.rot`` elements are rotated."""
    import torch
    calls, dev, handle = _read(torch, stream, layout)
    if calls is not None and table.__class__ is RopeTable:
        done = calls.rope(q, k, table.turns, table.interleaved, table.magnitude, q_weight, k_weight, eps, positions,
                          layout == "bnhd", q_out, k_out, dev, handle)
        if done.__class__ is tuple:
            return done
        if done is not None:
            _check("attn_rope", done)
    device, B, H, Hk, N, d, qs, ks = _rope_qk(q, k, layout)
    at, step = _rope_positions(device, positions, B, N)
    arg = _rope_arg(torch, device, d, table, q_weight, None if k is None else k_weight, eps)
    with _on_stream(stream):
        if q_out is None:
            q_out = torch.empty_like(q)
        if k_out is None and k is not None:
            k_out = torch.empty_like(k)
    qos = _rope_heads(device, "q_out", q_out, layout, q)[1]
    kos = _NO_STRIDES if k is None else _rope_heads(device, "k_out", k_out, layout, k)[1]
    _check("attn_rope", load_library().attn_rope(
        arg, q.data_ptr(), qs, q_out.data_ptr(), qos, _ptr(k), ks, None if k is None else k_out.data_ptr(), kos, at, step,
        B, H, Hk, N, d, _call_stream(torch, device.index, stream)))
    return q_out, k_out if k is not None else None


@functools.lru_cache(maxsize=256)
def rope_bwd_workspace_bytes(B: int, H: int, Hk: int, N: int, d: int) -> int:
    return int(load_library().attn_rope_bwd_workspace_bytes(*map(_c_int, (B, H, Hk, N, d))))


def rope_bwd(dq_out, dk_out, table, positions=None, q=None, k=None, q_weight=None, k_weight=None, eps: float = 1e-6,
             layout: str = "bhnd", dq=None, dk=None, dq_weight=None, dk_weight=None, workspace=None, stream=None):
    """Backward of ``rope``: (dQ, dK, gradient of q_weight, of k_weight), the latter fp32 [d], None
    without a weight.  dq_out and dk_out (or None) are the gradients of ``rope``'s outputs, q and k its
    inputs, which only a tensor with a weight needs; dq may be dq_out, dk dk_out.  ``workspace``:
    ``rope_bwd_workspace_bytes`` bytes, one for each call that may overlap."""
    import torch
    calls, dev, handle = _read(torch, stream, layout)
    if calls is not None and table.__class__ is RopeTable:
        ws = workspace
        if ws is None and not torch._C._cuda_isCurrentStreamCapturing():
            ws = _kept.__dict__.get((dev, handle))
        done = calls.rope_bwd(dq_out, dk_out, table.turns, table.interleaved, table.magnitude, q_weight, k_weight, eps,
                              positions, q, k, layout == "bnhd", dq, dk, dq_weight, dk_weight, ws, dev, handle)
        if done.__class__ is tuple:
            return done
        if done is not None:
            _check("attn_rope_bwd", done)
    device, B, H, Hk, N, d, gqs, gks = _rope_qk(dq_out, dk_out, layout, ("dq_out", "dk_out"))
    if dk_out is None:
        k = k_weight = None
    at, step = _rope_positions(device, positions, B, N)
    arg = _rope_arg(torch, device, d, table, q_weight, k_weight, eps)
    strides = []
    for name, x, w, like in (("q", q, q_weight, dq_out), ("k", k, k_weight, dk_out)):
        strides.append(_NO_STRIDES if w is None else _rope_heads(device, name, x, layout, like)[1])
    need = 0
    if q_weight is not None or k_weight is not None:
        need = rope_bwd_workspace_bytes(B, H, Hk, N, d)
        if need == 0:
            raise ValueError(f"invalid sizes: B {B}, H {H}, Hk {Hk}, N {N}, d {d}")
    handle = _call_stream(torch, device.index, stream)
    with _on_stream(stream):
        if dq is None:
            dq = torch.empty_like(dq_out)
        if dk is None and dk_out is not None:
            dk = torch.empty_like(dk_out)
        if dq_weight is None and q_weight is not None:
            dq_weight = torch.empty(d, dtype=torch.float32, device=device)
        if dk_weight is None and k_weight is not None:
            dk_weight = torch.empty(d, dtype=torch.float32, device=device)
    if workspace is not None and need:
        _explain_workspace(device, workspace, need)
    elif need:
        workspace = _call_workspace(torch, device.index, stream, handle, need)
    dqs = _rope_heads(device, "dq", dq, layout, dq_out)[1]
    dks = _NO_STRIDES if dk_out is None else _rope_heads(device, "dk", dk, layout, dk_out)[1]
    for name, w, g in (("dq_weight", q_weight, dq_weight), ("dk_weight", k_weight, dk_weight)):
        if w is not None:
            _explain_on(device, name, g, torch.float32, 1)
            if g.shape != (d,) or not g.is_contiguous():
                raise ValueError(f"{name} must be a contiguous [{d}]")
    _check("attn_rope_bwd", load_library().attn_rope_bwd(
        arg, _ptr(q if q_weight is not None else None), strides[0], dq_out.data_ptr(), gqs, dq.data_ptr(), dqs,
        _ptr(dq_weight if q_weight is not None else None), _ptr(k if k_weight is not None else None), strides[1],
        _ptr(dk_out), gks, _ptr(dk if dk_out is not None else None), dks,
        _ptr(dk_weight if k_weight is not None else None), _ptr(workspace if need else None), at, step, B, H, Hk, N, d, handle))
    return (dq, dk if dk_out is not None else None, dq_weight if q_weight is not None else None,
            dk_weight if k_weight is not None else None)


def cache_append_rope(q, k, v, table, k_pages, v_pages, k_scale, v_scale, page_table, seq_lens, new_lens=None,
                      q_weight=None, k_weight=None, eps: float = 1e-6, layout: str = "bhnd", q_out=None, stream=None):
    """``cache_append`` of keys that are normed (where k_weight is given) and rotated first, and the
    same of the new tokens' queries, in one launch; returns q_out, for ``fwd_cache``.

    q: bf16 [B, H, T, d] (``layout`` "bhnd") or [B, T, H, d] ("bnhd"); q_out may be q.  Token t of
    the new_lens[b] (default T) new ones is rotated at its position in the cache, seq_lens - new_lens
    + t.  Rows of q_out behind them are left as they were.  The rest as ``rope`` and ``cache_append``."""
    import torch
    calls, dev, handle = _read(torch, stream, layout)
    if calls is not None and table.__class__ is RopeTable:
        done = calls.cache_append_rope(q, k, v, table.turns, table.interleaved, table.magnitude, q_weight, k_weight, eps,
                                       k_pages, v_pages, k_scale, v_scale, page_table, seq_lens, new_lens,
                                       layout == "bnhd", q_out, dev, handle)
        if done.__class__ is int:
            _check("attn_cache_append_rope", done)
        elif done is not None:
            return done
    device, B, H, Hk, T, d, qs, ks = _rope_qk(q, k, layout)
    if k is None:
        raise ValueError("k must be a bf16 CUDA tensor")
    vs = _rope_heads(device, "v", v, layout, k)[1]
    arg = _rope_arg(torch, device, d, table, q_weight, k_weight, eps)
    cache = _cache_arg(torch, device.index, device, B, Hk, d, k_pages, v_pages, k_scale, v_scale, page_table, seq_lens,
                       new_lens, "new_lens")
    if q_out is None:
        with _on_stream(stream):
            q_out = torch.empty_like(q)
    qos = _rope_heads(device, "q_out", q_out, layout, q)[1]
    _check("attn_cache_append_rope", load_library().attn_cache_append_rope(
        cache, arg, q.data_ptr(), qs, q_out.data_ptr(), qos, k.data_ptr(), ks, v.data_ptr(), vs, _ptr(new_lens), B, H, Hk,
        T, d, _call_stream(torch, device.index, stream)))
    return q_out


# ---------------------------------------------------------------------------
# Sequences that share their first tokens
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=256)
def fwd_cache_prefix_workspace_bytes(B: int, H: int, Hk: int, T: int, d: int) -> int:
    return int(load_library().attn_fwd_cache_prefix_workspace_bytes(*map(_c_int, (B, H, Hk, T, d))))


def fwd_cache_prefix(q, k_pages, v_pages, k_scale, v_scale, page_table, seq_lens, prefix_lens, group_first=None,
                     q_lens=None, layout: str = "bhnd", scale: float | None = None, o=None, lse=None, workspace=None,
                     stream=None):
    """``fwd_cache`` for a batch whose sequences share their first tokens, which are read once for all
    where that pays: with at most 64 rows a sequence and key/value head (T * H / Hk), groups of six
    sequences or more on average, and a table that can hold 256 MB of keys and values.  Elsewhere the call
    is ``fwd_cache``.  Unused columns of the table count: hand in page_table[:, :n] with the columns that
    the longest sequence needs.

    prefix_lens: int32 [groups], tokens whose pages the sequences of a group share (their tables
    begin with the same pages); every query stands behind them.  A page that is still to be appended
    to is no shared one: where a prompt ends inside a page, each sequence has a copy of that page (codes
    and scales), and prefix_lens ends with the page before it (with pages of up to 128 tokens it may
    be the whole prompt: the last prefix_lens % 128 tokens are read through each sequence's own
    table).  group_first: int32 [groups + 1],
    ascending: group g is sequences group_first[g] .. group_first[g + 1] - 1 (default: one group of
    all).  Both stay on the device, as the lengths do.  ``workspace``:
    ``fwd_cache_prefix_workspace_bytes`` bytes, one for each call that may overlap.  The rest, and what
    is returned, as ``fwd_cache``."""
    import torch
    calls, dev, handle = _read(torch, stream, layout)
    if calls is not None:
        ws = workspace
        if ws is None and not torch._C._cuda_isCurrentStreamCapturing():
            ws = _kept.__dict__.get((dev, handle))
        if ws is not None:
            done = calls.fwd_cache_prefix(q, k_pages, v_pages, k_scale, v_scale, page_table, seq_lens, prefix_lens,
                                          group_first, q_lens, layout == "bnhd", scale, o, lse, ws, dev, handle)
            if done.__class__ is tuple:
                return done
            if done is not None:
                _check("attn_fwd_cache_prefix", done)
    device = _explain_device(q, "q")
    B, H, T, d = _layout_shape(q, layout)
    qs = _rope_heads(device, "q", q, layout)[1]
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("k_pages must be a tensor [pages, Hk, page_size, d]")
    Hk, dev = k_pages.shape[1], device.index
    cache = _cache_arg(torch, dev, device, B, Hk, d, k_pages, v_pages, k_scale, v_scale, page_table, seq_lens,
                       q_lens, "q_lens")
    _explain_on(device, "prefix_lens", prefix_lens, torch.int32, 1)
    groups = prefix_lens.shape[0]
    _explain_lens(device, "prefix_lens", prefix_lens, groups)
    if group_first is not None:
        _explain_lens(device, "group_first", group_first, groups + 1)
    if not 1 <= groups <= B or (group_first is None and groups != 1):
        raise ValueError(f"prefix_lens must be of 1 .. {B} groups, with group_first where there are several; got {groups}")
    need = fwd_cache_prefix_workspace_bytes(B, H, Hk, T, d)
    if need == 0:
        raise ValueError(f"invalid sizes: B {B}, H {H}, Hk {Hk}, T {T}, d {d}")
    handle = _call_stream(torch, dev, stream)
    with _on_stream(stream):
        if o is None:
            o = torch.empty_like(q)
        if lse is None:
            lse = torch.empty((B, H, T), dtype=torch.float32, device=device)
    if workspace is None:
        workspace = _call_workspace(torch, dev, stream, handle, need)
    _explain_like(device, "o", o, q)
    _explain_lse(device, lse, (B, H, T))
    if not _workspace_ok(torch, dev, workspace, need):
        _explain_workspace(device, workspace, need)
    _check("attn_fwd_cache_prefix", load_library().attn_fwd_cache_prefix(
        cache, _ptr(group_first), prefix_lens.data_ptr(), groups, q.data_ptr(), qs, o.data_ptr(), _strides4(o, layout),
        lse.data_ptr(), workspace.data_ptr(), _ptr(q_lens), B, H, Hk, T, d,
        1.0 / math.sqrt(d) if scale is None else float(scale), handle))
    return o, lse
