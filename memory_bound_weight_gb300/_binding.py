"""Thin ctypes binding of libmbw.so (include/mbw.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of libmbw.so. PyTorch supplies device memory and the current stream.
If the library is missing the calls raise; there is no fallback path.
"""
from __future__ import annotations

import collections
import contextlib
import ctypes
import os
import sys
import threading
import types

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmbw.so")

MBW_OK = 0
OP_GEMV_BF16 = 1
OP_GEMV_INT4_G64 = 2
OP_GEMV_INT4_AWQ_G128 = 3
OP_GEMM_SKINNY_BF16 = 4
OP_GEMV_INT8_PC = 5
FUSE_NORM = 0x100
FUSE_GLU = 0x200
FUSE_RESIDUAL = 0x400
REPACKED = 0x800

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t
_ST = ctypes.c_int

_lock = threading.Lock()
_lib = None


class MbwFusion(ctypes.Structure):
    """struct mbw_fusion of include/mbw.h."""
    _fields_ = [("norm_weight", ctypes.c_void_p), ("norm_eps", ctypes.c_float), ("residual", ctypes.c_void_p),
                ("up_weights", ctypes.c_void_p), ("up_scales", ctypes.c_void_p), ("up_zeros", ctypes.c_void_p)]


class MbwKv4Cache(ctypes.Structure):
    """struct mbw_kv4_cache of include/mbw.h."""
    _fields_ = [("pages", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("group", ctypes.c_int32)]


class MbwRope(ctypes.Structure):
    """struct mbw_rope of include/mbw.h."""
    _fields_ = [("cos_sin", ctypes.c_void_p), ("max_pos", ctypes.c_int64), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("positions", ctypes.c_void_p)]


# name -> (argtypes, restype)
SIGNATURES = {
    "gemv_bf16": ([_P, _P, _P, _I64, _I64, _P, _SZ, _P], _ST),
    "gemv_int4_g64": ([_P, _P, _P, _P, _I64, _I64, _P, _SZ, _P], _ST),
    "gemv_int4_awq_g128": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P], _ST),
    "gemv_int4_awq_g128_repacked": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P], _ST),
    "mbw_repack_int4": ([_P, _P, _I64, _I64, _P], _ST),
    "gemm_skinny_bf16": ([_P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P], _ST),
    "gemv_int8_pc": ([_P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P], _ST),
    "mbw_quantize_int8_pc": ([_P, _P, _P, _I64, _I64, _P], _ST),
    "gemv_fused": ([ctypes.c_int, _P, _P, _P, _P, _I64, _I64, _I64, ctypes.POINTER(MbwFusion), _P, _SZ, _P], _ST),
    "gemv_fused_awq_g128": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, ctypes.c_int, ctypes.POINTER(MbwFusion), _P, _SZ,
                             _P], _ST),
    "mbw_kv4_page_bytes": ([_I32, _I32, _I32, _I32], _SZ),
    "mbw_kv4_append": ([_P, _P, _I64, _P, _I64, _P, _P, _I64, _P, _I64, _I64, _P, _I64, _P], _ST),
    "mbw_kv4_gather": ([_P, _P, _P, _P, _I64, _P], _ST),
    "mbw_kv4_attention": ([_P, _P, _I64, _P, _I64, _P, _P, _I64, _I64, _P, _P, _I64, _I64, _I64, ctypes.c_float, _I64,
                           _P, _SZ, _P], _ST),
    "mbw_kv4_attention_workspace_bytes": ([_I32], _SZ),
    "mbw_token_logprobs": ([_P, ctypes.c_int, _I64, _P, _I64, _I64, ctypes.c_float, _I32, _P, _P, _P, _P, _P, _P, _SZ,
                            _P], _ST),
    "mbw_token_logprobs_workspace_bytes": ([], _SZ),
    "mbw_workspace_bytes": ([ctypes.c_int, _I64, _I64, _I64], _SZ),
    "mbw_dequant_int4_g64": ([_P, _P, _P, _I64, _I64, _P], _ST),
    "mbw_dequant_int4_awq_g128": ([_P, _P, _P, _P, _I64, _I64, _P], _ST),
    "mbw_set_output_fp32": ([ctypes.c_int], _ST),
    "mbw_autotune": ([ctypes.c_int, _I64, _I64, _I64, _P], _ST),
    "mbw_plan_candidates": ([ctypes.c_int, _I64, _I64, _I64], ctypes.c_int),
    "mbw_plan_select": ([ctypes.c_int, _I64, _I64, _I64, ctypes.c_int], _ST),
    "mbw_plan_index": ([ctypes.c_int, _I64, _I64, _I64], ctypes.c_int),
    "mbw_plan_describe": ([ctypes.c_int, _I64, _I64, _I64, ctypes.c_char_p, _SZ], _ST),
    "mbw_check_device_error": ([], _ST),
    "mbw_selftest_wait_expiry": ([_I64, _P], _ST),
    "mbw_inject_launch_failures": ([ctypes.c_int], _ST),
    "mbw_launch_count": ([], ctypes.c_uint64),
    "mbw_status_string": ([_ST], ctypes.c_char_p),
    "mbw_last_error": ([], ctypes.c_char_p),
}


class MbwError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str):
        super().__init__(f"{fn} failed: status {status} ({detail})")
        self.status = status
        self.detail = detail


def lib() -> ctypes.CDLL:
    """The loaded libmbw.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                       "`python -m memory_bound_weight_gb300.build`")
                L = ctypes.CDLL(LIB_PATH)
                for name, (args, res) in SIGNATURES.items():
                    f = getattr(L, name)
                    f.argtypes = args
                    f.restype = res
                _lib = L
    return _lib


def check(fn: str, status: int) -> None:
    if status != MBW_OK:
        L = lib()
        name = L.mbw_status_string(status).decode()
        detail = L.mbw_last_error().decode()
        raise MbwError(fn, status, f"{name}: {detail}")


def _torch():
    import torch

    return torch


def _stream_ptr(device) -> int:
    torch = _torch()
    return torch.cuda.current_stream(device).cuda_stream


def _need(t, name, dtype, ndim):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {t.dim()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _common_device(*ts):
    """The one device all given tensors (None skipped) are on."""
    devs = {t.device for t in ts if t is not None}
    if len(devs) != 1:
        raise ValueError(f"all tensors must be on one device, got {sorted(str(d) for d in devs)}")
    return devs.pop()


def _on_current_device(*ts):
    """All tensors on one CUDA device, the current one: the library plans and
    launches on the current device, and a kernel given another device's memory
    would fault."""
    torch = _torch()
    d = _common_device(*ts)
    cur = torch.cuda.current_device()
    if d.index != cur:
        raise ValueError(f"tensors are on {d} but the current CUDA device is cuda:{cur} (torch.cuda.set_device)")
    return d


def _need_shape(t, name, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


_tls = threading.local()


def _out_dtype():
    torch = _torch()
    return torch.float32 if getattr(_tls, "fp32", False) else torch.bfloat16


@contextlib.contextmanager
def output_fp32():
    """Within this block, calls on this thread write the fp32 accumulator (test hook)."""
    check("mbw_set_output_fp32", lib().mbw_set_output_fp32(1))
    _tls.fp32 = True
    try:
        yield
    finally:
        lib().mbw_set_output_fp32(0)
        _tls.fp32 = False


def _alloc_out(shape, like, out):
    torch = _torch()
    dt = _out_dtype()
    if out is None:
        return torch.empty(shape, dtype=dt, device=like.device)
    _need(out, "out", dt, len(shape))
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"out must have shape {tuple(shape)}")
    return out


def _ws(workspace):
    if workspace is None:
        return None, 0
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


# ----------------------------------------------------------------- calls ----
def gemv_bf16(W, x, out=None, workspace=None):
    """y = W . x; W bf16 (N, K), x bf16 (K,) -> y (N,)."""
    torch = _torch()
    _need(W, "W", torch.bfloat16, 2)
    _need(x, "x", torch.bfloat16, 1)
    N, K = W.shape
    if x.shape[0] != K:
        raise ValueError("x must have length K")
    y = _alloc_out((N,), W, out)
    _on_current_device(W, x, y, workspace)
    wp, wn = _ws(workspace)
    check("gemv_bf16", lib().gemv_bf16(W.data_ptr(), x.data_ptr(), y.data_ptr(), N, K, wp, wn,
                                       _stream_ptr(W.device)))
    return y


def gemv_int4_g64(Wq, scales, x, out=None, workspace=None):
    """y = W . x; Wq uint8 (N, K/2), scales fp16 (N, K/64), x bf16 (K,) -> y (N,)."""
    torch = _torch()
    _need(Wq, "Wq", torch.uint8, 2)
    _need(scales, "scales", torch.float16, 2)
    _need(x, "x", torch.bfloat16, 1)
    N = Wq.shape[0]
    K = x.shape[0]
    if Wq.shape[1] * 2 != K or tuple(scales.shape) != (N, K // 64):
        raise ValueError("shapes: Wq (N, K/2), scales (N, K/64), x (K,)")
    y = _alloc_out((N,), Wq, out)
    _on_current_device(Wq, scales, x, y, workspace)
    wp, wn = _ws(workspace)
    check("gemv_int4_g64", lib().gemv_int4_g64(Wq.data_ptr(), scales.data_ptr(), x.data_ptr(), y.data_ptr(),
                                               N, K, wp, wn, _stream_ptr(Wq.device)))
    return y


def gemv_int4_awq_g128(Wq, scales, zeros, X, out=None, workspace=None, repacked=False):
    """Y = X . W^T; Wq uint8 (N, K/2), scales fp16 (N, G), zeros uint8 (N, ceil(G/2)),
    X bf16 (M, K) or (K,) -> Y (M, N) or (N,). `repacked`: Wq is in the layout of
    repack_int4 (calls gemv_int4_awq_g128_repacked)."""
    torch = _torch()
    vec = X.dim() == 1
    X2 = X.unsqueeze(0) if vec else X
    _need(Wq, "Wq", torch.uint8, 2)
    _need(scales, "scales", torch.float16, 2)
    _need(zeros, "zeros", torch.uint8, 2)
    _need(X2, "X", torch.bfloat16, 2)
    M, K = X2.shape
    N = Wq.shape[0]
    G = K // 128
    if Wq.shape[1] * 2 != K or tuple(scales.shape) != (N, G) or tuple(zeros.shape) != (N, (G + 1) // 2):
        raise ValueError("shapes: Wq (N, K/2), scales (N, K/128), zeros (N, ceil(K/256)), X (M, K)")
    Y = _alloc_out((M, N), Wq, None if out is None else (out.unsqueeze(0) if vec else out))
    _on_current_device(Wq, scales, zeros, X2, Y, workspace)
    wp, wn = _ws(workspace)
    name = "gemv_int4_awq_g128_repacked" if repacked else "gemv_int4_awq_g128"
    check(name, getattr(lib(), name)(
        Wq.data_ptr(), scales.data_ptr(), zeros.data_ptr(), X2.data_ptr(), Y.data_ptr(), M, N, K, wp, wn,
        _stream_ptr(Wq.device)))
    return Y[0] if vec else Y


def repack_int4(Wq, out=None):
    """Canonical INT4 codes uint8 (N, K/2) -> the load-time repacked layout (a new
    tensor, or `out`, which may be Wq itself)."""
    torch = _torch()
    _need(Wq, "Wq", torch.uint8, 2)
    N, half = Wq.shape
    Wr = torch.empty_like(Wq) if out is None else out
    if Wr.shape != Wq.shape or Wr.dtype != torch.uint8 or not Wr.is_contiguous():
        raise ValueError("out must be a contiguous uint8 tensor of Wq's shape")
    _on_current_device(Wq, Wr)
    check("mbw_repack_int4", lib().mbw_repack_int4(Wq.data_ptr(), Wr.data_ptr(), N, 2 * half, _stream_ptr(Wq.device)))
    return Wr


def gemm_skinny_bf16(X, W, out=None, workspace=None):
    """Y = X . W^T; X bf16 (M, K), W bf16 (N, K) -> Y (M, N)."""
    torch = _torch()
    _need(X, "X", torch.bfloat16, 2)
    _need(W, "W", torch.bfloat16, 2)
    M, K = X.shape
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError("W must be (N, K)")
    Y = _alloc_out((M, N), W, out)
    _on_current_device(X, W, Y, workspace)
    wp, wn = _ws(workspace)
    check("gemm_skinny_bf16", lib().gemm_skinny_bf16(X.data_ptr(), W.data_ptr(), Y.data_ptr(), M, N, K, wp, wn,
                                                     _stream_ptr(W.device)))
    return Y


def gemv_int8_pc(Wq, scales, X, out=None, workspace=None):
    """Y = X . W^T; Wq int8 (N, K), scales fp32 (N,), X bf16 (M, K) or (K,) -> Y (M, N) or (N,)."""
    torch = _torch()
    vec = X.dim() == 1
    X2 = X.unsqueeze(0) if vec else X
    _need(Wq, "Wq", torch.int8, 2)
    _need(scales, "scales", torch.float32, 1)
    _need(X2, "X", torch.bfloat16, 2)
    M, K = X2.shape
    N = Wq.shape[0]
    if Wq.shape[1] != K or scales.shape[0] != N:
        raise ValueError("shapes: Wq (N, K), scales (N,), X (M, K)")
    Y = _alloc_out((M, N), Wq, None if out is None else (out.unsqueeze(0) if vec else out))
    _on_current_device(Wq, scales, X2, Y, workspace)
    wp, wn = _ws(workspace)
    check("gemv_int8_pc", lib().gemv_int8_pc(Wq.data_ptr(), scales.data_ptr(), X2.data_ptr(), Y.data_ptr(), M, N, K,
                                             wp, wn, _stream_ptr(Wq.device)))
    return Y[0] if vec else Y


def gemv_fused(op, W, scales, X, out=None, norm_weight=None, norm_eps=1e-6, residual=None, up_weights=None,
               up_scales=None, workspace=None):
    """One GEMV of format `op` (OP_GEMV_BF16 / _INT4_G64 / _INT8_PC) with optional fusions:
    RMSNorm prologue (norm_weight bf16 (K,)), gated SiLU epilogue (up_weights / up_scales, same
    layout as W / scales), residual add (residual bf16 shaped like the output; may be `out`).
    X bf16 (M, K) or (K,) -> Y (M, N) or (N,)."""
    torch = _torch()
    vec = X.dim() == 1
    X2 = X.unsqueeze(0) if vec else X
    _need(X2, "X", torch.bfloat16, 2)
    M, K = X2.shape
    N = W.shape[0]
    wdt, sdt, kdiv = {OP_GEMV_BF16: (torch.bfloat16, None, 1), OP_GEMV_INT4_G64: (torch.uint8, torch.float16, 2),
                      OP_GEMV_INT8_PC: (torch.int8, torch.float32, 1)}[op]
    _need(W, "W", wdt, 2)
    if W.shape[1] * kdiv != K:
        raise ValueError("W does not match K")
    sshape = None if sdt is None else ((N, K // 64) if op == OP_GEMV_INT4_G64 else (N,))
    if sdt is not None:
        _need(scales, "scales", sdt, len(sshape))
        _need_shape(scales, "scales", sshape)
    f = MbwFusion()
    if norm_weight is not None:
        _need(norm_weight, "norm_weight", torch.bfloat16, 1)
        if norm_weight.shape[0] != K:
            raise ValueError("norm_weight must have length K")
        f.norm_weight = norm_weight.data_ptr()
        f.norm_eps = float(norm_eps)
    if up_weights is not None:
        _need(up_weights, "up_weights", wdt, 2)
        if tuple(up_weights.shape) != tuple(W.shape):
            raise ValueError("up_weights must have W's shape")
        f.up_weights = up_weights.data_ptr()
        if sdt is not None:
            _need(up_scales, "up_scales", sdt, len(sshape))
            _need_shape(up_scales, "up_scales", sshape)
            f.up_scales = up_scales.data_ptr()
    Y = _alloc_out((M, N), X2, None if out is None else (out.unsqueeze(0) if vec else out))
    if residual is not None:
        r2 = residual.unsqueeze(0) if residual.dim() == 1 else residual
        _need(r2, "residual", torch.bfloat16, 2)
        if tuple(r2.shape) != (M, N):
            raise ValueError("residual must be shaped like the output")
        f.residual = r2.data_ptr()
    _on_current_device(W, scales if sdt is not None else None, X2, Y, norm_weight, residual, up_weights,
                       up_scales if (up_weights is not None and sdt is not None) else None, workspace)
    wp, wn = _ws(workspace)
    check("gemv_fused", lib().gemv_fused(op, W.data_ptr(), None if scales is None else scales.data_ptr(),
                                         X2.data_ptr(), Y.data_ptr(), M, N, K, ctypes.byref(f), wp, wn,
                                         _stream_ptr(X2.device)))
    return Y[0] if vec else Y


def gemv_fused_awq_g128(Wq, scales, zeros, X, out=None, norm_weight=None, norm_eps=1e-6, residual=None,
                        up_weights=None, up_scales=None, up_zeros=None, repacked=False, workspace=None):
    """gemv_int4_awq_g128 (Wq uint8 (N, K/2), scales fp16 (N, K/128), zeros uint8 (N, (K/128+1)/2); codes
    canonical or, with repacked=True, from repack_int4) with optional fusions: RMSNorm prologue
    (norm_weight bf16 (K,)), gated SiLU epilogue (up_weights / up_scales / up_zeros, same layouts),
    residual add (bf16 shaped like the output; may be `out`). X bf16 (M, K) or (K,) -> Y (M, N) or (N,)."""
    torch = _torch()
    vec = X.dim() == 1
    X2 = X.unsqueeze(0) if vec else X
    _need(X2, "X", torch.bfloat16, 2)
    M, K = X2.shape
    _need(Wq, "Wq", torch.uint8, 2)
    N = Wq.shape[0]
    if Wq.shape[1] * 2 != K:
        raise ValueError("Wq does not match K")
    G = K // 128
    _need(scales, "scales", torch.float16, 2)
    _need_shape(scales, "scales", (N, G))
    _need(zeros, "zeros", torch.uint8, 2)
    _need_shape(zeros, "zeros", (N, (G + 1) // 2))
    f = MbwFusion()
    if norm_weight is not None:
        _need(norm_weight, "norm_weight", torch.bfloat16, 1)
        if norm_weight.shape[0] != K:
            raise ValueError("norm_weight must have length K")
        f.norm_weight = norm_weight.data_ptr()
        f.norm_eps = float(norm_eps)
    if up_weights is not None:
        _need(up_weights, "up_weights", torch.uint8, 2)
        if tuple(up_weights.shape) != tuple(Wq.shape):
            raise ValueError("up_weights must have Wq's shape")
        _need(up_scales, "up_scales", torch.float16, 2)
        _need_shape(up_scales, "up_scales", (N, G))
        _need(up_zeros, "up_zeros", torch.uint8, 2)
        _need_shape(up_zeros, "up_zeros", (N, (G + 1) // 2))
        f.up_weights, f.up_scales, f.up_zeros = up_weights.data_ptr(), up_scales.data_ptr(), up_zeros.data_ptr()
    Y = _alloc_out((M, N), X2, None if out is None else (out.unsqueeze(0) if vec else out))
    if residual is not None:
        r2 = residual.unsqueeze(0) if residual.dim() == 1 else residual
        _need(r2, "residual", torch.bfloat16, 2)
        if tuple(r2.shape) != (M, N):
            raise ValueError("residual must be shaped like the output")
        f.residual = r2.data_ptr()
    _on_current_device(Wq, scales, zeros, X2, Y, norm_weight, residual, up_weights, up_scales, up_zeros, workspace)
    wp, wn = _ws(workspace)
    check("gemv_fused_awq_g128", lib().gemv_fused_awq_g128(Wq.data_ptr(), scales.data_ptr(), zeros.data_ptr(),
                                                           X2.data_ptr(), Y.data_ptr(), M, N, K, int(bool(repacked)),
                                                           ctypes.byref(f), wp, wn, _stream_ptr(X2.device)))
    return Y[0] if vec else Y


def quantize_int8_pc(W):
    """BF16 W (N, K) -> (Wq int8 (N, K), scales fp32 (N,)), scale = max|w| / 127 per row."""
    torch = _torch()
    _need(W, "W", torch.bfloat16, 2)
    N, K = W.shape
    _on_current_device(W)
    Wq = torch.empty((N, K), dtype=torch.int8, device=W.device)
    sc = torch.empty((N,), dtype=torch.float32, device=W.device)
    check("mbw_quantize_int8_pc", lib().mbw_quantize_int8_pc(W.data_ptr(), Wq.data_ptr(), sc.data_ptr(), N, K,
                                                             _stream_ptr(W.device)))
    return Wq, sc


def dequant_int4_g64(Wq, scales):
    torch = _torch()
    _need(Wq, "Wq", torch.uint8, 2)
    _need(scales, "scales", torch.float16, 2)
    N, K = Wq.shape[0], Wq.shape[1] * 2
    _need_shape(scales, "scales", (N, K // 64))
    _on_current_device(Wq, scales)
    out = torch.empty((N, K), dtype=torch.float32, device=Wq.device)
    check("mbw_dequant_int4_g64", lib().mbw_dequant_int4_g64(Wq.data_ptr(), scales.data_ptr(), out.data_ptr(),
                                                             N, K, _stream_ptr(Wq.device)))
    return out


def dequant_int4_awq_g128(Wq, scales, zeros):
    torch = _torch()
    _need(Wq, "Wq", torch.uint8, 2)
    _need(scales, "scales", torch.float16, 2)
    _need(zeros, "zeros", torch.uint8, 2)
    N, K = Wq.shape[0], Wq.shape[1] * 2
    G = K // 128
    _need_shape(scales, "scales", (N, G))
    _need_shape(zeros, "zeros", (N, (G + 1) // 2))
    _on_current_device(Wq, scales, zeros)
    out = torch.empty((N, K), dtype=torch.float32, device=Wq.device)
    check("mbw_dequant_int4_awq_g128", lib().mbw_dequant_int4_awq_g128(
        Wq.data_ptr(), scales.data_ptr(), zeros.data_ptr(), out.data_ptr(), N, K, _stream_ptr(Wq.device)))
    return out


# The calls below are made many times per token, so their checks read each tensor once and compare devices by number; what
# is wrong is told by the slower checks above.
_dtypes = None
_fast = None  # the compiled marshalling of these calls (csrc/fast_calls.cpp); False where it was not built or does not fit


def _load_fast():
    global _fast
    L = lib()
    if not isinstance(L, ctypes.CDLL):  # a stand-in for the library sees the calls as the Python functions make them
        return
    path = os.path.join(os.path.dirname(LIB_PATH), "_fast.so")
    if not os.path.exists(path):
        _fast = False
        return
    import importlib.machinery
    import importlib.util
    import warnings

    torch = _torch()  # the libraries it is linked to
    _fast = False
    try:
        loader = importlib.machinery.ExtensionFileLoader("_fast", path)
        mod = importlib.util.module_from_spec(importlib.util.spec_from_loader("_fast", loader))
        loader.exec_module(mod)
        here, its = f"{sys.implementation.cache_tag} torch {torch.__version__}", getattr(mod, "built_for", "another build")
        if its != here:
            raise ImportError(f"built for {its}, this is {here}")
    except (ImportError, OSError) as e:
        warnings.warn(f"{path} is not used, calls are marshalled in Python (build() makes it anew): {e}", RuntimeWarning)
        return
    mod.init(*(ctypes.cast(f, ctypes.c_void_p).value
               for f in (L.mbw_kv4_append, L.mbw_kv4_gather, L.mbw_kv4_attention, L.mbw_token_logprobs)))
    _fast = mod


def _types():
    global _dtypes
    if _dtypes is None:
        torch = _torch()
        _dtypes = (torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8, torch.empty)
    return _dtypes


def _device_index():
    global _device_index
    _device_index = _torch()._C._cuda_getDevice
    return _device_index()


def _raw_stream(index):
    global _raw_stream
    _raw_stream = _torch()._C._cuda_getCurrentRawStream
    return _raw_stream(index)


def _check_devices(*ts):
    """All tensors (None skipped) on the current CUDA device, whose number it returns."""
    cur = _device_index()
    for t in ts:
        if t is not None and t.get_device() != cur:
            _on_current_device(*ts)  # says which
    return cur


def _plain(t, name, dtype, ndim):
    """_need's checks; returns the shape."""
    try:
        shape = t.shape
        if t.dtype is dtype and t.is_cuda and len(shape) == ndim and t.is_contiguous():
            return shape
    except AttributeError:
        pass
    _need(t, name, dtype, ndim)
    return t.shape


def _vector(t, name, dtype, n):
    if _plain(t, name, dtype, 1)[0] != n:
        _need_shape(t, name, (n,))


class Kv4Cache:
    """4-bit paged key/value cache over `pages`, a contiguous uint8 tensor (num_pages,
    kv4_page_bytes(page_size, kv_heads, head_dim, group)) that the caller owns. It stays as it was made, and so
    must the tensor's memory; for other pages make another."""

    __slots__ = ("pages", "kv_heads", "head_dim", "page_size", "group", "_c", "_addr")

    def __init__(self, pages, kv_heads, head_dim, page_size=16, group=64):
        size = kv4_page_bytes(page_size, kv_heads, head_dim, group)
        num, got = _plain(pages, "pages", _types()[4], 2)
        if got != size:
            raise ValueError(f"pages must have {size} bytes per page, got {got}")
        c = MbwKv4Cache(pages.data_ptr(), num, page_size, kv_heads, head_dim, group)
        put = _kv4_cache_put
        put[0](self, pages), put[1](self, kv_heads), put[2](self, head_dim), put[3](self, page_size), put[4](self, group)
        put[5](self, c), put[6](self, ctypes.addressof(c))

    def __setattr__(self, name, value):
        raise AttributeError(f"a Kv4Cache stays as it was made; make another for other {name}")

    def __delattr__(self, name):
        raise AttributeError("a Kv4Cache stays as it was made")

    def _check(self):
        """The tensor still is what the cache was made over (its storage may have been changed or freed under it)."""
        if self.pages.data_ptr() != (self._c.pages or 0) or self.pages.numel() != self._c.num_pages * kv4_page_bytes(
                self.page_size, self.kv_heads, self.head_dim, self.group):
            raise ValueError("the cache's pages were moved or resized after it was made; make another Kv4Cache")


_kv4_cache_put = tuple(getattr(Kv4Cache, name).__set__ for name in Kv4Cache.__slots__)  # past its __setattr__


def kv4_page_bytes(page_size, kv_heads, head_dim, group=64):
    """Bytes of one page of a Kv4Cache (page_size a multiple of 16 up to 1024, head_dim 64, 128 or 256, group 32 or 64)."""
    if (page_size % 16 or not 16 <= page_size <= 1024 or not 1 <= kv_heads <= 1024 or head_dim not in (64, 128, 256)
            or group not in (32, 64)):
        raise ValueError("page_size must be a multiple of 16 up to 1024, head_dim 64, 128 or 256, group 32 or 64, "
                         "kv_heads 1 to 1024")
    return kv_heads * (page_size // 16) * (16 * head_dim + 128 * (head_dim // group))


def _need_rows(t, name, heads, dim):
    """bf16 (T, heads, dim), possibly rows of a wider matrix; returns (T, heads, the row stride in elements)."""
    try:
        shape, st = t.shape, t.stride()
        if t.dtype is _types()[0] and t.is_cuda and len(shape) == 3:
            n, h, w = shape
            if w == dim and (heads is None or h == heads) and st[2] == 1 and (st[1] == dim or h == 1):
                return n, h, st[0] if n > 1 else h * dim
    except AttributeError:
        pass
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != 3 or (heads is not None and t.shape[1] != heads) or t.shape[2] != dim:
        raise ValueError(f"{name} must have shape (T, {'heads' if heads is None else heads}, {dim}), got {tuple(t.shape)}")
    raise ValueError(f"{name} must have contiguous rows of heads")


def kv4_append(cache, k, v, slots, q=None, positions=None, cos_sin=None, interleaved=False, q_out=None):
    """Rotate T tokens' queries and keys by their position and store keys and values in the cache.
    k, v bf16 (T, kv_heads, head_dim), q bf16 (T, q_heads, head_dim) or None, each possibly a part of a
    wider QKV output; slots int64 (T,), page * page_size + place in the page, negative: not stored.
    positions int32 (T,) and cos_sin fp32 (max_pos, rotary_dim) (see rope_table) together, or neither:
    no rotation. Returns the rotated queries (`q_out`, which may be q, or a new tensor), None without q."""
    if _fast is None:
        _load_fast()
    if _fast:
        r = _fast.kv4_append(cache._addr, cache.pages, k, v, slots, q, positions, cos_sin, interleaved, q_out)
        if r is not None:
            return r[0] if r.__class__ is tuple else check("mbw_kv4_append", r)
    cache._check()
    bf16, f32, i32, i64, _, empty = _types()
    hk, d = cache.kv_heads, cache.head_dim
    T, _, ks = _need_rows(k, "k", hk, d)
    Tv, _, vs = _need_rows(v, "v", hk, d)
    if Tv != T:
        raise ValueError("k and v must have the same number of tokens")
    _vector(slots, "slots", i64, T)
    qp = op = None
    qs = os_ = hq = 0
    if q is not None:
        Tq, hq, qs = _need_rows(q, "q", None, d)
        if Tq != T:
            raise ValueError("q and k must have the same number of tokens")
        if q_out is None:
            q_out = empty((T, hq, d), dtype=bf16, device=q.device)
            os_ = hq * d
        else:
            To, _, os_ = _need_rows(q_out, "q_out", hq, d)
            if To != T:
                raise ValueError("q_out and q must have the same number of tokens")
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    rope = None
    if (positions is None) != (cos_sin is None):
        raise ValueError("positions and cos_sin go together")
    if positions is not None:
        _vector(positions, "positions", i32, T)
        most, dim = _plain(cos_sin, "cos_sin", f32, 2)
        rope = ctypes.byref(MbwRope(cos_sin.data_ptr(), most, dim, 1 if interleaved else 0, positions.data_ptr()))
    dev = _check_devices(cache.pages, k, v, slots, q, q_out, positions, cos_sin)
    st = lib().mbw_kv4_append(ctypes.byref(cache._c), k.data_ptr(), ks, v.data_ptr(), vs, slots.data_ptr(), qp, qs, op,
                              os_, hq, rope, T, _raw_stream(dev))
    if st:
        check("mbw_kv4_append", st)
    return q_out


def kv4_gather(cache, slots):
    """The keys and values the cache holds at `slots` int64 (T,), each bf16 (T, kv_heads, head_dim); zeros for a
    negative slot."""
    if _fast is None:
        _load_fast()
    if _fast:
        r = _fast.kv4_gather(cache._addr, cache.pages, slots)
        if r is not None:
            return r if r.__class__ is tuple else check("mbw_kv4_gather", r)
    cache._check()
    bf16, _, _, i64, _, empty = _types()
    T, = _plain(slots, "slots", i64, 1)
    dev = _check_devices(cache.pages, slots)
    shape, device = (T, cache.kv_heads, cache.head_dim), slots.device
    k, v = empty(shape, dtype=bf16, device=device), empty(shape, dtype=bf16, device=device)
    st = lib().mbw_kv4_gather(ctypes.byref(cache._c), slots.data_ptr(), k.data_ptr(), v.data_ptr(), T, _raw_stream(dev))
    if st:
        check("mbw_kv4_gather", st)
    return k, v


def kv4_attention_workspace(head_dim, device="cuda"):
    """A workspace for kv4_attention (zero, as it has to be before its first use); one per stream."""
    torch = _torch()
    return torch.zeros(int(lib().mbw_kv4_attention_workspace_bytes(head_dim)), dtype=torch.uint8, device=device)


def kv4_attention(cache, q, block_table, ctx_lens, q_starts=None, scale=None, window=0, out=None, return_lse=False,
                  workspace=None):
    """Attention of q bf16 (T, q_heads, head_dim), possibly a part of a wider matrix, over the cache.
    block_table int32 (B, width): each request's pages; ctx_lens int32 (B,): its tokens in the cache, the
    queries' own among them; q_starts int32 (B + 1,): where its queries begin in q, or None: T / B each.
    A query sees the keys up to its own position, with `window` > 0 only that many. scale: head_dim ** -0.5
    by default. Returns out (T, q_heads, head_dim), with return_lse also fp32 (T, q_heads). workspace: from
    kv4_attention_workspace; without one, long contexts are not split and take longer."""
    if _fast is None:
        _load_fast()
    if _fast and out is None and not getattr(_tls, "fp32", False):
        r = _fast.kv4_attention(cache._addr, cache.pages, q, block_table, ctx_lens, q_starts,
                                cache.head_dim ** -0.5 if scale is None else scale, window, return_lse, workspace)
        if r is not None:
            return check("mbw_kv4_attention", r) if r.__class__ is int else r
    cache._check()
    bf16, f32, i32, _, _, empty = _types()
    d = cache.head_dim
    T, hq, qs = _need_rows(q, "q", None, d)
    B, width = _plain(block_table, "block_table", i32, 2)
    _vector(ctx_lens, "ctx_lens", i32, B)
    sp = None
    if q_starts is not None:
        _vector(q_starts, "q_starts", i32, B + 1)
        sp = q_starts.data_ptr()
    os_ = hq * d
    wide = getattr(_tls, "fp32", False)  # output_fp32
    if out is None:
        out = empty((T, hq, d), dtype=f32 if wide else bf16, device=q.device)
    elif not wide:
        To, _, os_ = _need_rows(out, "out", hq, d)
        if To != T:
            raise ValueError("out and q must have the same number of tokens")
    else:
        out = _alloc_out((T, hq, d), q, out)
    lse = lp = None
    if return_lse:
        lse = empty((T, hq), dtype=f32, device=q.device)
        lp = lse.data_ptr()
    dev = _check_devices(cache.pages, q, block_table, ctx_lens, q_starts, out, workspace)
    wp, wn = _ws(workspace)
    st = lib().mbw_kv4_attention(
        ctypes.byref(cache._c), q.data_ptr(), qs, out.data_ptr(), os_, lp, block_table.data_ptr(), width, width,
        ctx_lens.data_ptr(), sp, B, T, hq, d ** -0.5 if scale is None else scale, window, wp, wn, _raw_stream(dev))
    if st:
        check("mbw_kv4_attention", st)
    return (out, lse) if return_lse else out


TokenLogprobs = collections.namedtuple("TokenLogprobs", "logprob rank entropy top_ids top_logprobs")


def token_logprobs_workspace(device="cuda"):
    """A workspace for token_logprobs (zero, as it has to be before its first use); one per stream."""
    torch = _torch()
    return torch.zeros(int(lib().mbw_token_logprobs_workspace_bytes()), dtype=torch.uint8, device=device)


def token_logprobs(logits, targets=None, top_k=0, scale=1.0, workspace=None):
    """What logits bf16 or fp32 (M, V) (rows may be apart) say about tokens, over scale * logits: the log
    probability fp32 (M,) and rank int32 (M,) of targets int32 (M,) (None without), the entropy fp32 (M,) in
    nats, the top_k (<= 32) most likely ids int32 (M, top_k) and their log probabilities fp32 (M, top_k).
    workspace: from token_logprobs_workspace; without one, few rows take longer."""
    if _fast is None:
        _load_fast()
    if _fast:
        r = _fast.token_logprobs(logits, targets, top_k, scale, workspace)
        if r is not None:
            return TokenLogprobs._make(r) if r.__class__ is tuple else check("mbw_token_logprobs", r)
    bf16, f32, i32, _, _, empty = _types()
    try:
        shape, dtype, device = logits.shape, logits.dtype, logits.device
    except AttributeError:
        raise TypeError("logits must be a torch.Tensor") from None
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    wide = dtype is f32
    if not wide and dtype is not bf16:
        raise TypeError(f"logits must be {bf16} or {f32}, got {dtype}")
    if len(shape) != 2 or (logits.stride(1) != 1 and shape[1] > 1):
        raise ValueError("logits must have 2 dimensions and contiguous rows")
    M, V = shape
    tp = lp = rank = lpp = rp = None
    if targets is not None:
        _vector(targets, "targets", i32, M)
    if not 0 <= top_k <= 32:
        raise ValueError("top_k must be 0 to 32")
    dev = _check_devices(logits, targets, workspace)
    if targets is not None:
        lp, rank = empty(M, dtype=f32, device=device), empty(M, dtype=i32, device=device)
        tp, lpp, rp = targets.data_ptr(), lp.data_ptr(), rank.data_ptr()
    ent = empty(M, dtype=f32, device=device)
    ids, tlp = empty((M, top_k), dtype=i32, device=device), empty((M, top_k), dtype=f32, device=device)
    wp, wn = _ws(workspace)
    st = lib().mbw_token_logprobs(logits.data_ptr(), 1 if wide else 0, logits.stride(0) if M > 1 else V, tp, M, V, scale,
                                  top_k, lpp, rp, ent.data_ptr(), ids.data_ptr(), tlp.data_ptr(), wp, wn, _raw_stream(dev))
    if st:
        check("mbw_token_logprobs", st)
    return TokenLogprobs(lp, rank, ent, ids, tlp)


def autotune(op: int, M: int, N: int, K: int) -> None:
    torch = _torch()
    check("mbw_autotune", lib().mbw_autotune(op, M, N, K, torch.cuda.current_stream().cuda_stream))


def plan_describe(op: int, M: int, N: int, K: int) -> str:
    buf = ctypes.create_string_buffer(256)
    check("mbw_plan_describe", lib().mbw_plan_describe(op, M, N, K, buf, 256))
    return buf.value.decode()


def plan_candidates(op: int, M: int, N: int, K: int) -> int:
    return int(lib().mbw_plan_candidates(op, M, N, K))


def plan_select(op: int, M: int, N: int, K: int, index: int) -> None:
    check("mbw_plan_select", lib().mbw_plan_select(op, M, N, K, index))


def plan_index(op: int, M: int, N: int, K: int) -> int:
    return int(lib().mbw_plan_index(op, M, N, K))


def workspace_bytes(op: int, M: int, N: int, K: int) -> int:
    return int(lib().mbw_workspace_bytes(op, M, N, K))


def launch_count() -> int:
    return int(lib().mbw_launch_count())


def check_device_error() -> None:
    check("mbw_check_device_error", lib().mbw_check_device_error())


def inject_launch_failures(count: int) -> None:
    """The next `count` launching calls on this thread raise MbwError with
    MBW_ERR_CUDA and launch nothing (host-side fault injection; 0 turns it off)."""
    check("mbw_inject_launch_failures", lib().mbw_inject_launch_failures(int(count)))


def selftest_wait_expiry(tries: int) -> None:
    """Launch, on the current stream, the two one-thread kernels whose bounded
    waits expire after `tries` rounds; the next check_device_error() raises
    MbwError with MBW_ERR_DEVICE_TIMEOUT."""
    check("mbw_selftest_wait_expiry", lib().mbw_selftest_wait_expiry(int(tries), _stream_ptr(None)))


class _Module(types.ModuleType):
    """This module: the package keeps the functions it was asked for (0.4 us an access otherwise), and what is set or
    deleted here afterwards changes there too."""

    def _forget(self, name):
        kept = vars(sys.modules[__package__])
        if name in kept and kept[name] is vars(self).get(name):
            del kept[name]  # found anew by its next access

    def __setattr__(self, name, value):
        self._forget(name)
        super().__setattr__(name, value)

    def __delattr__(self, name):
        self._forget(name)
        super().__delattr__(name)


sys.modules[__name__].__class__ = _Module
