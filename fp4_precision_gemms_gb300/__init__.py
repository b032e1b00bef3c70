"""GB300-native block-scaled (MXFP8 / MXFP4 / NVFP4 / MOSS two-level FP8) linear layer.

A thin ctypes binding over ``libmx_gb300.so`` (C ABI in ``include/mx.h``).  This
module only marshals arguments: every step of quantize, GEMM and the linear
layer's passes runs in the library's CUDA kernels.  PyTorch supplies device
memory and streams.  There is no CPU fallback: without the built library (see
``build()``) or an sm_103 GPU every call raises ``MXError``.
"""
from __future__ import annotations

import ctypes as C
import operator
import os
import threading
import warnings
from array import array
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmx_gb300.so")

FORMATS = {"mxfp8": 0, "mxfp4": 1, "nvfp4": 2, "moss": 3, "nvfp4_local": 4}
BLOCK = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16, "moss": 32, "nvfp4_local": 16}
FP4 = ("mxfp4", "nvfp4", "nvfp4_local")
ROUNDING = {"rne": 0, "sr": 1}
RULES = {"default": 0, "floor": 1, "ceil": 2, "nearest": 3}
DIRS = {"row": 0, "col": 1}
OUT = {torch.float32: 0, torch.bfloat16: 1}

MX_OK, MX_ERR_INVALID_ARG, MX_ERR_UNSUPPORTED, MX_ERR_ALIGNMENT = 0, 1, 2, 3
MX_ERR_CUDA, MX_ERR_TIMEOUT, MX_ERR_NO_DEVICE, MX_ERR_WORKSPACE = 4, 5, 6, 7

EXPORTED = ("mx_codes_bytes", "mx_sf_bytes", "mx_scale_count", "mx_amax", "mx_quantize", "mx_quantize_dual", "mx_dequantize", "mx_gemm",
            "mx_gemm_amax", "mx_gemm_quantized",
            "mx_linear_workspace_bytes", "mx_linear_fwd", "mx_linear_fwd_noalloc", "mx_linear_bwd",
            "mx_linear_saved_bytes", "mx_linear_fwd_save", "mx_linear_bwd_saved", "mx_strerror",
            "mx_act8_codes_bytes", "mx_act8_sf_bytes", "mx_act8_save", "mx_act8_restore", "mx_norm_fwd",
            "mx_norm_bwd_workspace_bytes", "mx_norm_bwd", "mx_act_fwd", "mx_act_bwd",
            "mx_gemm_gated", "mx_gated_workspace_bytes", "mx_gated_fwd", "mx_gated_fwd_save", "mx_gated_bwd",
            "mx_grad_norm_workspace_bytes", "mx_grad_norm", "mx_adamw_step",
            "mx_last_device_status", "mx_selftest_bounded_wait", "mx_launch_count",
            "mx_debug_divide", "mx_debug_set_quant_impl", "mx_debug_set_tile_fail_at", "mx_debug_set_norm_fail_at", "mx_debug_set_bwd_fork", "mx_debug_set_gemm_variant",
            "mx_debug_last_gemm_variant")


class MXError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        super().__init__(f"{what}: {strerror(code)} (mx_status {code})" if what else strerror(code))


class _CTensor(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("sf", C.c_void_p), ("amax", C.c_void_p),
                ("tensor_scale", C.c_void_p), ("rows", C.c_int64), ("k", C.c_int64),
                ("fmt", C.c_int32), ("block", C.c_int32), ("hadamard", C.c_int32),
                ("reserved", C.c_int32)]


class _CAct8(C.Structure):
    _fields_ = [("codes", C.c_void_p), ("sf", C.c_void_p), ("rows", C.c_int64), ("cols", C.c_int64)]


class _CGrad(C.Structure):
    _fields_ = [("data", C.c_void_p), ("n", C.c_int64), ("dtype", C.c_int32), ("reserved", C.c_int32)]


class _CAdamwTensor(C.Structure):
    _fields_ = [("param", C.c_void_p), ("grad", C.c_void_p), ("m", C.c_void_p), ("v", C.c_void_p),
                ("m_sf", C.c_void_p), ("v_sf", C.c_void_p), ("copy", C.c_void_p), ("n", C.c_int64),
                ("weight_decay", C.c_double), ("p_dtype", C.c_int32), ("g_dtype", C.c_int32), ("bits", C.c_int32),
                ("reserved", C.c_int32)]


class _CAdamwOpts(C.Structure):
    _fields_ = [("lr", C.c_double), ("beta1", C.c_double), ("beta2", C.c_double), ("eps", C.c_double),
                ("t", C.c_int64), ("lr_at", C.c_void_p), ("t_at", C.c_void_p), ("seed", C.c_uint64),
                ("rounding", C.c_int32), ("reserved", C.c_int32)]


class _CBwdOpts(C.Structure):
    _fields_ = [("wgrad_hadamard", C.c_int32), ("wgrad_dy_rounding", C.c_int32),
                ("seed", C.c_uint64), ("stream_id", C.c_uint32), ("reserved", C.c_int32)]


_lock = threading.Lock()
_lib = None


def build(force: bool = False) -> str:
    """Compile libmx_gb300.so in-tree for sm_103a (nvcc)."""
    from . import _build
    return _build.build(force=force)


def lib():
    """The loaded C library; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise MXError(MX_ERR_NO_DEVICE, f"{LIB_PATH} is not built (call build())")
            L = C.CDLL(LIB_PATH)
            p, i64, i32, u64, u32, sz = C.c_void_p, C.c_int64, C.c_int, C.c_uint64, C.c_uint32, C.c_size_t
            L.mx_codes_bytes.restype = sz
            L.mx_codes_bytes.argtypes = [i32, i64, i64]
            L.mx_sf_bytes.restype = sz
            L.mx_sf_bytes.argtypes = [i32, i64, i64]
            L.mx_scale_count.restype = sz
            L.mx_scale_count.argtypes = [i32, i64]
            L.mx_amax.restype = i32
            L.mx_amax.argtypes = [p, i64, i64, i64, p, p]
            L.mx_quantize.restype = i32
            L.mx_quantize.argtypes = [p, i64, i64, i64, i32, i32, i32, i32, i32, u64, u32, i32, p,
                                      C.POINTER(_CTensor), p]
            L.mx_quantize_dual.restype = i32
            L.mx_quantize_dual.argtypes = [p, i64, i64, i64, i32, i32, i32, u64, u32, i32, i32, i32, i32, p,
                                           C.POINTER(_CTensor), C.POINTER(_CTensor), p]
            L.mx_debug_set_quant_impl.restype = None
            L.mx_debug_set_quant_impl.argtypes = [i32]
            L.mx_debug_set_tile_fail_at.restype = None
            L.mx_debug_set_tile_fail_at.argtypes = [i64]
            L.mx_debug_set_norm_fail_at.restype = None
            L.mx_debug_set_norm_fail_at.argtypes = [i64]
            L.mx_debug_set_bwd_fork.restype = None
            L.mx_debug_set_bwd_fork.argtypes = [i32]
            L.mx_dequantize.restype = i32
            L.mx_dequantize.argtypes = [C.POINTER(_CTensor), p, p]
            L.mx_gemm.restype = i32
            L.mx_gemm.argtypes = [C.POINTER(_CTensor), C.POINTER(_CTensor), C.c_float, p, i64, i32, p]
            L.mx_gemm_amax.restype = i32
            L.mx_gemm_amax.argtypes = [C.POINTER(_CTensor), C.POINTER(_CTensor), C.c_float, p, i64, i32, p, p]
            L.mx_gemm_quantized.restype = i32
            L.mx_gemm_quantized.argtypes = [C.POINTER(_CTensor), C.POINTER(_CTensor), C.c_float,
                                            C.POINTER(_CTensor), p]
            L.mx_linear_workspace_bytes.restype = sz
            L.mx_linear_workspace_bytes.argtypes = [i64, i64, i64, i32, i32]
            L.mx_linear_fwd.restype = i32
            L.mx_linear_fwd.argtypes = [p, p, i64, i64, i64, i32, p, i32, p, sz, p]
            L.mx_linear_fwd_noalloc.restype = i32
            L.mx_linear_fwd_noalloc.argtypes = [p, p, i64, i64, i64, i32, p, i32, p]
            L.mx_linear_bwd.restype = i32
            L.mx_linear_bwd.argtypes = [p, p, p, i64, i64, i64, i32, C.POINTER(_CBwdOpts), p, i32, p,
                                        i32, p, sz, p]
            L.mx_linear_saved_bytes.restype = sz
            L.mx_linear_saved_bytes.argtypes = [i64, i64, i64, i32]
            L.mx_linear_fwd_save.restype = i32
            L.mx_linear_fwd_save.argtypes = [p, p, i64, i64, i64, i32, p, p, C.POINTER(_CBwdOpts), p, i32, p, sz,
                                             p, sz, p]
            L.mx_linear_bwd_saved.restype = i32
            L.mx_linear_bwd_saved.argtypes = [p, i64, i64, i64, i32, p, C.POINTER(_CBwdOpts), p, sz, p, i32, p, i32,
                                              p, sz, p]
            a8 = C.POINTER(_CAct8)
            for name in ("mx_act8_codes_bytes", "mx_act8_sf_bytes", "mx_norm_bwd_workspace_bytes"):
                getattr(L, name).restype = sz
                getattr(L, name).argtypes = [i64, i64]
            L.mx_act8_save.argtypes = [p, i64, i32, a8, p]
            L.mx_act8_restore.argtypes = [a8, p, i64, i32, p]
            L.mx_norm_fwd.argtypes = [p, i64, p, i64, i32, i64, i64, i32, p, p, i32, C.c_float, p, i64, p, i64, i32,
                                      p, p, a8, p, p]
            L.mx_norm_bwd.argtypes = [p, i64, i32, p, i64, a8, p, p, p, i32, i64, i64, i32, p, i64, p, i64, i32, p,
                                      p, p, p, sz, p]
            L.mx_act_fwd.argtypes = [p, i64, p, i64, i64, i64, i32, i32, p, i64, a8, a8, p, p]
            L.mx_act_bwd.argtypes = [p, i64, p, i64, p, i64, a8, a8, i64, i64, i32, i32, p, i64, p, i64, p, p]
            for name in ("mx_act8_save", "mx_act8_restore", "mx_norm_fwd", "mx_norm_bwd", "mx_act_fwd", "mx_act_bwd"):
                getattr(L, name).restype = i32
            t8 = C.POINTER(_CTensor)
            L.mx_gated_workspace_bytes.restype = sz
            L.mx_gated_workspace_bytes.argtypes = [i64, i64, i64, i32, i32]
            L.mx_gemm_gated.argtypes = [t8, t8, t8, i32, p, i64, a8, a8, p, p]
            L.mx_gated_fwd.argtypes = [p, i64, i64, i64, i64, i32, i32, p, t8, t8, p, i64, p, p, sz, p]
            L.mx_gated_fwd_save.argtypes = [p, i64, p, i64, i64, i64, i32, i32, p, p, C.POINTER(_CBwdOpts), p, i64, a8, a8,
                                            p, p, sz, p, sz, p]
            L.mx_gated_bwd.argtypes = [p, i64, i64, i64, i64, i32, i32, a8, a8, C.POINTER(_CBwdOpts), p, sz, p, i32, p,
                                       i32, p, sz, p]
            for name in ("mx_gemm_gated", "mx_gated_fwd", "mx_gated_fwd_save", "mx_gated_bwd"):
                getattr(L, name).restype = i32
            L.mx_grad_norm_workspace_bytes.restype = sz
            L.mx_grad_norm_workspace_bytes.argtypes = [i64]
            L.mx_grad_norm.restype = i32
            L.mx_grad_norm.argtypes = [C.POINTER(_CGrad), i64, C.c_double, p, p, sz, p]
            L.mx_adamw_step.restype = i32
            L.mx_adamw_step.argtypes = [C.POINTER(_CAdamwTensor), i64, C.POINTER(_CAdamwOpts), p, p, p]
            L.mx_strerror.restype = C.c_char_p
            L.mx_strerror.argtypes = [i32]
            L.mx_last_device_status.restype = i32
            L.mx_last_device_status.argtypes = [p]
            L.mx_selftest_bounded_wait.restype = i32
            L.mx_selftest_bounded_wait.argtypes = [u64, p]
            L.mx_launch_count.restype = u64
            L.mx_launch_count.argtypes = []
            L.mx_debug_divide.restype = i32
            L.mx_debug_divide.argtypes = [p, p, i64, p, p, p]
            L.mx_debug_set_gemm_variant.restype = None
            L.mx_debug_set_gemm_variant.argtypes = [i32]
            L.mx_debug_last_gemm_variant.restype = i32
            L.mx_debug_last_gemm_variant.argtypes = []
            _lib = L
    return _lib


def strerror(code: int) -> str:
    try:
        return lib().mx_strerror(int(code)).decode()
    except Exception:
        return f"mx_status {code}"


def _check(rc: int, what: str):
    if rc != MX_OK:
        raise MXError(rc, what)


def _stream(stream=None):
    if stream is None:
        if not torch.cuda.is_available():
            return None  # the library reports MX_ERR_NO_DEVICE
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def _on_gpu(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise MXError(MX_ERR_NO_DEVICE if not torch.cuda.is_available() else MX_ERR_INVALID_ARG,
                          "tensors must live on a CUDA device (there is no CPU path)")


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


class MXTensor:
    """A quantized K-major operand: codes, swizzled block scales, amax and tensor scale."""

    def __init__(self, fmt: str, rows: int, k: int, device=None):
        device = device or torch.device("cuda")
        self.fmt, self.rows, self.k = fmt, int(rows), int(k)
        self.block = BLOCK[fmt]
        self.hadamard = False
        L = lib()
        nc = L.mx_codes_bytes(FORMATS[fmt], self.rows, self.k)
        ns = L.mx_sf_bytes(FORMATS[fmt], self.rows, self.k)
        if (nc == 0 or ns == 0) and self.rows * self.k > 0:
            raise MXError(MX_ERR_INVALID_ARG, f"operand shape {rows}x{k} for {fmt}")
        kb = self.k // 2 if fmt in FP4 else self.k
        self.codes = torch.empty((self.rows, kb), dtype=torch.uint8, device=device)
        self.sf = torch.empty(max(ns, 1), dtype=torch.uint8, device=device)
        # amax and tensor scale: one each, or one per 128-row region (nvfp4_local)
        self.nscale = max(1, int(L.mx_scale_count(FORMATS[fmt], self.rows)))
        self.scalars = torch.zeros(2 * self.nscale, dtype=torch.float32, device=device)

    @property
    def amax(self):
        return self.scalars[0:self.nscale]

    @property
    def tensor_scale(self):
        return self.scalars[self.nscale:2 * self.nscale]

    def _c(self) -> _CTensor:
        t = _CTensor()
        _on_gpu(self.codes, self.sf, self.scalars)  # the library only reads and writes device memory
        t.codes = self.codes.data_ptr()
        t.sf = self.sf.data_ptr()
        t.amax = self.scalars.data_ptr()
        t.tensor_scale = self.scalars.data_ptr() + 4 * self.nscale
        t.rows, t.k = self.rows, self.k
        t.fmt, t.block, t.hadamard = FORMATS[self.fmt], self.block, int(self.hadamard)
        return t


def amax(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    _on_gpu(x, out)
    out = out if out is not None else torch.empty(1, dtype=torch.float32, device=x.device)
    _check(lib().mx_amax(_ptr(x), x.shape[0], x.shape[1], x.stride(0), _ptr(out), _stream(stream)),
           "mx_amax")
    return out


def quantize(x: torch.Tensor, fmt: str, direction: str = "row", rounding: str = "rne",
             rule: str = "default", seed: int = 0, stream_id: int = 0, hadamard: bool = False,
             amax_in: torch.Tensor | None = None, out: MXTensor | None = None, stream=None) -> MXTensor:
    """bf16 [R, C] -> block-scaled K-major operand (rowwise: [R, C]; colwise: [C, R])."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    _on_gpu(x, amax_in)
    R, Cc = x.shape
    rows, k = (R, Cc) if direction == "row" else (Cc, R)
    q = out if out is not None else MXTensor(fmt, rows, k, x.device)
    ct = q._c()
    rc = lib().mx_quantize(_ptr(x), R, Cc, x.stride(0), DIRS[direction], FORMATS[fmt], BLOCK[fmt],
                           ROUNDING[rounding], RULES[rule], seed, stream_id, int(bool(hadamard)),
                           _ptr(amax_in), C.byref(ct), _stream(stream))
    _check(rc, "mx_quantize")
    q.rows, q.k, q.hadamard = ct.rows, ct.k, bool(ct.hadamard)
    return q


def quantize_dual(x: torch.Tensor, fmt: str, rule: str = "default", seed: int = 0, stream_id: int = 0,
                  row_rounding: str = "rne", row_hadamard: bool = False, col_rounding: str = "rne",
                  col_hadamard: bool = False, amax_in: torch.Tensor | None = None,
                  row_out: MXTensor | None = None, col_out: MXTensor | None = None, stream=None):
    """One read of bf16 x [R, C] -> (rowwise operand [R, C], colwise operand [C, R])."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    _on_gpu(x, amax_in)
    R, Cc = x.shape
    qr = row_out if row_out is not None else MXTensor(fmt, R, Cc, x.device)
    qc = col_out if col_out is not None else MXTensor(fmt, Cc, R, x.device)
    cr, cc = qr._c(), qc._c()
    rc = lib().mx_quantize_dual(_ptr(x), R, Cc, x.stride(0), FORMATS[fmt], BLOCK[fmt], RULES[rule], seed,
                                stream_id, ROUNDING[row_rounding], int(bool(row_hadamard)),
                                ROUNDING[col_rounding], int(bool(col_hadamard)), _ptr(amax_in),
                                C.byref(cr), C.byref(cc), _stream(stream))
    _check(rc, "mx_quantize_dual")
    qr.rows, qr.k, qr.hadamard = cr.rows, cr.k, bool(cr.hadamard)
    qc.rows, qc.k, qc.hadamard = cc.rows, cc.k, bool(cc.hadamard)
    return qr, qc


QUANT_IMPLS = {"auto": 0, "direct": 1, "tile": 2}


def set_quant_impl(impl: str) -> None:
    """Choose the producer implementation (tests and tuning)."""
    lib().mx_debug_set_quant_impl(QUANT_IMPLS[impl])


def set_tile_fail_at(tile: int) -> None:
    """Test hook: the tile producer gives up its wait on this tile of each CTA (-1: off)."""
    lib().mx_debug_set_tile_fail_at(int(tile))


def set_norm_fail_at(row: int) -> None:
    """Test hook: the norm kernels give up their wait for this row of each CTA (-1: off)."""
    lib().mx_debug_set_norm_fail_at(int(row))


def set_bwd_fork(on: bool) -> None:
    """Whether linear_bwd / linear_bwd_saved run the weight gradient on the
    library's side stream (the default) or after the data gradient on the
    caller's stream.  Per host thread."""
    lib().mx_debug_set_bwd_fork(int(on))


def dequantize(q: MXTensor, stream=None) -> torch.Tensor:
    out = torch.empty((q.rows, q.k), dtype=torch.float32, device=q.codes.device)
    ct = q._c()
    _check(lib().mx_dequantize(C.byref(ct), _ptr(out), _stream(stream)), "mx_dequantize")
    return out


def gemm(a: MXTensor, b: MXTensor, extra_alpha: float = 1.0, out_dtype=torch.float32,
         out: torch.Tensor | None = None, stream=None, amax_out: torch.Tensor | None = None) -> torch.Tensor:
    """C[M, N] = alpha * dq(a) dq(b)^T on the tensor cores.  amax_out: an
    optional one-element fp32 device tensor that receives max |C| as written,
    reduced in the GEMM's epilogue."""
    _on_gpu(out, amax_out)
    out = out if out is not None else torch.empty((a.rows, b.rows), dtype=out_dtype,
                                                  device=a.codes.device)
    ca, cb = a._c(), b._c()
    if amax_out is None:
        rc = lib().mx_gemm(C.byref(ca), C.byref(cb), float(extra_alpha), _ptr(out), out.stride(0),
                           OUT[out.dtype], _stream(stream))
        _check(rc, "mx_gemm")
    else:
        if amax_out.dtype != torch.float32 or amax_out.numel() < 1:
            raise ValueError("amax_out must be a float32 tensor with at least one element")
        rc = lib().mx_gemm_amax(C.byref(ca), C.byref(cb), float(extra_alpha), _ptr(out), out.stride(0),
                                OUT[out.dtype], _ptr(amax_out), _stream(stream))
        _check(rc, "mx_gemm_amax")
    return out


def gemm_quantized(a: MXTensor, b: MXTensor, fmt: str = "mxfp8", extra_alpha: float = 1.0,
                   out: MXTensor | None = None, stream=None) -> MXTensor:
    """alpha * dq(a) dq(b)^T quantized in the GEMM epilogue into the rowwise MX
    operand (rows M = a.rows, K = N = b.rows) of format fmt (mxfp8 or mxfp4)."""
    out = out if out is not None else MXTensor(fmt, a.rows, b.rows, a.codes.device)
    ca, cb, co = a._c(), b._c(), out._c()
    _check(lib().mx_gemm_quantized(C.byref(ca), C.byref(cb), float(extra_alpha), C.byref(co), _stream(stream)),
           "mx_gemm_quantized")
    return out


PASSES = {"fwd": 0, "bwd": 1, "bwd_saved": 2}


def workspace_bytes(T: int, Kin: int, Nout: int, fmt: str, pass_: str = "fwd") -> int:
    return int(lib().mx_linear_workspace_bytes(T, Kin, Nout, FORMATS[fmt], PASSES[pass_]))


def saved_bytes(T: int, Kin: int, Nout: int, fmt: str) -> int:
    """Bytes of one layer's saved backward state (X^T and W^T operands)."""
    return int(lib().mx_linear_saved_bytes(T, Kin, Nout, FORMATS[fmt]))


def linear_fwd(X: torch.Tensor, W: torch.Tensor, fmt: str, out_dtype=torch.bfloat16,
               workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """Y = X W^T with X [T, Kin], W [Nout, Kin] (bf16, contiguous)."""
    _on_gpu(X, W, workspace, out)
    T, Kin = X.shape
    Nout = W.shape[0]
    n = workspace_bytes(T, Kin, Nout, fmt, "fwd")
    ws = workspace if workspace is not None else torch.empty(n, dtype=torch.uint8, device=X.device)
    Y = out if out is not None else torch.empty((T, Nout), dtype=out_dtype, device=X.device)
    rc = lib().mx_linear_fwd(_ptr(X), _ptr(W), T, Kin, Nout, FORMATS[fmt], _ptr(Y), OUT[Y.dtype],
                             _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "mx_linear_fwd")
    return Y


def linear_fwd_noalloc(X: torch.Tensor, W: torch.Tensor, fmt: str, out_dtype=torch.bfloat16,
                       out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """linear_fwd without a workspace: the library's fixed device array holds the
    quantized operands (for callers that cannot allocate; up to 32 MiB)."""
    _on_gpu(X, W, out)
    T, Kin = X.shape
    Nout = W.shape[0]
    Y = out if out is not None else torch.empty((T, Nout), dtype=out_dtype, device=X.device)
    rc = lib().mx_linear_fwd_noalloc(_ptr(X), _ptr(W), T, Kin, Nout, FORMATS[fmt], _ptr(Y),
                                     OUT[Y.dtype], _stream(stream))
    _check(rc, "mx_linear_fwd_noalloc")
    return Y


def linear_bwd(dY: torch.Tensor, X: torch.Tensor, W: torch.Tensor, fmt: str,
               wgrad_hadamard: bool = False, wgrad_dy_rounding: str = "rne", seed: int = 0,
               stream_id: int = 0, dx_dtype=torch.bfloat16, dw_dtype=torch.float32,
               need_dx: bool = True, need_dw: bool = True, workspace: torch.Tensor | None = None,
               dX: torch.Tensor | None = None, dW: torch.Tensor | None = None, stream=None):
    """dX = dY W and dW = dY^T X for the layer Y = X W^T."""
    _on_gpu(dY, X, W, workspace, dX, dW)
    T, Kin = X.shape
    Nout = W.shape[0]
    n = workspace_bytes(T, Kin, Nout, fmt, "bwd")
    ws = workspace if workspace is not None else torch.empty(n, dtype=torch.uint8, device=X.device)
    if need_dx and dX is None:
        dX = torch.empty((T, Kin), dtype=dx_dtype, device=X.device)
    if need_dw and dW is None:
        dW = torch.empty((Nout, Kin), dtype=dw_dtype, device=X.device)
    o = _CBwdOpts(int(bool(wgrad_hadamard)), ROUNDING[wgrad_dy_rounding], seed, stream_id, 0)
    rc = lib().mx_linear_bwd(_ptr(dY), _ptr(X), _ptr(W), T, Kin, Nout, FORMATS[fmt], C.byref(o),
                             _ptr(dX) if need_dx else None, OUT[dX.dtype] if need_dx else 0,
                             _ptr(dW) if need_dw else None, OUT[dW.dtype] if need_dw else 0,
                             _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "mx_linear_bwd")
    return dX, dW


def _bwd_opts(wgrad_hadamard, wgrad_dy_rounding, seed, stream_id):
    return _CBwdOpts(int(bool(wgrad_hadamard)), ROUNDING[wgrad_dy_rounding], seed, stream_id, 0)


def linear_fwd_save(X: torch.Tensor, W: torch.Tensor, fmt: str, out_dtype=torch.bfloat16,
                    wgrad_hadamard: bool = False, wgrad_dy_rounding: str = "rne", seed: int = 0,
                    stream_id: int = 0, x_amax: torch.Tensor | None = None, w_amax: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, saved: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, stream=None):
    """Y = X W^T plus the layer's saved backward state (one read each of X and W).
    Returns (Y, saved); pass `saved` and the same backward options to linear_bwd_saved."""
    _on_gpu(X, W, x_amax, w_amax, workspace, saved, out)
    T, Kin = X.shape
    Nout = W.shape[0]
    ws = workspace if workspace is not None else torch.empty(workspace_bytes(T, Kin, Nout, fmt, "fwd"),
                                                             dtype=torch.uint8, device=X.device)
    sv = saved if saved is not None else torch.empty(saved_bytes(T, Kin, Nout, fmt), dtype=torch.uint8,
                                                     device=X.device)
    Y = out if out is not None else torch.empty((T, Nout), dtype=out_dtype, device=X.device)
    o = _bwd_opts(wgrad_hadamard, wgrad_dy_rounding, seed, stream_id)
    rc = lib().mx_linear_fwd_save(_ptr(X), _ptr(W), T, Kin, Nout, FORMATS[fmt], _ptr(x_amax), _ptr(w_amax),
                                  C.byref(o), _ptr(Y), OUT[Y.dtype], _ptr(ws), ws.numel(), _ptr(sv), sv.numel(),
                                  _stream(stream))
    _check(rc, "mx_linear_fwd_save")
    return Y, sv


def linear_bwd_saved(dY: torch.Tensor, saved: torch.Tensor, Kin: int, fmt: str,
                     wgrad_hadamard: bool = False, wgrad_dy_rounding: str = "rne", seed: int = 0,
                     stream_id: int = 0, dy_amax: torch.Tensor | None = None, dx_dtype=torch.bfloat16,
                     dw_dtype=torch.float32, need_dx: bool = True, need_dw: bool = True,
                     workspace: torch.Tensor | None = None, dX: torch.Tensor | None = None,
                     dW: torch.Tensor | None = None, stream=None):
    """dX = dY W and dW = dY^T X from the state linear_fwd_save kept (one read of dY)."""
    _on_gpu(dY, saved, dy_amax, workspace, dX, dW)
    T, Nout = dY.shape
    ws = workspace if workspace is not None else torch.empty(workspace_bytes(T, Kin, Nout, fmt, "bwd_saved"),
                                                             dtype=torch.uint8, device=dY.device)
    if need_dx and dX is None:
        dX = torch.empty((T, Kin), dtype=dx_dtype, device=dY.device)
    if need_dw and dW is None:
        dW = torch.empty((Nout, Kin), dtype=dw_dtype, device=dY.device)
    o = _bwd_opts(wgrad_hadamard, wgrad_dy_rounding, seed, stream_id)
    rc = lib().mx_linear_bwd_saved(_ptr(dY), T, Kin, Nout, FORMATS[fmt], _ptr(dy_amax), C.byref(o), _ptr(saved),
                                   saved.numel(), _ptr(dX) if need_dx else None, OUT[dX.dtype] if need_dx else 0,
                                   _ptr(dW) if need_dw else None, OUT[dW.dtype] if need_dw else 0,
                                   _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "mx_linear_bwd_saved")
    return dX, dW


# ---------------------------------------------------------------- norm, activation, 8-bit checkpoints
def _cuda_calls(c):
    """(() -> the current device's index, (device index) -> cudaStream_t of its current
    stream) by torch's own short cuts in module c, or in public calls where it has none:
    those need CUDA only when they are made, so a torch without it can import this."""
    return (getattr(c, "_cuda_getDevice", torch.cuda.current_device),
            getattr(c, "_cuda_getCurrentRawStream", lambda index: torch.cuda.current_stream(index).cuda_stream))


_device_index, _raw_stream = _cuda_calls(torch._C)
_U8, _F32 = torch.uint8, torch.float32

NORMS = {"layer": 0, "rms": 1}
ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}


class Act8:
    """An 8-bit checkpoint of a matrix [rows, cols] (G = ceil(cols / 32)): E4M3
    codes uint8 [rows, 32 G] and exponent bytes uint8 [rows, G]; a value stands
    for code * 2^(byte - 127).  Made by act8_save, norm_fwd and act_fwd."""

    __slots__ = ("codes", "sf", "cols")

    def __init__(self, codes: torch.Tensor, sf: torch.Tensor, cols: int):
        self.codes, self.sf, self.cols = codes, sf, cols

    @staticmethod
    def empty(rows: int, cols: int, device=None) -> "Act8":
        device = device or torch.device("cuda")
        G = -(-cols // 32)
        return Act8(torch.empty((rows, 32 * G), dtype=torch.uint8, device=device),
                    torch.empty((rows, G), dtype=torch.uint8, device=device), cols)

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    def _c(self, dev, rows=None, cols=None) -> _CAct8:
        c, f = self.codes, self.sf
        n, G = c.shape[0], -(-self.cols // 32)
        if (c.dtype is not torch.uint8 or f.dtype is not torch.uint8 or c.shape != (n, 32 * G) or f.shape != (n, G)
                or not c.is_contiguous() or not f.is_contiguous()):
            raise MXError(MX_ERR_INVALID_ARG, "a checkpoint holds contiguous uint8 codes [rows, 32 G] and sf [rows, G]")
        if c.device != dev or f.device != dev:
            raise MXError(MX_ERR_INVALID_ARG, f"checkpoint on {c.device}, expected {dev}")
        if rows is not None and (n != rows or self.cols != cols):
            raise MXError(MX_ERR_INVALID_ARG, f"checkpoint of [{n}, {self.cols}], expected [{rows}, {cols}]")
        return _CAct8(c.data_ptr(), f.data_ptr(), n, self.cols)


class NormOut(NamedTuple):
    """norm_fwd's results: y; sum (the residual stream after the addition, or x
    itself); mean and rstd [rows] (None where not asked for; rms has no mean);
    saved (the checkpoint of sum, or None)."""
    y: torch.Tensor
    sum: torch.Tensor
    mean: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]
    saved: Optional[Act8]


class ActOut(NamedTuple):
    """act_fwd's results: h and the checkpoints of gate and up (or None)."""
    h: torch.Tensor
    gate: Optional[Act8]
    up: Optional[Act8]


def _first(t, what):
    """(pointer, row stride, rows, columns, device, type) of the matrix that a call goes by."""
    if not t.is_cuda:
        _on_gpu(t)
    if t.dim() != 2:
        raise MXError(MX_ERR_INVALID_ARG, f"{what} must be a matrix, not of shape {tuple(t.shape)}")
    dt = t.dtype
    if dt not in OUT:
        raise MXError(MX_ERR_INVALID_ARG, f"{what} has type {dt}, expected bfloat16 or float32")
    rows, cols = t.shape
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise MXError(MX_ERR_INVALID_ARG, f"{what} must have unit column stride")
    return t.data_ptr(), ld if rows > 1 else cols, rows, cols, t.device, dt


def _mat(t, rows, cols, dev, what, dtype=None):
    """(pointer, row stride) of a matrix after checking it."""
    if t.shape != (rows, cols):
        raise MXError(MX_ERR_INVALID_ARG, f"{what} has shape {tuple(t.shape)}, expected ({rows}, {cols})")
    dt = t.dtype
    if dt is not dtype and (dtype is not None or dt not in OUT):
        raise MXError(MX_ERR_INVALID_ARG, f"{what} has type {dt}, expected {dtype or 'bfloat16 or float32'}")
    if t.device != dev:
        raise MXError(MX_ERR_INVALID_ARG, f"{what} is on {t.device}, expected {dev}")
    ld, unit = t.stride()
    if unit != 1 and cols > 1:
        raise MXError(MX_ERR_INVALID_ARG, f"{what} must have unit column stride")
    return t.data_ptr(), ld if rows > 1 else cols


def _save_to(out, rows, cols, dev):
    """(checkpoint, its C form): a new one, or the one given after checking it."""
    if isinstance(out, Act8):
        return out, out._c(dev, rows, cols)
    G = (cols + 31) >> 5
    codes = torch.empty((rows, 32 * G), dtype=_U8, device=dev)
    sf = torch.empty((rows, G), dtype=_U8, device=dev)
    return Act8(codes, sf, cols), _CAct8(codes.data_ptr(), sf.data_ptr(), rows, cols)


def _vec(t, n, dev, what, dtype=torch.float32):
    """Pointer of a contiguous vector of n elements (None: absent)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != n or t.device != dev or not t.is_contiguous():
        raise MXError(MX_ERR_INVALID_ARG, f"{what} must be {n} contiguous {dtype} values on {dev}")
    return t.data_ptr()


def _params(weight, bias, cols, dev):
    """(weight pointer, bias pointer, their type's number)."""
    first = weight if weight is not None else bias
    if first is None:
        return None, None, 0
    if first.dtype not in OUT:
        raise MXError(MX_ERR_INVALID_ARG, f"weight and bias are bfloat16 or float32, not {first.dtype}")
    return (_vec(weight, cols, dev, "weight", first.dtype), _vec(bias, cols, dev, "bias", first.dtype),
            OUT[first.dtype])


def _run(dev, what, fn, *args):
    """One call of the library on the tensors' device and its current stream."""
    index = dev.index
    if index != _device_index():
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(index))
    else:
        rc = fn(*args, _raw_stream(index))
    if rc != MX_OK:
        raise MXError(rc, what)


def _look_up(table, key, what):
    if key not in table:
        raise MXError(MX_ERR_INVALID_ARG, f"{what} {key!r} is none of {', '.join(map(str, table))}")
    return table[key]


def act8_save(x: torch.Tensor, out: Act8 | None = None, stream=None) -> Act8:
    """The 8-bit checkpoint of a bf16 or fp32 matrix."""
    if stream is not None:  # also what is allocated here then belongs to that stream
        with torch.cuda.stream(stream):
            return act8_save(x, out)
    px, ldx, rows, cols, dev, dt = _first(x, "x")
    out, c = _save_to(out, rows, cols, dev)
    _run(dev, "mx_act8_save", lib().mx_act8_save, px, ldx, OUT[dt], c)
    return out


def act8_restore(a: Act8, out_dtype=torch.bfloat16, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values a checkpoint stands for, [rows, cols]."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return act8_restore(a, out_dtype, out)
    if not a.codes.is_cuda:
        _on_gpu(a.codes)
    rows, cols, dev = a.codes.shape[0], a.cols, a.codes.device
    c = a._c(dev)
    if out is None:
        number = _look_up(OUT, out_dtype, "out_dtype")
        out = torch.empty((rows, cols), dtype=out_dtype, device=dev)
        po, ldo = out.data_ptr(), cols
    else:
        po, ldo = _mat(out, rows, cols, dev, "out")
        number = OUT[out.dtype]
    _run(dev, "mx_act8_restore", lib().mx_act8_restore, c, po, ldo, number)
    return out


def norm_fwd(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
             kind: str = "layer", eps: float = 1e-5, residual: torch.Tensor | None = None,
             sum_out: torch.Tensor | None = None, save: bool | Act8 = False, amax_out: torch.Tensor | None = None,
             out_dtype=None, out: torch.Tensor | None = None, need_stats: bool = True,
             mean: torch.Tensor | None = None, rstd: torch.Tensor | None = None, stream=None) -> NormOut:
    """Layer norm (or RMS norm) of the rows of x [rows, cols], or of x +
    residual: y = (s - mean) * rstd * weight + bias.  sum_out may be x or
    residual itself.  save: True, or an Act8 to fill, keeps the 8-bit checkpoint
    of s for norm_bwd.  amax_out: one fp32 word that receives max |y|."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return norm_fwd(x, weight, bias, kind, eps, residual, sum_out, save, amax_out, out_dtype, out, need_stats,
                            mean, rstd)
    px, ldx, rows, cols, dev, dt = _first(x, "x")
    k = _look_up(NORMS, kind, "kind")
    pr = ps = pm = pt = saved = csaved = None
    ldr = lds = 0
    if residual is not None:
        pr, ldr = _mat(residual, rows, cols, dev, "residual", dt)
        if sum_out is None:
            sum_out = torch.empty((rows, cols), dtype=dt, device=dev)
            ps, lds = sum_out.data_ptr(), cols
        else:
            ps, lds = _mat(sum_out, rows, cols, dev, "sum_out", dt)
    elif sum_out is not None:
        raise MXError(MX_ERR_INVALID_ARG, "sum_out goes with residual")
    pw, pb, wt = _params(weight, bias, cols, dev)
    if out is None:
        ydt = out_dtype or dt
        yt = _look_up(OUT, ydt, "out_dtype")
        out = torch.empty((rows, cols), dtype=ydt, device=dev)
        py, ldy = out.data_ptr(), cols
    else:
        py, ldy = _mat(out, rows, cols, dev, "out")
        yt = OUT[out.dtype]
    if need_stats:
        if rstd is None:
            rstd = torch.empty(rows, dtype=_F32, device=dev)
        if mean is None and k == 0:
            mean = torch.empty(rows, dtype=_F32, device=dev)
    if rstd is not None:
        pt = _vec(rstd, rows, dev, "rstd")
    if k != 0:
        mean = None
    elif mean is not None:
        pm = _vec(mean, rows, dev, "mean")
    if save is not False and save is not None:
        saved, csaved = _save_to(save, rows, cols, dev)
    _run(dev, "mx_norm_fwd", lib().mx_norm_fwd, px, ldx, pr, ldr, OUT[dt], rows, cols, k, pw, pb, wt, eps, ps, lds,
         py, ldy, yt, pm, pt, csaved, _vec(amax_out, 1, dev, "amax_out") if amax_out is not None else None)
    return NormOut(out, sum_out if residual is not None else x, mean, rstd, saved)


def norm_bwd_workspace_bytes(rows: int, cols: int) -> int:
    return int(lib().mx_norm_bwd_workspace_bytes(rows, cols))


def norm_bwd(dy: torch.Tensor, x: torch.Tensor | Act8, rstd: torch.Tensor, mean: torch.Tensor | None = None,
             weight: torch.Tensor | None = None, kind: str = "layer", dres: torch.Tensor | None = None,
             need_dw: bool = True, need_db: bool | None = None, dx_dtype=None, dx: torch.Tensor | None = None,
             dw: torch.Tensor | None = None, db: torch.Tensor | None = None, amax_out: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None, stream=None):
    """(dx, dw, db) of norm_fwd.  x: the forward's sum, or its checkpoint.  dres:
    the gradient that reaches the residual stream past the norm, added to dx.
    need_db defaults to the kind's use of a bias (layer: True, rms: False);
    dw and db are fp32 (None where not asked for)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return norm_bwd(dy, x, rstd, mean, weight, kind, dres, need_dw, need_db, dx_dtype, dx, dw, db, amax_out,
                            workspace)
    pdy, lddy, rows, cols, dev, ydt = _first(dy, "dy")
    k = _look_up(NORMS, kind, "kind")
    px = x8 = pres = pm = pdw = pdb = pws = None
    ldx = ldres = n = 0
    if isinstance(x, Act8):
        x8 = x._c(dev, rows, cols)
        dt = dx.dtype if dx is not None else dx_dtype or (dres.dtype if dres is not None else ydt)
    else:
        dt = x.dtype
        px, ldx = _mat(x, rows, cols, dev, "x")
        if dx_dtype is not None and dx_dtype is not dt:
            raise MXError(MX_ERR_UNSUPPORTED, "dx has the type of x")
    number = _look_up(OUT, dt, "dx's type")
    if dx is None:
        dx = torch.empty((rows, cols), dtype=dt, device=dev)
        pdx, lddx = dx.data_ptr(), cols
    else:
        pdx, lddx = _mat(dx, rows, cols, dev, "dx", dt)
    if dres is not None:
        pres, ldres = _mat(dres, rows, cols, dev, "dres", dt)
    if rstd is None or (k == 0 and mean is None):
        raise MXError(MX_ERR_INVALID_ARG, "norm_bwd needs the forward's rstd, and its mean for a layer norm")
    if k == 0:
        pm = _vec(mean, rows, dev, "mean")
    pw, _, wt = _params(weight, None, cols, dev)
    if need_db is None:
        need_db = k == 0
    L = lib()
    if need_dw or need_db:
        if need_dw:
            if dw is None:
                dw = torch.empty(cols, dtype=_F32, device=dev)
            pdw = _vec(dw, cols, dev, "dw")
        if need_db:
            if db is None:
                db = torch.empty(cols, dtype=_F32, device=dev)
            pdb = _vec(db, cols, dev, "db")
        if workspace is None:
            n = L.mx_norm_bwd_workspace_bytes(rows, cols)
            workspace = torch.empty(n, dtype=_U8, device=dev)
        elif workspace.device != dev or not workspace.is_contiguous():
            raise MXError(MX_ERR_INVALID_ARG, f"workspace must be contiguous memory on {dev}")
        else:
            n = workspace.numel() * workspace.element_size()
        pws = workspace.data_ptr() if n else None
    _run(dev, "mx_norm_bwd", L.mx_norm_bwd, pdy, lddy, OUT[ydt], px, ldx, x8, pm, _vec(rstd, rows, dev, "rstd"), pw, wt,
         rows, cols, k, pres, ldres, pdx, lddx, number, pdw, pdb,
         _vec(amax_out, 1, dev, "amax_out") if amax_out is not None else None, pws, n)
    return dx, dw if need_dw else None, db if need_db else None


def act_fwd(gate: torch.Tensor, up: torch.Tensor | None = None, act: str = "silu", save: bool = False,
            gate8: Act8 | None = None, up8: Act8 | None = None, amax_out: torch.Tensor | None = None,
            out: torch.Tensor | None = None, stream=None) -> ActOut:
    """h = act(gate) * up, or act(gate) without up; gate and up may be views of
    the halves of one projection's output.  save (or gate8 / up8 to fill) keeps
    the 8-bit checkpoints that act_bwd reads.  amax_out: one fp32 word that
    receives max |h|."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return act_fwd(gate, up, act, save, gate8, up8, amax_out, out)
    pg, ldg, rows, cols, dev, dt = _first(gate, "gate")
    pu = c8 = cu8 = None
    ldu = 0
    if up is not None:
        pu, ldu = _mat(up, rows, cols, dev, "up", dt)
    if out is None:
        out = torch.empty((rows, cols), dtype=dt, device=dev)
        ph, ldh = out.data_ptr(), cols
    else:
        ph, ldh = _mat(out, rows, cols, dev, "out", dt)
    if save or gate8 is not None:
        gate8, c8 = _save_to(gate8, rows, cols, dev)
    if up8 is not None or (save and up is not None):
        up8, cu8 = _save_to(up8, rows, cols, dev)
    _run(dev, "mx_act_fwd", lib().mx_act_fwd, pg, ldg, pu, ldu, rows, cols, _look_up(ACTS, act, "act"), OUT[dt], ph, ldh,
         c8, cu8, _vec(amax_out, 1, dev, "amax_out") if amax_out is not None else None)
    return ActOut(out, gate8, up8)


def act_bwd(dh: torch.Tensor, gate: torch.Tensor | Act8, up: torch.Tensor | Act8 | None = None, act: str = "silu",
            amax_out: torch.Tensor | None = None, dgate: torch.Tensor | None = None,
            dup: torch.Tensor | None = None, stream=None):
    """(dgate, dup) of act_fwd from dh and its inputs, both kept or both as
    checkpoints (dup is None without up).  Without buffers given, dgate and dup
    are the halves of one [rows, 2 cols] tensor, as the projection's backward
    pass takes them.  amax_out: max over both."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return act_bwd(dh, gate, up, act, amax_out, dgate, dup)
    pdh, ldh, rows, cols, dev, dt = _first(dh, "dh")
    gated = up is not None
    pg = pu = g8 = u8 = None
    ldg = ldu = lddu = 0
    if isinstance(gate, Act8):
        g8 = gate._c(dev, rows, cols)
        if gated:
            if not isinstance(up, Act8):
                raise MXError(MX_ERR_INVALID_ARG, "gate and up are both kept or both checkpoints")
            u8 = up._c(dev, rows, cols)
    else:
        pg, ldg = _mat(gate, rows, cols, dev, "gate", dt)
        if gated:
            if isinstance(up, Act8):
                raise MXError(MX_ERR_INVALID_ARG, "gate and up are both kept or both checkpoints")
            pu, ldu = _mat(up, rows, cols, dev, "up", dt)
    pdu = None
    if dgate is None and dup is None and gated:
        both = torch.empty((rows, 2 * cols), dtype=dt, device=dev)
        dgate, dup = both[:, :cols], both[:, cols:]
        pdg = both.data_ptr()
        pdu = pdg + cols * both.element_size()
        lddg = lddu = 2 * cols
    else:
        if dgate is None:
            dgate = torch.empty((rows, cols), dtype=dt, device=dev)
        pdg, lddg = _mat(dgate, rows, cols, dev, "dgate", dt)
        if gated:
            dup = dup if dup is not None else torch.empty((rows, cols), dtype=dt, device=dev)
            pdu, lddu = _mat(dup, rows, cols, dev, "dup", dt)
        elif dup is not None:
            raise MXError(MX_ERR_INVALID_ARG, "dup goes with up")
    _run(dev, "mx_act_bwd", lib().mx_act_bwd, pdh, ldh, pg, ldg, pu, ldu, g8, u8, rows, cols,
         _look_up(ACTS, act, "act"), OUT[dt], pdg, lddg, pdu, lddu,
         _vec(amax_out, 1, dev, "amax_out") if amax_out is not None else None)
    return dgate, dup


# ---------------------------------------------------------------- gated feed-forward block
class GatedOut(NamedTuple):
    """gated_fwd_save's results: h; saved (the X^T and W^T operands) and the
    checkpoints of both projections' outputs, which gated_bwd reads."""
    h: torch.Tensor
    saved: torch.Tensor
    gate: Act8
    up: Act8


_BF16 = torch.bfloat16
_GATED_PASSES = {"fwd": 0, "bwd": 1, "fwd_quantized": 2}


def gated_workspace_bytes(T: int, Kin: int, F: int, fmt: str, pass_: str = "fwd") -> int:
    """Workspace of gated_fwd from W and gated_fwd_save ("fwd"), gated_bwd ("bwd") and
    gated_fwd from quantized weights ("fwd_quantized").  One for T tokens serves fewer, but
    for up to 64 tokens in one for more than 64: there, the larger of the sizes for 64 and T."""
    return int(lib().mx_gated_workspace_bytes(T, Kin, F, _look_up(FORMATS, fmt, "fmt"),
                                              _look_up(_GATED_PASSES, pass_, "pass_")))


def _memory(t, n, dev, what):
    """(tensor, pointer, bytes) of a buffer of at least n bytes: a new one, or the one given."""
    if t is None:
        t = torch.empty(n, dtype=_U8, device=dev)
    elif t.device != dev or not t.is_contiguous():
        raise MXError(MX_ERR_INVALID_ARG, f"{what} must be contiguous memory on {dev}")
    return t, t.data_ptr(), t.numel() * t.element_size()


def _bf16_rows(t, what):
    px, ld, rows, cols, dev, dt = _first(t, what)
    if dt is not _BF16:
        raise MXError(MX_ERR_INVALID_ARG, f"{what} has type {dt}, expected bfloat16")
    return px, ld, rows, cols, dev


def _gate_up(W, cols, dev):
    """(pointer of W [2 F, cols], F)."""
    if W.dim() != 2 or W.shape[0] % 2 or W.shape[1] != cols:
        raise MXError(MX_ERR_INVALID_ARG, f"W has shape {tuple(W.shape)}, expected (2 F, {cols})")
    if W.dtype is not _BF16 or W.device != dev or not W.is_contiguous():
        raise MXError(MX_ERR_INVALID_ARG, f"W must be contiguous bfloat16 on {dev}")
    return W.data_ptr(), W.shape[0] // 2


def _operand(q, fmt, cols, dev, what):
    if not isinstance(q, MXTensor) or q.fmt != fmt or q.k != cols or q.codes.device != dev:
        raise MXError(MX_ERR_INVALID_ARG, f"{what} must be an MXTensor of {fmt} with k = {cols} on {dev}")
    if not (q.sf.is_cuda and q.scalars.is_cuda):
        _on_gpu(q.sf, q.scalars)
    top = q.scalars.data_ptr()
    return _CTensor(q.codes.data_ptr(), q.sf.data_ptr(), top, top + 4 * q.nscale, q.rows, cols, FORMATS[fmt], q.block,
                    int(q.hadamard), 0)


def gated_weights(W: torch.Tensor, fmt: str, stream=None):
    """(gate, up): the two halves of W [2 F, Kin] (gate rows first) quantized once, for
    gated_fwd, under one tensor scale where the format has one."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gated_weights(W, fmt)
    _look_up(FORMATS, fmt, "fmt")
    if not W.is_cuda:
        _on_gpu(W)
    if W.dim() != 2:
        raise MXError(MX_ERR_INVALID_ARG, f"W must be a matrix, not of shape {tuple(W.shape)}")
    _, F = _gate_up(W, W.shape[1], W.device)
    with torch.cuda.device(W.device):
        top = amax(W) if fmt in ("nvfp4", "moss") else None
        return quantize(W[:F], fmt, amax_in=top), quantize(W[F:], fmt, amax_in=top)


def gemm_gated(a: MXTensor, gate: MXTensor, up: MXTensor, act: str = "silu", save: bool = False,
               amax_out: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> ActOut:
    """h = act(dq(a) dq(gate)^T) * (dq(a) dq(up)^T) in bfloat16, one kernel.  save keeps
    the 8-bit checkpoints of both products; amax_out: one fp32 word, max |h|."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gemm_gated(a, gate, up, act, save, amax_out, out)
    dev = a.codes.device
    ca, cg, cu = a._c(), _operand(gate, a.fmt, a.k, dev, "gate"), _operand(up, a.fmt, a.k, dev, "up")
    rows, F = a.rows, gate.rows
    if out is None:
        out = torch.empty((rows, -(-F // 8) * 8), dtype=_BF16, device=dev)[:, :F]
    ph, ldh = _mat(out, rows, F, dev, "out", _BF16)
    g8, c8 = _save_to(None, rows, F, dev) if save else (None, None)
    u8, cu8 = _save_to(None, rows, F, dev) if save else (None, None)
    _run(dev, "mx_gemm_gated", lib().mx_gemm_gated, ca, cg, cu, _look_up(ACTS, act, "act"), ph, -(-ldh // 8) * 8 if rows <= 1 else ldh,
         c8, cu8, _vec(amax_out, 1, dev, "amax_out") if amax_out is not None else None)
    return ActOut(out, g8, u8)


def gated_fwd(X: torch.Tensor, W, fmt: str, act: str = "silu", amax_out: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h [T, F] = act(X Wg^T) * (X Wu^T), X [T, Kin] bfloat16 quantized within the call.
    W: [2 F, Kin] bfloat16 (gate rows first), quantized within the call too, or
    gated_weights(W, fmt).  amax_out: one fp32 word, max |h| (the x_amax of the next
    linear).  The rows of h start at multiples of eight values."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gated_fwd(X, W, fmt, act, amax_out, workspace, out)
    px, ldx, T, Kin, dev = _bf16_rows(X, "X")
    number, kind = _look_up(FORMATS, fmt, "fmt"), _look_up(ACTS, act, "act")
    pw = cg = cu = None
    if isinstance(W, torch.Tensor):
        pw, F = _gate_up(W, Kin, dev)
    else:
        gate, up = W
        cg, cu = _operand(gate, fmt, Kin, dev, "gate"), _operand(up, fmt, Kin, dev, "up")
        F = gate.rows
    if out is None:
        out = torch.empty((T, -(-F // 8) * 8), dtype=_BF16, device=dev)
        if F % 8:
            out = out[:, :F]
    ph, ldh = _mat(out, T, F, dev, "out", _BF16)
    L = lib()
    workspace, pws, n = _memory(workspace, L.mx_gated_workspace_bytes(T, Kin, F, number, 2 if pw is None else 0), dev,
                                "workspace")
    _run(dev, "mx_gated_fwd", L.mx_gated_fwd, px, ldx, T, Kin, F, number, kind, pw, cg, cu, ph,
         -(-ldh // 8) * 8 if T <= 1 else ldh, _vec(amax_out, 1, dev, "amax_out") if amax_out is not None else None, pws, n)
    return out


def gated_fwd_save(X: torch.Tensor, W: torch.Tensor, fmt: str, act: str = "silu", wgrad_hadamard: bool = False,
                   wgrad_dy_rounding: str = "rne", seed: int = 0, stream_id: int = 0,
                   x_amax: torch.Tensor | None = None, w_amax: torch.Tensor | None = None,
                   amax_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   saved: torch.Tensor | None = None, gate8: Act8 | None = None, up8: Act8 | None = None,
                   out: torch.Tensor | None = None, stream=None) -> GatedOut:
    """gated_fwd from W [2 F, Kin], keeping what gated_bwd reads: the X^T and W^T
    operands (as linear_fwd_save does) and 8-bit checkpoints of both projections'
    outputs.  Pass the same backward options to gated_bwd."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gated_fwd_save(X, W, fmt, act, wgrad_hadamard, wgrad_dy_rounding, seed, stream_id, x_amax, w_amax,
                                  amax_out, workspace, saved, gate8, up8, out)
    px, ldx, T, Kin, dev = _bf16_rows(X, "X")
    number, kind = _look_up(FORMATS, fmt, "fmt"), _look_up(ACTS, act, "act")
    pw, F = _gate_up(W, Kin, dev)
    if out is None:
        out = torch.empty((T, F), dtype=_BF16, device=dev)
    ph, ldh = _mat(out, T, F, dev, "out", _BF16)
    L = lib()
    workspace, pws, n = _memory(workspace, L.mx_gated_workspace_bytes(T, Kin, F, number, 0), dev, "workspace")
    saved, psv, ns = _memory(saved, L.mx_linear_saved_bytes(T, Kin, 2 * F, number), dev, "saved")
    gate8, cg = _save_to(gate8, T, F, dev)
    up8, cu = _save_to(up8, T, F, dev)
    o = _CBwdOpts(int(bool(wgrad_hadamard)), _look_up(ROUNDING, wgrad_dy_rounding, "wgrad_dy_rounding"), seed, stream_id, 0)
    one = lambda t, what: _vec(t, 1, dev, what) if t is not None else None  # noqa: E731
    _run(dev, "mx_gated_fwd_save", L.mx_gated_fwd_save, px, ldx, pw, T, Kin, F, number, kind, one(x_amax, "x_amax"),
         one(w_amax, "w_amax"), o, ph, ldh, cg, cu, one(amax_out, "amax_out"), pws, n, psv, ns)
    return GatedOut(out, saved, gate8, up8)


def gated_bwd(dH: torch.Tensor, kept: GatedOut, Kin: int, fmt: str, act: str = "silu", wgrad_hadamard: bool = False,
              wgrad_dy_rounding: str = "rne", seed: int = 0, stream_id: int = 0, dx_dtype=torch.bfloat16,
              dw_dtype=torch.float32, need_dx: bool = True, need_dw: bool = True,
              workspace: torch.Tensor | None = None, dX: torch.Tensor | None = None,
              dW: torch.Tensor | None = None, stream=None):
    """(dX [T, Kin], dW [2 F, Kin]) of gated_fwd_save from dH [T, F] (bfloat16) and what
    it kept (kept.h is not read)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gated_bwd(dH, kept, Kin, fmt, act, wgrad_hadamard, wgrad_dy_rounding, seed, stream_id, dx_dtype, dw_dtype,
                             need_dx, need_dw, workspace, dX, dW)
    pd, ldd, T, F, dev = _bf16_rows(dH, "dH")
    number, kind = _look_up(FORMATS, fmt, "fmt"), _look_up(ACTS, act, "act")
    cg, cu = kept.gate._c(dev, T, F), kept.up._c(dev, T, F)
    pdx = pdw = None
    if need_dx:
        if dX is None:
            _look_up(OUT, dx_dtype, "dx_dtype")
            dX = torch.empty((T, Kin), dtype=dx_dtype, device=dev)
        pdx, ld = _mat(dX, T, Kin, dev, "dX")
        if ld != Kin:
            raise MXError(MX_ERR_INVALID_ARG, "dX must be contiguous")
    if need_dw:
        if dW is None:
            _look_up(OUT, dw_dtype, "dw_dtype")
            dW = torch.empty((2 * F, Kin), dtype=dw_dtype, device=dev)
        pdw, ld = _mat(dW, 2 * F, Kin, dev, "dW")
        if ld != Kin:
            raise MXError(MX_ERR_INVALID_ARG, "dW must be contiguous")
    L = lib()
    workspace, pws, n = _memory(workspace, L.mx_gated_workspace_bytes(T, Kin, F, number, 1), dev, "workspace")
    _, psv, ns = _memory(kept.saved, 0, dev, "saved")
    o = _CBwdOpts(int(bool(wgrad_hadamard)), _look_up(ROUNDING, wgrad_dy_rounding, "wgrad_dy_rounding"), seed, stream_id, 0)
    _run(dev, "mx_gated_bwd", L.mx_gated_bwd, pd, ldd, T, Kin, F, number, kind, cg, cu, o, psv, ns, pdx,
         OUT[dX.dtype] if need_dx else 0, pdw, OUT[dW.dtype] if need_dw else 0, pws, n)
    return (dX if need_dx else None), (dW if need_dw else None)


# ---------------------------------------------------------------- gradient norm and optimizer step
def _flat(t, what, dev=None):
    """(pointer, values, type's number) of one of many tensors after checking it."""
    if not t.is_cuda:
        _on_gpu(t)
    if t.dtype not in OUT:
        raise MXError(MX_ERR_INVALID_ARG, f"{what} has type {t.dtype}, expected bfloat16 or float32")
    if not t.is_contiguous():
        raise MXError(MX_ERR_INVALID_ARG, f"{what} must be contiguous")
    if dev is not None and t.device != dev:
        raise MXError(MX_ERR_INVALID_ARG, f"{what} is on {t.device}, expected {dev}")
    return t.data_ptr(), t.numel(), OUT[t.dtype]


_dtype_of = operator.attrgetter("dtype")


def _flats(ts, what, dev):
    """(pointers, sizes, types' numbers) of many tensors after checking them; by maps over
    torch's own methods, which for tens of tensors take a third of a loop's time."""
    try:
        if set(map(torch.Tensor.get_device, ts)) <= {dev.index} and all(map(torch.Tensor.is_contiguous, ts)):
            kinds = set(map(_dtype_of, ts))
            types = [OUT[kinds.pop()]] * len(ts) if len(kinds) == 1 else list(map(OUT.__getitem__, map(_dtype_of, ts)))
            return list(map(torch.Tensor.data_ptr, ts)), list(map(torch.Tensor.numel, ts)), types
    except (KeyError, TypeError):
        pass
    for t in ts:  # names what is wrong
        if not isinstance(t, torch.Tensor):
            raise MXError(MX_ERR_INVALID_ARG, f"{what} must be a tensor, not {type(t).__name__}")
        _flat(t, what, dev)
    raise MXError(MX_ERR_INVALID_ARG, f"{what} is not a plain tensor on {dev}")


def grad_norm(grads, max_norm: float | None = None, out: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """fp32 [norm, factor] of the gradients' values taken together, on the device:
    factor = min(1, max_norm / (norm + 1e-6)) (1 without max_norm), NaN when the
    norm is not finite.  out[1:] is what AdamW.step takes as grad_scale.  None
    among the gradients counts as zeros."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return grad_norm(grads, max_norm, out, workspace)
    given = [g for g in grads if g is not None]
    if not given and out is None:
        raise MXError(MX_ERR_INVALID_ARG, "grad_norm needs a gradient, or out")
    first = given[0] if given else out
    if not first.is_cuda:
        _on_gpu(first)
    dev, count = first.device, len(given)
    table = (_CGrad * count)()
    if count:
        pointers, sizes, types = _flats(given, "a gradient", dev)
        words = memoryview(table).cast("B").cast("q")
        words[0::3] = memoryview(array("q", pointers))
        words[1::3] = memoryview(array("q", sizes))
        words[2::3] = memoryview(array("q", types))  # the type in the low half, zero above
    L = lib()
    if out is None:
        out = torch.empty(2, dtype=_F32, device=dev)
        po = out.data_ptr()
    else:
        po = _vec(out, 2, dev, "out")
    if workspace is None:
        n = L.mx_grad_norm_workspace_bytes(count)
        workspace = torch.empty(n, dtype=_U8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise MXError(MX_ERR_INVALID_ARG, f"workspace must be contiguous memory on {dev}")
    else:
        n = workspace.numel() * workspace.element_size()
    _run(dev, "mx_grad_norm", L.mx_grad_norm, table, count, float("inf") if max_norm is None else max_norm, po,
         workspace.data_ptr(), n)
    return out


class AdamW:
    """AdamW over a list of tensors, one launch a step for those of a kind.

    params: contiguous bfloat16 or float32 tensors on one device, updated in place.
    weight_decay: one number, or one for each tensor.  state: "fp32", or "8bit"
    for moments in the checkpoints' format (m, and the root of v; 1.03 bytes each).
    copies: bfloat16 tensors (or None) beside float32 params, which a step fills
    with the rounded weights.  rounding: "rne", or "sr" for stochastic rounding of
    8-bit moments and of bfloat16 params by seed and step number.  Give 8-bit moments
    that train "sr": to nearest, which they have by default (with a warning), a root
    never falls and follows only gradients that move it by half a code, for a step
    moves it by 0.05 % with a beta2 of 0.999 and codes are 6 to 12 % apart.  capturable: the
    step number lives on the device, so that a step captured into a CUDA graph
    counts at each replay.

    m, v: the moments, one for each tensor (float32 views, or Act8 with one row;
    v holds roots there); m_all, v_all: the memory that holds them, each tensor's
    from the next multiple of 32 values.  t: the number of the last step (a step
    that a NaN grad_scale left without effect counts too).

    To save an optimizer keep m_all and v_all (with 8 bits their codes and sf) and
    t beside the params; to go on, make one over the same tensors with the same
    state, rounding and seed, copy the moments back into m_all and v_all, and set t.
    """

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.01,
                 state: str = "fp32", copies=None, rounding: str | None = None, seed: int = 0, capturable: bool = False):
        self.params = tuple(params)
        if not self.params:
            raise MXError(MX_ERR_INVALID_ARG, "AdamW needs a tensor")
        n = len(self.params)
        self.lr, self.betas, self.eps, self.seed = lr, tuple(betas), eps, int(seed)
        self.state = state
        bits = _look_up({"fp32": 32, "8bit": 8}, state, "state")
        self._rounding = _look_up(ROUNDING, "rne" if rounding is None else rounding, "rounding")
        if bits == 8 and rounding is None:
            warnings.warn("8-bit moments rounded to nearest: their roots follow only large gradients, and never fall; "
                          'give rounding="sr" (or "rne")', stacklevel=2)
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * n
        self.copies = tuple(copies) if copies is not None else (None,) * n
        if len(decay) != n or len(self.copies) != n:
            raise MXError(MX_ERR_INVALID_ARG, f"weight_decay and copies have one entry for each of the {n} tensors")
        self._t, self._t_dev = 0, None
        dev = self.device = self.params[0].device
        self._table = (_CAdamwTensor * n)()
        self._opts = _CAdamwOpts()
        groups = []
        for row, p, wd in zip(self._table, self.params, decay):
            row.param, row.n, row.p_dtype = _flat(p, "a parameter", dev)
            row.weight_decay, row.bits = wd, bits
            groups.append(-(-row.n // 32))
        G = sum(groups)
        if bits == 8:
            self.m_all, self.v_all = (Act8(torch.zeros((1, 32 * G), dtype=_U8, device=dev),
                                           torch.zeros((1, G), dtype=_U8, device=dev), 32 * G) for _ in range(2))
        else:
            self.m_all, self.v_all = (torch.zeros(32 * G, dtype=_F32, device=dev) for _ in range(2))
        self.m, self.v = [], []
        first = 0
        for row, p, g in zip(self._table, self.params, groups):
            for mine, everything, name in ((self.m, self.m_all, "m"), (self.v, self.v_all, "v")):
                if bits == 8:
                    a = Act8(everything.codes[:, 32 * first:32 * (first + g)], everything.sf[:, first:first + g], row.n)
                    setattr(row, name, a.codes.data_ptr())
                    setattr(row, name + "_sf", a.sf.data_ptr())
                else:
                    a = everything[32 * first:32 * first + row.n].view(p.shape)
                    setattr(row, name, a.data_ptr())
                mine.append(a)
            first += g
        if capturable:
            self._t_dev = torch.zeros(1, dtype=torch.int64, device=dev)
        self._sizes = [row.n for row in self._table]
        self._words = memoryview(self._table).cast("B").cast("q"), memoryview(self._table).cast("B").cast("i")
        self._check_written()

    def _number_is_free(self, what):
        """A number on the device is not read or set by the host while a graph is captured: the graph would hold it."""
        with torch.cuda.device(self.device):
            if torch.cuda.is_current_stream_capturing():
                raise MXError(MX_ERR_UNSUPPORTED, f"{what} while a graph is captured")

    @property
    def t(self) -> int:
        """The last step's number.  With capturable it is read from the device, behind what the current stream holds,
        and counts the replays of captured steps; setting it is ordered likewise."""
        if self._t_dev is None:
            return self._t
        self._number_is_free("the number is on the device and cannot be read")
        return int(self._t_dev)

    @t.setter
    def t(self, number):
        number = operator.index(number)
        if number < 0:
            raise MXError(MX_ERR_INVALID_ARG, "steps are numbered from 1")
        if self._t_dev is not None:
            self._number_is_free("the number cannot be set")
            self._t_dev.fill_(number)
        self._t = number

    def _check_written(self):
        """Takes the parameters' and copies' places; no two of what a step writes may share memory."""
        spans = []
        for row, p, c in zip(self._table, self.params, self.copies):
            at, n, dtype = _flat(p, "a parameter", self.device)
            if n != row.n or dtype != row.p_dtype:
                raise MXError(MX_ERR_INVALID_ARG, "a parameter changed its size or type")
            row.param = at
            spans.append((at, at + n * p.element_size()))
            row.copy = None
            if c is not None:
                if dtype != OUT[torch.float32]:
                    raise MXError(MX_ERR_UNSUPPORTED, "a copy goes with a float32 parameter")
                at, m, dtype = _flat(c, "a copy", self.device)
                if m != n or dtype != OUT[torch.bfloat16]:
                    raise MXError(MX_ERR_INVALID_ARG, "a copy is bfloat16 and has its parameter's size")
                row.copy = at
                spans.append((at, at + 2 * n))
        spans = sorted(s for s in spans if s[1] > s[0])
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise MXError(MX_ERR_INVALID_ARG, "parameters and copies must not share memory")
        self._written = self.params + tuple(c for c in self.copies if c is not None)
        self._where = list(map(torch.Tensor.data_ptr, self._written))

    def step(self, grads, grad_scale: torch.Tensor | None = None, amax_out: torch.Tensor | None = None, lr=None,
             t: int | None = None, stream=None) -> None:
        """One step.  grads: one for each tensor, with as many values in the same order, in
        memory that the step does not write (None: the tensor stays as it is).  grad_scale:
        one fp32 value on the device that multiplies them; NaN leaves every tensor as it is.  amax_out: fp32 [tensors], max |weight| of each
        copy (of the parameter without one), for its next quantization.  lr: a number,
        or one fp32 value on the device; the default is the optimizer's.  t: this
        step's number (from 1), in place of the count (with capturable, not while a
        graph is captured)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.step(grads, grad_scale, amax_out, lr, t)
        dev = self.device
        grads = list(grads)
        n = len(self.params)
        if len(grads) != n:
            raise MXError(MX_ERR_INVALID_ARG, f"{len(grads)} gradients for {n} tensors")
        if list(map(torch.Tensor.data_ptr, self._written)) != self._where:  # storage that was replaced
            self._check_written()
        given = [g for g in grads if g is not None]
        at = pointers, sizes, types = _flats(given, "a gradient", dev)
        if len(given) != n:  # a tensor without a gradient: no pointer
            where = iter(zip(*at))
            pointers, sizes, types = zip(*((0, m, 0) if g is None else next(where) for g, m in zip(grads, self._sizes)))
        if list(sizes) != self._sizes:
            raise MXError(MX_ERR_INVALID_ARG, "a gradient's size is not its tensor's")
        words, ints = self._words
        words[_CAdamwTensor.grad.offset // 8::C.sizeof(_CAdamwTensor) // 8] = memoryview(array("q", pointers))
        ints[_CAdamwTensor.g_dtype.offset // 4::C.sizeof(_CAdamwTensor) // 4] = memoryview(array("i", types))
        o = self._opts
        lr = self.lr if lr is None else lr
        o.lr_at = None
        if isinstance(lr, torch.Tensor):
            o.lr, o.lr_at = 0.0, _vec(lr, 1, dev, "lr")
        else:
            o.lr = lr
        o.beta1, o.beta2 = self.betas
        o.eps, o.seed, o.rounding = self.eps, self.seed, self._rounding
        count = self._t + 1 if t is None else int(t)
        if count < 1:
            raise MXError(MX_ERR_INVALID_ARG, "steps are numbered from 1")
        if self._t_dev is not None and t is not None:
            self._number_is_free("a step cannot be given its number")
        scale = _vec(grad_scale, 1, dev, "grad_scale") if grad_scale is not None else None
        top = _vec(amax_out, n, dev, "amax_out") if amax_out is not None else None
        if self._t_dev is not None:
            if t is None:
                self._t_dev.add_(1)
            else:
                before = self._t_dev.clone()
                self._t_dev.fill_(count)
            o.t_at = self._t_dev.data_ptr()
        o.t = count
        try:
            _run(dev, "mx_adamw_step", lib().mx_adamw_step, self._table, n, o, scale, top)
        except MXError:
            if self._t_dev is not None:
                if t is None:
                    self._t_dev.sub_(1)
                else:
                    self._t_dev.copy_(before)
            raise
        self._t = count


def last_device_status(stream=None) -> int:
    return int(lib().mx_last_device_status(_stream(stream)))


def selftest_bounded_wait(limit_ns: int, stream=None) -> int:
    return int(lib().mx_selftest_bounded_wait(int(limit_ns), _stream(stream)))


def launch_count() -> int:
    """Kernels the library has launched so far in this process."""
    return int(lib().mx_launch_count())


def debug_divide(v: torch.Tensor, d: torch.Tensor):
    """(fast, ieee) quotients of the quantizer's shared-divisor division."""
    _on_gpu(v, d)
    fast, ieee = torch.empty_like(v), torch.empty_like(v)
    _check(lib().mx_debug_divide(_ptr(v), _ptr(d), v.numel(), _ptr(fast), _ptr(ieee), _stream()),
           "mx_debug_divide")
    return fast, ieee


GEMM_VARIANTS = {"auto": 0, "cta_n128": 1, "cta_n256": 2, "pair": 3, "pair_ws": 4}


def set_gemm_variant(variant: str) -> None:
    """Force one GEMM kernel variant (tests and tuning); "auto" restores the default."""
    lib().mx_debug_set_gemm_variant(GEMM_VARIANTS[variant])


def last_gemm_variant() -> str:
    """The GEMM variant the most recent GEMM launch used (a GEMM_VARIANTS key)."""
    v = lib().mx_debug_last_gemm_variant()
    return {i: k for k, i in GEMM_VARIANTS.items()}.get(v, "none")
