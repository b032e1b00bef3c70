"""GB300-native block-scaled (MXFP8 / MXFP4 / NVFP4 / MOSS two-level FP8) linear layer.

A thin ctypes binding over ``libmx_gb300.so`` (C ABI in ``include/mx.h``).  This
module only marshals arguments: every step of quantize, GEMM and the linear
layer's passes runs in the library's CUDA kernels.  PyTorch supplies device
memory and streams.  There is no CPU fallback: without the built library (see
``build()``) or an sm_103 GPU every call raises ``MXError``.
"""
from __future__ import annotations

import ctypes as C
import os
import threading
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
