"""Python binding of libslope.so, the SLoPe 2:4 sparse linear layer for MI355X.

Argument marshalling only: every function below checks that its tensors are
contiguous device tensors, reads their shapes and dtypes, and calls the C ABI
function of the same name (declared in include/slope.h, slope_int8.h and slope_mx.h) on the
current HIP stream.  All computation happens in the library's HIP kernels; there is no
fallback.  If the shared library has not been built, every call raises.

Tensor conventions (see include/slope.h):
  dense matrices      torch.bfloat16, torch.float16 or torch.float32, row-major
  masks               torch.uint8, 1 = kept
  compressed values   [rows, cols/2], same dtype as the dense matrix
  compressed metadata [rows, ceil(cols/32)] torch.int32 holding the uint32 words
  adapter workspace   torch.uint8 (or any dtype) of slope_lowrank_workspace_bytes()
  wgrad workspace     torch.uint8 (or any dtype) of slope_wgrad_workspace_bytes()
  packed operands     torch.uint8 buffers of slope_packed_sparse_bytes() (sparse
                      tile chunks) or slope_packed_tokens_bytes() (token chunks)
"""
from __future__ import annotations

import array
import ctypes
import functools
import operator
import os
import struct

import torch

__all__ = [
    "SlopeError", "library", "library_path", "STATUS",
    "slope_version", "slope_compressed_sizes", "slope_lowrank_workspace_bytes",
    "slope_prune24", "slope_prune_nm", "slope_compress24", "slope_double_prune", "slope_spmm_fwd",
    "slope_spmm_bwd_dx", "slope_masked_wgrad", "slope_lowrank_add", "slope_wgrad_workspace_bytes",
    "slope_packed_tokens_bytes", "slope_pack_tokens", "slope_masked_wgrad_packed", "slope_wgrad_split_workspace_bytes",
    "slope_packed_sparse_bytes", "slope_pack_sparse", "slope_spmm_fwd_packed", "slope_spmm_bwd_dx_packed",
    "slope_spmm_fwd_packed_tokens", "slope_spmm_bwd_dx_packed_tokens",
    "slope_decode_workspace_bytes", "slope_spmm_fwd_decode", "slope_spmm_fwd_decode_noalloc",
    "DECODE_NOALLOC_SCRATCH_BYTES", "slope_lowrank_grads_workspace_bytes",
    "slope_lowrank_grads_packed", "slope_adamw", "slope_adamw_double_prune", "AdamWParams",
    "slope_double_prune_packed", "slope_adamw_double_prune_packed", "slope_prune_compress24", "EXPORTED_SYMBOLS",
    "slope_quantize_e4m3", "slope_packed_sparse_e4m3_bytes", "slope_pack_sparse_e4m3", "slope_spmm_e4m3_packed",
    "slope_rmsnorm", "slope_rmsnorm_bwd_workspace_bytes", "slope_rmsnorm_bwd", "slope_quantize_rows_i8",
    "slope_packed_sparse_i8_bytes", "slope_pack_sparse_i8", "slope_spmm_i8_packed", "slope_spmm_i8_decode",
    "I8_DECODE_MAX_TOKENS", "I8_MAX_COLS", "EXPORTED_SYMBOLS_INT8",
    "slope_adamw_multi", "slope_adamw8_double_prune_packed", "slope_adamw_moments", "slope_mxfp4_row_bytes", "slope_quantize_mxfp4", "slope_mxfp4_values",
    "slope_packed_sparse_mxfp4_bytes", "slope_pack_sparse_mxfp4",
    "slope_spmm_mxfp4_workspace_bytes", "slope_spmm_mxfp4_packed", "MX_BLOCK", "EXPORTED_SYMBOLS_MX",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libslope.so")

STATUS = {0: "SLOPE_OK", -1: "SLOPE_ERR_INVALID_ARG", -2: "SLOPE_ERR_SHAPE", -3: "SLOPE_ERR_ALIGN",
          -4: "SLOPE_ERR_WORKSPACE", -5: "SLOPE_ERR_HIP", -6: "SLOPE_ERR_UNSUPPORTED"}

_F32, _BF16, _F16 = 0, 1, 2
_i64, _vp, _i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
_P_I64 = ctypes.POINTER(ctypes.c_int64)


class AdamWParams(ctypes.Structure):
    """slope_adamw_params: hyper-parameters of one AdamW update (step counts from 1)."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64)]


_P_HP = ctypes.POINTER(AdamWParams)

# name -> (restype, argtypes)
_SIGS = {
    "slope_version": (ctypes.c_int, []),
    "slope_status_string": (ctypes.c_char_p, [_i32]),
    "slope_compressed_sizes": (_i32, [_i64, _i64, _P_I64, _P_I64]),
    "slope_lowrank_workspace_bytes": (_i32, [_i64, _i64, _i64, _i64, _P_I64]),
    "slope_prune24": (_i32, [_i32, _vp, _i64, _i64, _vp, _vp, _vp]),
    "slope_compress24": (_i32, [_i32, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp]),
    "slope_double_prune": (_i32, [_i32, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp]),
    "slope_spmm_fwd": (_i32, [_i32, _i32, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _vp]),
    "slope_spmm_bwd_dx": (_i32, [_i32, _i32, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _vp]),
    "slope_masked_wgrad": (_i32, [_i32, _i32, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _i32, _vp, _i64, _vp]),
    "slope_wgrad_workspace_bytes": (_i32, [_i64, _i64, _i64, _P_I64]),
    "slope_packed_tokens_bytes": (_i32, [_i64, _i64, _P_I64]),
    "slope_packed_sparse_bytes": (_i32, [_i64, _i64, _P_I64]),
    "slope_decode_workspace_bytes": (_i32, [_i64, _i64, _i64, _i64, _P_I64]),
    "slope_spmm_fwd_decode": (_i32, [_i32, _i32, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _vp,
                                     _vp]),
    "slope_spmm_fwd_decode_noalloc": (_i32, [_i32, _i32, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _vp,
                                             _vp]),
    "slope_pack_sparse": (_i32, [_i32, _vp, _vp, _i64, _i64, _vp, _i64, _vp]),
    "slope_spmm_fwd_packed": (_i32, [_i32, _i32, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _vp,
                                     _vp]),
    "slope_spmm_bwd_dx_packed": (_i32, [_i32, _i32, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _i64,
                                        _vp, _vp]),
    "slope_spmm_fwd_packed_tokens": (_i32, [_i32, _i32, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _vp,
                                            _i64, _vp, _vp, _i64, _vp]),
    "slope_spmm_bwd_dx_packed_tokens": (_i32, [_i32, _i32, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _vp,
                                               _i64, _vp, _vp, _i64, _vp]),
    "slope_lowrank_grads_workspace_bytes": (_i32, [_i64, _i64, _i64, _i64, _P_I64]),
    "slope_lowrank_grads_packed": (_i32, [_i32, _i32, _vp, _vp, _vp, _i64, _vp, _i64, _i64, _i64, _i64, _i64, _vp,
                                          _vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i32, _vp]),
    "slope_pack_tokens": (_i32, [_i32, _vp, _i64, _i64, _vp, _i64, _vp]),
    "slope_masked_wgrad_packed": (_i32, [_i32, _i32, _vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _i32,
                                         _vp, _i64, _vp]),
    "slope_wgrad_split_workspace_bytes": (_i32, [_i64, _i64, _i64, _P_I64]),
    "slope_lowrank_add": (_i32, [_i32, _i32, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _vp]),
    "slope_adamw": (_i32, [_i32, _i32, _vp, _vp, _vp, _vp, _i64, _P_HP, _vp]),
    "slope_adamw_double_prune": (_i32, [_i32, _i32, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _P_HP, _vp, _vp, _vp,
                                        _vp]),
    "slope_double_prune_packed": (_i32, [_i32, _vp, _vp, _i64, _i64, _vp, _i64, _vp]),
    "slope_prune_compress24": (_i32, [_i32, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _vp]),
    "slope_prune_nm": (_i32, [_i32, _vp, _i64, _i64, _i32, _i32, _vp, _vp, _vp]),
    "slope_adamw_double_prune_packed": (_i32, [_i32, _i32, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _P_HP, _vp, _i64,
                                               _vp, _i64, _vp]),
    "slope_quantize_e4m3": (_i32, [_i32, _vp, _i64, _vp, _vp, _vp]),
    "slope_packed_sparse_e4m3_bytes": (_i32, [_i64, _i64, _P_I64]),
    "slope_pack_sparse_e4m3": (_i32, [_i32, _vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp]),
    "slope_spmm_e4m3_packed": (_i32, [_i32, _vp, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp]),
}
EXPORTED_SYMBOLS = tuple(_SIGS)

# include/slope_int8.h
_f64 = ctypes.c_double
_SIGS_INT8 = {
    "slope_rmsnorm": (_i32, [_i32, _vp, _vp, _i32, _vp, _i64, _i64, _f64, _vp, _vp, _vp, _vp, _vp, _vp]),
    "slope_rmsnorm_bwd_workspace_bytes": (_i32, [_i64, _i64, _P_I64]),
    "slope_rmsnorm_bwd": (_i32, [_i32, _vp, _vp, _vp, _i32, _vp, _vp, _i64, _i64, _vp, _vp, _i32, _vp, _i64, _vp]),
    "slope_quantize_rows_i8": (_i32, [_i32, _vp, _i64, _i64, _vp, _vp, _vp]),
    "slope_packed_sparse_i8_bytes": (_i32, [_i64, _i64, _P_I64]),
    "slope_pack_sparse_i8": (_i32, [_i32, _vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp]),
    "slope_spmm_i8_packed": (_i32, [_i32, _vp, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp]),
    "slope_spmm_i8_decode": (_i32, [_i32, _vp, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp]),
}
EXPORTED_SYMBOLS_INT8 = tuple(_SIGS_INT8)

# include/slope_mx.h
_SIGS_MX = {
    "slope_adamw_multi": (_i32, [_i32, _i64, *[_vp] * 10, ctypes.c_uint64, _vp]),
    "slope_adamw8_double_prune_packed": (_i32, [_i32, _i32, *[_vp] * 7, _i64, _i64, _P_HP, ctypes.c_uint64, _vp, _i64,
                                                _vp, _i64, _vp]),
    "slope_adamw_moments": (_i32, [_i32, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp]),
    "slope_mxfp4_row_bytes": (_i32, [_i64, _P_I64, _P_I64]),
    "slope_quantize_mxfp4": (_i32, [_i32, _vp, _i64, _i64, _vp, _vp, _vp]),
    "slope_mxfp4_values": (_i32, [_i32, _vp, _vp, _i64, _i64, _vp, _vp]),
    "slope_packed_sparse_mxfp4_bytes": (_i32, [_i64, _i64, _P_I64]),
    "slope_pack_sparse_mxfp4": (_i32, [_i32, _vp, _vp, _i64, _i64, _vp, _i64, _vp]),
    "slope_spmm_mxfp4_workspace_bytes": (_i32, [_i64, _i64, _i64, _P_I64]),
    "slope_spmm_mxfp4_packed": (_i32, [_i32, _vp, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _vp]),
}
EXPORTED_SYMBOLS_MX = tuple(_SIGS_MX)

_lib = None


class SlopeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS.get(status, status)} ({_status_text(status)})")


def library() -> ctypes.CDLL:
    """The loaded libslope.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise RuntimeError(f"{library_path} is missing: build it first "
                               "(python -m sparse_gemm_02_amd.build); there is no fallback path")
        lib = ctypes.CDLL(library_path)
        for name, (res, args) in (*_SIGS.items(), *_SIGS_INT8.items(), *_SIGS_MX.items()):
            f = getattr(lib, name)
            f.restype, f.argtypes = res, args
        _lib = lib
    return _lib


def _status_text(status: int) -> str:
    try:
        return library().slope_status_string(status).decode()
    except Exception:  # pragma: no cover - library missing
        return "?"


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise SlopeError(fn, status)


def _dt(t) -> int:
    """Library dtype code of a tensor (or of a torch dtype)."""
    d = t if isinstance(t, torch.dtype) else t.dtype
    if d == torch.bfloat16:
        return _BF16
    if d == torch.float16:
        return _F16
    if d == torch.float32:
        return _F32
    raise TypeError(f"expected bfloat16, float16 or float32, got {d}")


def _p(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    if t.numel() and not t.is_cuda:
        raise ValueError("tensors must live in GPU memory")
    return t.data_ptr() if t.numel() else None


def _nn(t):
    """Pointer of a required tensor (a dummy non-null address for empty ones)."""
    p = _p(t)
    return p if p is not None else 256  # never dereferenced: the size is zero


def _adapter(L, R):
    """(L pointer, R pointer, r) of the adapter arguments.  Factors with no
    elements (K, N or r zero) make the adapter term zero and go as two NULLs; a
    single factor goes through as given, for the library to reject."""
    if L is None and R is None:
        return None, None, 0
    r = int(L.shape[1]) if L is not None else int(R.shape[0])
    if L is not None and R is not None and (L.numel() == 0 or R.numel() == 0):
        return None, None, r
    return _p(L), _p(R), r


def _nb(t):
    """Bytes of a buffer tensor (0 for None)."""
    return t.numel() * t.element_size() if t is not None else 0


def _s(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def slope_version() -> int:
    return library().slope_version()


def slope_compressed_sizes(rows: int, cols: int):
    nv, nm = ctypes.c_int64(), ctypes.c_int64()
    _check("slope_compressed_sizes", library().slope_compressed_sizes(rows, cols, ctypes.byref(nv), ctypes.byref(nm)))
    return nv.value, nm.value


def slope_lowrank_workspace_bytes(T: int, K: int, r: int, N: int) -> int:
    b = ctypes.c_int64()
    _check("slope_lowrank_workspace_bytes", library().slope_lowrank_workspace_bytes(T, K, r, N, ctypes.byref(b)))
    return b.value


def slope_prune24(W, mask, W_s=None, stream=None) -> None:
    rows, cols = W.shape
    _check("slope_prune24", library().slope_prune24(_dt(W), _nn(W), rows, cols, _nn(mask), _p(W_s), _s(stream)))


def slope_prune_nm(W, n, m, mask, W_s=None, stream=None) -> None:
    rows, cols = W.shape
    _check("slope_prune_nm", library().slope_prune_nm(_dt(W), _nn(W), rows, cols, n, m, _nn(mask), _p(W_s),
                                                      _s(stream)))


def slope_compress24(W, mask, values, meta, invalid=None, stream=None) -> None:
    rows, cols = W.shape
    _check("slope_compress24", library().slope_compress24(_dt(W), _nn(W), _nn(mask), rows, cols, _nn(values),
                                                          _nn(meta), _p(invalid), _s(stream)))


def slope_double_prune(values_s, meta_s, N, K, values_dpT, meta_dpT, mask_dpT=None, stream=None) -> None:
    _check("slope_double_prune", library().slope_double_prune(_dt(values_s), _nn(values_s), _nn(meta_s), N, K,
                                                              _nn(values_dpT), _nn(meta_dpT), _p(mask_dpT),
                                                              _s(stream)))


def slope_spmm_fwd(X, values_s, meta_s, N, Y, L=None, R=None, workspace=None, stream=None) -> None:
    T, K = X.shape
    pl, pr, r = _adapter(L, R)
    wb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("slope_spmm_fwd", library().slope_spmm_fwd(_dt(X), _dt(Y), _nn(X), T, K, _nn(values_s), _nn(meta_s), N,
                                                      pl, pr, r, _p(workspace), wb, _nn(Y), _s(stream)))


def slope_spmm_bwd_dx(dY, values_dpT, meta_dpT, K, dX, stream=None) -> None:
    T, N = dY.shape
    _check("slope_spmm_bwd_dx", library().slope_spmm_bwd_dx(_dt(dY), _dt(dX), _nn(dY), T, N, _nn(values_dpT),
                                                            _nn(meta_dpT), K, _nn(dX), _s(stream)))


def slope_wgrad_workspace_bytes(T: int, N: int, K: int) -> int:
    b = ctypes.c_int64()
    _check("slope_wgrad_workspace_bytes", library().slope_wgrad_workspace_bytes(T, N, K, ctypes.byref(b)))
    return b.value


def slope_masked_wgrad(dY, X, meta_s, dW_values, dW_dense=None, accumulate=False, workspace=None,
                       stream=None) -> None:
    T, N = dY.shape
    K = X.shape[1]
    wb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("slope_masked_wgrad", library().slope_masked_wgrad(_dt(dY), _dt(dW_values), _nn(dY), _nn(X), T, N, K,
                                                              _nn(meta_s), _nn(dW_values), _p(dW_dense),
                                                              int(bool(accumulate)), _p(workspace), wb,
                                                              _s(stream)))


def slope_packed_sparse_bytes(rows: int, cols: int) -> int:
    b = ctypes.c_int64()
    _check("slope_packed_sparse_bytes", library().slope_packed_sparse_bytes(rows, cols, ctypes.byref(b)))
    return b.value


def slope_pack_sparse(values, meta, rows, cols, packed, stream=None) -> None:
    nb = packed.numel() * packed.element_size()
    _check("slope_pack_sparse", library().slope_pack_sparse(_dt(values), _nn(values), _nn(meta), rows, cols,
                                                            _nn(packed), nb, _s(stream)))


def slope_spmm_fwd_packed(X, packed_s, N, Y, L=None, R=None, workspace=None, stream=None) -> None:
    T, K = X.shape
    pl, pr, r = _adapter(L, R)
    wb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("slope_spmm_fwd_packed", library().slope_spmm_fwd_packed(_dt(X), _dt(Y), _nn(X), T, K, _nn(packed_s),
                                                                    _nb(packed_s), N, pl, pr, r, _p(workspace),
                                                                    wb, _nn(Y), _s(stream)))


def slope_spmm_fwd_packed_tokens(X, packed_s, N, Y, X_packed, L=None, R=None, workspace=None, stream=None) -> None:
    T, K = X.shape
    pl, pr, r = _adapter(L, R)
    wb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("slope_spmm_fwd_packed_tokens",
           library().slope_spmm_fwd_packed_tokens(_dt(X), _dt(Y), _nn(X), T, K, _nn(packed_s), _nb(packed_s), N, pl,
                                                  pr, r, _p(workspace), wb, _nn(Y), _nn(X_packed), _nb(X_packed),
                                                  _s(stream)))


def slope_decode_workspace_bytes(T: int, K: int, r: int, N: int) -> int:
    b = ctypes.c_int64()
    _check("slope_decode_workspace_bytes", library().slope_decode_workspace_bytes(T, K, r, N, ctypes.byref(b)))
    return b.value


def slope_spmm_fwd_decode(X, packed_s, N, Y, workspace, L=None, R=None, stream=None) -> None:
    T, K = X.shape
    pl, pr, r = _adapter(L, R)
    wb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("slope_spmm_fwd_decode", library().slope_spmm_fwd_decode(_dt(X), _dt(Y), _nn(X), T, K, _nn(packed_s),
                                                                    _nb(packed_s), N, pl, pr, r, _p(workspace),
                                                                    wb, _nn(Y), _s(stream)))


DECODE_NOALLOC_SCRATCH_BYTES = 32 << 20   # SLOPE_DECODE_NOALLOC_SCRATCH_BYTES


def slope_spmm_fwd_decode_noalloc(X, packed_s, N, Y, L=None, R=None, stream=None) -> None:
    """slope_spmm_fwd_decode without a workspace: the library's static scratch."""
    T, K = X.shape
    pl, pr, r = _adapter(L, R)
    _check("slope_spmm_fwd_decode_noalloc", library().slope_spmm_fwd_decode_noalloc(
        _dt(X), _dt(Y), _nn(X), T, K, _nn(packed_s), _nb(packed_s), N, pl, pr, r, _nn(Y), _s(stream)))


def slope_spmm_bwd_dx_packed(dY, packed_dpT, K, dX, L=None, R=None, workspace=None, stream=None) -> None:
    T, N = dY.shape
    pl, pr, r = _adapter(L, R)
    wb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("slope_spmm_bwd_dx_packed", library().slope_spmm_bwd_dx_packed(_dt(dY), _dt(dX), _nn(dY), T, N,
                                                                          _nn(packed_dpT), _nb(packed_dpT), K, pl,
                                                                          pr, r, _p(workspace), wb, _nn(dX),
                                                                          _s(stream)))


def slope_spmm_bwd_dx_packed_tokens(dY, packed_dpT, K, dX, dY_packed, L=None, R=None, workspace=None,
                                    stream=None) -> None:
    T, N = dY.shape
    pl, pr, r = _adapter(L, R)
    wb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("slope_spmm_bwd_dx_packed_tokens",
           library().slope_spmm_bwd_dx_packed_tokens(_dt(dY), _dt(dX), _nn(dY), T, N, _nn(packed_dpT),
                                                     _nb(packed_dpT), K, pl, pr, r, _p(workspace), wb, _nn(dX),
                                                     _nn(dY_packed), _nb(dY_packed), _s(stream)))


def slope_lowrank_grads_workspace_bytes(T: int, K: int, r: int, N: int) -> int:
    b = ctypes.c_int64()
    _check("slope_lowrank_grads_workspace_bytes",
           library().slope_lowrank_grads_workspace_bytes(T, K, r, N, ctypes.byref(b)))
    return b.value


def slope_lowrank_grads_packed(X, dY, X_packed, dY_packed, L, R, workspace, dL, dR, accumulate=False,
                               fwd_workspace=None, bwd_workspace=None, stream=None) -> None:
    T, K = X.shape
    N = dY.shape[1]
    r = int(L.shape[1])
    wb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("slope_lowrank_grads_packed", library().slope_lowrank_grads_packed(
        _dt(X), _dt(dL), _nn(X), _nn(dY), _nn(X_packed), _nb(X_packed), _nn(dY_packed), _nb(dY_packed), T, K, r, N,
        _nn(L), _nn(R), _p(fwd_workspace), _nb(fwd_workspace), _p(bwd_workspace), _nb(bwd_workspace), _p(workspace),
        wb, _nn(dL), _nn(dR), int(bool(accumulate)), _s(stream)))


def slope_packed_tokens_bytes(T: int, C: int) -> int:
    b = ctypes.c_int64()
    _check("slope_packed_tokens_bytes", library().slope_packed_tokens_bytes(T, C, ctypes.byref(b)))
    return b.value


def slope_pack_tokens(M, packed, stream=None) -> None:
    T, C = M.shape
    nb = packed.numel() * packed.element_size()
    _check("slope_pack_tokens", library().slope_pack_tokens(_dt(M), _nn(M), T, C, _nn(packed), nb, _s(stream)))


def slope_wgrad_split_workspace_bytes(T: int, N: int, K: int) -> int:
    b = ctypes.c_int64()
    _check("slope_wgrad_split_workspace_bytes", library().slope_wgrad_split_workspace_bytes(T, N, K, ctypes.byref(b)))
    return b.value


def slope_masked_wgrad_packed(dY_packed, X_packed, T, N, K, meta_s, dW_values, dW_dense=None, accumulate=False,
                              stream=None, in_dtype=None, split_workspace=None) -> None:
    """in_dtype: torch dtype the packed operands hold (the chunks do not record
    it); defaults to dW_values' dtype when that is 16-bit, else bfloat16.
    split_workspace: optional buffer of slope_wgrad_split_workspace_bytes()."""
    if in_dtype is None:
        in_dtype = dW_values.dtype if dW_values.dtype in (torch.bfloat16, torch.float16) else torch.bfloat16
    _check("slope_masked_wgrad_packed", library().slope_masked_wgrad_packed(
        _dt(in_dtype), _dt(dW_values), _nn(dY_packed), _nb(dY_packed), _nn(X_packed), _nb(X_packed), T, N, K,
        _nn(meta_s), _nn(dW_values), _p(dW_dense), int(bool(accumulate)), _p(split_workspace), _nb(split_workspace),
        _s(stream)))


def slope_lowrank_add(X, L, R, workspace, Y, stream=None) -> None:
    T, K = X.shape
    r, N = R.shape
    wb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("slope_lowrank_add", library().slope_lowrank_add(_dt(X), _dt(Y), _nn(X), _nn(L), _nn(R), T, K, r, N,
                                                            _p(workspace), wb, _nn(Y), _s(stream)))


def _hp(step, lr, beta1, beta2, eps, weight_decay):
    return AdamWParams(float(lr), float(beta1), float(beta2), float(eps), float(weight_decay), int(step))


def _f32(t):
    if t.dtype != torch.float32:
        raise TypeError(f"optimizer moments must be float32, got {t.dtype}")
    return _nn(t)


def slope_adamw(params, grads, m, v, step, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01,
                stream=None) -> None:
    """One AdamW step on params (updated in place) with float32 moments m, v."""
    n = params.numel()
    if grads.numel() != n or m.numel() != n or v.numel() != n:
        raise ValueError("params, grads, m and v must have the same number of elements")
    hp = _hp(step, lr, beta1, beta2, eps, weight_decay)
    _check("slope_adamw", library().slope_adamw(_dt(params), _dt(grads), _nn(params), _nn(grads), _f32(m), _f32(v),
                                                n, ctypes.byref(hp), _s(stream)))


def slope_prune_compress24(W, values, meta, mask=None, packed=None, stream=None) -> None:
    """Magnitude 2:4 prune and compression of W [rows, cols] in one pass, with
    the mask and W_s's tile-chunk form as optional outputs."""
    rows, cols = W.shape
    nb = packed.numel() * packed.element_size() if packed is not None else 0
    _check("slope_prune_compress24", library().slope_prune_compress24(
        _dt(W), _nn(W), rows, cols, _p(mask), _nn(values), _nn(meta), _p(packed), nb, _s(stream)))


def slope_double_prune_packed(values_s, meta_s, N, K, packed_dpT, stream=None) -> None:
    """The double prune of W_s written straight to W_dp^T's tile-chunk form."""
    nb = packed_dpT.numel() * packed_dpT.element_size()
    _check("slope_double_prune_packed", library().slope_double_prune_packed(
        _dt(values_s), _nn(values_s), _nn(meta_s), N, K, _nn(packed_dpT), nb, _s(stream)))


def slope_adamw_double_prune_packed(values_s, meta_s, dW_values, m, v, N, K, packed_s, packed_dpT, step, lr,
                                    beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, stream=None) -> None:
    """AdamW on the compressed values of W_s (in place, and inside its tile
    chunks packed_s), then the double prune of the updated W_s into the tile
    chunks packed_dpT."""
    n = values_s.numel()
    if dW_values.numel() != n or m.numel() != n or v.numel() != n:
        raise ValueError("values_s, dW_values, m and v must have the same number of elements")
    hp = _hp(step, lr, beta1, beta2, eps, weight_decay)
    _check("slope_adamw_double_prune_packed", library().slope_adamw_double_prune_packed(
        _dt(values_s), _dt(dW_values), _nn(values_s), _nn(meta_s), _nn(dW_values), _f32(m), _f32(v), N, K,
        ctypes.byref(hp), _nn(packed_s), packed_s.numel() * packed_s.element_size(), _nn(packed_dpT),
        packed_dpT.numel() * packed_dpT.element_size(), _s(stream)))


def slope_adamw_double_prune(values_s, meta_s, dW_values, m, v, N, K, values_dpT, meta_dpT, step, lr, beta1=0.9,
                             beta2=0.999, eps=1e-8, weight_decay=0.01, mask_dpT=None, stream=None) -> None:
    """AdamW on the compressed values of W_s (in place), then the double prune of the updated W_s."""
    n = values_s.numel()
    if dW_values.numel() != n or m.numel() != n or v.numel() != n:
        raise ValueError("values_s, dW_values, m and v must have the same number of elements")
    hp = _hp(step, lr, beta1, beta2, eps, weight_decay)
    _check("slope_adamw_double_prune", library().slope_adamw_double_prune(
        _dt(values_s), _dt(dW_values), _nn(values_s), _nn(meta_s), _nn(dW_values), _f32(m), _f32(v), N, K,
        ctypes.byref(hp), _nn(values_dpT), _nn(meta_dpT), _p(mask_dpT), _s(stream)))



# ------------------------------------------------------------------ 8-bit (E4M3) variant
# Codes travel as torch.uint8 tensors; scales as one-element torch.float32 tensors.

def slope_quantize_e4m3(M, scale, q, stream=None) -> None:
    """scale[0] <- 448 / amax(|M|); q <- E4M3 codes of M * scale (same shape as M)."""
    if q.dtype != torch.uint8 or q.numel() != M.numel():
        raise ValueError("q must be a uint8 tensor with as many elements as M")
    if scale.dtype != torch.float32:
        raise TypeError("scale must be float32")
    _check("slope_quantize_e4m3", library().slope_quantize_e4m3(_dt(M), _nn(M), M.numel(), _nn(scale), _nn(q),
                                                                _s(stream)))


def slope_packed_sparse_e4m3_bytes(rows: int, cols: int) -> int:
    b = ctypes.c_int64()
    _check("slope_packed_sparse_e4m3_bytes", library().slope_packed_sparse_e4m3_bytes(rows, cols, ctypes.byref(b)))
    return b.value


def slope_pack_sparse_e4m3(values, meta, rows, cols, scale, packed, stream=None) -> None:
    """E4M3 tile chunks of a compressed 16-bit matrix, with its scale in scale[0]."""
    if scale.dtype != torch.float32:
        raise TypeError("scale must be float32")
    _check("slope_pack_sparse_e4m3", library().slope_pack_sparse_e4m3(_dt(values), _nn(values), _nn(meta), rows, cols,
                                                                      _nn(scale), _nn(packed), _nb(packed),
                                                                      _s(stream)))


def slope_spmm_e4m3_packed(Xq, x_scale, packed_w, w_scale, N, Y, stream=None) -> None:
    """Y [T, N] = (Xq . W_q^T) / (x_scale * w_scale) on E4M3 operands."""
    if Xq.dtype != torch.uint8:
        raise TypeError("Xq must hold uint8 E4M3 codes")
    T, K = Xq.shape
    _check("slope_spmm_e4m3_packed", library().slope_spmm_e4m3_packed(_dt(Y), _nn(Xq), _nn(x_scale), T, K,
                                                                      _nn(packed_w), _nb(packed_w), _nn(w_scale), N,
                                                                      _nn(Y), _s(stream)))


# ------------------------------------------------------------------ RMS norm, row-scaled int8 codes and products
# Codes travel as torch.int8 tensors, scales as torch.float32 tensors with one
# element for each token or channel.  These calls check shapes, dtypes and that
# all tensors are on one device, and run on that device's current stream (the
# caller's current device may be another) unless `stream` says otherwise.

I8_DECODE_MAX_TOKENS = 64   # SLOPE_I8_DECODE_MAX_TOKENS
I8_MAX_COLS = 1 << 18       # SLOPE_I8_MAX_COLS


# The calls of a few-token step are bound by the host, so the checks below are
# written for the path where they pass: torch's own handles of the current stream
# and device (its Python functions build a Stream object first: 2 us of a 10 us
# call), one comparison chain a tensor, one dict look-up a dtype.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_CODES = {torch.float32: _F32, torch.bfloat16: _BF16, torch.float16: _F16}
_i8, _f32t = torch.int8, torch.float32


def _code(dtype):
    c = _CODES.get(dtype)
    return _dt(dtype) if c is None else c          # _dt raises


def _rows(t, name):
    """(T, K) of a matrix with one token per row."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must have two dimensions [T, K], got shape {tuple(shape)}")
    return shape


def _place(index):
    return "the CPU" if index < 0 else f"GPU {index}"


def _arg(t, name, shape, dtype, dev):
    """Address of a contiguous tensor of this shape and dtype on device `dev`."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr() or 256                 # no elements: never dereferenced
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {_place(t.get_device())}, not on {_place(dev)}")


def _buffer(t, name, dev):
    """(address, bytes) of a contiguous scratch or operand buffer on device `dev`."""
    if t is None:
        return None, 0
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {_place(t.get_device())}, not on {_place(dev)}")
    return t.data_ptr() or 256, t.nbytes


def _on_device(fn, dev, stream, *args):
    """The library's fn(*args, stream) on device `dev`."""
    if dev < 0:
        raise ValueError("tensors must live in GPU memory")
    s = _raw_stream(dev) if stream is None else stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    f = getattr(_lib or library(), fn)
    if dev == _device_now():
        st = f(*args, s)
    else:
        with torch.cuda.device(dev):
            st = f(*args, s)
    if st != 0:
        raise SlopeError(fn, st)


def slope_rmsnorm(X, gamma, eps, residual=None, H=None, Y=None, q=None, q_scale=None, rstd=None, stream=None) -> None:
    """h = X + residual; Y = h * rstd * gamma; q, q_scale its int8 codes and
    scales; H, Y, (q, q_scale) and rstd are outputs, each may be None.  gamma:
    X's dtype or float32, or None for ones."""
    T, K = shape = _rows(X, "X")
    dt, d = X.dtype, X.get_device()
    gdt = dt if gamma is None else gamma.dtype
    _on_device("slope_rmsnorm", d, stream, _code(dt), _arg(X, "X", shape, dt, d),
               None if residual is None else _arg(residual, "residual", shape, dt, d), _code(gdt),
               None if gamma is None else _arg(gamma, "gamma", (K,), gdt, d), T, K, eps,
               None if H is None else _arg(H, "H", shape, dt, d), None if Y is None else _arg(Y, "Y", shape, dt, d),
               None if q is None else _arg(q, "q", shape, _i8, d),
               None if q_scale is None else _arg(q_scale, "q_scale", (T,), _f32t, d),
               None if rstd is None else _arg(rstd, "rstd", (T,), _f32t, d))


def slope_rmsnorm_bwd_workspace_bytes(T: int, K: int) -> int:
    b = ctypes.c_int64()
    _check("slope_rmsnorm_bwd_workspace_bytes", library().slope_rmsnorm_bwd_workspace_bytes(T, K, ctypes.byref(b)))
    return b.value


def slope_rmsnorm_bwd(dY, H, rstd, gamma, dX=None, dgamma=None, workspace=None, dH=None, accumulate=False,
                      stream=None) -> None:
    """dX = gradient of X and residual (with dH, the gradient reaching h by other
    ways, added); dgamma (added to with accumulate).  workspace:
    slope_rmsnorm_bwd_workspace_bytes(T, K) bytes, needed with dgamma."""
    T, K = shape = _rows(dY, "dY")
    dt, d = dY.dtype, dY.get_device()
    gdt = gamma.dtype if gamma is not None else dgamma.dtype if dgamma is not None else dt
    wp, wb = _buffer(workspace, "workspace", d)
    _on_device("slope_rmsnorm_bwd", d, stream, _code(dt), _arg(dY, "dY", shape, dt, d), _arg(H, "H", shape, dt, d),
               _arg(rstd, "rstd", (T,), _f32t, d), _code(gdt),
               None if gamma is None else _arg(gamma, "gamma", (K,), gdt, d),
               None if dH is None else _arg(dH, "dH", shape, dt, d), T, K,
               None if dX is None else _arg(dX, "dX", shape, dt, d),
               None if dgamma is None else _arg(dgamma, "dgamma", (K,), gdt, d), int(bool(accumulate)), wp, wb)


def slope_quantize_rows_i8(X, q, scale, stream=None) -> None:
    """int8 codes q [T, K] and scales [T] of the rows of a bf16 or fp16 X [T, K]."""
    T, K = shape = _rows(X, "X")
    d = X.get_device()
    _on_device("slope_quantize_rows_i8", d, stream, _code(X.dtype), _arg(X, "X", shape, X.dtype, d), T, K,
               _arg(q, "q", shape, _i8, d), _arg(scale, "scale", (T,), _f32t, d))


def slope_packed_sparse_i8_bytes(rows: int, cols: int) -> int:
    b = ctypes.c_int64()
    _check("slope_packed_sparse_i8_bytes", library().slope_packed_sparse_i8_bytes(rows, cols, ctypes.byref(b)))
    return b.value


def slope_pack_sparse_i8(values, meta, rows, cols, w_scale, packed, stream=None) -> None:
    """int8 tile chunks of a compressed 16-bit matrix, with its rows' scales in w_scale [rows]."""
    d = values.get_device()
    pp, pb = _buffer(packed, "packed", d)
    _on_device("slope_pack_sparse_i8", d, stream, _code(values.dtype),
               _arg(values, "values", (rows, cols // 2), values.dtype, d),
               _arg(meta, "meta", (rows, (cols // 4 + 7) // 8), torch.int32, d), rows, cols,
               _arg(w_scale, "w_scale", (rows,), _f32t, d), pp, pb)


def _spmm_i8(fn, Xq, x_scale, packed_w, w_scale, N, Y, stream):
    T, K = shape = _rows(Xq, "Xq")
    d = Xq.get_device()
    pp, pb = _buffer(packed_w, "packed_w", d)
    odt = Y.dtype
    _on_device(fn, d, stream, _code(odt), _arg(Xq, "Xq", shape, _i8, d), _arg(x_scale, "x_scale", (T,), _f32t, d), T, K,
               pp, pb, _arg(w_scale, "w_scale", (N,), _f32t, d), N, _arg(Y, "Y", (T, N), odt, d))


def slope_spmm_i8_packed(Xq, x_scale, packed_w, w_scale, N, Y, stream=None) -> None:
    """Y [T, N] = (Xq . W_q^T) * x_scale[t] * w_scale[n] on int8 codes, any T."""
    _spmm_i8("slope_spmm_i8_packed", Xq, x_scale, packed_w, w_scale, N, Y, stream)


def slope_spmm_i8_decode(Xq, x_scale, packed_w, w_scale, N, Y, stream=None) -> None:
    """slope_spmm_i8_packed for at most I8_DECODE_MAX_TOKENS tokens: the same result, bit for bit."""
    _spmm_i8("slope_spmm_i8_decode", Xq, x_scale, packed_w, w_scale, N, Y, stream)


# ------------------------------------------------------------------ microscaled formats
# Codes and scales travel as torch.uint8 tensors.  As above these calls check shapes,
# dtypes and devices, and run on the tensors' device.

MX_BLOCK = 32               # SLOPE_MX_BLOCK

_u8 = torch.uint8


_numel, _data_ptr, _get_device = torch.Tensor.numel, torch.Tensor.data_ptr, torch.Tensor.get_device
_is_contiguous, _dtype_of = torch.Tensor.is_contiguous, operator.attrgetter("dtype")


_HP_PACK = struct.Struct("=dddddq").pack            # AdamWParams' bytes, made faster


def _multi_refuse(i, p, g, m, v, me, ve, dev, mdt):
    """Raises what tensor i of a list is refused for, if it is."""
    n = p.numel()
    for name, t in (("params", p), ("grads", g), ("m", m), ("v", v), ("m_exp", me), ("v_exp", ve)):
        if t is None:
            continue
        name = f"{name}[{i}]"
        want = -(-n // MX_BLOCK) if "_exp" in name else n
        if t.numel() != want:
            raise ValueError(f"{name} must have {want} elements, got {t.numel()}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {_place(t.get_device())}, not on {_place(dev)}")
    _dt(p), _dt(g)
    for name, t, dtype in (("m", m, mdt), ("v", v, mdt), ("m_exp", me, _u8), ("v_exp", ve, _u8)):
        if t is not None and t.dtype is not dtype:
            raise TypeError(f"{name}[{i}] must be {dtype}, got {t.dtype}")


def slope_adamw_multi(params, grads, m, v, step, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, m_exp=None,
                      v_exp=None, seed=0, stream=None) -> None:
    """One AdamW step on lists of tensors (weights and moments updated in place).
    With float32 moments m, v: slope_adamw's results on each.  With uint8 codes
    m, v and the scales of their blocks of 32 in m_exp, v_exp: 8-bit moments,
    rounded stochastically with random bits from `seed` (another for each step)."""
    count = len(params)
    if count == 0:
        if grads or m or v or m_exp or v_exp:
            raise ValueError("the lists must have the same length")
        return
    eight = m_exp is not None or v_exp is not None
    mes, ves = (m_exp, v_exp) if eight else (m, v)
    if mes is None or ves is None:
        raise ValueError("8-bit moments need both m_exp and v_exp")
    if not len(grads) == len(m) == len(v) == len(mes) == len(ves) == count:
        raise ValueError("the lists must have the same length")
    # one pass over all the tensors for each question (7 tensors of 8-bit state: 22 us tensor by tensor)
    every = [*params, *grads, *m, *v]
    scales = [*m_exp, *v_exp] if eight else []
    dev, mdt = params[0].get_device(), _u8 if eight else _f32t
    sizes = list(map(_numel, every))
    of = sizes[:count]
    dtypes = list(map(_dtype_of, every))
    codes = list(map(_CODES.get, dtypes[:2 * count]))
    everything = every + scales
    if not (sizes == of * 4 and None not in codes and dtypes[2 * count:].count(mdt) == 2 * count
            and all(map(_is_contiguous, everything)) and set(map(_get_device, everything)) == {dev}
            and (not eight or (list(map(_numel, scales)) == [-(-n // MX_BLOCK) for n in of] * 2
                               and list(map(_dtype_of, scales)).count(_u8) == 2 * count))):
        for i in range(count):
            _multi_refuse(i, params[i], grads[i], m[i], v[i], mes[i] if eight else None, ves[i] if eight else None, dev,
                          mdt)
        raise ValueError("the lists are not accepted")
    of += map(_data_ptr, everything)
    table, kinds = array.array("q", of), array.array("i", codes)
    at, kind_at, size = table.buffer_info()[0], kinds.buffer_info()[0], 8 * count
    _on_device("slope_adamw_multi", dev, stream, 8 if eight else 32, count, kind_at, kind_at + 4 * count, at + size,
               at + 2 * size, at + 3 * size, at + 4 * size, at + 5 * size if eight else None,
               at + 6 * size if eight else None, at, _HP_PACK(lr, beta1, beta2, eps, weight_decay, int(step)),
               int(seed) & (2 ** 64 - 1))


def slope_adamw8_double_prune_packed(values_s, meta_s, dW_values, m, m_exp, v, v_exp, N, K, packed_s, packed_dpT, step,
                                     lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, seed=0, stream=None) -> None:
    """slope_adamw_multi with 8-bit moments on the compressed values of W_s (in place, and inside its
    tile chunks packed_s), then the double prune of the updated W_s into the tile chunks packed_dpT."""
    n, d = N * K // 2, values_s.get_device()
    flat = lambda t, name, size, dtype: _arg(t.reshape(-1) if t.is_contiguous() else t, name, (size,), dtype, d)
    vdt, gdt = values_s.dtype, dW_values.dtype
    ps, pb = _buffer(packed_s, "packed_s", d)
    qs, qb = _buffer(packed_dpT, "packed_dpT", d)
    hp = _hp(step, lr, beta1, beta2, eps, weight_decay)
    _on_device("slope_adamw8_double_prune_packed", d, stream, _code(vdt), _code(gdt), flat(values_s, "values_s", n, vdt),
               flat(meta_s, "meta_s", N * -(-K // 32), torch.int32), flat(dW_values, "dW_values", n, gdt),
               flat(m, "m", n, _u8), flat(m_exp, "m_exp", -(-n // MX_BLOCK), _u8), flat(v, "v", n, _u8),
               flat(v_exp, "v_exp", -(-n // MX_BLOCK), _u8), N, K, ctypes.byref(hp), int(seed) & (2 ** 64 - 1), ps, pb, qs, qb)


def slope_adamw_moments(m, m_exp, v, v_exp, m_out=None, v_out=None, stream=None) -> None:
    """The values of 8-bit moments as bfloat16 or float32 (m_out, v_out; one
    moment may be left out: None for its three tensors)."""
    first = m if m is not None else v
    if first is None:
        raise ValueError("give one moment at least")
    n, d = first.numel(), first.get_device()
    out = m_out if m_out is not None else v_out
    odt = _f32t if out is None else out.dtype
    blocks = -(-n // MX_BLOCK)

    def flat(t, name, size, dtype):
        if t is None:
            return None
        if t.dtype is dtype and t.numel() == size and t.get_device() == d and t.is_contiguous():
            return t.data_ptr() or 256             # no elements: never dereferenced
        return _arg(t.reshape(-1) if t.is_contiguous() else t, name, (size,), dtype, d)

    _on_device("slope_adamw_moments", d, stream, _code(odt), flat(m, "m", n, _u8), flat(m_exp, "m_exp", blocks, _u8),
               flat(v, "v", n, _u8), flat(v_exp, "v_exp", blocks, _u8), n, flat(m_out, "m_out", n, odt),
               flat(v_out, "v_out", n, odt))


def _rows_fit(codes, exps, other, name, T, K, d):
    """Raises unless codes and exps are T 4-bit rows of K values on device d, and the other operand, on d, is
    contiguous.  (One test for what fits; addresses of no elements, 0, are passed as 256: never dereferenced.)"""
    nc, ne = 64 * -(-K // 128), 16 * -(-K // 512)
    if not (codes.dtype is _u8 and exps.dtype is _u8 and codes.shape == (T, nc) and exps.shape == (T, ne)
            and codes.is_contiguous() and exps.is_contiguous() and other.is_contiguous()
            and codes.get_device() == d and exps.get_device() == d):
        if not other.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        _arg(codes, "codes", (T, nc), _u8, d), _arg(exps, "exps", (T, ne), _u8, d)


@functools.lru_cache(maxsize=4096)
def slope_mxfp4_row_bytes(K: int):
    """(bytes of codes, bytes of scales) of one row of K 4-bit values."""
    c, e = ctypes.c_int64(), ctypes.c_int64()
    _check("slope_mxfp4_row_bytes", library().slope_mxfp4_row_bytes(K, ctypes.byref(c), ctypes.byref(e)))
    return c.value, e.value


def slope_quantize_mxfp4(X, codes, exps, stream=None) -> None:
    """4-bit codes [T, code bytes] and scales [T, scale bytes] (slope_mxfp4_row_bytes)
    of the rows of X [T, K]."""
    T, K = _rows(X, "X")
    d = X.get_device()
    _rows_fit(codes, exps, X, "X", T, K, d)
    _on_device("slope_quantize_mxfp4", d, stream, _code(X.dtype), X.data_ptr() or 256, T, K, codes.data_ptr() or 256,
               exps.data_ptr() or 256)


def slope_mxfp4_values(codes, exps, out, stream=None) -> None:
    """out [T, K] <- the values of 4-bit rows."""
    T, K = _rows(out, "out")
    d = out.get_device()
    _rows_fit(codes, exps, out, "out", T, K, d)
    _on_device("slope_mxfp4_values", d, stream, _code(out.dtype), codes.data_ptr() or 256, exps.data_ptr() or 256, T, K,
               out.data_ptr() or 256)


def slope_packed_sparse_mxfp4_bytes(rows: int, cols: int) -> int:
    b = ctypes.c_int64()
    _check("slope_packed_sparse_mxfp4_bytes", library().slope_packed_sparse_mxfp4_bytes(rows, cols, ctypes.byref(b)))
    return b.value


def slope_pack_sparse_mxfp4(values, meta, rows, cols, packed, stream=None) -> None:
    """4-bit tile chunks of a compressed 16-bit matrix."""
    d = values.get_device()
    pp, pb = _buffer(packed, "packed", d)
    _on_device("slope_pack_sparse_mxfp4", d, stream, _code(values.dtype),
               _arg(values, "values", (rows, cols // 2), values.dtype, d),
               _arg(meta, "meta", (rows, (cols // 4 + 7) // 8), torch.int32, d), rows, cols, pp, pb)


def slope_spmm_mxfp4_workspace_bytes(T: int, K: int, N: int) -> int:
    """Bytes of workspace that make the product fastest on the current device."""
    b = ctypes.c_int64()
    _check("slope_spmm_mxfp4_workspace_bytes", library().slope_spmm_mxfp4_workspace_bytes(T, K, N, ctypes.byref(b)))
    return b.value


@functools.lru_cache(maxsize=4096)
def _spmm_mxfp4_workspace(dev, T, K, N):
    with torch.cuda.device(dev):
        return slope_spmm_mxfp4_workspace_bytes(T, K, N)


def slope_spmm_mxfp4_packed(codes, exps, K, packed_w, N, Y, workspace=None, stream=None) -> None:
    """Y [T, N] = Xq . W_q^T on 4-bit rows of K values and a 2:4 weight's 4-bit chunks, any T.  Without a
    workspace the call takes one of slope_spmm_mxfp4_workspace_bytes (an allocation of the current
    stream), but not where `stream` is given: then its sums are in another order where a
    workspace would have split K, and it is slower.  A workspace of that size gives
    the same bits on every stream."""
    T = _rows(codes, "codes")[0]
    d = codes.get_device()
    pp, pb = _buffer(packed_w, "packed_w", d)
    _rows_fit(codes, exps, Y, "Y", T, K, d)
    if Y.shape != (T, N) or Y.get_device() != d:
        _arg(Y, "Y", (T, N), Y.dtype, d)
    if workspace is None and stream is None and 1 < T <= 64 and d >= 0:
        need = _spmm_mxfp4_workspace(d, T, K, N)
        if need:
            workspace = torch.empty(need, dtype=_u8, device=codes.device)
    wp, wb = (None, 0) if workspace is None else _buffer(workspace, "workspace", d)
    _on_device("slope_spmm_mxfp4_packed", d, stream, _code(Y.dtype), codes.data_ptr() or 256, exps.data_ptr() or 256, T, K,
               pp, pb, N, Y.data_ptr() or 256, wp, wb)
