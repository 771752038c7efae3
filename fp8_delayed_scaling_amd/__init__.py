"""fp8_delayed_scaling_amd -- FP8 per-tensor delayed scaling on AMD MI355X (gfx950).

A thin ctypes binding of ``libfp8ds.so`` (the HIP kernels behind the C ABI of
``include/fp8ds.h``).  Every function here has the name of its C entry point and only
marshals arguments: it reads sizes, strides and pointers off torch tensors, picks the
stream, calls the library and turns a non-zero status into an exception.  All arithmetic
runs in the library's kernels; PyTorch only supplies device memory and streams.

The library must be built (``__graft_entry__.build()`` or ``python -m
fp8_delayed_scaling_amd.build``); importing this package without it raises immediately,
there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional, Sequence

import torch

__all__ = [
    "E4M3", "E5M2", "OUT_BF16", "OUT_FP32", "Fp8dsError", "lib", "library_path",
    "fp8ds_status_string", "fp8ds_version",
    "fp8_cast_amax", "fp8_cast_transpose", "fp8_dbias_workspace_bytes", "fp8_dbias_cast_transpose",
    "fp8_dbias_cast_transpose_noalloc", "fp8_scale_update", "fp8_gemm_bias", "fp8_gemm_bias_chunked", "fp8_gemm_bias_fp8", "fp8_transpose",
    "fp8_linear_fwd", "fp8_linear_bwd", "prepare", "Prepared",
    "NORM_RMS", "NORM_LAYER", "fp8_norm_residual_fwd", "fp8_norm_residual_workspace_bytes", "fp8_norm_residual_bwd",
    "fp8_moe_capacity", "fp8_moe_workspace_bytes", "fp8_moe_plan", "fp8_moe_sort_cast", "fp8_moe_sort_codes",
    "fp8_moe_sort_bf16", "fp8_moe_combine", "fp8_moe_weight_grad", "fp8_grouped_gemm", "fp8_grouped_wgrad",
    "fp8_attention_workspace_bytes", "fp8_attention_fwd", "fp8_attention_bwd_workspace_bytes", "fp8_attention_bwd",
    "fp8_moe_route_workspace_bytes", "fp8_moe_route", "fp8_moe_route_bwd",
]

E4M3 = 0
E5M2 = 1
NORM_RMS = 0
NORM_LAYER = 1
OUT_BF16 = 0
OUT_FP32 = 1

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libfp8ds.so")


class Fp8dsError(RuntimeError):
    """A libfp8ds call returned a non-zero status."""

    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


_lib = None
P = ctypes.c_void_p
I64 = ctypes.c_int64
I32 = ctypes.c_int32
F32 = ctypes.c_float
INT = ctypes.c_int
SZ = ctypes.c_size_t



class _Heads(ctypes.Structure):
    """fp8ds_heads: tokens of heads, strides in elements."""
    _fields_ = [("data", P), ("token_stride", I64), ("head_stride", I64)]


_SIGS = {
    "fp8ds_status_string": ([INT], ctypes.c_char_p),
    "fp8ds_version": ([], INT),
    "fp8_cast_amax": ([P, I64, P, INT, P, P, P, P, P], INT),
    "fp8_cast_transpose": ([P, I64, I64, P, INT, P, P, P, P, P, P], INT),
    "fp8_dbias_workspace_bytes": ([I64, I64], SZ),
    "fp8_dbias_cast_transpose": ([P, I64, I64, P, INT, P, P, P, P, P, P, SZ, P], INT),
    "fp8_dbias_cast_transpose_noalloc": ([P, I64, I64, P, INT, P, P, P, P, P, P], INT),
    "fp8_scale_update": ([P, I64, I64, P, P, P, I32, P], INT),
    "fp8_gemm_bias": ([P, INT, P, I64, P, INT, P, I64, P, P, I64, INT, I64, I64, I64, P], INT),
    "fp8_gemm_bias_chunked": ([P, INT, P, I64, P, INT, P, I64, P, P, I64, INT, I64, I64, I64, INT, P, P], INT),
    "fp8_gemm_bias_fp8": ([P, INT, P, I64, P, INT, P, I64, P, P, I64, INT, P, P, P, I64, I64, I64, P], INT),
    "fp8_transpose": ([P, I64, I64, P, P, P], INT),
    "fp8_linear_fwd": ([P, P, P, I64, I64, I64, P, P, P, P, P, P, P, P, P, P, P, P, P], INT),
    "fp8_linear_bwd": ([P, I64, I64, I64, P, P, P, P, P, P, P, SZ, P, P, P, P, P, P, INT, P], INT),
    "fp8_norm_residual_fwd": ([P, P, P, P, I64, P, F32, P, P, P, P, P, P, P, P, INT, P, P, INT, F32, I64, I64, P], INT),
    "fp8_norm_residual_workspace_bytes": ([I64, I64, I64], SZ),
    "fp8_norm_residual_bwd": ([P, P, P, P, P, P, I64, F32, P, P, P, P, P, P, P, P, P, P, P, P, SZ, INT, I64, I64, P],
                              INT),
    "fp8_moe_capacity": ([I64, I64, I64, I64], I64),
    "fp8_moe_workspace_bytes": ([I64, I64, I64], SZ),
    "fp8_moe_plan": ([P, I64, I64, I64, I64, I64, P, P, P, P, SZ, P], INT),
    "fp8_moe_sort_cast": ([P, I64, P, I64, I64, P, P, INT, P, P, P, P, I64, P], INT),
    "fp8_moe_sort_codes": ([P, I64, P, I64, I64, P, P, I64, P], INT),
    "fp8_moe_sort_bf16": ([P, I64, P, I64, I64, P, P, I64, P], INT),
    "fp8_moe_combine": ([P, I64, P, P, I64, I64, P, I64, P], INT),
    "fp8_moe_weight_grad": ([P, P, I64, P, I64, I64, P, I64, P], INT),
    "fp8_grouped_gemm": ([P, INT, P, I64, P, INT, P, I64, I64, P, I64, P, I64, INT, I64, I64, I64, P], INT),
    "fp8_grouped_wgrad": ([P, INT, P, I64, P, INT, P, I64, P, I64, P, INT, I64, I64, I64, P], INT),
    "fp8_attention_workspace_bytes": ([I64] * 6, SZ),
    "fp8_attention_fwd": ([_Heads] * 4 + [P, P, P, INT, P, P, P, P] + [I64] * 6 + [F32, INT, I64, P, SZ, P], INT),
    "fp8_attention_bwd_workspace_bytes": ([I64] * 6, SZ),
    "fp8_attention_bwd": ([_Heads] * 5 + [P] + [_Heads] * 3 + [P, P] + [I64] * 6 + [F32, INT, I64, P, SZ, P], INT),
    "fp8_moe_route_workspace_bytes": ([I64, I64], SZ),
    "fp8_moe_route": ([P, INT, I64, I64, I64, I64, INT, P, P, P, P, P, P, P, SZ, P], INT),
    "fp8_moe_route_bwd": ([P, INT, I64, I64, I64, I64, INT, P, P, P, P, P, P, P, I64, P], INT),
}


def lib() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise RuntimeError(
                f"{library_path} is not built: run `python -c 'import __graft_entry__ as g; g.build()'` "
                "(the FP8 path has no fallback)")
        L = ctypes.CDLL(library_path)
        for name, (argtypes, restype) in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = argtypes
            fn.restype = restype
        _lib = L
    return _lib


def fp8ds_status_string(status: int) -> str:
    return lib().fp8ds_status_string(int(status)).decode()


def fp8ds_version() -> int:
    return int(lib().fp8ds_version())


_calls = None


def _native():
    """The module of csrc/call.cpp, which takes the block operators' calls when every argument is as it should be."""
    global _calls
    if _calls is None:
        lib()
        try:
            from . import _call
        except ImportError as e:
            raise RuntimeError("the module of csrc/call.cpp is not built: run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`") from e
        _calls = _call
    return _calls


# ----------------------------------------------------------------------------- marshalling

def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensor arguments must live on the GPU")
    return t.data_ptr()


def _stream(s) -> Optional[int]:
    if s is None:
        if torch.cuda.is_initialized():      # the current stream's handle, without building a Stream object
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(status: int):
    if status != 0:
        raise Fp8dsError(status, fp8ds_status_string(status))


class _Tls(threading.local):
    rec = None             # the list prepare() records into, on this thread only


_tls = _Tls()
_HOST = object()           # stands for the pointer of a tensor that is not on the GPU (see _arg)


def _invoke(name: str, *cargs):
    """Call entry point ``name`` with marshalled arguments, or hand them to prepare()."""
    rec = _tls.rec
    if rec is not None:
        if _HOST in cargs:
            raise ValueError("tensor arguments must live on the GPU")
        rec.append((name, cargs))
        return
    try:
        status = getattr(_lib or lib(), name)(*cargs)
    except ctypes.ArgumentError:
        if _HOST in cargs:
            raise ValueError("tensor arguments must live on the GPU") from None
        raise
    if status != 0:
        _check(status)


class Prepared:
    """One entry-point call whose checks and marshalling ran once, in prepare(): calling it
    repeats only the C call, with the same device pointers, sizes and stream (or ``stream``).
    It keeps the tensors it was prepared with alive; they must keep their storage (no resize,
    no set_) for as long as it is used."""

    def __init__(self, name: str, cargs, keep):
        self.name = name
        self._fn = getattr(lib(), name)
        self._args = tuple(cargs)
        self._keep = keep

    def __call__(self, stream=None):
        a = self._args if stream is None else self._args[:-1] + (_stream(stream),)
        status = self._fn(*a)
        if status != 0:
            raise Fp8dsError(status, fp8ds_status_string(status))


def prepare(fn, *args, **kwargs) -> Prepared:
    """Run the binding ``fn`` (one of the entry points above) on these arguments up to the C call
    and return that call, ready to repeat: for layers small enough that the binding's per-call
    checks cost more host time than the launch itself.  The stream is the one ``fn`` would have
    used (the current stream unless ``stream=`` is given) unless the call passes another."""
    rec = []
    _tls.rec = rec
    try:
        fn(*args, **kwargs)
    finally:
        _tls.rec = None
    if len(rec) != 1:
        raise ValueError(f"{getattr(fn, '__name__', fn)} is not a single library call")
    name, cargs = rec[0]
    return Prepared(name, cargs, (args, kwargs))


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)


_F32 = (torch.float32,)
_U8 = (torch.uint8,)
_I32 = (torch.int32,)


def _want(t, dtypes, name, contiguous=True, shape=None, min_numel=None, required=False):
    """Check a tensor argument before its pointer goes to the library, which cannot see sizes:
    dtype, density, and the exact ``shape`` or at least ``min_numel`` elements.  A plain int is
    a raw device pointer and is passed through unchecked."""
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return
    if isinstance(t, int):
        return
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError(f"{name} must hold at least {min_numel} elements, got {t.numel()}")


def _arg(t, dtypes, shape, name, required=False):
    """Check a dense tensor argument of exactly ``shape`` as _want does, and return its pointer.  One
    that is not on the GPU gives _HOST, which _invoke refuses after all arguments' own checks."""
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return None
    if t.__class__ is int:
        return t
    if t.dtype not in dtypes or t.shape != shape or not t.is_contiguous():
        _want(t, dtypes, name, shape=shape)
    return t.data_ptr() if t.is_cuda else _HOST


def _some(t, dtypes, least, name):
    """As _arg, for a dense tensor (or None) of any shape with at least ``least`` elements."""
    if t is None or t.__class__ is int:
        return t
    if t.dtype not in dtypes or not t.is_contiguous() or t.numel() < least:
        _want(t, dtypes, name, min_numel=least)
    return t.data_ptr() if t.is_cuda else _HOST


def _workspace_bytes(workspace) -> int:
    """Size of a dbias workspace tensor in bytes (0 for None); it must be one dense block."""
    if workspace is None:
        return 0
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.numel() * workspace.element_size()


def _scalars(**kw):
    """float32 device scalars (scale, inverse scale, amax slot, noop flag): one element each."""
    for name, t in kw.items():
        _want(t, _F32, name, min_numel=1)


# ----------------------------------------------------------------------------- entry points

def fp8_cast_amax(x, scale, fmt, out, scale_inv_out=None, amax_slot=None, noop=None, stream=None):
    """Cast bfloat16 ``x`` to FP8 codes ``out`` with amax capture (see include/fp8ds.h)."""
    _want(x, _BF16, "x", required=True)
    _want(out, _U8, "out", required=True)
    if out.numel() != x.numel():
        raise ValueError("out must have x's number of elements")
    _scalars(scale=scale, scale_inv_out=scale_inv_out, amax_slot=amax_slot, noop=noop)
    _invoke("fp8_cast_amax", _ptr(x), x.numel(), _ptr(scale), int(fmt), _ptr(out), _ptr(scale_inv_out),
                               _ptr(amax_slot), _ptr(noop), _stream(stream))


def fp8_cast_transpose(x, scale, fmt, out, out_t, scale_inv_out=None, amax_slot=None, noop=None, stream=None):
    """Cast a 2-D bfloat16 ``x`` [R, C] to ``out`` [R, C] and its transpose ``out_t`` [C, R]."""
    _want(x, _BF16, "x", required=True)
    R, C = x.shape
    _want(out, _U8, "out", shape=(R, C), required=True)
    _want(out_t, _U8, "out_t", shape=(C, R), required=True)
    _scalars(scale=scale, scale_inv_out=scale_inv_out, amax_slot=amax_slot, noop=noop)
    _invoke("fp8_cast_transpose", _ptr(x), R, C, _ptr(scale), int(fmt), _ptr(out), _ptr(out_t),
                                    _ptr(scale_inv_out), _ptr(amax_slot), _ptr(noop), _stream(stream))


def fp8_dbias_workspace_bytes(rows: int, cols: int) -> int:
    return int(lib().fp8_dbias_workspace_bytes(int(rows), int(cols)))


def fp8_dbias_cast_transpose(dy, scale, fmt, out, out_t, dbias, workspace, scale_inv_out=None, amax_slot=None,
                             stream=None):
    """dbias = column sums of ``dy`` plus its cast+transpose (see include/fp8ds.h).

    ``workspace``: at least ``fp8_dbias_workspace_bytes(rows, cols)`` bytes, zero-filled before
    its first use (``torch.zeros``); every call leaves its counter bytes zero again."""
    _want(dy, _BF16, "dy", required=True)
    R, C = dy.shape
    _want(dbias, _F32, "dbias", shape=(C,), required=True)
    _want(out, _U8, "out", shape=(R, C))
    _want(out_t, _U8, "out_t", shape=(C, R))
    ws_bytes = _workspace_bytes(workspace)
    _scalars(scale=scale, scale_inv_out=scale_inv_out, amax_slot=amax_slot)
    _invoke("fp8_dbias_cast_transpose", _ptr(dy), R, C, _ptr(scale), int(fmt), _ptr(out), _ptr(out_t),
                                          _ptr(scale_inv_out), _ptr(amax_slot), _ptr(dbias), _ptr(workspace),
                                          ws_bytes, _stream(stream))


def fp8_dbias_cast_transpose_noalloc(dy, scale, fmt, out, out_t, dbias, scale_inv_out=None, amax_slot=None,
                                     stream=None):
    """fp8_dbias_cast_transpose without a workspace: the partial sums go to the library's static
    per-GPU scratch (no allocation; calls overlapping on one GPU race; see include/fp8ds.h)."""
    _want(dy, _BF16, "dy", required=True)
    R, C = dy.shape
    _want(dbias, _F32, "dbias", shape=(C,), required=True)
    _want(out, _U8, "out", shape=(R, C))
    _want(out_t, _U8, "out_t", shape=(C, R))
    _scalars(scale=scale, scale_inv_out=scale_inv_out, amax_slot=amax_slot)
    _invoke("fp8_dbias_cast_transpose_noalloc", _ptr(dy), R, C, _ptr(scale), int(fmt), _ptr(out), _ptr(out_t),
                                                  _ptr(scale_inv_out), _ptr(amax_slot), _ptr(dbias),
                                                  _stream(stream))


def fp8_scale_update(amax_history, scale, scale_inv, fmts: Sequence[int], margin: int = 0, stream=None):
    """One delayed-scaling step for the T tensors of ``amax_history`` [L, T]."""
    _want(amax_history, _F32, "amax_history", required=True)
    L, T = amax_history.shape
    _want(scale, _F32, "scale", min_numel=T, required=True)
    _want(scale_inv, _F32, "scale_inv", min_numel=T, required=True)
    if len(fmts) != T:
        raise ValueError("one format per tensor")
    f = (ctypes.c_int32 * T)(*[int(v) for v in fmts])
    _invoke("fp8_scale_update", _ptr(amax_history), L, T, _ptr(scale), _ptr(scale_inv),
                                  ctypes.cast(f, ctypes.c_void_p), int(margin), _stream(stream))


def _out_dtype(D):
    if D.dtype == torch.bfloat16:
        return OUT_BF16
    if D.dtype == torch.float32:
        return OUT_FP32
    raise TypeError("D must be bfloat16 or float32")


def _gemm_args(A, fa, a_scale_inv, B, fb, b_scale_inv, bias, D):
    _want(A, _U8, "A", contiguous=False, required=True)
    _want(B, _U8, "B", contiguous=False, required=True)
    M, K = A.shape
    N, K2 = B.shape
    if K != K2:
        raise ValueError("A and B must share K")
    _want(bias, _BF16, "bias", shape=(N,))
    if tuple(D.shape) != (M, N):
        raise ValueError("D must be [M, N]")
    for t, nm in ((A, "A"), (B, "B"), (D, "D")):
        if t.numel() and t.stride(1) != 1:
            raise ValueError(f"{nm} rows must be contiguous")
    _scalars(a_scale_inv=a_scale_inv, b_scale_inv=b_scale_inv)
    return (_ptr(A), int(fa), _ptr(a_scale_inv), A.stride(0), _ptr(B), int(fb), _ptr(b_scale_inv), B.stride(0),
            _ptr(bias), _ptr(D), D.stride(0), _out_dtype(D), M, N, K)


def fp8_gemm_bias(A, fa, a_scale_inv, B, fb, b_scale_inv, bias, D, stream=None):
    """D = (A B^T) * a_scale_inv * b_scale_inv + bias, A [M, K] and B [N, K] FP8 codes."""
    _invoke("fp8_gemm_bias", *_gemm_args(A, fa, a_scale_inv, B, fb, b_scale_inv, bias, D), _stream(stream))


def fp8_gemm_bias_fp8(A, fa, a_scale_inv, B, fb, b_scale_inv, bias, D, d_fmt, d_scale, d_scale_inv_out=None,
                      d_amax_slot=None, stream=None):
    """FP8-output GEMM: D = codes of ((A B^T) * a_scale_inv * b_scale_inv + bias) * d_scale, with the
    output's amax folded into ``d_amax_slot`` and 1/d_scale written to ``d_scale_inv_out``."""
    _want(D, _U8, "D", contiguous=False, required=True)
    _want(A, _U8, "A", contiguous=False, required=True)
    _want(B, _U8, "B", contiguous=False, required=True)
    M, K = A.shape
    N, K2 = B.shape
    if K != K2:
        raise ValueError("A and B must share K")
    _want(bias, _BF16, "bias", shape=(N,))
    _scalars(a_scale_inv=a_scale_inv, b_scale_inv=b_scale_inv, d_scale=d_scale, d_scale_inv_out=d_scale_inv_out,
             d_amax_slot=d_amax_slot)
    if tuple(D.shape) != (M, N):
        raise ValueError("D must be [M, N]")
    for t, nm in ((A, "A"), (B, "B"), (D, "D")):
        if t.numel() and t.stride(1) != 1:
            raise ValueError(f"{nm} rows must be contiguous")
    _invoke("fp8_gemm_bias_fp8", _ptr(A), int(fa), _ptr(a_scale_inv), A.stride(0), _ptr(B), int(fb),
                                   _ptr(b_scale_inv), B.stride(0), _ptr(bias), _ptr(D), D.stride(0), int(d_fmt),
                                   _ptr(d_scale), _ptr(d_scale_inv_out), _ptr(d_amax_slot), M, N, K,
                                   _stream(stream))


def fp8_transpose(x8, out_t, noop=None, stream=None):
    """Transpose cache of an existing FP8 tensor: out_t [C, R] = x8 [R, C]^T (codes copied)."""
    _want(x8, _U8, "x8", required=True)
    R, C = x8.shape
    _want(out_t, _U8, "out_t", shape=(C, R), required=True)
    _scalars(noop=noop)
    _invoke("fp8_transpose", _ptr(x8), R, C, _ptr(out_t), _ptr(noop), _stream(stream))


def fp8_gemm_bias_chunked(A, fa, a_scale_inv, B, fb, b_scale_inv, bias, D, n_chunks: int,
                          chunk_streams=None, stream=None):
    """The N-chunked GEMM: chunk c on ``chunk_streams[c]`` with its own bias offset."""
    arr = None
    if chunk_streams is not None:
        if len(chunk_streams) < n_chunks:
            raise ValueError("one stream per chunk")
        arr = (ctypes.c_void_p * n_chunks)(*[_stream(s) for s in chunk_streams[:n_chunks]])
    _invoke("fp8_gemm_bias_chunked", *_gemm_args(A, fa, a_scale_inv, B, fb, b_scale_inv, bias, D),
                                       int(n_chunks), None if arr is None else ctypes.cast(arr, ctypes.c_void_p),
                                       _stream(stream))


def fp8_linear_fwd(x, w, bias, x_scale, x_amax, x8, x8_t, x_scale_inv, w_scale, w_amax, w8, w8_t, w_scale_inv,
                   w_noop, y, stream=None):
    """Forward of the FP8 linear layer: casts of x and W, then y = x8 W8^T + bias."""
    _want(x, _BF16, "x", required=True)
    _want(w, _BF16, "w", required=True)
    M, K = x.shape
    N, K2 = w.shape
    if K != K2:
        raise ValueError("x [M, K] and w [N, K] must share K")
    _want(y, (torch.bfloat16,), "y", shape=(M, N), required=True)
    _want(bias, _BF16, "bias", shape=(N,))
    _want(x8, _U8, "x8", shape=(M, K), required=True)
    _want(x8_t, _U8, "x8_t", shape=(K, M))
    _want(w8, _U8, "w8", shape=(N, K), required=True)
    _want(w8_t, _U8, "w8_t", shape=(K, N), required=True)
    _scalars(x_scale=x_scale, x_amax=x_amax, x_scale_inv=x_scale_inv, w_scale=w_scale, w_amax=w_amax,
             w_scale_inv=w_scale_inv, w_noop=w_noop)
    _invoke("fp8_linear_fwd", _ptr(x), _ptr(w), _ptr(bias), M, N, K, _ptr(x_scale), _ptr(x_amax), _ptr(x8),
                                _ptr(x8_t), _ptr(x_scale_inv), _ptr(w_scale), _ptr(w_amax), _ptr(w8), _ptr(w8_t),
                                _ptr(w_scale_inv), _ptr(w_noop), _ptr(y), _stream(stream))


def fp8_linear_bwd(dy, K, dy_scale, dy_amax, dy8, dy8_t, dy_scale_inv, dbias, workspace, x8_t, x_scale_inv, w8_t,
                   w_scale_inv, dx, dw, stream=None):
    """Backward of the FP8 linear layer: dbias + cast+transpose of dy, dgrad and wgrad GEMMs.

    ``workspace`` (with ``dbias``): zero-filled before its first use, as for
    ``fp8_dbias_cast_transpose``."""
    _want(dy, _BF16, "dy", required=True)
    M, N = dy.shape
    K = int(K)
    _want(dy8, _U8, "dy8", shape=(M, N), required=True)
    _want(dy8_t, _U8, "dy8_t", shape=(N, M), required=True)
    _want(dbias, _F32, "dbias", shape=(N,))
    _want(x8_t, _U8, "x8_t", shape=(K, M), required=True)
    _want(w8_t, _U8, "w8_t", shape=(K, N), required=True)
    _want(dx, (torch.bfloat16,), "dx", shape=(M, K), required=True)
    _want(dw, (torch.bfloat16, torch.float32), "dw", shape=(N, K), required=True)
    ws_bytes = _workspace_bytes(workspace)
    _scalars(dy_scale=dy_scale, dy_amax=dy_amax, dy_scale_inv=dy_scale_inv, x_scale_inv=x_scale_inv,
             w_scale_inv=w_scale_inv)
    _invoke("fp8_linear_bwd", _ptr(dy), M, N, int(K), _ptr(dy_scale), _ptr(dy_amax), _ptr(dy8), _ptr(dy8_t),
                                _ptr(dy_scale_inv), _ptr(dbias), _ptr(workspace), ws_bytes, _ptr(x8_t),
                                _ptr(x_scale_inv), _ptr(w8_t), _ptr(w_scale_inv), _ptr(dx), _ptr(dw),
                                _out_dtype(dw), _stream(stream))


# ------------------------------------------------------- the operators around the linear layer

def _gate_arg(gate, M, H):
    """Pointer and number of the gates."""
    if gate is None:
        return None, 0
    _want(gate, _BF16, "gate")
    if gate.dim() != 2 or gate.shape[1] != H or gate.shape[0] < 1 or M % gate.shape[0] != 0:
        raise ValueError(f"gate must be [G, {H}] with G dividing the {M} rows, got {tuple(gate.shape)}")
    return gate.data_ptr() if gate.is_cuda else _HOST, gate.shape[0]


def fp8_norm_residual_fwd(block_out, w_post, b_post, gate, resid, alpha, x, post_stats, w_pre, b_pre, pre_stats, h,
                          h8=None, scale=None, fmt=E4M3, scale_inv_out=None, amax_slot=None, kind=NORM_RMS, eps=1e-5,
                          stream=None):
    """x = alpha * resid + gate * (norm(block_out) * w_post + b_post), h = norm(x) * w_pre + b_pre as bfloat16
    ``h`` and / or FP8 codes ``h8`` (see include/fp8ds.h for what may be None).

    ``post_stats`` / ``pre_stats``: float32, rows values (RMS) or 2 * rows (layer: 1 / deviation, then mean)."""
    if _tls.rec is None and (_calls or _native()).norm_fwd(
            block_out, w_post, b_post, gate, resid, alpha, x, post_stats, w_pre, b_pre, pre_stats, h, h8, scale, fmt,
            scale_inv_out, amax_slot, kind, eps, stream):
        return
    ref, name = (resid, "resid") if block_out is None else (block_out, "block_out")
    _want(ref, _BF16, name, required=True)
    shape = ref.shape
    M, H = shape
    row = (H,)
    stats = 2 * M if kind == NORM_LAYER else M
    p_gate, G = _gate_arg(gate, M, H)
    _invoke("fp8_norm_residual_fwd", _arg(block_out, _BF16, shape, "block_out"), _arg(w_post, _BF16, row, "w_post"),
            _arg(b_post, _BF16, row, "b_post"), p_gate, G, _arg(resid, _BF16, shape, "resid"), float(alpha),
            _arg(x, _BF16, shape, "x", block_out is not None), _some(post_stats, _F32, stats, "post_stats"),
            _arg(w_pre, _BF16, row, "w_pre"), _arg(b_pre, _BF16, row, "b_pre"), _some(pre_stats, _F32, stats, "pre_stats"),
            _arg(h, _BF16, shape, "h"), _arg(h8, _U8, shape, "h8"), _some(scale, _F32, 1, "scale"), int(fmt),
            _some(scale_inv_out, _F32, 1, "scale_inv_out"), _some(amax_slot, _F32, 1, "amax_slot"), int(kind), float(eps),
            M, H, _stream(stream))


def fp8_norm_residual_workspace_bytes(rows: int, width: int, n_gates: int) -> int:
    return int(lib().fp8_norm_residual_workspace_bytes(int(rows), int(width), int(n_gates)))


def fp8_norm_residual_bwd(dh, dx, block_out, w_post, b_post, gate, alpha, x, post_stats, w_pre, pre_stats, d_block,
                          d_resid, dw_post, db_post, dgate, dw_pre, db_pre, workspace, kind=NORM_RMS, stream=None):
    """Gradients of fp8_norm_residual_fwd: ``dh`` of h, ``dx`` of x (either may be None), from the x and the
    statistics that the forward wrote.  ``workspace``: ``fp8_norm_residual_workspace_bytes(rows, width, gates)``."""
    if _tls.rec is None and (_calls or _native()).norm_bwd(
            dh, dx, block_out, w_post, b_post, gate, alpha, x, post_stats, w_pre, pre_stats, d_block, d_resid, dw_post,
            db_post, dgate, dw_pre, db_pre, workspace, kind, stream):
        return
    ref = dh if dh is not None else dx
    _want(ref, _BF16, "dh" if dh is not None else "dx", required=True)
    shape = ref.shape
    M, H = shape
    row = (H,)
    stats = 2 * M if kind == NORM_LAYER else M
    p_gate, G = _gate_arg(gate, M, H)
    ws_bytes = _workspace_bytes(workspace)
    _invoke("fp8_norm_residual_bwd", _arg(dh, _BF16, shape, "dh"), _arg(dx, _BF16, shape, "dx"),
            _arg(block_out, _BF16, shape, "block_out"), _arg(w_post, _BF16, row, "w_post"), _arg(b_post, _BF16, row, "b_post"),
            p_gate, G, float(alpha), _arg(x, _BF16, shape, "x"), _some(post_stats, _F32, stats, "post_stats"),
            _arg(w_pre, _BF16, row, "w_pre"), _some(pre_stats, _F32, stats, "pre_stats"), _arg(d_block, _BF16, shape, "d_block"),
            _arg(d_resid, _BF16, shape, "d_resid"), _arg(dw_post, _F32, row, "dw_post"), _arg(db_post, _F32, row, "db_post"),
            _arg(dgate, _F32, (max(G, 1), H), "dgate"), _arg(dw_pre, _F32, row, "dw_pre"), _arg(db_pre, _F32, row, "db_pre"),
            _ptr(workspace), ws_bytes, int(kind), M, H, _stream(stream))


def fp8_moe_capacity(T: int, top: int, E: int, align: int = 16) -> int:
    """Rows of the sorted buffers that hold any routing of T tokens to ``top`` of E experts each."""
    n = int(lib().fp8_moe_capacity(int(T), int(top), int(E), int(align)))
    if n < 0:
        raise ValueError(f"no plan for T={T}, top={top}, E={E}, align={align} (1 <= E <= 1024, align a multiple of 16 "
                         "up to 1024)")
    return n


def fp8_moe_workspace_bytes(T: int, top: int, E: int) -> int:
    return int(lib().fp8_moe_workspace_bytes(int(T), int(top), int(E)))


def fp8_moe_plan(experts, E: int, align: int, offsets, src, slot, workspace=None, stream=None):
    """Sort the choices ``experts`` [T, top] (int32; outside [0, E): dropped) by expert: ``offsets`` [E + 1],
    ``src`` [capacity], ``slot`` [T, top] (see include/fp8ds.h)."""
    if _tls.rec is None and (_calls or _native()).moe_plan(experts, E, align, offsets, src, slot, workspace, stream):
        return
    _want(experts, _I32, "experts", required=True)
    if experts.dim() != 2:
        raise ValueError("experts must be [T, top]")
    shape = experts.shape
    T, k = shape
    _want(src, _I32, "src", required=True)
    ws_bytes = _workspace_bytes(workspace)
    _invoke("fp8_moe_plan", _arg(experts, _I32, shape, "experts"), T, k, int(E), int(align), src.numel(),
            _arg(offsets, _I32, (int(E) + 1,), "offsets", True), _arg(src, _I32, src.shape, "src"),
            _arg(slot, _I32, shape, "slot", True), _ptr(workspace), ws_bytes, _stream(stream))


def _sort_args(x, dtypes, src, top, weights, out, out_dtypes, out_t):
    """Sizes T, width and capacity, and the five pointers."""
    _want(x, dtypes, "x", required=True)
    _want(src, _I32, "src", required=True)
    if x.dim() != 2:
        raise ValueError("x must be [T, width]")
    T, H = x.shape
    cap = src.numel()
    return (T, H, cap, _arg(x, dtypes, x.shape, "x"), _arg(src, _I32, src.shape, "src"),
            _arg(weights, _F32, (T, int(top)), "weights"), _arg(out, out_dtypes, (cap, H), "out", True),
            _arg(out_t, _U8, (H, cap), "out_t"))


def fp8_moe_sort_cast(x, src, top: int, weights, scale, fmt, out, out_t=None, scale_inv_out=None, amax_slot=None,
                      stream=None):
    """Rows of bfloat16 ``x`` in expert order, times ``weights`` (or None), as FP8 codes and their transpose."""
    if _tls.rec is None and (_calls or _native()).moe_sort_cast(
            x, src, top, weights, scale, fmt, out, out_t, scale_inv_out, amax_slot, stream):
        return
    T, H, cap, p_x, p_src, p_w, p_out, p_out_t = _sort_args(x, _BF16, src, top, weights, out, _U8, out_t)
    _invoke("fp8_moe_sort_cast", p_x, T, p_src, cap, int(top), p_w, _some(scale, _F32, 1, "scale"), int(fmt), p_out, p_out_t,
            _some(scale_inv_out, _F32, 1, "scale_inv_out"), _some(amax_slot, _F32, 1, "amax_slot"), H, _stream(stream))


def fp8_moe_sort_codes(x8, src, top: int, out, out_t=None, stream=None):
    """Rows of FP8 codes in expert order, and their transpose (codes copied; padding rows are zero)."""
    if _tls.rec is None and (_calls or _native()).moe_sort_codes(x8, src, top, out, out_t, stream):
        return
    T, H, cap, p_x, p_src, _, p_out, p_out_t = _sort_args(x8, _U8, src, top, None, out, _U8, out_t)
    _invoke("fp8_moe_sort_codes", p_x, T, p_src, cap, int(top), p_out, p_out_t, H, _stream(stream))


def fp8_moe_sort_bf16(x, src, top: int, weights, out, stream=None):
    """Rows of bfloat16 ``x`` in expert order, times ``weights`` (or None)."""
    T, H, cap, p_x, p_src, p_w, p_out, _ = _sort_args(x, _BF16, src, top, weights, out, _BF16, None)
    _invoke("fp8_moe_sort_bf16", p_x, T, p_src, cap, int(top), p_w, p_out, H, _stream(stream))


def _back_args(ys, slot):
    """Sizes and the two pointers."""
    _want(ys, _BF16, "ys", required=True)
    _want(slot, _I32, "slot", required=True)
    if ys.dim() != 2 or slot.dim() != 2:
        raise ValueError("ys must be [capacity, width] and slot [T, top]")
    return (*ys.shape, *slot.shape, _arg(ys, _BF16, ys.shape, "ys"), _arg(slot, _I32, slot.shape, "slot"))


def fp8_moe_combine(ys, slot, weights, y, stream=None):
    """y[t] = sum over j of weights[t, j] * ys[slot[t, j]] (weights None: 1)."""
    if _tls.rec is None and (_calls or _native()).moe_combine(ys, slot, weights, y, stream):
        return
    cap, H, T, k, p_ys, p_slot = _back_args(ys, slot)
    _invoke("fp8_moe_combine", p_ys, cap, p_slot, _arg(weights, _F32, (T, k), "weights"), T, k, _arg(y, _BF16, (T, H), "y", True),
            H, _stream(stream))


def fp8_moe_weight_grad(dy, ys, slot, dweights, stream=None):
    """dweights[t, j] = <dy[t], ys[slot[t, j]]>, 0 for a dropped choice."""
    if _tls.rec is None and (_calls or _native()).moe_weight_grad(dy, ys, slot, dweights, stream):
        return
    cap, H, T, k, p_ys, p_slot = _back_args(ys, slot)
    _invoke("fp8_moe_weight_grad", _arg(dy, _BF16, (T, H), "dy", True), p_ys, cap, p_slot, T, k,
            _arg(dweights, _F32, (T, k), "dweights", True), H, _stream(stream))


def _rows_dense(**kw):
    for name, t in kw.items():
        if t.numel() and t.stride(-1) != 1:
            raise ValueError(f"{name} rows must be contiguous")


def fp8_grouped_gemm(A, fa, a_scale_inv, B, fb, b_scale_inv, offsets, D, stream=None):
    """D[r] = A[r] B[e]^T * a_scale_inv * b_scale_inv for the rows r in [offsets[e], offsets[e + 1]):
    A [cap, K] and B [E, N, K] FP8 codes (B may be a strided view), D [cap, N] bfloat16 or float32."""
    if _tls.rec is None and (_calls or _native()).grouped_gemm(
            A, fa, a_scale_inv, B, fb, b_scale_inv, offsets, D, stream):
        return
    _want(A, _U8, "A", contiguous=False, required=True)
    _want(B, _U8, "B", contiguous=False, required=True)
    if A.dim() != 2 or B.dim() != 3 or A.shape[1] != B.shape[2]:
        raise ValueError("A [cap, K] and B [E, N, K] must share K")
    cap, K = A.shape
    E, N = B.shape[:2]
    p_off = _arg(offsets, _I32, (E + 1,), "offsets", True)
    if D.shape != (cap, N):
        raise ValueError(f"D must be [{cap}, {N}]")
    _rows_dense(A=A, B=B, D=D)
    dtype = _out_dtype(D)
    _invoke("fp8_grouped_gemm", _ptr(A), int(fa), _some(a_scale_inv, _F32, 1, "a_scale_inv"), A.stride(0), _ptr(B), int(fb),
            _some(b_scale_inv, _F32, 1, "b_scale_inv"), B.stride(1), B.stride(0), p_off, E, _ptr(D), D.stride(0), dtype, cap, N,
            K, _stream(stream))


def fp8_grouped_wgrad(At, fa, a_scale_inv, Bt, fb, b_scale_inv, offsets, dW, stream=None):
    """dW[e] = At[:, rows of e] Bt[:, rows of e]^T * a_scale_inv * b_scale_inv: At [N, cap] and Bt [K, cap] FP8
    codes (the transposes of the sorted rows), dW [E, N, K] bfloat16 or float32."""
    if _tls.rec is None and (_calls or _native()).grouped_wgrad(
            At, fa, a_scale_inv, Bt, fb, b_scale_inv, offsets, dW, stream):
        return
    _want(At, _U8, "At", contiguous=False, required=True)
    _want(Bt, _U8, "Bt", contiguous=False, required=True)
    if At.dim() != 2 or Bt.dim() != 2 or At.shape[1] != Bt.shape[1]:
        raise ValueError("At [N, cap] and Bt [K, cap] must share the sorted rows")
    N, cap = At.shape
    K = Bt.shape[0]
    _want(offsets, _I32, "offsets", required=True)
    E = offsets.numel() - 1
    _want(dW, (torch.bfloat16, torch.float32), "dW", required=True)
    p_dw = _arg(dW, (torch.bfloat16, torch.float32), (E, N, K), "dW")
    _rows_dense(At=At, Bt=Bt)
    _invoke("fp8_grouped_wgrad", _ptr(At), int(fa), _some(a_scale_inv, _F32, 1, "a_scale_inv"), At.stride(0), _ptr(Bt), int(fb),
            _some(b_scale_inv, _F32, 1, "b_scale_inv"), Bt.stride(0), _ptr(offsets), E, p_dw, _out_dtype(dW), cap, N, K,
            _stream(stream))


def fp8_attention_workspace_bytes(Tq: int, Tk: int, batch: int, Hq: int, Hkv: int, D: int) -> int:
    return int(lib().fp8_attention_workspace_bytes(int(Tq), int(Tk), int(batch), int(Hq), int(Hkv), int(D)))


def fp8_attention_bwd_workspace_bytes(Tq: int, Tk: int, batch: int, Hq: int, Hkv: int, D: int) -> int:
    return int(lib().fp8_attention_bwd_workspace_bytes(int(Tq), int(Tk), int(batch), int(Hq), int(Hkv), int(D)))


def _heads(t, T, H, D, name, required=True):
    """[T, H, D] bfloat16 with strides of its own, the elements of a head one behind the other."""
    _want(t, _BF16, name, contiguous=False, shape=(T, H, D), required=required)
    if t is None:
        return _Heads(None, D, D)
    if t.numel() and t.stride(2) != 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    if not t.is_cuda:
        return _HOST
    return _Heads(t.data_ptr(), t.stride(0) if T > 1 else D, t.stride(1) if H > 1 else D)


def _attention_sizes(q, k, offsets_q, offsets_k, batch):
    """Tq, Hq, D, Tk, Hkv, the number of sequences and the offsets' pointers."""
    _want(q, _BF16, "q", contiguous=False, required=True)
    _want(k, _BF16, "k", contiguous=False, required=True)
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [tokens, heads, head size]")
    if (offsets_q is None) != (offsets_k is None):
        raise ValueError("offsets_q and offsets_k go together")
    if offsets_q is not None:
        _want(offsets_q, _I32, "offsets_q")
        if offsets_q.numel() < 1:
            raise ValueError("offsets_q must hold at least one element")
        batch = offsets_q.numel() - 1
    row = (int(batch) + 1,)
    return (*q.shape, k.shape[0], k.shape[1], int(batch), _arg(offsets_q, _I32, row, "offsets_q"),
            _arg(offsets_k, _I32, row, "offsets_k"))


def fp8_attention_fwd(q, k, v, out, lse=None, offsets_q=None, offsets_k=None, batch: int = 1, causal: bool = True,
                      window: int = 0, softmax_scale=None, out8=None, scale=None, fmt=E4M3, scale_inv_out=None,
                      amax_slot=None, workspace=None, stream=None):
    """Attention of ``q`` [Tq, Hq, D] over ``k``, ``v`` [Tk, Hkv, D] (any token and head strides) into ``out`` (or
    None), ``lse`` [Hq, Tq] and FP8 codes ``out8`` [Tq, Hq * D]; sequences by offsets, or ``batch`` equal ones;
    ``softmax_scale`` None: D ** -0.5 (see include/fp8ds.h)."""
    if _tls.rec is None and (_calls or _native()).attention_fwd(
            q, k, v, out, lse, offsets_q, offsets_k, batch, causal, window, softmax_scale, out8, scale, fmt, scale_inv_out,
            amax_slot, workspace, stream):
        return
    Tq, Hq, D, Tk, Hkv, B, p_oq, p_ok = _attention_sizes(q, k, offsets_q, offsets_k, batch)
    ws_bytes = _workspace_bytes(workspace)
    _invoke("fp8_attention_fwd", _heads(q, Tq, Hq, D, "q"), _heads(k, Tk, Hkv, D, "k"), _heads(v, Tk, Hkv, D, "v"),
            _heads(out, Tq, Hq, D, "out", required=False), _arg(lse, _F32, (Hq, Tq), "lse"),
            _arg(out8, _U8, (Tq, Hq * D), "out8"), _some(scale, _F32, 1, "scale"), int(fmt),
            _some(scale_inv_out, _F32, 1, "scale_inv_out"), _some(amax_slot, _F32, 1, "amax_slot"), p_oq, p_ok, B, Tq, Tk,
            Hq, Hkv, D, D ** -0.5 if softmax_scale is None else float(softmax_scale), int(bool(causal)), int(window),
            _ptr(workspace), ws_bytes, _stream(stream))


def fp8_attention_bwd(dout, q, k, v, out, lse, dq, dk, dv, workspace, offsets_q=None, offsets_k=None, batch: int = 1,
                      causal: bool = True, window: int = 0, softmax_scale=None, stream=None):
    """Gradients of fp8_attention_fwd into ``dq``, ``dk``, ``dv`` (bfloat16, any token and head strides), from the
    ``out`` and ``lse`` that it wrote (see include/fp8ds.h)."""
    if _tls.rec is None and (_calls or _native()).attention_bwd(
            dout, q, k, v, out, lse, dq, dk, dv, workspace, offsets_q, offsets_k, batch, causal, window, softmax_scale,
            stream):
        return
    Tq, Hq, D, Tk, Hkv, B, p_oq, p_ok = _attention_sizes(q, k, offsets_q, offsets_k, batch)
    ws_bytes = _workspace_bytes(workspace)
    _invoke("fp8_attention_bwd", _heads(dout, Tq, Hq, D, "dout"), _heads(q, Tq, Hq, D, "q"), _heads(k, Tk, Hkv, D, "k"),
            _heads(v, Tk, Hkv, D, "v"), _heads(out, Tq, Hq, D, "out"), _arg(lse, _F32, (Hq, Tq), "lse", True),
            _heads(dq, Tq, Hq, D, "dq"), _heads(dk, Tk, Hkv, D, "dk"), _heads(dv, Tk, Hkv, D, "dv"), p_oq, p_ok, B, Tq, Tk,
            Hq, Hkv, D, D ** -0.5 if softmax_scale is None else float(softmax_scale), int(bool(causal)), int(window),
            _ptr(workspace), ws_bytes, _stream(stream))


def fp8_moe_route_workspace_bytes(T: int, E: int) -> int:
    return int(lib().fp8_moe_route_workspace_bytes(int(T), int(E)))


def _logits(t, name):
    """[T, E] float32 or bfloat16 rows with unit stride: pointer, type, row stride."""
    _want(t, (torch.float32, torch.bfloat16), name, contiguous=False, required=True)
    if t.dim() != 2:
        raise ValueError(f"{name} must be [T, E]")
    if t.numel() and t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} rows must be contiguous")
    return t.data_ptr() if t.is_cuda else _HOST, _out_dtype(t), t.stride(0) if t.shape[0] > 1 else t.shape[1]


def fp8_moe_route(logits, experts, weights, lse, counts, prob_sum, loss, workspace=None, normalise: bool = True, stream=None):
    """The choice of experts from the router's ``logits`` [T, E] (float32 or bfloat16, rows with unit stride):
    ``experts`` [T, top] int32 as fp8_moe_plan reads them, ``weights`` [T, top], ``lse`` [T], ``counts`` [E + 1] int32,
    ``prob_sum`` [E] and the balance ``loss`` [1] (see include/fp8ds.h)."""
    if _tls.rec is None and (_calls or _native()).moe_route(logits, experts, weights, lse, counts, prob_sum, loss, workspace,
                                                            normalise, stream):
        return
    p_l, dtype, ld = _logits(logits, "logits")
    _want(experts, _I32, "experts", required=True)
    if experts.dim() != 2:
        raise ValueError("experts must be [T, top]")
    (T, E), top = logits.shape, experts.shape[1]
    ws_bytes = _workspace_bytes(workspace)
    _invoke("fp8_moe_route", p_l, dtype, ld, T, E, top, int(bool(normalise)), _arg(experts, _I32, (T, top), "experts"),
            _arg(weights, _F32, (T, top), "weights", True), _arg(lse, _F32, (T,), "lse", True),
            _arg(counts, _I32, (E + 1,), "counts", True), _arg(prob_sum, _F32, (E,), "prob_sum", True),
            _some(loss, _F32, 1, "loss"), _ptr(workspace), ws_bytes, _stream(stream))


def fp8_moe_route_bwd(logits, experts, weights, lse, counts, dweights, dloss, dlogits, normalise: bool = True, stream=None):
    """Gradient of fp8_moe_route: ``dlogits`` (as ``logits``) from ``dweights`` [T, top] and ``dloss`` [1], either of
    which may be None; experts, weights, lse, counts: what the forward wrote."""
    if _tls.rec is None and (_calls or _native()).moe_route_bwd(logits, experts, weights, lse, counts, dweights, dloss,
                                                                dlogits, normalise, stream):
        return
    p_l, dtype, ld = _logits(logits, "logits")
    p_d, dtype_d, ld_d = _logits(dlogits, "dlogits")
    if dtype != dtype_d or logits.shape != dlogits.shape:
        raise ValueError("dlogits must have the type and shape of logits")
    _want(experts, _I32, "experts", required=True)
    if experts.dim() != 2:
        raise ValueError("experts must be [T, top]")
    (T, E), top = logits.shape, experts.shape[1]
    _invoke("fp8_moe_route_bwd", p_l, dtype, ld, T, E, top, int(bool(normalise)), _arg(experts, _I32, (T, top), "experts"),
            _arg(weights, _F32, (T, top), "weights", True), _arg(lse, _F32, (T,), "lse", True),
            _arg(counts, _I32, (E + 1,), "counts", True), _arg(dweights, _F32, (T, top), "dweights"),
            _some(dloss, _F32, 1, "dloss"), p_d, ld_d, _stream(stream))
