"""Products grouped by expert, their weight gradient, and the 8-bit product
(include/grouped_gemm.h; argument marshalling only).

A layer of experts sorts its rows by expert and describes the sorting by
``offsets``, an int32 GPU tensor of E + 1 row numbers: expert e owns the rows
``offsets[e]:offsets[e + 1]``.  The offsets are read on the GPU, so no call waits
for a router's counts.  Every call writes its output tensor in place, is
asynchronous on ``stream`` (default: torch's current stream) and returns the
output.
"""
from __future__ import annotations

import ctypes

import torch

from .binding import _f32, _i32, _i64, _lib, _stream_handle, _vp

_SIGS = {
    "gemm_grouped": ([_i32, _i32, _i32, _i32, _vp, _i64, _i64, _i64, _f32, _vp, _i64, _vp, _i64, _i64,
                      _f32, _vp, _i64, _vp], ctypes.c_int),
    "gemm_grouped_wgrad": ([_i32, _i32, _i32, _vp, _i64, _i64, _i64, _f32, _vp, _i64, _vp, _i64, _f32,
                            _vp, _i64, _i64, _vp], ctypes.c_int),
    "quantize_rows": ([_i32, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp], ctypes.c_int),
    "igemm": ([_i32, _i32, _vp, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _i64,
               _vp], ctypes.c_int),
    "gemm_grouped_plan": ([_i32, _i32, _i32, _i32, _i64, _i64, _i64, ctypes.POINTER(_i32)], _i64),
    "gemm_grouped_status_string": ([ctypes.c_int], ctypes.c_char_p),
}
for _name, (_args, _res) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res

_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_INT8 = {torch.int8: 3}
_FORMS = {"nt": 0, "nn": 1, "tn": 2}


class GroupedGemmError(RuntimeError):
    def __init__(self, call: str, status: int):
        self.status = status
        msg = _lib.gemm_grouped_status_string(status).decode()
        if status == 4:
            msg += f" (hipError_t {_lib.sgemm_last_hip_error()})"
        super().__init__(f"{call} status {status}: {msg}")


def exported_symbols():
    """Names declared in include/grouped_gemm.h that the library must export."""
    return sorted(_SIGS)


def plan(form: str, dtype, groups: int, M: int, N: int, K: int, out=None) -> dict:
    """The tile and workgroups of a product; form "nt", "nn" or "tn" as the
    kernels see it (transposed weights, plain weights, weight gradient); out is
    the output's type (default: the operands', bfloat16 for int8)."""
    tile = (_i32 * 2)()
    out = out or (torch.bfloat16 if dtype is torch.int8 else dtype)
    grid = _lib.gemm_grouped_plan(_FORMS[form], {**_TYPES, **_INT8}[dtype], _TYPES[out], groups, M, N, K, tile)
    if grid < 0:
        raise ValueError("bad arguments")
    return {"BM": tile[0], "BN": tile[1], "grid": grid}


def _matrix(t, name, types, dev):
    """(type code, leading dimension) of a 2-D tensor with unit column stride
    on GPU `dev` (any GPU when None); raises on anything else."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = types.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be one of {[str(d) for d in types]}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU device")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} is on another device")
    rows, cols = t.shape
    s0, s1 = t.stride()
    if cols > 1 and s1 != 1:
        raise ValueError(f"{name} must have unit column stride (row-major)")
    if rows > 1:
        if s0 < cols:
            raise ValueError(f"{name}: rows overlap (row stride {s0} < {cols} columns)")
        return code, s0 if s0 > 1 else 1
    return code, cols if cols > 1 else 1


def _stack(t, name, types, dev, grouped):
    """(type code, leading dimension, group stride, groups, rows, columns) of a
    stack of matrices: 3-D when grouped, 2-D otherwise."""
    if not grouped:
        code, ld = _matrix(t, name, types, dev)
        return (code, ld, 0, 1, *t.shape)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D (experts, rows, columns) when offsets are given")
    groups, rows, cols = t.shape
    if groups == 0:
        raise ValueError(f"{name} holds no expert")
    code, ld = _matrix(t[0], name, types, dev)
    return code, ld, t.stride(0) if groups > 1 else 0, groups, rows, cols


def _offsets(offsets, groups, dev):
    """Pointer of the group offsets (None: one group of all rows)."""
    if offsets is None:
        return None
    if not isinstance(offsets, torch.Tensor) or offsets.dtype is not torch.int32:
        raise TypeError("offsets must be an int32 torch.Tensor")
    if offsets.dim() != 1 or offsets.numel() != groups + 1 or (offsets.stride(0) != 1):
        raise ValueError(f"offsets must be {groups + 1} consecutive row numbers for {groups} experts")
    if offsets.get_device() != dev or not offsets.is_cuda:
        raise ValueError("offsets must be on the operands' device")
    return offsets.data_ptr()


def _call(name, dev, *args):
    fn = getattr(_lib, name)
    if dev == torch.cuda.current_device():
        rc = fn(*args)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args)
    if rc != 0:
        raise GroupedGemmError(name, rc)


def _out_type(code, out, name):
    if out != code and out != 0:
        raise TypeError(f"{name} must have the operands' type or be float32")


def gemm_grouped(X, W, offsets, Y, alpha=1.0, beta=0.0, transpose_w=False, stream=None):
    """Y[r] <- alpha * X[r] @ W[e] + beta * Y[r] for every row r of every expert e.

    X is M x K, W is E x K x N (E x N x K with ``transpose_w``, which is also the
    input gradient dX = dY @ W[e].T), Y is M x N; float32, bfloat16 or float16,
    Y of the operands' type or float32.  Sums are float32.  With ``offsets``
    None, W is one 2-D matrix.  Rows of Y that no expert owns keep their values.
    """
    code, ldx = _matrix(X, "X", _TYPES, None)
    dev = X.get_device()
    wcode, ldw, stride, groups, rows, cols = _stack(W, "W", _TYPES, dev, offsets is not None)
    out, ldy = _matrix(Y, "Y", _TYPES, dev)
    M, K = X.shape
    K2, N = (cols, rows) if transpose_w else (rows, cols)
    if wcode != code:
        raise TypeError("X and W must have the same type")
    _out_type(code, out, "Y")
    if K2 != K or tuple(Y.shape) != (M, N):
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}, Y {tuple(Y.shape)}")
    _call("gemm_grouped", dev, code, out, 1 if transpose_w else 0, groups, _offsets(offsets, groups, dev),
          M, N, K, alpha, X.data_ptr(), ldx, W.data_ptr(), ldw, stride, beta, Y.data_ptr(), ldy,
          _stream_handle(X.device, stream))
    return Y


def gemm_grouped_wgrad(X, dY, offsets, dW, alpha=1.0, beta=0.0, stream=None):
    """dW[e] <- alpha * X[rows of e].T @ dY[rows of e] + beta * dW[e] for every expert e.

    X is M x K, dY is M x N, dW is E x K x N (2-D with ``offsets`` None), of the
    operands' type or float32; sums are float32.  For weights stored N x K pass
    dY and X in each other's place.  An expert without rows gets beta * dW[e].
    """
    code, ldx = _matrix(X, "X", _TYPES, None)
    dev = X.get_device()
    ycode, lddy = _matrix(dY, "dY", _TYPES, dev)
    out, lddw, stride, groups, K2, N2 = _stack(dW, "dW", _TYPES, dev, offsets is not None)
    M, K = X.shape
    M2, N = dY.shape
    if ycode != code:
        raise TypeError("X and dY must have the same type")
    _out_type(code, out, "dW")
    if M2 != M or K2 != K or N2 != N:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, dY {tuple(dY.shape)}, dW {tuple(dW.shape)}")
    _call("gemm_grouped_wgrad", dev, code, out, groups, _offsets(offsets, groups, dev), M, N, K, alpha,
          X.data_ptr(), ldx, dY.data_ptr(), lddy, beta, dW.data_ptr(), lddw, stride,
          _stream_handle(X.device, stream))
    return dW


def _scales(t, name, shape, dev):
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32:
        raise TypeError(f"{name} must be a float32 torch.Tensor")
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous with shape {shape}, got {tuple(t.shape)}")
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name} must be on the operands' device")
    return t.data_ptr()


def quantize_rows(X, Q, scale, stream=None):
    """Bring every row of X (M x K) to 8 bits: scale[r] = max|X[r]| / 127 and Q[r]
    the nearest integers to 127 * X[r] / max|X[r]|, ties to even.

    A row of zeros gets scale 0, a row that holds an infinity or NaN scale NaN
    and codes 0.  Weights are brought to 8 bits by the same call, a channel a
    row.  Returns (Q, scale).
    """
    code, ldx = _matrix(X, "X", _TYPES, None)
    dev = X.get_device()
    _, ldq = _matrix(Q, "Q", _INT8, dev)
    M, K = X.shape
    if tuple(Q.shape) != (M, K):
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, Q {tuple(Q.shape)}")
    _call("quantize_rows", dev, code, M, K, X.data_ptr(), ldx, Q.data_ptr(), ldq,
          _scales(scale, "scale", (M,), dev), _stream_handle(X.device, stream))
    return Q, scale


def igemm(A, scale_a, B, scale_b, C, bias=None, offsets=None, stream=None):
    """C[r, n] <- (A[r] . B[e, n]) * scale_a[r] * scale_b[e, n] + bias[e, n].

    A is M x K and B is N x K (E x N x K with ``offsets``), both int8, as
    :func:`quantize_rows` writes them; scale_b and bias are N (E x N).  Sums are
    exact 32-bit integers.  C is float32, bfloat16 or float16.
    """
    grouped = offsets is not None
    _, lda = _matrix(A, "A", _INT8, None)
    dev = A.get_device()
    _, ldb, stride, groups, N, K2 = _stack(B, "B", _INT8, dev, grouped)
    out, ldc = _matrix(C, "C", _TYPES, dev)
    M, K = A.shape
    if K2 != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shape mismatch: A {tuple(A.shape)}, B {tuple(B.shape)}, C {tuple(C.shape)}")
    per = (groups, N) if grouped else (N,)
    _call("igemm", dev, out, groups, _offsets(offsets, groups, dev), M, N, K, A.data_ptr(), lda,
          _scales(scale_a, "scale_a", (M,), dev), B.data_ptr(), ldb, stride,
          _scales(scale_b, "scale_b", per, dev),
          None if bias is None else _scales(bias, "bias", per, dev), C.data_ptr(), ldc,
          _stream_handle(A.device, stream))
    return C
