"""Products grouped by expert, their weight gradient, and the 8-bit product
(include/grouped_gemm.h).  csrc/torch_calls.cpp checks and marshals the tensors.

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

from .binding import _f32, _i32, _i64, _lib, _vp


class _Missing:
    """In place of the module where it cannot be loaded: any call says why."""

    def __init__(self, error):
        self._why = f"{error}; run `python -m fp32_gemm_amd.build`"

    def __getattr__(self, name):
        raise ImportError(f"{name}: {self._why}")


try:
    from . import _torch_calls  # after the library, which it links to
except ImportError as error:
    _torch_calls = _Missing(error)

_SIGS = {
    "gemm_grouped": ([_i32, _i32, _i32, _i32, _vp, _i64, _i64, _i64, _f32, _vp, _i64, _vp, _i64, _i64,
                      _f32, _vp, _i64, _vp], ctypes.c_int),
    "gemm_grouped_wgrad": ([_i32, _i32, _i32, _vp, _i64, _i64, _i64, _f32, _vp, _i64, _vp, _i64, _f32,
                            _vp, _i64, _i64, _vp], ctypes.c_int),
    "quantize_rows": ([_i32, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp], ctypes.c_int),
    "igemm": ([_i32, _i32, _vp, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _i64,
               _vp], ctypes.c_int),
    "gemm_grouped_plan": ([_i32, _i32, _i32, _i32, _i64, _i64, _i64, ctypes.POINTER(_i32)], _i64),
    "gemm_grouped_tile": ([_i32, _i32, _i32, _i32, _i64, _i64, _i64], _i32),
    "gemm_grouped_tiles": ([_i32, _i32], _i32),
    "gemm_grouped_tile_order": ([_i32, _i32, _i32, _i32, _vp, _i64, _i64, _i64, _i64, _i64, _vp], _i64),
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


TILES = ("256x256", "128x128", "128x128 deep", "64x64", "16x32", "16x16")


def plan(form: str, dtype, groups: int, M: int, N: int, K: int, out=None) -> dict:
    """The tile and workgroups of a product; form "nt", "nn" or "tn" as the
    kernels see it (transposed weights, plain weights, weight gradient); out is
    the output's type (default: the operands', bfloat16 for int8)."""
    tile = (_i32 * 2)()
    out = out or (torch.bfloat16 if dtype is torch.int8 else dtype)
    args = (_FORMS[form], {**_TYPES, **_INT8}[dtype], _TYPES[out], groups, M, N, K)
    grid = _lib.gemm_grouped_plan(*args, tile)
    if grid < 0:
        raise ValueError("bad arguments")
    return {"BM": tile[0], "BN": tile[1], "grid": grid, "tile": TILES[_lib.gemm_grouped_tile(*args)]}


def tiles(form: str, dtype) -> list:
    """The tiles that a form and type can run with."""
    bits = _lib.gemm_grouped_tiles(_FORMS[form], {**_TYPES, **_INT8}[dtype])
    if bits < 0:
        raise ValueError("bad arguments")
    return [name for i, name in enumerate(TILES) if bits >> i & 1]


def tile_order(form: str, dtype, tile: str, offsets, M: int, N: int, K: int, first=0, count=None) -> list:
    """(group, first row, end of the group's rows, column) of each workgroup's
    tile, group -1 where it has none; offsets is a list, or None for one group of
    M rows.  For weight gradients the first row is the row tile and the end 0."""
    at = None if offsets is None else (_i32 * len(offsets))(*offsets)
    groups = 1 if offsets is None else len(offsets) - 1
    args = (_FORMS[form], {**_TYPES, **_INT8}[dtype], TILES.index(tile), groups, at, M, N, K, first)
    n = _lib.gemm_grouped_tile_order(*args, 0, None)
    if n < 0:
        raise ValueError("bad arguments")
    count = max(0, n - first) if count is None else min(count, max(0, n - first))
    order = (_i32 * (4 * count))()
    _lib.gemm_grouped_tile_order(*args, count, order)
    return [tuple(order[4 * i:4 * i + 4]) for i in range(count)]


def gemm_grouped(X, W, offsets, Y, alpha=1.0, beta=0.0, transpose_w=False, stream=None):
    """Y[r] <- alpha * X[r] @ W[e] + beta * Y[r] for every row r of every expert e.

    X is M x K, W is E x K x N (E x N x K with ``transpose_w``, which is also the
    input gradient dX = dY @ W[e].T), Y is M x N; float32, bfloat16 or float16,
    Y of the operands' type or float32.  Sums are float32.  With ``offsets``
    None, W is one 2-D matrix.  Rows of Y that no expert owns keep their values.
    """
    status = _torch_calls.gemm_grouped(X, W, offsets, Y, alpha, beta, transpose_w, stream)
    if status:
        raise GroupedGemmError("gemm_grouped", status)
    return Y


def gemm_grouped_wgrad(X, dY, offsets, dW, alpha=1.0, beta=0.0, stream=None):
    """dW[e] <- alpha * X[rows of e].T @ dY[rows of e] + beta * dW[e] for every expert e.

    X is M x K, dY is M x N, dW is E x K x N (2-D with ``offsets`` None), of the
    operands' type or float32; sums are float32.  For weights stored N x K pass
    dY and X in each other's place.  An expert without rows gets beta * dW[e].
    """
    status = _torch_calls.gemm_grouped_wgrad(X, dY, offsets, dW, alpha, beta, stream)
    if status:
        raise GroupedGemmError("gemm_grouped_wgrad", status)
    return dW


def quantize_rows(X, Q, scale, stream=None):
    """Bring every row of X (M x K) to 8 bits: scale[r] = max|X[r]| / 127 and Q[r]
    the nearest integers to 127 * X[r] / max|X[r]|, ties to even.

    A row of zeros gets scale 0, a row that holds an infinity or NaN scale NaN
    and codes 0.  Weights are brought to 8 bits by the same call, a channel a
    row.  Returns (Q, scale).
    """
    status = _torch_calls.quantize_rows(X, Q, scale, stream)
    if status:
        raise GroupedGemmError("quantize_rows", status)
    return Q, scale


def igemm(A, scale_a, B, scale_b, C, bias=None, offsets=None, stream=None):
    """C[r, n] <- (A[r] . B[e, n]) * scale_a[r] * scale_b[e, n] + bias[e, n].

    A is M x K and B is N x K (E x N x K with ``offsets``), both int8, as
    :func:`quantize_rows` writes them; scale_b and bias are N (E x N).  Sums are
    exact 32-bit integers.  C is float32, bfloat16 or float16.
    """
    status = _torch_calls.igemm(A, scale_a, B, scale_b, C, bias, offsets, stream)
    if status:
        raise GroupedGemmError("igemm", status)
    return C
