"""The norm in front of a layer's products, with its gradient, and a whole layer of
experts for a few tokens (include/layer_ops.h).  csrc/torch_calls.cpp checks and
marshals the tensors.

Every call writes its output tensors in place, is asynchronous on ``stream``
(default: torch's current stream) and returns what it wrote.  Where a call needs a
workspace and none is given, it takes one from torch for the length of the call.
"""
from __future__ import annotations

import ctypes

from .binding import _f32, _i32, _i64, _lib, _vp
from .grouped import _torch_calls

_SIGS = {
    "rms_norm": ([_i32, _i32, _i32, _i64, _i64, _f32, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp,
                  _vp], ctypes.c_int),
    "rms_norm_grad": ([_i32, _i32, _i32, _i64, _i64, _f32, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _vp,
                       _i64, _vp], ctypes.c_int),
    "rms_norm_grad_workspace": ([_i64, _i64], _i64),
    "expert_layer": ([_i32, _i32, _i32, _i32, _i64, _i64, _i64, _i32, _i32, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _vp,
                      _vp, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _vp], ctypes.c_int),
    "expert_layer_workspace": ([_i32, _i64, _i64, _i64, _i32], _i64),
    "layer_status_string": ([ctypes.c_int], ctypes.c_char_p),
}
for _name, (_args, _res) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res


class LayerError(RuntimeError):
    def __init__(self, call: str, status: int):
        self.status = status
        msg = _lib.layer_status_string(status).decode()
        if status == 4:
            msg += f" (hipError_t {_lib.sgemm_last_hip_error()})"
        super().__init__(f"{call} status {status}: {msg}")


def exported_symbols():
    """Names declared in include/layer_ops.h that the library must export."""
    return sorted(_SIGS)


def rms_norm(X, weight, Y=None, residual=None, H=None, Q=None, scale=None, eps=1e-6, stream=None):
    """H <- X + residual, Y <- H / sqrt(mean(H ** 2) + eps) * weight, row by row, and
    (Q, scale) <- Y in 8 bits as :func:`quantize_rows` would bring it there.

    X, residual and H are M x K, float32, bfloat16 or float16; Y has their type or is
    float32, and so has weight (K values; None: ones).  Q is int8, scale float32.
    Y, H, and Q with scale are each written if given, Y and Q from the sum before it is
    rounded to H.  H may be X or residual itself.  Returns Y, or (Q, scale) without Y.
    """
    status = _torch_calls.rms_norm(X, weight, Y, residual, H, Q, scale, eps, stream)
    if status:
        raise LayerError("rms_norm", status)
    return (Q, scale) if Y is None else Y


def rms_norm_grad(dY, X, weight, dX, dweight=None, residual_grad=None, eps=1e-6, workspace=None, stream=None):
    """The gradient of :func:`rms_norm` where X (M x K) is what was normed, its H.

    dX gets the gradient of X, with residual_grad, what reaches X by other ways, added
    if given; it may be dY or residual_grad itself.  dweight gets the weight's gradient
    (K values of X's type or float32), summed in float32 in a fixed order.  workspace:
    uint8, ``layers.rms_norm_grad_workspace(M, K)`` bytes.  Returns (dX, dweight).
    """
    status = _torch_calls.rms_norm_grad(dY, X, weight, dX, dweight, residual_grad, eps, workspace, stream)
    if status:
        raise LayerError("rms_norm_grad", status)
    return dX, dweight


def rms_norm_grad_workspace(M: int, K: int) -> int:
    """Bytes of the workspace that :func:`rms_norm_grad` needs for a weight's gradient."""
    need = _lib.rms_norm_grad_workspace(M, K)
    if need < 0:
        raise ValueError("bad arguments")
    return need


def expert_layer(X, ids, share, W_in, W_out, Y, scale_in=None, scale_out=None, gated=True, workspace=None,
                 stream=None):
    """Y[t] <- sum over j of share[t, j] * W_out[e] @ h, e = ids[t, j], for up to 64 tokens
    (and 512 choices in all), in two kernels that read each named expert's weights once for each
    16 of its tokens.

    h = silu(u[:F]) * u[F:] with u = W_in[e] @ X[t] and W_in E x 2F x D, or, without
    ``gated``, h = silu(u) and W_in E x F x D; W_out is E x D x F.  h is held in 32 bits.
    X is T x D, float32, bfloat16 or float16, Y T x D of its type or float32.  ids (int32)
    and share (float32) are T x top; an id that is no expert's counts for nothing.  The
    weights have X's type, or are int8 with float32 scales E x rows as
    :func:`quantize_rows` writes them, or uint8 with scales as :func:`quantize_mx4` writes
    them.  workspace: uint8, ``layers.expert_layer_workspace(X, ids, F)`` bytes.
    """
    status = _torch_calls.expert_layer(X, ids, share, W_in, W_out, Y, scale_in, scale_out, gated, workspace, stream)
    if status:
        raise LayerError("expert_layer", status)
    return Y


def expert_layer_workspace(X, ids, F: int) -> int:
    """Bytes of the workspace that :func:`expert_layer` needs with a hidden width of F."""
    from .grouped import _TYPES
    need = _lib.expert_layer_workspace(_TYPES[X.dtype], X.shape[0], X.shape[1], F, ids.shape[1])
    if need < 0:
        raise ValueError("bad arguments")
    return need
