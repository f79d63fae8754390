"""ctypes binding of include/dspark_head.h (argument marshalling only): the
drafter head's loss and gradient, the residual stream's norm and dropout.

As in ``dspark``: every function has the name of the C entry point it calls
and passes ``torch`` tensors as raw device pointers with the current CUDA
stream; there is no CPU or PyTorch fallback.  Shapes, types and layouts that
the C call cannot see from a pointer are checked here (``ValueError``).
"""
from __future__ import annotations

import ctypes
import os
import re

from . import dspark as _d
from .dspark import (BF16, F32, _F, _I32, _I64, _P, _SZ, _U32, _check, _nbytes,
                     _ptr, _stream, new_workspace)

HEADER = os.path.join(os.path.dirname(_d.HERE), "include", "dspark_head.h")

_SIGS = {
    "dspark_head_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32]),
    "dspark_head_loss": (_I32, [_P, _I64, _P, _P, _P, _P, _P, _I32, _I32, _I32,
                                _I32, _P, _P, _P, _SZ, _P]),
    "dspark_head_loss_grad": (_I32, [_P, _I64, _P, _P, _P, _P, _P, _P, _P, _I32,
                                     _I32, _I32, _I32, _P, _I64, _P, _P, _P, _P,
                                     _SZ, _P]),
    "dspark_residual_norm": (_I32, [_P, _I64, _P, _I64, _P, _I32, _I32, _I32, _F,
                                    _F, ctypes.c_uint64, _U32, _P, _I64, _P, _I64,
                                    _I32, _I32, _P, _P, _P]),
    "dspark_norm_workspace_size": (_SZ, [_I32, _I32]),
    "dspark_residual_norm_grad": (_I32, [_P, _I64, _P, _I64, _P, _I64, _P, _P,
                                         _I32, _I32, _I32, _F, ctypes.c_uint64,
                                         _U32, _P, _I64, _P, _I64, _P, _P, _SZ,
                                         _P]),
    "dspark_dropout": (_I32, [_P, _I64, _P, _I64, _I32, _I32, _I32, _F,
                              ctypes.c_uint64, _U32, _P, _I64, _P]),
}

E4M3 = 2

__all__ = sorted(_SIGS) + ["new_workspace"]

_lib = None


def header_functions() -> list[str]:
    """Names of the entry points declared in include/dspark_head.h."""
    with open(HEADER) as f:
        txt = f.read()
    return sorted(set(re.findall(r"DSPARK_API\s+[\w\s\*]+?\b(dspark_\w+)\s*\(", txt)))


def load() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = _d.load()
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _want(name, t, shape, dtype, rows_strided=False):
    """t is a tensor of this shape and type, contiguous (or, where rows may
    be apart, with contiguous rows)."""
    if t is None:
        raise ValueError(f"{name} is required")
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{name} must be {tuple(shape)} {dtype}, got "
                         f"{tuple(t.shape)} {t.dtype}")
    ok = t.stride(-1) == 1 or t.shape[-1] == 1 if rows_strided else t.is_contiguous()
    if not ok:
        raise ValueError(f"{name} must be contiguous" + (" along its rows" if rows_strided else ""))


def _row_stride(t):
    # the stride of a dimension with one entry means nothing
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


# ------------------------------------------------------------------- loss
def dspark_head_workspace_size(M: int, vocab: int, d: int, rank: int, grad: bool) -> int:
    return int(load().dspark_head_workspace_size(M, vocab, d, rank, int(bool(grad))))


def _head_dims(h, W, U, V, prev, target):
    import torch
    if h.dim() != 2 or W.dim() != 2:
        raise ValueError("h and W must be 2-D")
    (M, d), vocab = h.shape, W.shape[0]
    rank = 0 if V is None else V.shape[1]
    _want("h", h, (M, d), torch.bfloat16, rows_strided=True)
    _want("W", W, (vocab, d), torch.bfloat16)
    if rank:
        _want("U", U, (vocab, rank), torch.bfloat16)
        _want("V", V, (vocab, rank), torch.bfloat16)
        _want("prev", prev, (M,), torch.int32)
    _want("target", target, (M,), torch.int32)
    return M, vocab, d, rank


def dspark_head_loss(h, W, U, V, prev, target, loss, lse, workspace, *,
                     stream=None, raise_on_error=True) -> int:
    """h [M, d] bf16 (rows may be apart), W [vocab, d] bf16, U/V [vocab, rank]
    bf16 or None, prev/target [M] int32 (target < 0: ignored), loss/lse [M]
    fp32 (out), workspace of dspark_head_workspace_size bytes."""
    import torch
    M, vocab, d, rank = _head_dims(h, W, U, V, prev, target)
    _want("loss", loss, (M,), torch.float32)
    _want("lse", lse, (M,), torch.float32)
    code = load().dspark_head_loss(
        _ptr(h), _row_stride(h), _ptr(W), _ptr(U), _ptr(V), _ptr(prev),
        _ptr(target), M, vocab, d, rank, _ptr(loss), _ptr(lse),
        _ptr(workspace), _nbytes(workspace), _stream(stream))
    return _check("dspark_head_loss", code, raise_on_error)


def dspark_head_loss_grad(h, W, U, V, prev, target, lse, dloss, dh, dW, dU, dV,
                          workspace, *, stream=None, raise_on_error=True) -> int:
    """Gradients of sum_i dloss_i loss_i: dh [M, d] (rows may be apart), dW
    [vocab, d], dU/dV [vocab, rank] or None, all bf16 and written in full; lse
    [M] as written by dspark_head_loss, dloss [M] fp32."""
    import torch
    M, vocab, d, rank = _head_dims(h, W, U, V, prev, target)
    _want("lse", lse, (M,), torch.float32)
    _want("dloss", dloss, (M,), torch.float32)
    _want("dh", dh, (M, d), torch.bfloat16, rows_strided=True)
    _want("dW", dW, (vocab, d), torch.bfloat16)
    if rank:
        _want("dU", dU, (vocab, rank), torch.bfloat16)
        _want("dV", dV, (vocab, rank), torch.bfloat16)
    code = load().dspark_head_loss_grad(
        _ptr(h), _row_stride(h), _ptr(W), _ptr(U), _ptr(V), _ptr(prev),
        _ptr(target), _ptr(lse), _ptr(dloss), M, vocab, d, rank, _ptr(dh),
        _row_stride(dh), _ptr(dW), _ptr(dU), _ptr(dV), _ptr(workspace),
        _nbytes(workspace), _stream(stream))
    return _check("dspark_head_loss_grad", code, raise_on_error)


# -------------------------------------------------------- residual stream
def _dtype(name, t):
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _rows(name, t, like, required=False):
    """(pointer, row stride) of a [M, d] tensor of like's type, or of None."""
    if t is None and not required:
        return None, 0
    _want(name, t, like.shape, like.dtype, rows_strided=True)
    return _ptr(t), _row_stride(t)


def _matrix(name, t):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    return t.shape


def dspark_residual_norm(x, residual, gain, r, y, scale=None, rstd=None, *, eps,
                         group=0, p=0.0, seed=0, offset=0, stream=None,
                         raise_on_error=True) -> int:
    """r = residual + dropout(x), y = r / rms(r) * gain.  x, residual (or None)
    and r (or None) [M, d] bf16 or fp32 (rows may be apart), gain [d]; y of the
    same type, or float8_e4m3fn with scale [M, 1] (group 0) or [M, ceil(d /
    128)] (group 128) fp32; rstd [M] fp32 or None."""
    import torch
    M, d = _matrix("x", x)
    dt = _dtype("x", x)
    px, sx = _rows("x", x, x)
    pres, sres = _rows("residual", residual, x)
    pr, sr = _rows("r", r, x)
    _want("gain", gain, (d,), x.dtype)
    if rstd is not None:
        _want("rstd", rstd, (M,), torch.float32)
    ydt = dt
    if y is not None and y.dtype == torch.float8_e4m3fn:
        ydt = E4M3
        _want("y", y, (M, d), y.dtype, rows_strided=True)
        n = -(-d // group) if group > 0 else 1
        if scale is None or scale.dim() != 2:
            raise ValueError("scale must be 2-D with an 8-bit y")
        _want("scale", scale, (M, n), torch.float32)
    else:
        _rows("y", y, x, required=True)
    code = load().dspark_residual_norm(
        px, sx, pres, sres, _ptr(gain), dt, M, d, float(eps), float(p), int(seed),
        int(offset), pr, sr, _ptr(y), _row_stride(y), ydt, int(group), _ptr(scale),
        _ptr(rstd), _stream(stream))
    return _check("dspark_residual_norm", code, raise_on_error)


def dspark_norm_workspace_size(M: int, d: int) -> int:
    return int(load().dspark_norm_workspace_size(M, d))


def dspark_residual_norm_grad(dy, dr, r, gain, rstd, dx, dresidual, dgain, workspace,
                              *, p=0.0, seed=0, offset=0, stream=None,
                              raise_on_error=True) -> int:
    """dr' = dr + the norm's gradient of dy; dresidual = dr', dx =
    dropout(dr'), dgain = the gain's gradient.  dr, dx, dresidual and dgain may
    be None; everything of r's type but rstd [M] fp32 (as written by
    dspark_residual_norm)."""
    import torch
    M, d = _matrix("r", r)
    dt = _dtype("r", r)
    pdy, sdy = _rows("dy", dy, r, required=True)
    pdr, sdr = _rows("dr", dr, r)
    pr, sr = _rows("r", r, r)
    pdx, sdx = _rows("dx", dx, r)
    pds, sds = _rows("dresidual", dresidual, r)
    _want("gain", gain, (d,), r.dtype)
    _want("rstd", rstd, (M,), torch.float32)
    if dgain is not None:
        _want("dgain", dgain, (d,), r.dtype)
    code = load().dspark_residual_norm_grad(
        pdy, sdy, pdr, sdr, pr, sr, _ptr(gain), _ptr(rstd), dt, M, d, float(p),
        int(seed), int(offset), pdx, sdx, pds, sds, _ptr(dgain), _ptr(workspace),
        _nbytes(workspace), _stream(stream))
    return _check("dspark_residual_norm_grad", code, raise_on_error)


def dspark_dropout(x, residual, y, *, p, seed, offset, stream=None,
                   raise_on_error=True) -> int:
    """y = residual + dropout(x) ([M, d] bf16 or fp32; residual may be None);
    seed (uint64) and offset (uint32) as in include/dspark_head.h."""
    M, d = _matrix("x", x)
    dt = _dtype("x", x)
    px, sx = _rows("x", x, x)
    pres, sres = _rows("residual", residual, x)
    py, sy = _rows("y", y, x, required=True)
    code = load().dspark_dropout(px, sx, pres, sres, dt, M, d, float(p), int(seed),
                                 int(offset), py, sy, _stream(stream))
    return _check("dspark_dropout", code, raise_on_error)
