"""ctypes binding of include/dspark_head.h (argument marshalling only): the
drafter head's loss and gradient.

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
from .dspark import _F, _I32, _I64, _P, _SZ, _check, _nbytes, _ptr, _stream, new_workspace

HEADER = os.path.join(os.path.dirname(_d.HERE), "include", "dspark_head.h")

_SIGS = {
    "dspark_head_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32]),
    "dspark_head_loss": (_I32, [_P, _I64, _P, _P, _P, _P, _P, _I32, _I32, _I32,
                                _I32, _P, _P, _P, _SZ, _P]),
    "dspark_head_loss_grad": (_I32, [_P, _I64, _P, _P, _P, _P, _P, _P, _P, _I32,
                                     _I32, _I32, _I32, _P, _I64, _P, _P, _P, _P,
                                     _SZ, _P]),
}

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
