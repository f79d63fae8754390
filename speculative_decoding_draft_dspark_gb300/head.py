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

import torch

from . import dspark as _d
from .dspark import (BF16, F32, DsparkError, _F, _I32, _I64, _P, _SZ, _U32, _nbytes,
                     new_workspace)

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
_device_now = torch._C._cuda_getDevice


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


def _place(name, t):
    """The GPU of a call's first tensor: the current one, whose stream it takes."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be on the GPU")
    if dev != _device_now():
        raise ValueError(f"{name} must be on the current GPU ({_device_now()}), not GPU {dev}")
    return dev


def _refuse(name, t, shape, dtype, dev):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.get_device() < 0:
        raise ValueError(f"{name} must be on the GPU")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on GPU {dev} as the others, not GPU {t.get_device()}")
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{name} must be {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")
    raise ValueError(f"{name} must be contiguous (a matrix: along its rows)")


def _flat(name, t, shape, dtype, dev):
    """Pointer of a contiguous tensor of this shape and type."""
    if (t is None or t.dtype is not dtype or t.shape != shape or not t.is_contiguous()
            or t.get_device() != dev):
        _refuse(name, t, shape, dtype, dev)
    return t.data_ptr()


def _rows(name, t, shape, dtype, dev):
    """(pointer, row stride) of a matrix of this shape and type whose rows are
    contiguous; (None, 0) for None."""
    if t is None:
        return None, 0
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _refuse(name, t, shape, dtype, dev)
    s, one = t.stride()
    if one != 1 and shape[1] > 1:
        _refuse(name, t, shape, dtype, dev)
    # the stride of a dimension with one entry means nothing
    return t.data_ptr(), s if shape[0] > 1 else shape[1]


def _space(workspace, dev):
    """(pointer, bytes) of a workspace."""
    if workspace is None or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on GPU {dev}")
    return workspace.data_ptr(), _nbytes(workspace)


_I32_MAX = (1 << 31) - 1


def _matrix(name, t):
    if t is None or t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, columns = shape = t.shape
    if rows > _I32_MAX or columns > _I32_MAX:
        raise ValueError(f"{name}'s rows and columns must be below 2^31, got {tuple(shape)}")
    return shape


def _whole(name, value, bits):
    """A whole number of so many bits; more would be cut off on the way to C."""
    if not 0 <= value < 1 << bits:
        raise ValueError(f"{name} must be in [0, 2^{bits}), got {value}")
    return value


def _mask(seed, offset):
    return _whole("seed", seed, 64), _whole("offset", offset, 32)


_TYPES = {torch.bfloat16: BF16, torch.float32: F32}


def _dtype(name, t):
    dt = _TYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return dt


def _stream(stream):
    # the current stream's handle without the Stream object around it: the
    # object costs as long as a small call's kernel
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(_device_now())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _done(name, code, raise_on_error):
    if code and raise_on_error:
        raise DsparkError(name, code)
    return code


# ------------------------------------------------------------------- loss
def dspark_head_workspace_size(M: int, vocab: int, d: int, rank: int, grad: bool) -> int:
    if max(M, vocab, d, rank) >= 1 << 31:
        return 0                                   # as for all that is not supported
    return int(load().dspark_head_workspace_size(M, vocab, d, rank, int(bool(grad))))


def _head_inputs(h, W, U, V, prev, target):
    M, d = _matrix("h", h)
    vocab, dw = _matrix("W", W)
    if (U is None) != (V is None):
        raise ValueError("U and V are required together (or neither)")
    rank = 0 if V is None else _matrix("V", V)[1]
    bf16, i32 = torch.bfloat16, torch.int32
    dev = _place("h", h)
    ph, sh = _rows("h", h, (M, dw), bf16, dev)
    pw = _flat("W", W, (vocab, dw), bf16, dev)
    pu = pv = pp = None
    if rank:
        pu = _flat("U", U, (vocab, rank), bf16, dev)
        pv = _flat("V", V, (vocab, rank), bf16, dev)
        pp = _flat("prev", prev, (M,), i32, dev)
    pt = _flat("target", target, (M,), i32, dev)
    return (ph, sh, pw, pu, pv, pp, pt), (M, vocab, d, rank), dev


def dspark_head_loss(h, W, U, V, prev, target, loss, lse, workspace, *,
                     stream=None, raise_on_error=True) -> int:
    """h [M, d] bf16 (rows may be apart), W [vocab, d] bf16, U/V [vocab, rank]
    bf16 or None, prev/target [M] int32 (target < 0: ignored), loss/lse [M]
    fp32 (out), workspace of dspark_head_workspace_size bytes."""
    x, dims, dev = _head_inputs(h, W, U, V, prev, target)
    rows = (dims[0],)
    code = (_lib or load()).dspark_head_loss(
        *x, *dims, _flat("loss", loss, rows, torch.float32, dev),
        _flat("lse", lse, rows, torch.float32, dev), *_space(workspace, dev),
        _stream(stream))
    return _done("dspark_head_loss", code, raise_on_error)


def dspark_head_loss_grad(h, W, U, V, prev, target, lse, dloss, dh, dW, dU, dV,
                          workspace, *, stream=None, raise_on_error=True) -> int:
    """Gradients of sum_i dloss_i loss_i: dh [M, d] (rows may be apart), dW
    [vocab, d], dU/dV [vocab, rank] or None, all bf16 and written in full; lse
    [M] as written by dspark_head_loss, dloss [M] fp32."""
    x, dims, dev = _head_inputs(h, W, U, V, prev, target)
    M, vocab, d, rank = dims
    bf16 = torch.bfloat16
    pdh, sdh = _rows("dh", dh, (M, d), bf16, dev)
    pdu = pdv = None
    if rank:
        pdu = _flat("dU", dU, (vocab, rank), bf16, dev)
        pdv = _flat("dV", dV, (vocab, rank), bf16, dev)
    code = (_lib or load()).dspark_head_loss_grad(
        *x, _flat("lse", lse, (M,), torch.float32, dev),
        _flat("dloss", dloss, (M,), torch.float32, dev), *dims, pdh, sdh,
        _flat("dW", dW, (vocab, d), bf16, dev), pdu, pdv, *_space(workspace, dev),
        _stream(stream))
    return _done("dspark_head_loss_grad", code, raise_on_error)


# -------------------------------------------------------- residual stream
def dspark_residual_norm(x, residual, gain, r, y, scale=None, rstd=None, *, eps,
                         group=0, p=0.0, seed=0, offset=0, stream=None,
                         raise_on_error=True) -> int:
    """r = residual + dropout(x), y = r / rms(r) * gain.  x, residual (or None)
    and r (or None) [M, d] bf16 or fp32 (rows may be apart), gain [d]; y of the
    same type, or float8_e4m3fn with scale [M, 1] (group 0) or [M, ceil(d /
    128)] (group 128) fp32; rstd [M] fp32 or None."""
    shape = M, d = _matrix("x", x)
    dev = _place("x", x)
    ydt = dt = _dtype("x", x)
    ty = t = x.dtype
    px, sx = _rows("x", x, shape, t, dev)
    ps, ss = _rows("residual", residual, shape, t, dev)
    pr, sr = _rows("r", r, shape, t, dev)
    pscale = prstd = None
    _whole("group", group, 31)
    if y is not None and y.dtype is torch.float8_e4m3fn:
        ydt, ty = E4M3, y.dtype
        n = -(-d // group) if group > 0 else 1
        pscale = _flat("scale", scale, (M, n), torch.float32, dev)
    py, sy = _rows("y", y, shape, ty, dev)
    if rstd is not None:
        prstd = _flat("rstd", rstd, (M,), torch.float32, dev)
    code = (_lib or load()).dspark_residual_norm(
        px, sx, ps, ss, _flat("gain", gain, (d,), t, dev), dt, M, d, eps, p, *_mask(seed, offset),
        pr, sr, py, sy, ydt, group, pscale, prstd, _stream(stream))
    return _done("dspark_residual_norm", code, raise_on_error)


def dspark_norm_workspace_size(M: int, d: int) -> int:
    if max(M, d) >= 1 << 31:
        return 0
    return int(load().dspark_norm_workspace_size(M, d))


def dspark_residual_norm_grad(dy, dr, r, gain, rstd, dx, dresidual, dgain, workspace,
                              *, p=0.0, seed=0, offset=0, stream=None,
                              raise_on_error=True) -> int:
    """dr' = dr + the norm's gradient of dy; dresidual = dr', dx =
    dropout(dr'), dgain = the gain's gradient.  dr, dx, dresidual and dgain may
    be None; everything of r's type but rstd [M] fp32 (as written by
    dspark_residual_norm)."""
    shape = M, d = _matrix("r", r)
    dev = _place("r", r)
    dt, t = _dtype("r", r), r.dtype
    pg = None if dgain is None else _flat("dgain", dgain, (d,), t, dev)
    code = (_lib or load()).dspark_residual_norm_grad(
        *_rows("dy", dy, shape, t, dev), *_rows("dr", dr, shape, t, dev),
        *_rows("r", r, shape, t, dev),
        _flat("gain", gain, (d,), t, dev), _flat("rstd", rstd, (M,), torch.float32, dev),
        dt, M, d, p, *_mask(seed, offset), *_rows("dx", dx, shape, t, dev),
        *_rows("dresidual", dresidual, shape, t, dev), pg, *_space(workspace, dev),
        _stream(stream))
    return _done("dspark_residual_norm_grad", code, raise_on_error)


def dspark_dropout(x, residual, y, *, p, seed, offset, stream=None,
                   raise_on_error=True) -> int:
    """y = residual + dropout(x) ([M, d] bf16 or fp32; residual may be None);
    seed (uint64) and offset (uint32) as in include/dspark_head.h."""
    shape = M, d = _matrix("x", x)
    dev = _place("x", x)
    t = x.dtype
    code = (_lib or load()).dspark_dropout(
        *_rows("x", x, shape, t, dev), *_rows("residual", residual, shape, t, dev),
        _dtype("x", x), M, d, p, *_mask(seed, offset), *_rows("y", y, shape, t, dev),
        _stream(stream))
    return _done("dspark_dropout", code, raise_on_error)
