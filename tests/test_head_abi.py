"""include/dspark_head.h: every declared entry point is exported and bound,
workspace sizes grow with what they hold, and bad arguments are rejected on
the host before anything is launched (so these run without a GPU)."""
import ctypes

import pytest

import __graft_entry__
from speculative_decoding_draft_dspark_gb300 import dspark as D
from speculative_decoding_draft_dspark_gb300 import head as H

FAKE = 1 << 20  # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return H.load()


def test_exports_every_header_function(lib):
    names = H.header_functions()
    assert set(names) == set(H._SIGS)
    for n in names:
        assert hasattr(lib, n), n


def test_head_workspace_size(lib):
    f = H.dspark_head_workspace_size
    assert f(1792, 262144, 2048, 256, True) >= f(1792, 262144, 2048, 256, False) > 1792 * 2304 * 2
    assert f(7168, 262144, 2048, 256, False) > f(1792, 262144, 2048, 256, False)
    assert f(1, 1, 8, 0, True) > 0
    for bad in ((0, 10, 8, 0), (1, 0, 8, 0), (1, 10, 12, 0), (1, 10, 8, 12), (1, 10, 8, 264),
                (1, 10, 8, -8), (1, 10, 65544, 0), ((1 << 20) + 1, 10, 8, 0), (1, 1 << 30, 8, 0),
                (1 << 20, (1 << 30) - 1, 8, 0)):
        assert f(*bad, True) == 0, bad


def _loss(lib, **kw):
    a = dict(h=FAKE, hs=64, W=FAKE, U=FAKE, V=FAKE, prev=FAKE, target=FAKE, M=4, vocab=1000, d=64,
             rank=16, loss=FAKE, lse=FAKE, ws=FAKE, wsb=1 << 40, stream=None)
    a.update(kw)
    return lib.dspark_head_loss(*a.values())


def _grad(lib, **kw):
    a = dict(h=FAKE, hs=64, W=FAKE, U=FAKE, V=FAKE, prev=FAKE, target=FAKE, lse=FAKE, dloss=FAKE,
             M=4, vocab=1000, d=64, rank=16, dh=FAKE, dhs=64, dW=FAKE, dU=FAKE, dV=FAKE, ws=FAKE,
             wsb=1 << 40, stream=None)
    a.update(kw)
    return lib.dspark_head_loss_grad(*a.values())


@pytest.mark.parametrize("call", [_loss, _grad])
@pytest.mark.parametrize("kw,code", [
    (dict(h=None), D.ERR_INVALID_ARG),
    (dict(W=None), D.ERR_INVALID_ARG),
    (dict(U=None), D.ERR_INVALID_ARG),
    (dict(V=None), D.ERR_INVALID_ARG),
    (dict(prev=None), D.ERR_INVALID_ARG),
    (dict(target=None), D.ERR_INVALID_ARG),
    (dict(lse=None), D.ERR_INVALID_ARG),
    (dict(M=0), D.ERR_INVALID_ARG),
    (dict(vocab=0), D.ERR_INVALID_ARG),
    (dict(rank=-8), D.ERR_INVALID_ARG),
    (dict(d=60, hs=64), D.ERR_UNSUPPORTED),
    (dict(rank=20), D.ERR_UNSUPPORTED),
    (dict(rank=264), D.ERR_UNSUPPORTED),
    (dict(M=(1 << 20) + 1), D.ERR_UNSUPPORTED),
    (dict(vocab=1 << 30), D.ERR_UNSUPPORTED),
    (dict(hs=56), D.ERR_INVALID_ARG),
    (dict(hs=68), D.ERR_INVALID_ARG),
    (dict(h=FAKE + 8), D.ERR_INVALID_ARG),
    (dict(W=FAKE + 8), D.ERR_INVALID_ARG),
    (dict(U=FAKE + 2), D.ERR_INVALID_ARG),
    (dict(target=FAKE + 2), D.ERR_INVALID_ARG),
    (dict(ws=None), D.ERR_WORKSPACE),
    (dict(ws=FAKE + 16), D.ERR_WORKSPACE),
    (dict(wsb=4096), D.ERR_WORKSPACE),
])
def test_head_validation(lib, call, kw, code):
    assert call(lib, **kw) == code


@pytest.mark.parametrize("kw", [
    dict(dloss=None), dict(dh=None), dict(dW=None), dict(dU=None), dict(dV=None),
    dict(dh=FAKE + 8), dict(dW=FAKE + 8), dict(dV=FAKE + 4), dict(dhs=56), dict(dhs=68),
])
def test_head_grad_validation(lib, kw):
    assert _grad(lib, **kw) == D.ERR_INVALID_ARG


def test_loss_workspace_is_not_enough_for_the_gradient(lib):
    small = H.dspark_head_workspace_size(4, 1000, 64, 16, False)
    assert H.dspark_head_workspace_size(4, 1000, 64, 16, True) > small
    assert _grad(lib, wsb=small) == D.ERR_WORKSPACE
    assert _loss(lib, loss=None) == D.ERR_INVALID_ARG


def test_binding_checks_shapes_and_types():
    torch = pytest.importorskip("torch")
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    f = lambda n: torch.zeros(n)  # noqa: E731
    ok = dict(h=z(4, 64), W=z(100, 64), U=z(100, 16), V=z(100, 16), prev=i(4), target=i(4),
              loss=f(4), lse=f(4), workspace=z(8))
    for kw in (dict(h=z(4, 32)), dict(h=z(4, 64, t=torch.float32)), dict(W=z(64, 100).T),
               dict(U=z(99, 16)), dict(U=None), dict(prev=i(3)),
               dict(target=torch.zeros(4, dtype=torch.int64)), dict(loss=f(5)), dict(lse=i(4)),
               dict(h=z(64, 4).T)):
        with pytest.raises(ValueError):
            H.dspark_head_loss(**{**ok, **kw})


# -------------------------------------------------------- residual stream
def _norm(lib, **kw):
    a = dict(x=FAKE, xs=64, res=FAKE, ress=64, gain=FAKE, dt=D.BF16, M=4, d=64, eps=1e-6, p=0.0,
             seed=1, offset=0, r=FAKE, rs=64, y=FAKE, ys=64, ydt=D.BF16, group=0, scale=None,
             rstd=FAKE, stream=None)
    a.update(kw)
    return lib.dspark_residual_norm(*a.values())


def _norm_grad(lib, **kw):
    a = dict(dy=FAKE, dys=64, dr=FAKE, drs=64, r=FAKE, rs=64, gain=FAKE, rstd=FAKE, dt=D.F32, M=4,
             d=64, p=0.0, seed=1, offset=0, dx=FAKE, dxs=64, ds=FAKE, dss=64, dgain=FAKE, ws=FAKE,
             wsb=1 << 30, stream=None)
    a.update(kw)
    return lib.dspark_residual_norm_grad(*a.values())


def _drop(lib, **kw):
    a = dict(x=FAKE, xs=64, res=FAKE, ress=64, dt=D.BF16, M=4, d=64, p=0.1, seed=1, offset=0, y=FAKE,
             ys=64, stream=None)
    a.update(kw)
    return lib.dspark_dropout(*a.values())


@pytest.mark.parametrize("call", [_norm, _norm_grad, _drop])
@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), D.ERR_INVALID_ARG),
    (dict(M=0), D.ERR_INVALID_ARG),
    (dict(d=0), D.ERR_INVALID_ARG),
    (dict(d=32769), D.ERR_UNSUPPORTED),
    (dict(p=-0.1), D.ERR_INVALID_ARG),
    (dict(p=1.5), D.ERR_INVALID_ARG),
    (dict(p=float("nan")), D.ERR_INVALID_ARG),
])
def test_residual_stream_validation(lib, call, kw, code):
    assert call(lib, **kw) == code


@pytest.mark.parametrize("call,kw,code", [
    (_norm, dict(x=None), D.ERR_INVALID_ARG),
    (_norm, dict(gain=None), D.ERR_INVALID_ARG),
    (_norm, dict(y=None), D.ERR_INVALID_ARG),
    (_norm, dict(xs=63), D.ERR_INVALID_ARG),
    (_norm, dict(ress=10), D.ERR_INVALID_ARG),
    (_norm, dict(rs=63), D.ERR_INVALID_ARG),
    (_norm, dict(ys=63), D.ERR_INVALID_ARG),
    (_norm, dict(x=FAKE + 1), D.ERR_INVALID_ARG),
    (_norm, dict(eps=-1.0), D.ERR_INVALID_ARG),
    (_norm, dict(eps=float("inf")), D.ERR_INVALID_ARG),
    (_norm, dict(ydt=D.F32), D.ERR_INVALID_ARG),
    (_norm, dict(ydt=H.E4M3), D.ERR_INVALID_ARG),                 # no scale
    (_norm, dict(ydt=H.E4M3, scale=FAKE, group=64), D.ERR_UNSUPPORTED),
    (_norm_grad, dict(dy=None), D.ERR_INVALID_ARG),
    (_norm_grad, dict(r=None), D.ERR_INVALID_ARG),
    (_norm_grad, dict(rstd=None), D.ERR_INVALID_ARG),
    (_norm_grad, dict(gain=FAKE + 2), D.ERR_INVALID_ARG),
    (_norm_grad, dict(dxs=60), D.ERR_INVALID_ARG),
    (_norm_grad, dict(ws=None), D.ERR_WORKSPACE),
    (_norm_grad, dict(ws=FAKE + 128), D.ERR_WORKSPACE),
    (_norm_grad, dict(wsb=256), D.ERR_WORKSPACE),
    (_drop, dict(x=None), D.ERR_INVALID_ARG),
    (_drop, dict(y=None), D.ERR_INVALID_ARG),
    (_drop, dict(ys=8), D.ERR_INVALID_ARG),
])
def test_residual_stream_arguments(lib, call, kw, code):
    assert call(lib, **kw) == code


def test_norm_workspace_size(lib):
    f = H.dspark_norm_workspace_size
    assert f(1, 8) >= 256 + 32 and f(15360, 2048) > f(1, 2048)
    assert f(0, 8) == f(1, 0) == f(1, 40000) == 0
