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
                (1, 10, 8, -8), (1, 10, 65544, 0), ((1 << 20) + 1, 10, 8, 0), (1, 1 << 30, 8, 0)):
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
