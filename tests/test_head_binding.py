"""The checks that speculative_decoding_draft_dspark_gb300.head makes of its
arguments, one at a time, and what it passes on.  The tensors are stand-ins that
say they are on GPU 0 and the library only records its calls, so that each check
is reached on a machine without a GPU."""
import pytest

torch = pytest.importorskip("torch")

from speculative_decoding_draft_dspark_gb300 import head as H  # noqa: E402

BF16, F32, I32, F8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


class Tensor:
    """Shape, strides, type and place of a tensor, without its memory."""
    at = 1 << 20

    def __init__(self, *shape, dtype=BF16, strides=None, device=0):
        self.shape, self.dtype, self.device_index = torch.Size(shape), dtype, device
        dense, n = [], 1
        for s in reversed(shape):
            dense.insert(0, n)
            n *= s
        self.strides = tuple(strides or dense)
        self.dense = self.strides == tuple(dense)
        self.is_cuda = device >= 0
        Tensor.at += 1 << 12
        self.pointer = Tensor.at

    def dim(self):
        return len(self.shape)

    def stride(self):
        return self.strides

    def is_contiguous(self):
        return self.dense

    def get_device(self):
        return self.device_index

    def data_ptr(self):
        return self.pointer

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return 1


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(H, "_lib", lib)
    monkeypatch.setattr(H, "_device_now", lambda: 0)
    return lib


def loss_arguments(M=4, vocab=100, d=64, rank=16):
    return dict(h=Tensor(M, d), W=Tensor(vocab, d), U=Tensor(vocab, rank), V=Tensor(vocab, rank),
                prev=Tensor(M, dtype=I32), target=Tensor(M, dtype=I32), loss=Tensor(M, dtype=F32),
                lse=Tensor(M, dtype=F32), workspace=Tensor(1 << 20), stream=1)


def grad_arguments(M=4, vocab=100, d=64, rank=16):
    a = loss_arguments(M, vocab, d, rank)
    del a["loss"]
    return dict(a, dloss=Tensor(M, dtype=F32), dh=Tensor(M, d), dW=Tensor(vocab, d),
                dU=Tensor(vocab, rank), dV=Tensor(vocab, rank))


def norm_arguments(M=4, d=64, dtype=BF16):
    return dict(x=Tensor(M, d, dtype=dtype), residual=Tensor(M, d, dtype=dtype),
                gain=Tensor(d, dtype=dtype), r=Tensor(M, d, dtype=dtype), y=Tensor(M, d, dtype=dtype),
                rstd=Tensor(M, dtype=F32), eps=1e-6, stream=1)


def norm_grad_arguments(M=4, d=64, dtype=BF16):
    m = lambda: Tensor(M, d, dtype=dtype)  # noqa: E731
    return dict(dy=m(), dr=m(), r=m(), gain=Tensor(d, dtype=dtype), rstd=Tensor(M, dtype=F32),
                dx=m(), dresidual=m(), dgain=Tensor(d, dtype=dtype), workspace=Tensor(1 << 20), stream=1)


def dropout_arguments(M=4, d=64, dtype=BF16):
    m = lambda: Tensor(M, d, dtype=dtype)  # noqa: E731
    return dict(x=m(), residual=m(), y=m(), p=0.1, seed=1, offset=2, stream=1)


CALLS = {"loss": (H.dspark_head_loss, loss_arguments), "grad": (H.dspark_head_loss_grad, grad_arguments),
         "norm": (H.dspark_residual_norm, norm_arguments),
         "norm_grad": (H.dspark_residual_norm_grad, norm_grad_arguments),
         "dropout": (H.dspark_dropout, dropout_arguments)}


def refused(lib, call, match, **changed):
    fn, arguments = CALLS[call]
    with pytest.raises(ValueError, match=match):
        fn(**{**arguments(), **changed})
    assert not lib.calls


@pytest.mark.parametrize("call", list(CALLS))
def test_what_is_right_is_passed_on(lib, call):
    fn, arguments = CALLS[call]
    assert fn(**arguments()) == 0
    assert len(lib.calls) == 1


@pytest.mark.parametrize("call,name,tensor,match", [
    ("loss", "h", Tensor(4, 32), "h must be"),
    ("loss", "h", Tensor(4, 64, dtype=F32), "h must be"),
    ("loss", "h", Tensor(4, 64, strides=(1, 4)), "h must be contiguous"),
    ("loss", "W", Tensor(100, 64, strides=(72, 1)), "W must be contiguous"),
    ("loss", "U", Tensor(99, 16), "U must be"),
    ("loss", "prev", Tensor(3, dtype=I32), "prev must be"),
    ("loss", "prev", None, "prev is required"),
    ("loss", "target", Tensor(4, dtype=torch.int64), "target must be"),
    ("loss", "loss", Tensor(5, dtype=F32), "loss must be"),
    ("loss", "lse", Tensor(4, dtype=I32), "lse must be"),
    ("grad", "dloss", Tensor(4), "dloss must be"),
    ("grad", "dh", Tensor(4, 64, dtype=F32), "dh must be"),
    ("grad", "dW", Tensor(64, 100), "dW must be"),
    ("grad", "dU", None, "dU is required"),
    ("grad", "dV", Tensor(100, 8), "dV must be"),
    ("norm", "x", Tensor(4, 64, dtype=torch.float16), "x must be bfloat16 or float32"),
    ("norm", "residual", Tensor(4, 63), "residual must be"),
    ("norm", "gain", Tensor(64, dtype=F32), "gain must be"),
    ("norm", "r", Tensor(4, 64, strides=(64, 2)), "r must be contiguous"),
    ("norm", "y", Tensor(4, 64, dtype=F32), "y must be"),
    ("norm", "y", Tensor(4, 64, dtype=F8), "scale is required"),
    ("norm", "rstd", Tensor(4, 1, dtype=F32), "rstd must be"),
    ("norm_grad", "dy", Tensor(5, 64), "dy must be"),
    ("norm_grad", "dgain", Tensor(64, dtype=F32), "dgain must be"),
    ("dropout", "y", Tensor(4, 64, dtype=F32), "y must be"),
])
def test_shapes_types_and_layouts(lib, call, name, tensor, match):
    refused(lib, call, match, **{name: tensor})


@pytest.mark.parametrize("group,shape,right", [(0, (4, 1), True), (128, (4, 3), True), (128, (4, 1), False),
                                               (0, (4, 3), False), (128, (4, 2), False)])
def test_scales_have_a_column_for_each_group(lib, group, shape, right):
    a = dict(norm_arguments(d=300), y=Tensor(4, 300, dtype=F8), group=group, scale=Tensor(*shape, dtype=F32))
    if right:
        assert H.dspark_residual_norm(**a) == 0
    else:
        with pytest.raises(ValueError, match="scale must be"):
            H.dspark_residual_norm(**a)


def test_rows_apart_are_passed_on(lib):
    H.dspark_head_loss(**{**loss_arguments(), "h": Tensor(4, 64, strides=(1003, 1))})
    assert lib.calls[0][1][1] == 1003


@pytest.mark.parametrize("pitch", [1003, 64, 1, 0])
def test_one_row_has_no_stride(lib, pitch):
    """A slice of one row has its buffer's pitch as the stride, or any other (an
    expanded one 0): the row's width is passed on instead."""
    row = dict(strides=(pitch, 1))
    H.dspark_head_loss_grad(**{**grad_arguments(M=1), "h": Tensor(1, 64, **row), "dh": Tensor(1, 64, **row)})
    H.dspark_residual_norm(**{**norm_arguments(M=1), "x": Tensor(1, 64, **row), "y": Tensor(1, 64, **row)})
    (_, grad), (_, norm) = lib.calls
    assert grad[1] == grad[14] == 64
    assert norm[1] == norm[15] == 64


@pytest.mark.parametrize("call", ["loss", "grad"])
@pytest.mark.parametrize("missing", ["U", "V"])
def test_one_factor_alone_is_refused(lib, call, missing):
    refused(lib, call, "U and V are required together", **{missing: None})


def test_no_factors_are_rank_0(lib):
    H.dspark_head_loss(**{**loss_arguments(), "U": None, "V": None, "prev": None})
    assert lib.calls[0][1][3:6] == (None, None, None) and lib.calls[0][1][10] == 0


@pytest.mark.parametrize("call", ["norm", "norm_grad", "dropout"])
@pytest.mark.parametrize("name,value", [("offset", 1 << 32), ("offset", -1), ("seed", 1 << 64), ("seed", -1)])
def test_a_mask_that_would_wrap_is_refused(lib, call, name, value):
    """C takes the low bits: (seed, offset + 2^32) would draw (seed, offset)'s mask."""
    refused(lib, call, f"{name} must be in", **{name: value})


def test_the_last_mask_is_passed_on(lib):
    H.dspark_dropout(**{**dropout_arguments(), "seed": (1 << 64) - 1, "offset": (1 << 32) - 1})
    assert lib.calls[0][1][8:10] == ((1 << 64) - 1, (1 << 32) - 1)


def test_dimensions_that_would_wrap_are_refused(lib):
    """2^32 + 4 rows would be computed as 4, and a group of 2^32 + 128 as 128 with
    scales for one."""
    many = (1 << 32) + 4
    refused(lib, "dropout", "x's rows", x=Tensor(many, 64), residual=None, y=Tensor(many, 64))
    refused(lib, "loss", "W's rows", W=Tensor(many, 64), U=None, V=None)
    refused(lib, "norm", "group must be in", y=Tensor(4, 64, dtype=F8), group=(1 << 32) + 128,
            scale=Tensor(4, 1, dtype=F32))
    assert H.dspark_head_workspace_size(many, 100, 64, 0, True) == 0
    assert H.dspark_head_workspace_size(4, many, 64, 0, True) == 0
    assert H.dspark_norm_workspace_size(many, 64) == 0
    assert not lib.calls


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("device", [-1, 1])
def test_every_tensor_is_on_the_current_gpu(lib, call, device):
    """One tensor at a time on the CPU or on another GPU, the workspace too."""
    fn, arguments = CALLS[call]
    for name, t in arguments().items():
        if isinstance(t, Tensor):
            with pytest.raises(ValueError, match=f"^{name} must be .*GPU"):
                fn(**{**arguments(), name: Tensor(*t.shape, dtype=t.dtype, device=device)})
    assert not lib.calls


def test_all_tensors_on_another_gpu_than_the_current(lib):
    a = {k: Tensor(*t.shape, dtype=t.dtype, device=1) if isinstance(t, Tensor) else t
         for k, t in dropout_arguments().items()}
    with pytest.raises(ValueError, match="x must be on the current GPU"):
        H.dspark_dropout(**a)


@pytest.mark.parametrize("call", ["loss", "grad", "norm_grad"])
def test_a_workspace_is_contiguous(lib, call):
    refused(lib, call, "workspace must be", workspace=Tensor(64, 64, strides=(128, 1)))
    refused(lib, call, "workspace must be", workspace=None)
