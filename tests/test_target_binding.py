"""The checks that speculative_decoding_draft_dspark_gb300.target makes of its
arguments, one at a time, and what it passes on: with stand-ins for tensors on GPU 0
and a library that only records its calls."""
import pytest

torch = pytest.importorskip("torch")

from speculative_decoding_draft_dspark_gb300 import target as T  # noqa: E402
from test_head_binding import Library, Tensor  # noqa: E402

BF16, F32, I32, I64, U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(T, "_lib", lib)
    import speculative_decoding_draft_dspark_gb300.head as H
    monkeypatch.setattr(H, "_device_now", lambda: 0)
    return lib


def i32(*shape, **kw):
    return Tensor(*shape, dtype=I32, **kw)


def rows_arguments(N=3, K=7, rows=20):
    return dict(draft_len=i32(N), sampling_mask=Tensor(N, dtype=U8), chunk_len=i32(N), ctx_len=i32(N),
                tree=Tensor(N, K + 1, dtype=I64), tokens=i32(N, 50), draft_tokens=i32(N, K), page_count=i32(N),
                free_pages=i32(30), free_count=i32(1), block_table=i32(N, 9), page_count_out=i32(N),
                free_count_out=i32(1), cu_rows=i32(N + 1), cu_out=i32(N + 1), row_request=i32(rows),
                position=i32(rows), slot=i32(rows), row_token=i32(rows), out_row=i32(rows), workspace=Tensor(256),
                page_size=16, num_pages=40, stream=1)


def rotary_arguments(R=5, Hq=4, Hk=2, d=64, dtype=BF16):
    t = lambda h: Tensor(R, h, d, dtype=dtype)  # noqa: E731
    return dict(q=t(Hq), k=t(Hk), position=i32(R), turns=Tensor(d // 2, dtype=I64), q_out=t(Hq), k_out=t(Hk),
                n_rows=i32(1), stream=1)


def append_arguments(R=5, Hq=4, Hk=2, d=64, dtype=BF16):
    t = lambda h: Tensor(R, h, d, dtype=dtype)  # noqa: E731
    return dict(q=t(Hq), k=t(Hk), v=t(Hk), position=i32(R), slot=i32(R), turns=Tensor(d // 2, dtype=I64),
                q_out=t(Hq), k_cache=Tensor(10, 16, Hk, d, dtype=dtype), v_cache=Tensor(10, 16, Hk, d, dtype=dtype),
                n_rows=i32(1), stream=1)


def attention_arguments(N=3, R=5, Hq=4, Hk=2, d=64):
    return dict(q=Tensor(R, Hq, d), k_cache=Tensor(10, 16, Hk, d), v_cache=Tensor(10, 16, Hk, d),
                block_table=i32(N, 9), ctx_len=i32(N), cu_rows=i32(N + 1), tree=Tensor(N, 4, dtype=I64),
                out=Tensor(R, Hq, d), lse=Tensor(R, Hq, dtype=F32), workspace=Tensor(1 << 20), max_len=2, scale=0.1,
                stream=1)


def adjust_arguments(N=3, R=5, vocab=100, K=7, dtype=BF16):
    t = lambda *s: Tensor(*s, dtype=F32)  # noqa: E731
    logits = Tensor(R, vocab, dtype=dtype)
    return dict(logits=logits, cu_rows=i32(N + 1), tokens=i32(N, 30), hist_len=i32(N), prompt_len=i32(N),
                draft_tokens=i32(N, K), tree=Tensor(N, K + 1, dtype=I64), out=Tensor(R, vocab, dtype=dtype),
                workspace=Tensor(256), repetition=t(N), frequency=t(N), presence=t(N), bias_token=i32(N, 4),
                bias_value=t(N, 4), bias_count=i32(N), mask=i32(2, 4), mask_index=i32(R), stream=1)


CALLS = {"rows": (T.dspark_step_rows, rows_arguments), "rotary": (T.dspark_rotary, rotary_arguments),
         "append": (T.dspark_rotary_append, append_arguments),
         "attention": (T.dspark_tree_attention, attention_arguments),
         "adjust": (T.dspark_adjust_logits, adjust_arguments)}


@pytest.mark.parametrize("call", list(CALLS))
def test_what_is_right_is_passed_on(lib, call):
    fn, arguments = CALLS[call]
    assert fn(**arguments()) == 0
    (name, args), = lib.calls
    assert name == fn.__name__ and len(args) == len(T._SIGS[name][1])


@pytest.mark.parametrize("call,name,tensor,match", [
    ("rows", "draft_len", i32(4), "draft_len must be"),
    ("rows", "draft_len", Tensor(3, dtype=I64), "draft_len must be"),
    ("rows", "sampling_mask", i32(3), "sampling_mask must be"),
    ("rows", "tree", Tensor(2, 8, dtype=I64), "tree must be"),
    ("rows", "tree", i32(3, 8), "tree must be"),
    ("rows", "tokens", None, "required together"),
    ("rows", "row_token", None, "required together"),
    ("rows", "tokens", i32(3, 50, strides=(1, 3)), "tokens must be contiguous"),
    ("rows", "position", i32(19), "position must be"),
    ("rows", "out_row", None, "out_row is required"),
    ("rows", "cu_rows", i32(3), "cu_rows must be"),
    ("rows", "block_table", i32(2, 9), "block_table must be"),
    ("rows", "free_count", i32(2), "free_count must be"),
    ("rows", "draft_tokens", i32(3), "draft_tokens must be 2-D"),
    ("rotary", "q", Tensor(5, 4, 64, dtype=torch.float16), "q must be bfloat16 or float32"),
    ("rotary", "k", Tensor(5, 2, 32), "k must be"),
    ("rotary", "k", Tensor(4, 2, 64), "k must be"),
    ("rotary", "k", Tensor(5, 2, 64, dtype=F32), "k must be"),
    ("rotary", "q_out", None, "q and q_out are required together"),
    ("rotary", "k_out", Tensor(5, 3, 64), "k_out must be"),
    ("rotary", "q", Tensor(5, 4, 64, strides=(256, 1, 4)), "q must be contiguous along"),
    ("rotary", "position", Tensor(5, dtype=I64), "position must be"),
    ("rotary", "turns", Tensor(32, dtype=F32), "turns must be"),
    ("rotary", "n_rows", i32(2), "n_rows must be"),
    ("append", "v", Tensor(5, 4, 64), "v must be"),
    ("append", "k", Tensor(4, 2, 64), "k must be"),
    ("append", "slot", i32(4), "slot must be"),
    ("append", "k_cache", Tensor(10, 16, 4, 64), "k_cache must be"),
    ("append", "v_cache", Tensor(9, 16, 2, 64), "v_cache must be"),
    ("append", "v_cache", Tensor(10, 16, 2, 64, strides=(4096, 128, 64, 1)), "the same strides"),
    ("append", "k_cache", Tensor(10, 2, 64), "k_cache must be 4-D"),
    ("attention", "q", Tensor(5, 4, 64, dtype=F32), "q must be"),
    ("attention", "out", Tensor(5, 4, 32), "out must be"),
    ("attention", "lse", Tensor(5, 4), "lse must be"),
    ("attention", "k_cache", Tensor(10, 16, 2, 32), "k_cache must be"),
    ("attention", "v_cache", Tensor(10, 16, 2, 64, dtype=F32), "v_cache must be"),
    ("attention", "ctx_len", i32(4), "ctx_len must be"),
    ("attention", "cu_rows", i32(3), "cu_rows must be"),
    ("attention", "tree", Tensor(3, 4), "tree must be"),
    ("adjust", "logits", Tensor(5, 100, dtype=torch.float16), "logits must be"),
    ("adjust", "out", Tensor(5, 99), "out must be"),
    ("adjust", "out", None, "out is required"),
    ("adjust", "cu_rows", i32(3), "cu_rows must be"),
    ("adjust", "hist_len", None, "hist_len is required"),
    ("adjust", "draft_tokens", i32(2, 7), "draft_tokens must be"),
    ("adjust", "repetition", Tensor(3), "repetition must be"),
    ("adjust", "bias_value", None, "required together"),
    ("adjust", "bias_count", None, "required together"),
    ("adjust", "bias_token", None, "required together"),
    ("adjust", "bias_value", Tensor(3, 5, dtype=F32), "bias_value must be"),
    ("adjust", "mask", i32(2, 3), "mask must have 4 words"),
    ("adjust", "mask", None, "mask_index needs a mask"),
    ("adjust", "mask_index", None, "mask must have a row for each"),
    ("adjust", "mask_index", i32(4), "mask_index must be"),
])
def test_shapes_types_and_layouts(lib, call, name, tensor, match):
    fn, arguments = CALLS[call]
    with pytest.raises(ValueError, match=match):
        fn(**{**arguments(), name: tensor})
    assert not lib.calls


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("device", [-1, 1])
def test_every_tensor_is_on_the_current_gpu(lib, call, device):
    fn, arguments = CALLS[call]
    for name, t in arguments().items():
        if isinstance(t, Tensor):
            with pytest.raises(ValueError, match=f"^{name} must be .*GPU"):
                fn(**{**arguments(), name: Tensor(*t.shape, dtype=t.dtype, device=device)})
    assert not lib.calls


@pytest.mark.parametrize("call,name,value", [
    ("rows", "page_size", 1 << 32), ("rows", "num_pages", -1), ("attention", "max_len", (1 << 32) + 1)])
def test_numbers_that_c_would_cut_off(lib, call, name, value):
    fn, arguments = CALLS[call]
    with pytest.raises(ValueError, match=f"{name} must be in"):
        fn(**{**arguments(), name: value})
    assert not lib.calls


def test_what_may_be_left_out(lib):
    T.dspark_step_rows(**{**rows_arguments(), "sampling_mask": None, "chunk_len": None, "tree": None, "tokens": None,
                          "row_token": None})
    T.dspark_rotary(**{**rotary_arguments(), "q": None, "q_out": None, "n_rows": None})
    T.dspark_tree_attention(**{**attention_arguments(), "tree": None, "lse": None})
    none = dict.fromkeys(("prompt_len", "draft_tokens", "tree", "repetition", "frequency", "presence", "bias_token",
                          "bias_value", "bias_count", "mask", "mask_index"))
    T.dspark_adjust_logits(**{**adjust_arguments(), **none})
    assert [len(a) for _, a in lib.calls] == [len(T._SIGS[n][1]) for n, _ in lib.calls]


def test_strides_are_passed_on(lib):
    q = Tensor(5, 4, 64, strides=(1000, 72, 1))
    cache = dict(strides=(9000, 64, 1024, 1))
    T.dspark_tree_attention(**{**attention_arguments(), "q": q, "k_cache": Tensor(10, 16, 2, 64, **cache),
                               "v_cache": Tensor(10, 16, 2, 64, **cache),
                               "block_table": i32(3, 9, strides=(20, 1))})
    a = lib.calls[0][1]
    assert a[1:3] == (1000, 72) and a[5:8] == (9000, 64, 1024) and a[11] == 20


@pytest.mark.parametrize("pitch", [1003, 64, 1, 0])
def test_a_dimension_of_one_has_no_stride(lib, pitch):
    """One row, one head, one page: whatever the stride says, sizes are passed on."""
    one = Tensor(1, 1, 64, strides=(pitch, pitch, 1))
    T.dspark_rotary(**{**rotary_arguments(R=1, Hq=1, Hk=1), "q": one, "q_out": one})
    a = lib.calls[0][1]
    assert a[1:3] == (64, 64)
    c = Tensor(1, 16, 1, 64, strides=(pitch, 64, pitch, 1))
    T.dspark_rotary_append(**{**append_arguments(Hk=1), "k_cache": c, "v_cache": c})
    assert lib.calls[1][1][-6:-3] == (1024, 64, 64)


def test_the_bits_of_a_bool_mask(lib):
    class Bool(Tensor):
        def view(self, dtype):
            return Tensor(*self.shape, dtype=dtype)
    assert T.dspark_step_rows(**{**rows_arguments(), "sampling_mask": Bool(3, dtype=torch.bool)}) == 0
