"""The target step's entry points: declared, exported, bound, and their host
checks, which come before any CUDA call (so these run without a GPU)."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

import __graft_entry__  # noqa: E402
from speculative_decoding_draft_dspark_gb300 import dspark as D  # noqa: E402
from speculative_decoding_draft_dspark_gb300 import target as T  # noqa: E402

FAKE = 1 << 20  # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return T.load()


def test_exports_every_header_function(lib):
    assert T.header_functions() == sorted(T._SIGS)
    for n in T._SIGS:
        assert hasattr(lib, n), n


OK_ARGS = {
    "dspark_step_rows": dict(
        draft_len=FAKE, mask=None, chunk=None, ctx=FAKE, tree=None, tree_width=0, tokens=FAKE, tokens_stride=100,
        tokens_width=100, draft=FAKE, N=4, K=7, page_count=FAKE, free=FAKE, free_max=10, free_count=FAKE,
        page_size=16, num_pages=100, table=FAKE, table_stride=8, max_pages=8, page_count_out=FAKE,
        free_count_out=FAKE, cu_rows=FAKE, cu_out=FAKE, max_rows=32, request=FAKE, position=FAKE, slot=FAKE,
        token=FAKE, out_row=FAKE, ws=FAKE, wsb=256, stream=None),
    "dspark_rotary": dict(
        q=FAKE, qs=512, qh=64, Hq=8, k=FAKE, ks=128, kh=64, Hk=2, dtype=D.BF16, R=4, d=64, position=FAKE, n=None,
        turns=FAKE, rot=64, inter=0, inverse=0, amplitude=1.0, qo=FAKE, qos=512, qoh=64, ko=FAKE, kos=128, koh=64,
        stream=None),
    "dspark_rotary_append": dict(
        q=FAKE, qs=512, qh=64, Hq=8, k=FAKE, ks=128, kh=64, v=FAKE, vs=128, vh=64, Hk=2, dtype=D.BF16, R=4, d=64,
        position=FAKE, slot=FAKE, n=None, turns=FAKE, rot=64, inter=0, amplitude=1.0, qo=FAKE, qos=512, qoh=64,
        kc=FAKE, vc=FAKE, page_stride=16 * 128, token_stride=128, head_stride=64, page_size=16, pages=10,
        stream=None),
    "dspark_tree_attention": dict(
        q=FAKE, qs=512, qh=64, kc=FAKE, vc=FAKE, page_stride=16 * 128, token_stride=128, head_stride=64,
        page_size=16, pages=10, table=FAKE, table_stride=8, max_pages=8, ctx=FAKE, cu=FAKE, tree=None, tree_width=0,
        N=4, R=4, max_len=1, Hq=8, Hk=2, d=64, scale=0.125, out=FAKE, os=512, oh=64, lse=None, ws=FAKE, wsb=1 << 40,
        stream=None),
    "dspark_adjust_logits": dict(
        logits=FAKE, stride=1000, dtype=D.BF16, R=4, vocab=1000, cu=FAKE, N=4, tokens=FAKE, tokens_stride=50,
        tokens_width=50, hist=FAKE, prompt=None, draft=FAKE, K=7, tree=None, tree_width=0, rep=None, freq=None,
        pres=None, bt=None, bv=None, bc=None, bw=0, mask=None, ms=0, mr=0, mi=None, out=FAKE, os=1000, ws=FAKE,
        wsb=256, stream=None),
}

I, U, W = D.ERR_INVALID_ARG, D.ERR_UNSUPPORTED, D.ERR_WORKSPACE


@pytest.mark.parametrize("fn,kw,code", [
    ("dspark_step_rows", dict(draft_len=None), I),
    ("dspark_step_rows", dict(ctx=None), I),
    ("dspark_step_rows", dict(draft=None), I),
    ("dspark_step_rows", dict(out_row=FAKE + 2), I),
    ("dspark_step_rows", dict(N=0), I),
    ("dspark_step_rows", dict(K=64), U),
    ("dspark_step_rows", dict(N=16385), U),
    ("dspark_step_rows", dict(max_rows=0), I),
    ("dspark_step_rows", dict(max_rows=(1 << 22) + 1), U),
    ("dspark_step_rows", dict(page_size=8), U),
    ("dspark_step_rows", dict(page_size=48), U),
    ("dspark_step_rows", dict(page_size=512), U),
    ("dspark_step_rows", dict(page_size=0), I),
    ("dspark_step_rows", dict(num_pages=1 << 27), U),
    ("dspark_step_rows", dict(max_pages=1 << 27, table_stride=1 << 27), U),
    ("dspark_step_rows", dict(table_stride=7), I),
    ("dspark_step_rows", dict(tree=FAKE, tree_width=0), I),
    ("dspark_step_rows", dict(tree=FAKE + 4, tree_width=8), I),
    ("dspark_step_rows", dict(tree=FAKE, tree_width=65), U),
    ("dspark_step_rows", dict(tokens=None), I),
    ("dspark_step_rows", dict(tokens_stride=99), I),
    ("dspark_step_rows", dict(free=None), I),
    ("dspark_step_rows", dict(ws=None), W),
    ("dspark_step_rows", dict(wsb=128), W),
    ("dspark_rotary", dict(dtype=2), I),
    ("dspark_rotary", dict(q=None), I),
    ("dspark_rotary", dict(ko=None), I),
    ("dspark_rotary", dict(rot=63), I),
    ("dspark_rotary", dict(rot=66), I),
    ("dspark_rotary", dict(rot=0), I),
    ("dspark_rotary", dict(R=-1), I),
    ("dspark_rotary", dict(d=1026, qs=9000, qh=1026, ks=9000, kh=1026, qos=9000, qoh=1026, kos=9000, koh=1026), U),
    ("dspark_rotary", dict(turns=None), I),
    ("dspark_rotary", dict(position=None), I),
    ("dspark_rotary", dict(amplitude=math.nan), I),
    ("dspark_rotary", dict(qos=64), I),              # rows of the output overlap
    ("dspark_rotary", dict(qos=576), I),             # in place, rows elsewhere
    ("dspark_rotary", dict(koh=128, kos=256), I),
    ("dspark_rotary", dict(qh=63), I),
    ("dspark_rotary_append", dict(v=None), I),
    ("dspark_rotary_append", dict(slot=None), I),
    ("dspark_rotary_append", dict(kc=None), I),
    ("dspark_rotary_append", dict(Hk=0), I),
    ("dspark_rotary_append", dict(token_stride=64), I),   # tokens overlap heads
    ("dspark_rotary_append", dict(page_size=24), U),
    ("dspark_rotary_append", dict(pages=0), I),
    ("dspark_tree_attention", dict(Hq=7), I),
    ("dspark_tree_attention", dict(Hq=512, Hk=2, qs=512 * 64, os=512 * 64), U),   # a group of 256
    ("dspark_tree_attention", dict(d=260), U),
    ("dspark_tree_attention", dict(d=60), U),
    ("dspark_tree_attention", dict(d=0), I),
    ("dspark_tree_attention", dict(q=FAKE + 8), I),
    ("dspark_tree_attention", dict(qs=516), I),
    ("dspark_tree_attention", dict(kc=FAKE + 8), I),
    ("dspark_tree_attention", dict(token_stride=132), I),
    ("dspark_tree_attention", dict(scale=math.inf), I),
    ("dspark_tree_attention", dict(scale=-1.0), I),
    ("dspark_tree_attention", dict(scale=0.0), I),
    ("dspark_tree_attention", dict(scale=1e-40), I),
    ("dspark_tree_attention", dict(scale=3e38), I),
    ("dspark_tree_attention", dict(max_len=0), I),
    ("dspark_tree_attention", dict(R=0), I),
    ("dspark_tree_attention", dict(N=16385), U),
    ("dspark_tree_attention", dict(cu=None), I),
    ("dspark_tree_attention", dict(table_stride=7), I),
    ("dspark_tree_attention", dict(tree=FAKE, tree_width=65), U),
    ("dspark_tree_attention", dict(page_size=100), U),
    ("dspark_tree_attention", dict(max_pages=1 << 26, table_stride=1 << 26), U),
    ("dspark_tree_attention", dict(os=64), I),
    ("dspark_tree_attention", dict(ws=None), W),
    ("dspark_tree_attention", dict(ws=FAKE + 64), W),
    ("dspark_tree_attention", dict(wsb=256), W),
    ("dspark_adjust_logits", dict(dtype=2), I),
    ("dspark_adjust_logits", dict(logits=None), I),
    ("dspark_adjust_logits", dict(stride=999, os=999), I),
    ("dspark_adjust_logits", dict(os=1008), I),           # in place, rows elsewhere
    ("dspark_adjust_logits", dict(vocab=1 << 30, stride=1 << 30, os=1 << 30), U),
    ("dspark_adjust_logits", dict(K=64), U),
    ("dspark_adjust_logits", dict(tokens_width=(1 << 26) + 1, tokens_stride=1 << 27), U),
    ("dspark_adjust_logits", dict(draft=None), I),
    ("dspark_adjust_logits", dict(tokens=None), I),
    ("dspark_adjust_logits", dict(hist=None), I),
    ("dspark_adjust_logits", dict(bw=4), I),
    ("dspark_adjust_logits", dict(bw=1025, bt=FAKE, bv=FAKE, bc=FAKE), U),
    ("dspark_adjust_logits", dict(mask=FAKE, ms=31, mr=4), I),
    ("dspark_adjust_logits", dict(mask=FAKE, ms=32, mr=0), I),
    ("dspark_adjust_logits", dict(wsb=128), W),
])
def test_refusals(lib, fn, kw, code):
    assert getattr(lib, fn)(*{**OK_ARGS[fn], **kw}.values()) == code


def test_no_rows_and_no_heads_launch_nothing(lib):
    """An empty tensor has no pointer; so these run without a GPU."""
    ok = OK_ARGS["dspark_rotary"]
    empty = dict(q=None, k=None, qo=None, ko=None, position=None)
    assert lib.dspark_rotary(*{**ok, **empty, "R": 0}.values()) == D.OK
    no_heads = dict(q=None, k=None, qo=None, ko=None, Hq=0, Hk=0, qs=0, ks=0, qos=0, kos=0)
    assert lib.dspark_rotary(*{**ok, **no_heads}.values()) == D.OK
    ok = OK_ARGS["dspark_rotary_append"]
    assert lib.dspark_rotary_append(*{**ok, "q": None, "k": None, "v": None, "R": 0}.values()) == D.OK


def test_workspace_sizes(lib):
    size = T.dspark_attention_workspace_size
    assert size(4, 8, 32, 8, 128) > 640 * 32 * 128 * 4
    assert size(4, 1, 32, 8, 128) < size(4, 8, 32, 8, 128) < size(4, 1000, 32, 8, 128) == size(9, 9999, 32, 8, 128)
    for bad in ((0, 1, 8, 8, 64), (1, 0, 8, 8, 64), (1, 1, 7, 2, 64), (1, 1, 8, 8, 65), (1, 1, 8, 8, 512),
                (1 << 32, 1, 8, 8, 64)):
        assert size(*bad) == 0


def turns_of(freq):
    t = freq / (2.0 * math.pi)
    return t - math.floor(t)


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 10000.0), (50, 500000.0), (128, 1.5)])
def test_rotary_table(lib, rot, base):
    got = T.dspark_rotary_table(rot, base)
    assert got.shape == (rot // 2,)
    for i, x in enumerate(got.tolist()):
        want = turns_of(base ** (-2.0 * i / rot))
        assert abs((x % (1 << 64)) / 2.0 ** 64 - want) <= 2.0 ** -50


def test_rotary_table_scalings(lib):
    rot, base = 128, 10000.0
    plain = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    lin = T.dspark_rotary_table(rot, base, scaling=T.ROPE_LINEAR, factor=4.0).tolist()
    parts = T.dspark_rotary_table(rot, base, scaling=T.ROPE_BY_PARTS, factor=32.0, original=4096, low=1,
                                  high=32).tolist()
    turn = T.dspark_rotary_table(rot, base, scaling=T.ROPE_BY_TURNS, factor=8.0, original=8192, low=1,
                                 high=4).tolist()
    lo = max(0, math.floor(rot * math.log(4096 / (32 * 2 * math.pi)) / (2 * math.log(base))))
    hi = min(rot // 2 - 1, math.ceil(rot * math.log(4096 / (2 * math.pi)) / (2 * math.log(base))))
    assert 0 < lo < hi < rot // 2 - 1
    for i, f in enumerate(plain):
        w = min(1.0, max(0.0, (i - lo) / (hi - lo)))
        s = min(1.0, max(0.0, (8192 * f / (2 * math.pi) - 1) / 3))
        for got, want in ((lin[i], f / 4), (parts[i], f * (1 - w) + f / 32 * w), (turn[i], f * s + f / 8 * (1 - s))):
            assert abs(got / 2.0 ** 64 - turns_of(want)) <= 2.0 ** -50


@pytest.mark.parametrize("rot,base,kw", [
    (7, 1e4, {}), (0, 1e4, {}), (8, 1.0, {}), (8, math.inf, {}), (8, 1e4, dict(scaling=4)),
    (8, 1e4, dict(scaling=1, factor=0.0)), (8, 1e4, dict(scaling=2, factor=2.0)),
    (8, 1e4, dict(scaling=3, factor=2.0, original=10, low=4, high=4)), (1026, 1e4, {})])
def test_rotary_table_refusals(lib, rot, base, kw):
    with pytest.raises(D.DsparkError):
        T.dspark_rotary_table(rot, base, **kw)


def test_c_entry_survives_null(lib):
    assert lib.dspark_rotary_table(8, ctypes.c_double(1e4), 0, 1.0, 0.0, 0.0, 0.0, None) == I


@pytest.mark.parametrize("rot,base,original,factor,low,high,kept", [
    (128, 10000.0, 65536, 4.0, 1, 32, 0.31),         # the ramp ends two pairs behind the last
    (64, 10000.0, 65536, 4.0, 1, 32, None), (64, 100.0, 4096, 8.0, 1, 32, None), (16, 10000.0, 131072, 16.0, 1, 32, None)])
def test_a_ramp_that_ends_behind_the_last_pair(lib, rot, base, original, factor, low, high, kept):
    """The ramp's end is cut at rot - 1, not at the last pair, whose frequency is then
    stretched in part only."""
    got = T.dspark_rotary_table(rot, base, scaling=T.ROPE_BY_PARTS, factor=factor, original=original, low=low,
                                high=high).tolist()
    edge = lambda b: rot * math.log(original / (2 * math.pi * b)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(0, math.floor(edge(high))), min(rot - 1, math.ceil(edge(low)))
    assert lo < rot // 2 - 1 < hi
    for i, x in enumerate(got):
        f, w = base ** (-2.0 * i / rot), min(1.0, max(0.0, (i - lo) / (hi - lo)))
        assert abs(x / 2.0 ** 64 - turns_of(f * (1 - w) + f / factor * w)) <= 2.0 ** -50
    if kept:
        last = base ** (-2.0 * (rot // 2 - 1) / rot) / (2 * math.pi)
        assert abs(got[-1] / 2.0 ** 64 / last - kept) < 1e-6


@pytest.mark.parametrize("scaling", [T.ROPE_LINEAR, T.ROPE_BY_PARTS, T.ROPE_BY_TURNS])
def test_a_frequency_that_overflows_is_refused(lib, scaling):
    """1 / 1e-310 is no number in 64 bits, and has no fraction of a turn."""
    with pytest.raises(D.DsparkError):
        T.dspark_rotary_table(8, 1e4, scaling=scaling, factor=1e-310, original=4096, low=1, high=32)
