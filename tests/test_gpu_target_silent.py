"""Counts, lengths and pages out of range: what is left out or clamped is said in the
status word, as well where everything else goes on."""
import pytest

torch = pytest.importorskip("torch")

import test_gpu_target_adjust as logits  # noqa: E402
import test_gpu_target_attention as attention  # noqa: E402
import test_gpu_target_rows as steps  # noqa: E402
from speculative_decoding_draft_dspark_gb300 import dspark as D  # noqa: E402
from speculative_decoding_draft_dspark_gb300 import target as T  # noqa: E402

pytestmark = pytest.mark.gpu
I32 = torch.int32


def step(change, status, in_place=False):
    c = steps.make(6, 3, 16, 8, 2, prompts=0.0, ctx=50)
    change(c)
    want, table = steps.expected(c)
    s = steps.put(c)
    if "free_count" in c:
        s["free_count"].fill_(c["free_count"])
    out = dict(page_count_out=s["page_count"], free_count_out=s["free_count"]) if in_place else {}
    steps.call(c, s, **out)
    steps.same(c, s, want, table, *(("page_count", "free_count") if in_place else ()))
    assert D.dspark_read_status(s["ws"]) == status


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("count", [-1, -(1 << 31), 9, (1 << 31) - 1])
def test_page_counts(count, in_place):
    def change(c):
        c["page_count"][2] = count
        # so many pages are in its row of the table, or none
        c["table"][2] = [k % 5 for k in range(8)] if count > 0 else [steps.LEFT] * 8
    step(change, T.DEV_LEN_OOR, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_a_free_count_past_the_list(in_place):
    step(lambda c: c.update(free_count=len(c["free"]) + 1), T.DEV_LEN_OOR, in_place)


def test_a_negative_free_count():
    def change(c):
        c["free"], c["free_count"] = [], -3
        c["page_count"] = [8] * 6
        c["table"] = [[k for k in range(8)] for _ in range(6)]
    step(change, T.DEV_LEN_OOR)


@pytest.mark.parametrize("bad", [-7, -1, -(1 << 31), "num_pages", (1 << 31) - 1])
@pytest.mark.parametrize("own", [True, False])
def test_a_free_list_with_pages_that_are_not_there(bad, own):
    """Popped for a row, or for a page before the request's first row."""
    def change(c):
        c["ctx_len"] = [16, 5, 5, 5, 5, 5]
        c["page_count"] = [1 if own else 0, 1, 1, 1, 1, 1]
        c["table"] = [[n if k < c["page_count"][n] else steps.LEFT for k in range(8)] for n in range(6)]
        c["free"][-1] = c["num_pages"] if bad == "num_pages" else bad
    step(change, T.DEV_PAGE_OOR)


@pytest.mark.parametrize("dtype", [logits.BF16, logits.F32])
@pytest.mark.parametrize("count,as_if", [(-1, 0), (-(1 << 31), 0), (6, 5), ((1 << 31) - 1, 5)])
def test_bias_counts(count, as_if, dtype):
    c = logits.Case([3, 2], 700, dtype)
    c.a["bias_count"] = torch.tensor([2, count], dtype=I32)
    s = c.call(c.gpu())
    c.a["bias_count"][1] = as_if
    c.check(s, status=T.DEV_LEN_OOR)


@pytest.mark.parametrize("heads", [4, 96])      # few packed rows, and more than a block
@pytest.mark.parametrize("ctx", [-1, -(1 << 31)])
def test_negative_lengths(ctx, heads):
    c = attention.Case([(0, 3), (40, 2), (0, 0)], heads=heads, kv=2)
    s = c.gpu()
    s["ctx"][0] = ctx
    c.call(s)
    c.check(s, status=T.DEV_LEN_OOR)
    c = attention.Case([(40, 2), (0, 0)])        # of a request without rows: no matter
    s = c.gpu()
    s["ctx"][1] = ctx
    c.call(s)
    c.check(s)
