"""dspark_step_rows against its plain form: whole numbers, equal."""
import random

import pytest

torch = pytest.importorskip("torch")

import target_ref as ref  # noqa: E402
from speculative_decoding_draft_dspark_gb300 import dspark as D  # noqa: E402
from speculative_decoding_draft_dspark_gb300 import target as T  # noqa: E402

pytestmark = pytest.mark.gpu
I32 = torch.int32
LEFT = -77   # what is not written


def make(N, K, page, max_pages, seed, *, tree=False, prompts=0.2, chunk=40, ctx=200, extra_pages=500, max_rows=None,
         mask=True, owned="exact"):
    r = random.Random(seed)
    c = dict(N=N, K=K, page=page, max_pages=max_pages)
    c["draft_len"] = [r.randint(0, K) for _ in range(N)]
    c["mask"] = [int(r.random() >= prompts) for _ in range(N)] if mask else None
    c["chunk_len"] = [r.randint(0, chunk) for _ in range(N)]
    c["ctx_len"] = [r.choice([0, r.randint(0, ctx), page * r.randint(0, ctx // page)]) for _ in range(N)]
    g = torch.Generator().manual_seed(seed)
    c["tree"] = ref.tree_masks(g, N, K + 1) if tree else None
    if tree and mask:
        for n in range(N):
            if not c["mask"][n] or r.random() < 0.2:
                c["tree"][n] = 0      # a chain
    c["tokens"] = [[r.randint(0, 999) for _ in range(ctx + chunk + 1)] for _ in range(N)]
    c["draft_tokens"] = [[r.randint(0, 999) for _ in range(K)] for _ in range(N)]
    have = [min(-(-x // page), max_pages) for x in c["ctx_len"]]
    c["page_count"] = [min(max_pages, max(0, h + {"exact": 0, "more": r.randint(0, 2), "less": -r.randint(0, 2)}[owned]))
                       for h in have]
    c["num_pages"] = sum(c["page_count"]) + extra_pages + 1
    ids = list(range(c["num_pages"]))
    r.shuffle(ids)
    c["table"] = [[ids.pop() if k < c["page_count"][n] else LEFT for k in range(max_pages)] for n in range(N)]
    c["free"] = ids[:extra_pages]
    c["max_rows"] = max_rows or N * max(K + 1, chunk) + 5
    return c


def expected(c):
    table = [list(x) for x in c["table"]]
    want = ref.rows(c["draft_len"], c["mask"], c["chunk_len"], c["ctx_len"],
                    None if c["tree"] is None else c["tree"].tolist(), c["tokens"], c["draft_tokens"],
                    c["page_count"], c["free"], c["page"], c["max_pages"], c["num_pages"], c["max_rows"], table)
    return want, table


def put(c):
    t = lambda x, dt=I32: torch.tensor(x, dtype=dt, device="cuda")  # noqa: E731
    N, most = c["N"], c["max_rows"]
    s = {k: t(c[k]) for k in ("draft_len", "chunk_len", "ctx_len", "tokens", "draft_tokens", "page_count")}
    s["mask"] = None if c["mask"] is None else t(c["mask"], torch.uint8)
    s["tree"] = None if c["tree"] is None else c["tree"].cuda()
    s["free_pages"] = t(c["free"] if c["free"] else [0])
    s["free_count"] = t([len(c["free"])])
    wide = torch.full((N, c["max_pages"] + 3), LEFT, dtype=I32, device="cuda")    # rows apart
    wide[:, :c["max_pages"]] = t(c["table"])
    s["wide"], s["table"] = wide, wide[:, :c["max_pages"]]
    s["page_count_out"], s["free_count_out"] = (torch.full((n,), LEFT, dtype=I32, device="cuda") for n in (N, 1))
    s["cu_rows"], s["cu_out"] = (torch.full((N + 1,), LEFT, dtype=I32, device="cuda") for _ in range(2))
    for k in ("row_request", "position", "slot", "row_token", "out_row"):
        s[k] = torch.full((most,), LEFT, dtype=I32, device="cuda")
    s["ws"] = T.new_workspace(256)
    return s


def call(c, s, **kw):
    a = {**s, **kw}
    T.dspark_step_rows(a["draft_len"], a["mask"], a["chunk_len"], a["ctx_len"], a["tree"], a["tokens"],
                       a["draft_tokens"], a["page_count"], a["free_pages"], a["free_count"], a["table"],
                       a["page_count_out"], a["free_count_out"], a["cu_rows"], a["cu_out"], a["row_request"],
                       a["position"], a["slot"], a["row_token"], a["out_row"], a["ws"], page_size=c["page"],
                       num_pages=c["num_pages"])


def same(c, s, want, table, page_count="page_count_out", free_count="free_count_out"):
    assert s["cu_rows"].tolist() == want["cu_rows"]
    assert s["cu_out"].tolist() == want["cu_out"]
    for k in ("row_request", "position", "slot", "row_token", "out_row"):
        got = s[k].tolist()
        assert got[:len(want[k])] == want[k], k
        assert set(got[len(want[k]):]) <= {LEFT}, k
    assert s[page_count].tolist() == want["page_count"]
    assert s[free_count].tolist() == [want["free_count"]]
    assert s["table"].tolist() == table
    assert (s["wide"][:, c["max_pages"]:] == LEFT).all()


@pytest.mark.parametrize("kw", [
    dict(N=1, K=1, page=16, max_pages=20, prompts=0.0),
    dict(N=3, K=7, page=16, max_pages=20),
    dict(N=8, K=7, page=32, max_pages=9, mask=False),
    dict(N=33, K=15, page=16, max_pages=40, tree=True),
    dict(N=257, K=63, page=64, max_pages=10, tree=True, ctx=400),
    dict(N=1024, K=15, page=16, max_pages=40, extra_pages=9000),
    dict(N=1100, K=5, page=256, max_pages=3, extra_pages=3000),
    dict(N=40, K=7, page=16, max_pages=40, owned="more"),
    dict(N=40, K=7, page=16, max_pages=40, owned="less"),
    dict(N=5, K=3, page=128, max_pages=30, prompts=1.0, chunk=1500, ctx=300),
])
def test_rows(kw):
    for seed in range(3):
        c = make(seed=seed, **kw)
        want, table = expected(c)
        s = put(c)
        call(c, s)
        same(c, s, want, table)
        assert D.dspark_read_status(s["ws"]) == 0


def test_the_largest_batch():
    c = make(16384, 1, 16, 3, 1, ctx=40, chunk=5, extra_pages=20000)
    want, table = expected(c)
    s = put(c)
    call(c, s)
    same(c, s, want, table)


@pytest.mark.parametrize("N,max_rows", [(20, 37), (20, 1), (600, 5000), (2000, 4097)])
def test_rows_past_the_buffers_are_cut_off(N, max_rows):
    c = make(N, 7, 16, 20, 5, max_rows=max_rows, extra_pages=8000)
    want, table = expected(c)
    s = put(c)
    call(c, s)
    same(c, s, want, table)
    assert bool(D.dspark_read_status(s["ws"]) & T.DEV_ROWS_SHORT) == (want["cu_rows"][-1] == max_rows)


@pytest.mark.parametrize("extra", [0, 1, 7])
def test_a_free_list_that_runs_out(extra):
    c = make(30, 7, 16, 20, 6, extra_pages=extra)
    want, table = expected(c)
    assert -1 in want["slot"]
    s = put(c)
    call(c, s)
    same(c, s, want, table)
    assert D.dspark_read_status(s["ws"]) == T.DEV_PAGES_SHORT


def test_a_table_that_is_too_short():
    c = make(12, 7, 16, 5, 7, ctx=160)
    want, table = expected(c)
    assert -1 in want["slot"]
    s = put(c)
    call(c, s)
    same(c, s, want, table)
    assert D.dspark_read_status(s["ws"]) & T.DEV_PAGES_SHORT


def test_in_place_over_steps():
    """The counts given back in place: a second step goes on from the first."""
    c = make(300, 15, 16, 60, 8, extra_pages=9000, max_rows=8000)
    s = put(c)
    for _ in range(3):
        want, table = expected(c)
        call(c, s, page_count_out=s["page_count"], free_count_out=s["free_count"])
        same(c, s, want, table, "page_count", "free_count")
        c["page_count"], c["table"] = want["page_count"], table
        c["free"] = c["free"][:want["free_count"]]
        c["ctx_len"] = [x + want["cu_rows"][n + 1] - want["cu_rows"][n] for n, x in enumerate(c["ctx_len"])]
        s["ctx_len"].copy_(torch.tensor(c["ctx_len"], dtype=I32))
        for k in ("row_request", "position", "slot", "row_token", "out_row"):
            s[k].fill_(LEFT)


def test_lengths_and_pages_out_of_range():
    c = make(4, 3, 16, 8, 9, prompts=0.0, ctx=50)
    c["draft_len"], c["ctx_len"] = [-5, 99, 2, 0], [-3, 20, 33, 10]
    c["page_count"] = [0, 2, 3, 1]
    ids = iter(range(100))
    c["table"] = [[next(ids) if k < c["page_count"][n] else LEFT for k in range(8)] for n in range(4)]
    c["num_pages"], c["free"] = 600, list(range(100, 140))
    c["table"][1][1], c["table"][2][2] = 600, -4
    want, table = expected(c)
    s = put(c)
    call(c, s)
    same(c, s, want, table)
    assert D.dspark_read_status(s["ws"]) == T.DEV_LEN_OOR | T.DEV_PAGE_OOR


def test_lengths_that_add_up_to_more_than_32_bits():
    c = make(64, 3, 16, 8, 10, max_rows=100)
    c["mask"], c["chunk_len"] = [0] * 64, [(1 << 31) - 1] * 64
    c["ctx_len"][0] = 0
    c["page_count"][0] = 0
    c["table"][0] = [LEFT] * 8
    want, table = expected(c)
    s = put(c)
    call(c, s)
    same(c, s, want, table)


def test_without_tokens_and_chunks():
    c = make(9, 4, 16, 20, 11)
    c["chunk_len"] = [0] * 9
    want, table = expected(c)
    s = put(c)
    call(c, s, tokens=None, row_token=None, chunk_len=None)
    want["row_token"] = []
    same(c, s, want, table)


def test_in_a_graph_on_another_stream():
    c = make(50, 7, 16, 30, 12)
    want, table = expected(c)
    s = put(c)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        call(c, s)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call(c, s)
    for _ in range(2):
        for k in ("row_request", "position", "slot", "row_token", "out_row", "cu_rows", "cu_out"):
            s[k].fill_(LEFT)
        graph.replay()
        same(c, s, want, table)
