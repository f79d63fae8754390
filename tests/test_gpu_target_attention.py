"""dspark_tree_attention against softmax attention in 64 bits.

Tolerances.  P is rounded to bf16 for its product with V (2^-8 of each weight, so of
sum p |v|), and the output once (2^-8 of itself).  A score is a sum of d products of
bf16 numbers, exact in fp32, added up in fp32 with truncation: at most d / 16 + 1
additions of 16, each off by 2^-22 of the sum of |q k| at most, taken as 2^-17 of
scale * sum |q k| for d <= 256 (17 additions are 2^-17.9); the scaling, the exponential and the fp32 sums of up to
some thousand terms in chains of 64 and fewer are below 2^-18.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import target_ref as ref  # noqa: E402
from speculative_decoding_draft_dspark_gb300 import dspark as D  # noqa: E402
from speculative_decoding_draft_dspark_gb300 import target as T  # noqa: E402

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
HALF = torch.finfo(BF16).eps / 2


class Case:
    """Requests of (ctx, rows) over a shuffled paged cache; every slot that no
    request owns holds NaN."""

    def __init__(self, requests, heads=4, kv=2, d=64, page=16, tree=None, seed=0, layout="nhd", tail=3, spread=1.0,
                 pages=None):
        g = torch.Generator().manual_seed(seed)
        self.page, self.d, self.heads = page, d, heads
        self.ctx = [c for c, _ in requests]
        counts = [r for _, r in requests]
        self.cu = [0]
        for r in counts:
            self.cu.append(self.cu[-1] + r)
        R = self.cu[-1] + tail
        self.q = (torch.randn(R, heads, d, generator=g) * spread).to(BF16)
        ends = [max(c, 0) + r for c, r in requests]
        self.max_len = max(max(counts), 1)
        width = max(-(-e // page) for e in ends) + 1
        total = sum(-(-e // page) for e in ends) + 2
        ids = torch.randperm(total, generator=g).int()
        self.table = torch.full((len(requests), width), -5, dtype=torch.int32)
        self.k, self.v = (torch.full((total, page, kv, d), math.nan).to(BF16) for _ in range(2))
        at = 0
        for n, e in enumerate(ends):
            for k in range(-(-e // page)):
                id = int(ids[at])
                at += 1
                self.table[n, k] = id
                here = min(page, e - k * page)
                self.k[id, :here] = torch.randn(here, kv, d, generator=g).to(BF16)
                self.v[id, :here] = torch.randn(here, kv, d, generator=g).to(BF16)
        self.tree = ref.tree_masks(g, len(requests), tree) if isinstance(tree, int) else tree
        self.scale = 1.0 / math.sqrt(d)
        self.layout = layout

    def gpu(self):
        s = {}
        if self.layout == "hnd":
            s["k"], s["v"] = (x.transpose(1, 2).contiguous().cuda().transpose(1, 2) for x in (self.k, self.v))
        elif self.layout == "pair":
            both = torch.stack([self.k, self.v], 1).cuda()
            s["k"], s["v"] = both[:, 0], both[:, 1]
        else:
            s["k"], s["v"] = self.k.cuda(), self.v.cuda()
        if self.layout == "nhd":
            s["q"] = self.q.cuda()
        else:                       # rows apart, as in a fused projection
            wide = torch.randn(len(self.q), self.heads + 2, self.d).to(BF16)
            wide[:, :self.heads] = self.q
            s["q"] = wide.cuda()[:, :self.heads]
        s["table"], s["ctx"] = self.table.cuda(), torch.tensor(self.ctx, dtype=torch.int32, device="cuda")
        s["cu"] = torch.tensor(self.cu, dtype=torch.int32, device="cuda")
        s["tree"] = None if self.tree is None else self.tree.cuda()
        s["out"] = torch.full(self.q.shape, 5.0, dtype=BF16, device="cuda")
        s["lse"] = torch.full(self.q.shape[:2], 5.0, device="cuda")
        kv = self.k.shape[2]
        s["ws"] = T.new_workspace(T.dspark_attention_workspace_size(len(self.ctx), self.max_len, self.heads, kv,
                                                                    self.d))
        return s

    def call(self, s, **kw):
        a = {**s, **kw}
        T.dspark_tree_attention(a["q"], a["k"], a["v"], a["table"], a["ctx"], a["cu"], a["tree"], a["out"], a["lse"],
                                a["ws"], max_len=a.get("max_len", self.max_len), scale=self.scale)
        return s

    def score_error(self):
        """scale * sum |q k| at most, by 2^-17."""
        big = float(torch.nan_to_num(self.k.double(), nan=0.0, posinf=0.0, neginf=0.0).abs().amax())
        return 2.0 ** -17 * self.scale * float(self.q.double().abs().sum(-1).amax()) * big

    def check(self, s, status=0):
        assert D.dspark_read_status(s["ws"]) == status
        R = self.cu[-1]
        want, lse, size = ref.attention(self.q, self.k, self.v, self.table, self.ctx, self.cu, self.tree, self.scale)
        out, got = s["out"].cpu().double(), s["lse"].cpu().double()
        assert (out[R:] == 5.0).all() and (got[R:] == 5.0).all()
        out, got, want, lse, size = out[:R], got[:R], want[:R], lse[:R], size[:R]
        e = self.score_error() + 2.0 ** -18
        fine = want.isfinite()
        assert torch.equal(fine, out.isfinite())
        tol = HALF * want.abs() + size * (HALF + 2 * e)
        bad = ((out - want).abs() > tol * 1.001) & fine
        assert not bad.any(), (bad.nonzero()[:5], out[bad][:5], want[bad][:5])
        none = lse == -math.inf
        assert torch.equal(none, got == -math.inf)
        ok = lse.isfinite()
        assert torch.equal(ok, got.isfinite())
        assert ((got - lse).abs()[ok] <= e + lse.abs()[ok] * 2.0 ** -22).all()

    def run(self, status=0, **kw):
        s = self.call(self.gpu(), **kw)
        self.check(s, status)
        return s


@pytest.mark.parametrize("requests", [
    [(0, 1)], [(1, 1)], [(15, 1)], [(16, 1)], [(63, 1)], [(64, 1)], [(63, 2)], [(127, 1), (128, 1), (129, 1)],
    [(0, 5), (100, 0), (64, 8), (1000, 1), (0, 0), (17, 3)], [(3000, 1)], [(700, 8)] * 3,
    [(i % 97, 1 + i % 4) for i in range(60)]])
@pytest.mark.parametrize("page", [16, 64])
def test_chains(requests, page):
    Case(requests, page=page).run()


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (6, 2), (8, 8), (32, 8), (48, 1), (128, 1), (5, 5)])
def test_groups_of_heads(heads, kv):
    Case([(70, 9), (5, 1), (200, 3)], heads=heads, kv=kv).run()


@pytest.mark.parametrize("d", [8, 24, 64, 72, 80, 128, 136, 192, 256])
def test_heads_widths(d):
    Case([(100, 7), (1, 1), (300, 2)], d=d, seed=d).run()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", ["nhd", "hnd", "pair"])
def test_pages_and_layouts(page, layout):
    Case([(page * 2 - 1, 3), (page, 1), (page * 3 + 5, 20)], page=page, layout=layout, d=128).run()


@pytest.mark.parametrize("requests,heads,kv,d", [
    ([(0, 130)], 1, 1, 64), ([(50, 200)], 4, 1, 64), ([(0, 300)], 4, 4, 128), ([(129, 65), (3, 129)], 6, 2, 64),
    ([(0, 70)], 5, 1, 256), ([(10, 40), (2, 1), (0, 100)], 16, 2, 128)])
def test_chunks_of_prompts(requests, heads, kv, d):
    """More rows than a tile holds, with and without a context."""
    Case(requests, heads=heads, kv=kv, d=d).run()


@pytest.mark.parametrize("width", [1, 2, 7, 25, 64])
@pytest.mark.parametrize("ctx", [0, 1, 40, 63, 64, 500])
def test_trees(width, ctx):
    Case([(ctx, width), (max(ctx - 1, 0), min(width, 3)), (ctx, width)], tree=width, heads=8, kv=2, seed=width).run()


def test_rows_that_attend_nothing_or_not_themselves():
    """With no context, rows whose mask is 0 or reaches past the request's rows are 0
    and their lse -inf; a mask may be anything, also without the row itself."""
    m = torch.tensor([[1, 0, 1 << 40, 0b110, 0b1010, -(1 << 63)]])
    c = Case([(0, 6)], tree=m, heads=2, kv=1)
    s = c.run()
    assert (s["out"][1:3] == 0).all() and (s["lse"][1:3] == -math.inf).all()
    c = Case([(0, 6), (33, 6)], tree=torch.cat([m, m]), heads=2, kv=1)
    c.run()


def test_masks_that_make_a_chain():
    """More rows than masks, or no bit 0 in the first: chains, among trees."""
    m = ref.tree_masks(torch.Generator().manual_seed(1), 4, 5)
    m[2] &= ~1
    Case([(20, 5), (20, 6), (20, 5), (0, 40)], tree=m).run()


def test_one_long_context_is_split():
    """As long as all CTAs together, and a cut that falls into a short one."""
    Case([(20000, 1)], heads=8, kv=1, d=128).run()
    Case([(37, 1), (9001, 2), (5, 1), (4000, 1)], heads=4, kv=2).run()


def test_many_requests():
    Case([(i * 7 % 41, i % 3) for i in range(500)], heads=2, kv=1).run()


def test_large_scores():
    """A softmax that is one token's, whose maximum grows from tile to tile."""
    c = Case([(900, 3)], spread=30.0)
    c.run()
    n = 900
    for t in range(n):       # growing along the context
        id = int(c.table[0, t // c.page])
        c.k[id, t % c.page] = (c.k[id, t % c.page].float() * (1 + t / 50)).to(BF16)
    c.run()


def test_the_types_lowest_values():
    """Scores as large as fp32 holds, both ways, do not overflow: q k about 1e38."""
    c = Case([(130, 2)], heads=1, kv=1)
    c.q[:] = 0
    c.q[:, :, 0] = 1e19
    c.k[..., 1:] = 0
    for t in range(132):
        c.k[int(c.table[0, t // 16]), t % 16, 0, 0] = -1e19 if t % 2 else 1e18
    want, lse, _ = ref.attention(c.q, c.k, c.v, c.table, c.ctx, c.cu, None, c.scale)
    s = c.call(c.gpu())
    # equal scores at the top: a mean of every second value, to P's and the output's rounding
    got = s["out"][:2].cpu().double()
    assert ((got - want[:2]).abs() <= 2 * HALF * (1 + want[:2].abs())).all()
    assert ((s["lse"][:2].cpu().double() / lse[:2] - 1).abs() < 2.0 ** -20).all()


@pytest.mark.parametrize("tree", [None, 12])
@pytest.mark.parametrize("ctx", [0, 30, 64])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("heads", [6, 32])
def test_what_is_not_attended_has_no_effect(tree, ctx, value, heads):
    """A token of the step with bad keys and values changes the rows that attend it,
    and no bit of the others; with 36 packed rows, and with 192."""
    requests = [(ctx, 12), (ctx + 3, 12)]
    half = heads // 2
    c = Case(requests, tree=tree, heads=heads, kv=2, d=128)
    clean = c.call(c.gpu())
    for which in ("k", "v", "both"):
        for j in (0, 4, 11):
            d = Case(requests, tree=tree, heads=heads, kv=2, d=128)
            t = ctx + j
            id = int(d.table[0, t // 16])
            if which != "v":
                d.k[id, t % 16, 0, 5] = value
            if which != "k":
                d.v[id, t % 16, 0, 7] = value
            s = d.call(d.gpu())
            masks = None if tree is None else [int(x) for x in d.tree[0]]
            for r in range(24):
                hit = r < 12 and j in ref.attended(masks, 12, r)
                if not hit:
                    assert torch.equal(s["out"][r], clean["out"][r]) and torch.equal(s["lse"][r], clean["lse"][r])
                else:
                    assert torch.equal(s["out"][r, half:], clean["out"][r, half:])     # the other key head
                    if which == "v":
                        assert not s["out"][r, :half, 7].isfinite().any()
                        assert torch.equal(s["out"][r, :half, 8:], clean["out"][r, :half, 8:])
                        assert torch.equal(s["lse"][r], clean["lse"][r])


def test_bad_values_in_the_context_reach_every_row():
    c = Case([(100, 5)], heads=2, kv=1)
    id = int(c.table[0, 3])
    c.v[id, 2, 0, 9], c.v[id, 4, 0, 11] = math.inf, math.nan
    s = c.call(c.gpu())
    assert (s["out"][:5, :, 9] == math.inf).all() and s["out"][:5, :, 11].isnan().all()
    other = [i for i in range(64) if i not in (9, 11)]
    assert s["out"][:5, :, other].isfinite().all()


@pytest.mark.parametrize("heads,kv,page", [(4, 2, 16), (48, 1, 16), (96, 1, 64)])
def test_pages_that_are_not_there_are_left_out(heads, kv, page):
    c = Case([(page * 12, 4), (page * 5 + 10, 2)], heads=heads, kv=kv, page=page)
    c.table[0, 3], c.table[0, 7], c.table[1, 0] = -1, len(c.k), 1 << 30
    c.run(status=T.DEV_PAGE_OOR)
    c = Case([(40, 3)])
    c.table[:] = -1           # nothing left: as if it attended nothing
    s = c.run(status=T.DEV_PAGE_OOR)
    assert (s["out"][:3] == 0).all()


def test_a_table_that_ends_early():
    c = Case([(200, 4), (30, 2)])
    s = c.gpu()
    s["table"] = s["table"][:, :10]      # rows stay apart
    c.call(s)
    c.table = c.table[:, :10]
    c.check(s, status=T.DEV_PAGE_OOR)


def test_lengths_out_of_range():
    c = Case([(-7, 3), (20, 6), (50, 2)])
    s = c.gpu()
    c.call(s, max_len=4)
    assert D.dspark_read_status(s["ws"]) == T.DEV_LEN_OOR
    assert (s["out"][7:9] == 5.0).all()           # rows 4 and 5 of the second request
    c.cu = [0, 3, 7, 7]
    full = Case([(-7, 3), (20, 6), (50, 2)])
    want, _, size = ref.attention(full.q, full.k, full.v, full.table, full.ctx, [0, 3, 9, 11], None, full.scale)
    got = s["out"].cpu().double()
    for r in (0, 1, 2, 3, 4, 5, 6, 9, 10):
        assert ((got[r] - want[r]).abs() <= HALF * want[r].abs() + size[r] * (HALF + 2.0 ** -8)).all()


def test_offsets_outside_the_rows():
    """cu_rows that are not within [0, R] stay within it."""
    c = Case([(20, 2), (30, 3)], tail=2)
    c.max_len = 5
    s = c.gpu()
    s["cu"] = torch.tensor([0, 2, 1 << 30], dtype=torch.int32, device="cuda")
    c.call(s)
    assert torch.equal(s["out"][:2], c.call(c.gpu())["out"][:2])


def test_the_same_bits_every_time():
    c = Case([(3000, 2), (50, 30), (700, 1)], heads=8, kv=2, d=128)
    s = c.gpu()
    first = None
    for _ in range(20):
        s["out"].fill_(5.0)
        c.call(s)
        got = s["out"].clone(), s["lse"].clone()
        first = first or got
        assert torch.equal(first[0], got[0]) and torch.equal(first[1], got[1])


def test_without_lse():
    c = Case([(100, 3)])
    s = c.gpu()
    c.call(s, lse=None)
    assert (s["lse"] == 5.0).all()
    s["lse"] = c.call(c.gpu())["lse"]
    c.check(s)


def test_two_streams_and_graphs():
    """Two calls at once with a workspace each, then replays of both as graphs, with
    lengths that change in between."""
    cases = [Case([(900, 4), (70, 2)], heads=8, kv=1, d=128, seed=1), Case([(2000, 1)], heads=4, kv=4, seed=2)]
    states = [c.gpu() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, st in zip(cases, states, streams):
            with torch.cuda.stream(st):
                c.call(s)
    torch.cuda.synchronize()
    for c, s in zip(cases, states):
        c.check(s)
    graphs = []
    for c, s in zip(cases, states):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call(s)
        graphs.append(g)
    cases[0].ctx, cases[1].ctx = [850, 64], [1]
    for c, s in zip(cases, states):
        s["ctx"].copy_(torch.tensor(c.ctx, dtype=torch.int32))
    torch.cuda.synchronize()
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for c, s in zip(cases, states):
        c.check(s)


def test_a_cache_past_32_bits():
    c = Case([(60, 3)], heads=2, kv=1)
    s = c.gpu()
    n = len(c.k)
    stride = (1 << 32) // n // 64 * 64 + (1 << 20)
    buf = torch.zeros(n * stride + 2 * (1 << 20), dtype=BF16, device="cuda")
    assert n * stride > 1 << 32
    for name, at in (("k", 0), ("v", 1 << 19)):
        view = buf[at:].as_strided(c.k.shape, (stride, 64, 64, 1), at)
        view.copy_(s[name])
        s[name] = view
    c.call(s)
    c.check(s)


def test_a_run_of_decoding_steps_matches_a_chunk():
    """One token at a time, and all at once: the same attention."""
    c = Case([(100, 9)], heads=8, kv=2, d=128)
    s = c.call(c.gpu())
    for j in range(9):
        one = c.gpu()
        one["cu"] = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        one["ctx"] += j
        one["q"] = one["q"][j:j + 1]
        one["out"], one["lse"] = one["out"][:1], one["lse"][:1]
        c.call(one, max_len=1)
        assert ((one["lse"][0] - s["lse"][j]).abs() < 2 * c.score_error()).all()
        assert ((one["out"][0].float() - s["out"][j].float()).abs() <= 4 * HALF * (1 + s["out"][j].float().abs())).all()


@pytest.mark.parametrize("requests,heads,kv,d,tree,page", [
    ([(3000, 1), (500, 40), (0, 200), (64, 8), (900, 33)], 8, 2, 128, None, 16),
    ([(300, 25), (0, 25), (64, 3), (127, 25)], 32, 1, 64, 25, 32),
    ([(5000, 64), (10, 64)], 32, 4, 128, 64, 64),
    ([(130, 17), (2000, 2)], 128, 1, 80, None, 256),
    ([(2500, 300)], 1, 1, 64, None, 128)])
def test_few_and_many_packed_rows_together(requests, heads, kv, d, tree, page):
    """Requests for both kernels in one call, and cut items of both."""
    Case(requests, heads=heads, kv=kv, d=d, tree=tree, page=page).run()


def test_many_packed_rows_the_same_bits_every_time():
    """Blocks of rows whose products follow each other in tensor memory."""
    c = Case([(700, 130), (64, 40), (0, 90), (2000, 3)], heads=16, kv=4, d=128)
    s = c.call(c.gpu())
    c.check(s)
    first = s["out"].clone(), s["lse"].clone()
    for _ in range(300):
        s["out"].fill_(5.0)
        c.call(s)
        assert torch.equal(first[0], s["out"]) and torch.equal(first[1], s["lse"])


def test_bad_values_in_a_chunk_of_a_prompt():
    """Rows before a token with bad values are as they were, bit for bit, in a chunk
    that takes several blocks."""
    requests = [(70, 150)]
    clean = Case(requests, heads=8, kv=2)
    a = clean.call(clean.gpu())
    for j in (0, 63, 64, 100, 149):
        c = Case(requests, heads=8, kv=2)
        t = 70 + j
        c.v[int(c.table[0, t // 16]), t % 16, 1, 3] = math.nan
        s = c.call(c.gpu())
        assert torch.equal(s["out"][:j], a["out"][:j])
        assert s["out"][j:150, 4:, 3].isnan().all() and s["out"][j:150, 4:, 4:].isfinite().all()
        assert torch.equal(s["out"][:150, :4], a["out"][:150, :4]) and torch.equal(s["lse"], a["lse"])


def test_no_rows_at_all():
    c = Case([(5, 0), (0, 0), (100, 0)], heads=8, kv=2)
    s = c.call(c.gpu())
    assert (s["out"] == 5.0).all() and (s["lse"] == 5.0).all() and D.dspark_read_status(s["ws"]) == 0


def test_thousands_of_requests():
    c = Case([(i % 23, 1 + (i % 50 == 0)) for i in range(4000)], heads=2, kv=1, d=64)
    c.run()


def test_the_largest_length():
    """ctx_len at the end of 32 bits: as one that fills the table."""
    c = Case([(150, 3), (20, 2)])
    full = Case([(150, 3), (20, 2)])
    for x in (c.k, c.v, full.k, full.v):
        x.nan_to_num_(0.0)            # what no request wrote counts here
    s, t = c.gpu(), full.gpu()
    s["ctx"][0] = (1 << 31) - 1
    t["ctx"][0] = c.table.shape[1] * 16
    c.call(s)
    full.call(t)
    assert D.dspark_read_status(s["ws"]) == D.dspark_read_status(t["ws"]) == T.DEV_PAGE_OOR
    assert torch.equal(s["out"], t["out"]) and torch.equal(s["lse"], t["lse"])
    assert s["out"].isfinite().all()
