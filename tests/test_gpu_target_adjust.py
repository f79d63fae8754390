"""dspark_adjust_logits against the formula in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")

import target_ref as ref  # noqa: E402
from speculative_decoding_draft_dspark_gb300 import dspark as D  # noqa: E402
from speculative_decoding_draft_dspark_gb300 import target as T  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Case:
    def __init__(self, counts, vocab, dtype=BF16, K=7, width=60, tree=False, seed=0, bias=5, masked=True, prompt=True,
                 penalties=True, tail=2, few=30):
        g = torch.Generator().manual_seed(seed)
        N = len(counts)
        self.dtype, self.vocab = dtype, vocab
        self.cu = [0]
        for r in counts:
            self.cu.append(self.cu[-1] + r)
        R = self.cu[-1] + tail
        self.logits = (torch.randn(R, vocab, generator=g) * 3).to(dtype)
        some = torch.randint(0, vocab, (few,), generator=g)
        some[0], some[-1] = 0, vocab - 1
        pick = lambda *s: some[torch.randint(0, few, s, generator=g)].int()  # noqa: E731
        a = self.a = {"tokens": pick(N, width), "hist_len": torch.randint(0, width + 1, (N,), generator=g, dtype=I32)}
        a["prompt_len"] = torch.randint(0, width + 1, (N,), generator=g, dtype=I32) if prompt else None
        a["draft_tokens"] = pick(N, K) if K else None
        a["tree"] = ref.tree_masks(g, N, K + 1) if tree else None
        for k in ("repetition", "frequency", "presence"):
            a[k] = torch.rand(N, generator=g) * 2 + (0.5 if k == "repetition" else -0.5) if penalties else None
        if bias:
            a["bias_token"] = torch.cat([pick(N, bias - bias // 2), torch.randint(0, vocab, (N, bias // 2), generator=g,
                                                                                   dtype=I32)], 1)
            a["bias_value"] = torch.randn(N, bias, generator=g)
            a["bias_count"] = torch.randint(0, bias + 1, (N,), generator=g, dtype=I32)
        if masked:
            m = max(1, R // 2)
            words = (vocab + 31) // 32
            a["mask"] = torch.randint(-(1 << 31), 1 << 31, (m, words), generator=g).int()
            a["mask"][torch.rand(m, words, generator=g) < 0.3] = 0
            a["mask"][torch.rand(m, words, generator=g) < 0.3] = -1
            a["mask_index"] = torch.randint(-1, m, (R,), generator=g, dtype=I32)

    def gpu(self, in_place=True, pad=0):
        s = {k: None if v is None else v.cuda() for k, v in self.a.items()}
        wide = torch.full((len(self.logits), self.vocab + pad), 7.0, dtype=self.dtype, device="cuda")
        s["wide"], s["logits"] = wide, wide[:, :self.vocab]
        s["logits"].copy_(self.logits)
        s["out"] = s["logits"] if in_place else torch.full_like(self.logits, 9.0, device="cuda")
        s["cu"] = torch.tensor(self.cu, dtype=I32, device="cuda")
        s["ws"] = T.new_workspace(256)
        return s

    def call(self, s):
        T.dspark_adjust_logits(s["logits"], s["cu"], s["tokens"], s["hist_len"], s["prompt_len"], s["draft_tokens"],
                               s["tree"], s["out"], s["ws"], **{k: s.get(k) for k in (
                                   "repetition", "frequency", "presence", "bias_token", "bias_value", "bias_count",
                                   "mask", "mask_index")})
        return s

    def check(self, s, in_place=True, status=0):
        """Six operations in fp32 (and the sum of a token's biases), each off by 2^-24
        of what it is applied to, and the rounding to the type."""
        assert D.dspark_read_status(s["ws"]) == status
        want, size = ref.adjust(self.logits, self.cu, **self.a)
        got, R = s["out"].cpu().double(), self.cu[-1]
        tail = self.logits[R:].double() if in_place else torch.full((len(got) - R, self.vocab), 9.0, dtype=torch.float64)
        assert torch.equal(got[R:], tail)
        got, want, size = got[:R], want[:R], size[:R]
        cut = want == -math.inf
        assert torch.equal(cut, got == -math.inf)
        tol = want.abs() * torch.finfo(self.dtype).eps / 2 + 16 * 2.0 ** -24 * size
        changed = want != self.logits[:R].double()
        assert torch.equal(got[~changed], want[~changed])
        assert ((got - want).abs() <= tol)[~cut].all()
        if s["wide"].shape[1] > self.vocab:
            assert (s["wide"][:, self.vocab:] == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("vocab,pad", [(1, 0), (31, 0), (32, 5), (100, 28), (8192, 0), (8193, 0), (8200, 8), (20011, 3),
                                       (32768, 0)])
def test_sizes(vocab, pad, in_place, dtype):
    for tree in (False, True):
        c = Case([3, 0, 8, 1], vocab, dtype, tree=tree, seed=vocab)
        c.check(c.call(c.gpu(in_place, pad)), in_place)


@pytest.mark.parametrize("kw", [
    dict(bias=0, masked=False), dict(bias=0), dict(masked=False), dict(penalties=False), dict(prompt=False),
    dict(K=0), dict(K=63, counts=[64, 1, 30], tree=True), dict(K=63, counts=[64, 1, 30]), dict(bias=300, few=40),
    dict(width=5000, few=900, counts=[8]), dict(width=20000, few=2900, counts=[4, 1], bias=50),
    dict(width=20000, few=2900, counts=[4, 9], tree=True), dict(bias=1024, few=900), dict(counts=[1] * 300, K=1), dict(counts=[40], K=5),
    dict(penalties=False, bias=0)])
def test_parts(kw):
    kw = dict(kw)
    for in_place in (True, False):
        c = Case(kw.pop("counts", [5, 2, 8]) if "counts" in kw else [5, 2, 8], 3001, **kw)
        c.check(c.call(c.gpu(in_place)), in_place)


def test_a_token_many_times():
    """The whole history, the drafts and every bias one token: counts, and an ordered sum."""
    c = Case([8], 50, F32, width=3000, bias=100)
    for k in ("tokens", "draft_tokens", "bias_token"):
        c.a[k].fill_(17)
    c.a["hist_len"].fill_(3000)
    c.a["prompt_len"].fill_(10)
    c.a["bias_count"].fill_(100)
    c.a["mask_index"].fill_(-1)
    s = c.call(c.gpu())
    want, size = ref.adjust(c.logits, c.cu, **c.a)
    # the biases' sum: 100 additions
    assert ((s["out"][:8].cpu().double() - want[:8]).abs() <= 120 * 2.0 ** -24 * size[:8]).all()


def test_special_logits():
    """NaN stays NaN unless masked, infinities as the formula has them."""
    c = Case([4], 640, masked=True, bias=0, few=600, width=400)
    c.logits[:, ::7], c.logits[:, 1::7], c.logits[:, 2::7] = math.nan, math.inf, -math.inf
    c.logits[:, 3::7] = torch.finfo(BF16).min
    s = c.call(c.gpu())
    want, _ = ref.adjust(c.logits, c.cu, **c.a)
    got = s["out"][:4].cpu().double()
    want = want[:4]
    assert torch.equal(got.isnan(), want.isnan())
    big = want.abs() > torch.finfo(BF16).max
    assert torch.equal(got[big].sign(), want[big].sign())
    lost = (want == -math.inf) & ~big
    assert not lost.any()


def test_a_mask_that_forbids_everything():
    c = Case([2], 9000, masked=True)
    c.a["mask"].zero_()
    c.a["mask_index"].zero_()
    s = c.call(c.gpu())
    assert (s["out"][:2] == -math.inf).all()
    c.check(s)


def test_tokens_and_indices_out_of_range():
    c = Case([3, 3], 100, K=4)
    a = c.a
    a["tokens"][0, 0], a["tokens"][1, 0], a["draft_tokens"][0, 0], a["bias_token"][1, 0] = -1, 100, 1 << 30, -(1 << 31)
    a["hist_len"].fill_(60)
    a["bias_count"].fill_(5)
    c.check(c.call(c.gpu()), status=D.DEV_TOKEN_OOR)
    c = Case([3, 3], 100)
    c.a["hist_len"][0], c.a["hist_len"][1] = 61, -1
    c.a["mask_index"][1] = 1000
    s = c.call(c.gpu())
    c.a["hist_len"][0], c.a["hist_len"][1] = 60, 0
    c.check(s, status=T.DEV_LEN_OOR)


def test_the_same_bits_every_time():
    c = Case([8] * 20, 30000, few=3000, width=2000, bias=60)
    s = c.gpu(False)
    first = None
    for _ in range(10):
        c.call(s)
        first = s["out"].clone() if first is None else first
        assert torch.equal(first, s["out"])


def test_in_a_graph_with_lengths_that_change():
    c = Case([5, 3], 5000)
    s = c.gpu(False)
    c.call(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(s)
    c.a["hist_len"] = torch.tensor([3, 55], dtype=I32)
    s["hist_len"].copy_(c.a["hist_len"])
    g.replay()
    c.check(s, False)


def test_rows_past_32_bits():
    """A row stride that puts the last row 2^32 elements in."""
    c = Case([4], 3000, tail=0)
    s = c.gpu()
    stride = (1 << 32) // 3 + 8
    big = torch.zeros(3 * stride + 3000, dtype=BF16, device="cuda").as_strided((4, 3000), (stride, 1))
    big.copy_(c.logits)
    s["logits"] = s["out"] = big
    c.call(s)
    c.check(s)


def test_a_request_with_most_of_the_rows():
    """Its rows times its distinct tokens, one CTA's work by the average request, are
    more than 2^31.  A single fp32 subtraction: exact but for the rounding to bf16."""
    N, rows, vocab = 304, 270000, 8192
    R = rows + N - 1
    g = torch.Generator(device="cuda").manual_seed(0)
    s = {"logits": torch.empty(R, vocab, dtype=BF16, device="cuda").normal_(generator=g)}
    before, s["out"], s["ws"] = s["logits"].clone(), s["logits"], T.new_workspace(256)
    s["cu"] = torch.cat([torch.zeros(1), torch.arange(N) + rows]).to(I32).cuda()
    s["tokens"] = torch.randperm(vocab, generator=g, device="cuda").to(I32).expand(N, vocab).contiguous()
    s["hist_len"] = torch.full((N,), vocab, dtype=I32, device="cuda")
    s["prompt_len"] = s["draft_tokens"] = s["tree"] = None
    s["presence"] = torch.linspace(0.5, 1.5, N, device="cuda")
    Case.call(None, s)
    assert D.dspark_read_status(s["ws"]) == 0
    pres = torch.cat([s["presence"][:1].expand(rows), s["presence"][1:]])
    for a in range(0, R, 30000):
        b = slice(a, min(R, a + 30000))
        assert torch.equal(s["out"][b], (before[b].float() - pres[b, None]).to(BF16))


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("counts,kw", [
    ([64, 1, 30], dict(K=63, tree=True)), ([64, 1, 30], dict(K=63)), ([8], dict(width=5000, few=900)),
    ([4, 1], dict(width=20000, few=2900, bias=50)), ([4, 9], dict(width=20000, few=2900, tree=True)),
    ([1] * 300, dict(K=1)), ([40], dict(K=5)), ([0, 0, 3], dict(K=2))])
def test_rows_of_a_request(counts, kw, dtype, in_place):
    c = Case(counts, 3001, dtype, **kw)
    c.check(c.call(c.gpu(in_place)), in_place)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bias", [0, 5])
def test_infinities_and_overflows(bias, dtype, in_place):
    """Every entry: infinities and NaN as in 64 bits; what is past the type's largest
    value by more than half a step, an infinity of its sign; all else to the usual bounds.
    Between them, within the 16 * 2^-24 of fp32's operations, either."""
    c = Case([4], 640, dtype, masked=True, bias=bias, few=600, width=400)
    top = torch.finfo(dtype)
    c.logits[:, ::7], c.logits[:, 1::7], c.logits[:, 2::7] = math.nan, math.inf, -math.inf
    c.logits[:, 3::7], c.logits[:, 4::14] = top.min, top.max
    s = c.call(c.gpu(in_place))
    want, size = ref.adjust(c.logits, c.cu, **c.a)
    got, want, size = s["out"][:4].cpu().double(), want[:4], size[:4]
    assert torch.equal(got.isnan(), want.isnan())
    cut = want.isinf()
    assert cut.any() and torch.equal(got[cut], want[cut])
    edge = top.max * (1.0 + top.eps / 4)                    # half a step past the largest value
    finite = want.isfinite()
    past, within = finite & (want.abs() > edge * (1 + 2.0 ** -20)), finite & (want.abs() < edge * (1 - 2.0 ** -20))
    assert past.any() and within.any()
    assert torch.equal(got[past], want[past].sign() * math.inf)
    tol = want.abs() * top.eps / 2 + 16 * 2.0 ** -24 * size
    assert ((got - want).abs() <= tol)[within].all()


@pytest.mark.parametrize("in_place", [True, False])
def test_columns_of_a_wide_text_buffer(in_place):
    """As many as the histories may reach, and all of them: the same bits."""
    c = Case([3, 8, 1], 20011, width=300)
    outs = []
    for narrow in (True, False):
        s = c.gpu(in_place)
        wide = torch.full((3, 20000), 77, dtype=I32, device="cuda")
        wide[:, :300] = s["tokens"]
        s["tokens"] = wide[:, :300] if narrow else wide
        c.check(c.call(s), in_place)
        outs.append(s["out"].clone())
    assert torch.equal(*outs)
