"""Inputs that the kernel just before wrote, other ones in every call and nothing
between the calls: operators of several kernels, whose later ones may begin early."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_target_adjust import BF16, Case as Logits  # noqa: E402
from test_gpu_target_attention import Case as Rows  # noqa: E402

pytestmark = pytest.mark.gpu
CALLS = 60


@pytest.mark.parametrize("counts", [[3], [8, 1] * 30])
@pytest.mark.parametrize("in_place", [True, False])
def test_logits(counts, in_place):
    """Lengths, texts, drafts, biases and the rows' offsets, and masks of a few rows: the
    first kernel takes a few CTAs, the second one all SMs."""
    cases = [Logits(counts if k == 0 else counts[::-1], 3001, BF16, seed=k) for k in range(2)]
    states = [c.gpu(in_place) for c in cases]
    wanted = []
    for c, s in zip(cases, states):
        c.call(s)
        torch.cuda.synchronize()
        c.check(s, in_place)
        wanted.append(s["out"].clone())
    s = cases[0].gpu(in_place)
    names = [k for k, v in s.items() if v is not None and k not in ("wide", "logits", "out", "ws")]
    raw = [c.logits.cuda() for c in cases]
    got = torch.empty(CALLS, *wanted[0].shape, dtype=BF16, device="cuda")
    for i in range(CALLS):
        s["logits"].copy_(raw[i % 2])
        s["out"].fill_(9.0) if not in_place else None
        for k in names:
            s[k].copy_(states[i % 2][k])
        cases[0].call(s)
        got[i].copy_(s["out"])
    for i in range(CALLS):
        assert torch.equal(got[i], wanted[i % 2]), i


@pytest.mark.parametrize("requests", [
    [(900, 40), (30, 2), (0, 70), (500, 1)],      # few and many packed rows: both kernels
    [(900, 40), (30, 2), (500, 1)],               # the same of trees
    [(3000, 1)], [(700, 90)]])
def test_attention(requests):
    """Lengths, pages, offsets, queries and trees: the second kernel plans its own part."""
    width = max(r for _, r in requests) if max(r for _, r in requests) <= 64 else None
    cases = [Rows(requests if k == 0 else [(c // 2, r) for c, r in requests], heads=16, kv=4, d=128, seed=k,
                  tree=width) for k in range(2)]
    size = max(len(c.k) for c in cases), max(c.table.shape[1] for c in cases)
    for c in cases:                    # one cache and one table for both
        pad = size[0] - len(c.k)
        c.k, c.v = (torch.cat([x, x.new_full((pad, *x.shape[1:]), float("nan"))]) for x in (c.k, c.v))
        c.table = torch.nn.functional.pad(c.table, (0, size[1] - c.table.shape[1]), value=-5)
    states = [c.gpu() for c in cases]
    wanted = []
    for c, s in zip(cases, states):
        c.call(s)
        torch.cuda.synchronize()
        c.check(s)
        wanted.append((s["out"].clone(), s["lse"].clone()))
    s = cases[0].gpu()
    names = [k for k, v in s.items() if v is not None and k not in ("out", "lse", "ws")]
    got = [torch.empty(CALLS, *x.shape, dtype=x.dtype, device="cuda") for x in wanted[0]]
    for i in range(CALLS):
        s["out"].fill_(5.0), s["lse"].fill_(5.0)
        for k in names:
            s[k].copy_(states[i % 2][k])
        cases[0].call(s)
        got[0][i].copy_(s["out"]), got[1][i].copy_(s["lse"])
    for i in range(CALLS):
        assert torch.equal(got[0][i], wanted[i % 2][0]) and torch.equal(got[1][i], wanted[i % 2][1]), i
