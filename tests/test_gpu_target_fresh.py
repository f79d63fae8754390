"""Inputs that the kernel just before wrote, other ones in every call and nothing
between the calls: operators of several kernels, whose later ones may begin early."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_target_adjust import BF16, Case as Logits  # noqa: E402

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
