"""dspark_rotary at angles near 0, where sin t is t: relative to itself."""
import math

import pytest

torch = pytest.importorskip("torch")

from speculative_decoding_draft_dspark_gb300 import target as T  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("base,factor", [(10000.0, 1.0), (500000.0, 8.0), (1e7, 64.0)])
def test_small_angles(base, factor, interleaved):
    """Pairs (0, 1): a' = -sin t.  The angle is off by 2^-24 of itself (fp32), sincospi by
    2 units in the last place (2^-22), the product by 2^-24 and the table's entry, at least
    2e-10 of a turn, by 2^-64 of a turn, 2^-31: 2^-21 together."""
    rot = 128
    position = torch.tensor([1, -1, 3, 17, 1000], dtype=torch.int32)
    q = torch.zeros(5, 1, rot)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    q[..., b] = 1.0
    turns = T.dspark_rotary_table(rot, base, scaling=T.ROPE_LINEAR, factor=factor).cuda()
    freq = torch.tensor([base ** (-2.0 * i / rot) / factor for i in range(rot // 2)], dtype=torch.float64)
    assert freq.min() / (2 * math.pi) > 2e-10
    angle = position.double()[:, None] * freq
    small = angle.abs() < 0.1
    assert small.sum() > 100
    out = torch.empty(5, 1, rot, device="cuda")
    T.dspark_rotary(q.cuda(), None, position.cuda(), turns, out, None, interleaved=interleaved)
    got, want = out.cpu().double()[:, 0, a], -torch.sin(angle)
    assert ((got - want).abs() <= 2.0 ** -21 * want.abs())[small].all()
