"""dspark_rotary and dspark_rotary_append against the formula in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")

import target_ref as ref  # noqa: E402
from speculative_decoding_draft_dspark_gb300 import target as T  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def case(R, Hq, Hk, d, rot, dtype, seed=0, fused=True, reach=100000):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(R, (Hq + 2 * Hk) * d, generator=g).to(dtype)
    position = torch.randint(0, reach, (R,), generator=g, dtype=torch.int32)
    dev = qkv.cuda()
    cut = lambda x, lo, h: x[:, lo * d:(lo + h) * d].reshape(R, h, d)  # noqa: E731
    host = [cut(qkv, lo, h) for lo, h in ((0, Hq), (Hq, Hk), (Hq + Hk, Hk))]
    gpu = [x.cuda() for x in host] if not fused else \
        [dev[:, lo * d:(lo + h) * d].view(R, h, d) for lo, h in ((0, Hq), (Hq, Hk), (Hq + Hk, Hk))]
    turns = T.dspark_rotary_table(rot, 10000.0)
    freq = torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    return host, gpu, position, turns.cuda(), freq


def close(got, want, x, dtype):
    """A rounding to the type, and in fp32 two products and a sum of terms as large
    as the pair, with a sine and cosine off by 2^-22 (the angle's fraction of a turn
    to 2^-25 times 2 pi, and sincospi's own 2^-23)."""
    size = x.to(torch.float64).abs().amax(-1, keepdim=True) * math.sqrt(2.0)
    tol = want.abs() * torch.finfo(dtype).eps / 2 + size * (2.0 ** -21)
    assert got.shape == want.shape and got.dtype == dtype
    assert ((got.cpu().to(torch.float64) - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("R,Hq,Hk,d,rot", [
    (1, 1, 1, 2, 2), (5, 4, 2, 64, 64), (7, 3, 1, 128, 64), (64, 32, 8, 128, 128), (3, 5, 5, 75, 50), (9, 2, 2, 80, 36),
    (2, 6, 3, 256, 256), (2, 2, 1, 1024, 1024), (33, 2, 1, 96, 8), (300, 1, 1, 40, 40)])
def test_rotary(R, Hq, Hk, d, rot, interleaved, dtype):
    (q, k, _), (gq, gk, _), pos, turns, freq = case(R, Hq, Hk, d, rot, dtype)
    qo, ko = (torch.full(x.shape, 9.0, dtype=dtype, device="cuda") for x in (q, k))
    for inverse, amplitude in ((False, 1.0), (True, 1.25)):
        T.dspark_rotary(gq, gk, pos.cuda(), turns, qo, ko, interleaved=interleaved, inverse=inverse,
                        amplitude=amplitude)
        for x, y in ((q, qo), (k, ko)):
            want = ref.rotate(x, pos, freq, rot, interleaved, amplitude, inverse)
            close(y, want, x * amplitude, dtype)


@pytest.mark.parametrize("offset", [0, 1, 3, 8])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_alignment_in_place_and_strides(dtype, offset):
    """Heads outermost, rows that begin anywhere, and the output on the input."""
    g = torch.Generator().manual_seed(offset)
    base = torch.randn(3 * 11 * 64 + 16, generator=g).to(dtype)
    x = base[offset:offset + 3 * 11 * 64].view(3, 11, 64).transpose(0, 1)     # [11, 3, 64]
    gx = base.cuda()[offset:offset + 3 * 11 * 64].view(3, 11, 64).transpose(0, 1)
    pos = torch.randint(0, 5000, (11,), generator=g, dtype=torch.int32)
    turns = T.dspark_rotary_table(64, 10000.0).cuda()
    freq = torch.tensor([10000.0 ** (-2.0 * i / 64) for i in range(32)], dtype=torch.float64)
    T.dspark_rotary(None, gx, pos.cuda(), turns, None, gx)
    close(gx, ref.rotate(x, pos, freq, 64, False), x, dtype)


def test_far_and_negative_positions():
    """An angle of position 2^31 - 1 is as good as one of position 1: to the 2^-53
    that the table's frequency is known to, times the position."""
    pos = torch.tensor([0, 1, -1, (1 << 20) + 1, -(1 << 30), (1 << 31) - 1], dtype=torch.int32)
    g = torch.Generator().manual_seed(3)
    q = torch.randn(6, 2, 128, generator=g)
    freq = torch.tensor([10000.0 ** (-2.0 * i / 128) for i in range(64)], dtype=torch.float64)
    out = torch.empty(6, 2, 128, device="cuda")
    T.dspark_rotary(q.cuda(), None, pos.cuda(), T.dspark_rotary_table(128, 10000.0).cuda(), out, None)
    # the reference's own angle in 64 bits: 2^31 * 2^-53 = 2^-22 at the far end
    close(out, ref.rotate(q, pos, freq, 128, False), q * 2, F32)


def test_gradient():
    """The inverse is the transpose (<R x, y> = <x, R' y>), and what differences give."""
    (q, _, _), (gq, _, _), pos, turns, freq = case(6, 4, 1, 64, 48, F32)
    y = torch.randn(6, 4, 64, generator=torch.Generator().manual_seed(9))
    for inter in (False, True):
        fwd, bwd = torch.empty(6, 4, 64, device="cuda"), torch.empty(6, 4, 64, device="cuda")
        kw = dict(interleaved=inter, amplitude=1.3)
        T.dspark_rotary(gq, None, pos.cuda(), turns, fwd, None, **kw)
        T.dspark_rotary(y.cuda(), None, pos.cuda(), turns, bwd, None, inverse=True, **kw)
        a = (fwd.cpu().double() * y.double()).sum()
        b = (q.double() * bwd.cpu().double()).sum()
        # 1536 products, each operand off by 2^-21 of a value of a few
        assert abs(a - b) < 1536 * 20 * 2.0 ** -21
        # differences: the map is linear, so a step of 1 along e_i gives R's column
        e = torch.zeros(6, 4, 64)
        e[2, 1, 17] = 1.0
        moved = torch.empty(6, 4, 64, device="cuda")
        T.dspark_rotary((q + e).cuda(), None, pos.cuda(), turns, moved, None, **kw)
        diff = ((moved - fwd).cpu().double() * y.double()).sum()
        assert abs(diff - bwd[2, 1, 17].item()) < 64 * 20 * 2.0 ** -21


def test_nan_stays_in_its_pair():
    (q, _, _), (gq, _, _), pos, turns, freq = case(3, 2, 1, 64, 64, BF16, fused=False)
    clean = torch.empty_like(gq)
    T.dspark_rotary(gq, None, pos.cuda(), turns, clean, None)
    gq[1, 1, 5] = math.nan
    got = torch.empty_like(gq)
    T.dspark_rotary(gq, None, pos.cuda(), turns, got, None)
    bad = got.isnan().nonzero().tolist()
    assert bad == [[1, 1, 5], [1, 1, 37]]
    keep = ~got.isnan()
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("R,Hq,Hk,d,rot,page,layout", [
    (1, 4, 1, 64, 64, 16, "nhd"), (64, 32, 8, 128, 128, 16, "nhd"), (37, 6, 2, 80, 36, 32, "hnd"),
    (100, 4, 4, 128, 64, 128, "pair"), (5, 3, 3, 75, 50, 256, "nhd")])
def test_append(R, Hq, Hk, d, rot, page, layout, interleaved, dtype):
    (q, k, v), (gq, gk, gv), pos, turns, freq = case(R, Hq, Hk, d, rot, dtype)
    pages = R // page * 2 + 3
    if layout == "nhd":
        kc, vc = (torch.full((pages, page, Hk, d), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    elif layout == "hnd":
        kc, vc = (torch.full((pages, Hk, page, d), 7.0, dtype=dtype, device="cuda").transpose(1, 2) for _ in range(2))
    else:       # keys and values of a page side by side
        both = torch.full((pages, 2, page, Hk, d), 7.0, dtype=dtype, device="cuda")
        kc, vc = both[:, 0], both[:, 1]
    g = torch.Generator().manual_seed(1)
    slot = torch.randperm(pages * page, generator=g)[:R].int()
    if R > 4:
        slot[1], slot[3] = -1, pages * page
    qo = torch.empty(R, Hq, d, dtype=dtype, device="cuda")
    T.dspark_rotary_append(gq, gk, gv, pos.cuda(), slot.cuda(), turns, qo, kc, vc, interleaved=interleaved)
    close(qo, ref.rotate(q, pos, freq, rot, interleaved), q, dtype)
    wk = torch.full((pages * page, Hk, d), 7.0, dtype=torch.float64)
    wv, written = wk.clone(), torch.zeros(pages * page, dtype=torch.bool)
    rk = ref.rotate(k, pos, freq, rot, interleaved)
    for r, s in enumerate(slot.tolist()):
        if 0 <= s < pages * page:
            wk[s], wv[s], written[s] = rk[r], v[r].double(), True
    flat = lambda x: x.reshape(pages * page, Hk, d).cpu()  # noqa: E731
    close(flat(kc)[written], wk[written], wk[written], dtype)
    assert torch.equal(flat(kc)[~written].double(), wk[~written])
    assert torch.equal(flat(vc).double(), wv)


def test_rows_behind_the_last_are_left():
    (q, k, v), (gq, gk, gv), pos, turns, freq = case(20, 2, 1, 64, 64, BF16)
    kc, vc = (torch.full((4, 16, 1, 64), 7.0, dtype=BF16, device="cuda") for _ in range(2))
    qo = torch.full((20, 2, 64), 7.0, dtype=BF16, device="cuda")
    n = torch.tensor([13], dtype=torch.int32, device="cuda")
    slot = torch.arange(20, dtype=torch.int32, device="cuda")
    T.dspark_rotary_append(gq, gk, gv, pos.cuda(), slot, turns, qo, kc, vc, n_rows=n)
    assert (qo[13:] == 7.0).all() and (kc.view(64, 64)[13:] == 7.0).all() and (vc.view(64, 64)[13:] == 7.0).all()
    close(qo[:13], ref.rotate(q[:13], pos[:13], freq, 64, False), q[:13], BF16)
    out = torch.full((20, 2, 64), 7.0, dtype=BF16, device="cuda")
    T.dspark_rotary(gq, None, pos.cuda(), turns, out, None, n_rows=n)
    assert (out[13:] == 7.0).all() and torch.equal(out[:13], qo[:13])


def test_a_cache_past_32_bits():
    """2^32 elements in: pages that lie 2 GB apart."""
    (q, k, v), (gq, gk, gv), pos, turns, freq = case(32, 1, 1, 64, 64, BF16)
    buf = torch.empty(5 << 30, dtype=BF16, device="cuda")
    both = buf.as_strided((5, 16, 1, 64), (1 << 30, 64, 64, 1)), buf[1 << 20:].as_strided((5, 16, 1, 64),
                                                                                        (1 << 30, 64, 64, 1))
    slot = torch.arange(48, 80, dtype=torch.int32)
    qo = torch.empty(32, 1, 64, dtype=BF16, device="cuda")
    T.dspark_rotary_append(gq, gk, gv, pos.cuda(), slot.cuda(), turns, qo, *both)
    close(both[0][3:].reshape(32, 1, 64), ref.rotate(k, pos, freq, 64, False), k, BF16)
    assert torch.equal(both[1][3:].reshape(32, 1, 64).cpu(), v)


def test_no_rows():
    turns = T.dspark_rotary_table(64, 10000.0).cuda()
    e = torch.empty(0, 2, 64, dtype=BF16, device="cuda")
    T.dspark_rotary(e, None, torch.empty(0, dtype=torch.int32, device="cuda"), turns, e, None)


def test_in_a_graph():
    (q, k, v), (gq, gk, gv), pos, turns, freq = case(9, 2, 1, 64, 64, BF16)
    out = torch.empty(9, 2, 64, dtype=BF16, device="cuda")
    gpos = pos.cuda()
    T.dspark_rotary(gq, None, gpos, turns, out, None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        T.dspark_rotary(gq, None, gpos, turns, out, None)
    gpos.add_(5)
    graph.replay()
    close(out, ref.rotate(q, pos + 5, freq, 64, False), q, BF16)


# rows from which a CTA takes 2, 4 or 8 of them, and CTAs that end in part
@pytest.mark.parametrize("R", [1215, 1216, 1217, 2435, 4871])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("Hq,Hk,d,rot", [(2, 1, 64, 64), (3, 2, 75, 50), (2, 2, 80, 40), (1, 1, 128, 128), (3, 1, 40, 2)])
def test_several_rows_of_a_cta(R, Hq, Hk, d, rot, interleaved, dtype):
    (q, k, v), (gq, gk, gv), pos, turns, freq = case(R, Hq, Hk, d, rot, dtype, seed=R)
    want = [ref.rotate(x, pos, freq, rot, interleaved, 1.25) for x in (q, k)]
    kw = dict(interleaved=interleaved, amplitude=1.25)
    page, gpos = 16, pos.cuda()
    pages = R // page + 2
    slot = torch.randperm(pages * page, generator=torch.Generator().manual_seed(R))[:R].int()
    slot[5], slot[R - 2], slot[R // 2] = -1, pages * page, -(1 << 31)
    for n in (None, R - 1, R - 9, 4, 1, 0):             # that end in and between CTAs
        last = R if n is None else n
        n_rows = None if n is None else torch.tensor([n], dtype=torch.int32, device="cuda")
        qo, ko = (torch.full(x.shape, 7.0, dtype=dtype, device="cuda") for x in (q, k))
        T.dspark_rotary(gq, gk, gpos, turns, qo, ko, n_rows=n_rows, **kw)
        for y, w, x in ((qo, want[0], q), (ko, want[1], k)):
            close(y[:last], w[:last], x[:last] * 1.25, dtype)
            assert (y[last:] == 7.0).all()
        kc, vc = (torch.full((pages, page, Hk, d), 7.0, dtype=dtype, device="cuda") for _ in range(2))
        q2 = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
        T.dspark_rotary_append(gq, gk, gv, gpos, slot.cuda(), turns, q2, kc, vc, n_rows=n_rows, **kw)
        assert torch.equal(q2, qo)
        wk, wv = (torch.full((pages * page, Hk, d), 7.0, dtype=dtype) for _ in range(2))
        there = (slot >= 0) & (slot < pages * page) & (torch.arange(R) < last)
        wk[slot[there].long()], wv[slot[there].long()] = ko.cpu()[there], v[there]
        assert torch.equal(kc.cpu().view(-1, Hk, d), wk) and torch.equal(vc.cpu().view(-1, Hk, d), wv)
