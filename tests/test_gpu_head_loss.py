"""The head's loss and gradient on the GPU against the formulas in 64 bits.

Error bounds (derived, per element):
* z: bf16 products are exact in fp32 and are summed in fp32, 16 at a time:
  |dz| <= (D / 16 + 5) 2^-23 sum_j |A_j B_j|.
* lse: |dz| plus the exponential's and logarithm's rounding,
  2^-20 (1 + max |z|).
* a gradient: G is rounded to bf16 (8 significant bits: at most 2^-8 of each
  entry) and carries the relative error of exp, |dz| + |dlse|; the product's
  sums are fp32 and the result is rounded to bf16 once (2^-8 of it):
  2^-8 |ref| + (2^-8 + |dz| + |dlse| + K/16 2^-23) sum |G| |B|.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def make(M, vocab, d, rank, ignored=0.0, seed=0, sd=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = {"h": (n(M, d) * sd).bfloat16(), "W": (n(vocab, d) * 2.0 / d ** 0.5).bfloat16(),
         "U": (n(vocab, rank) * 0.3).bfloat16() if rank else None,
         "V": (n(vocab, rank) * 0.3).bfloat16() if rank else None,
         "prev": torch.randint(0, vocab, (M,), generator=g, dtype=torch.int32) if rank else None,
         "target": torch.randint(0, vocab, (M,), generator=g, dtype=torch.int32)}
    k = int(M * ignored)
    x["target"][torch.randperm(M, generator=g)[:k]] = -1
    x["dloss"] = torch.full((M,), 1.0 / max(M - k, 1))
    return x


def reference(x):
    """Loss, lse, gradients in 64 bits, and the magnitudes the bounds need."""
    import torch
    f = torch.float64
    ok = (x["target"] >= 0) & (x["target"] < x["W"].shape[0])
    t = x["target"].long().clamp(0, x["W"].shape[0] - 1)
    A, B = x["h"].to(f), x["W"].to(f)
    if x["U"] is not None:
        pv = x["prev"].long()
        pv = torch.where((pv < 0) | (pv >= x["U"].shape[0]), 0, pv)
        A = torch.cat([A, x["U"][pv].to(f)], 1)
        B = torch.cat([B, x["V"].to(f)], 1)
    A = torch.where(ok[:, None], A, torch.zeros((), dtype=f))
    z = A @ B.T
    lse = torch.logsumexp(z, 1)
    zt = z[torch.arange(len(t)), t]
    G = (z - lse[:, None]).exp()
    G[torch.arange(len(t)), t] -= 1.0
    G *= torch.where(ok, x["dloss"].to(f), 0.0)[:, None]
    d = x["h"].shape[1]
    D = A.shape[1]
    dA, dB = G @ B, G.T @ A
    mA, mB = G.abs() @ B.abs(), G.abs().T @ A.abs()
    dz = (D / 16 + 5) * 2.0 ** -23 * (A.abs() @ B.abs().T).amax(1)     # per row
    dl = dz + 2.0 ** -20 * (1 + z.abs().amax(1))
    r = {"loss": torch.where(ok, lse - zt, 0.0), "lse": torch.where(ok, lse, 0.0),
         "dh": dA[:, :d], "dW": dB[:, :d]}
    eps = (dz + dl).amax().item() if len(dz) else 0.0
    tol = {"loss": dz + dl, "lse": dl}
    rel = 2.0 ** -8 + eps + max(B.shape[0], A.shape[0]) / 16 * 2.0 ** -23
    mags = {"dh": mA[:, :d], "dW": mB[:, :d]}
    if x["U"] is not None:
        vocab, rank = x["U"].shape
        r["dV"], mags["dV"] = dB[:, d:], mB[:, d:]
        r["dU"] = torch.zeros(vocab, rank, dtype=f).index_add_(0, pv, dA[:, d:])
        mags["dU"] = torch.zeros(vocab, rank, dtype=f).index_add_(0, pv, mA[:, d:])
    for k, m in mags.items():
        tol[k] = 2.0 ** -8 * r[k].abs() + rel * m
    return r, tol


def run(x, h=None, dh=None, stream=None, grad=True):
    import torch
    from speculative_decoding_draft_dspark_gb300 import head as H
    c = {k: (v.cuda() if v is not None else None) for k, v in x.items()}
    if h is not None:
        c["h"] = h
    (M, d), vocab = x["h"].shape, x["W"].shape[0]
    rank = 0 if x["U"] is None else x["U"].shape[1]
    full = lambda *s: torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    o = {"loss": torch.full((M,), 7.0, device="cuda"), "lse": torch.full((M,), 7.0, device="cuda"),
         "dh": full(M, d) if dh is None else dh, "dW": full(vocab, d)}
    if rank:
        o["dU"], o["dV"] = full(vocab, rank), full(vocab, rank)
    ws = H.new_workspace(H.dspark_head_workspace_size(M, vocab, d, rank, True))
    H.dspark_head_loss(c["h"], c["W"], c["U"], c["V"], c["prev"], c["target"], o["loss"], o["lse"],
                       ws, stream=stream)
    if grad:
        H.dspark_head_loss_grad(c["h"], c["W"], c["U"], c["V"], c["prev"], c["target"], o["lse"],
                                c["dloss"], o["dh"], o["dW"], o.get("dU"), o.get("dV"), ws,
                                stream=stream)
    torch.cuda.synchronize()
    from speculative_decoding_draft_dspark_gb300 import dspark as D
    o["status"] = D.dspark_read_status(ws)
    return {k: v.cpu() if hasattr(v, "cpu") else v for k, v in o.items()}


def check(got, ref, tol, keys=None):
    for k in keys or ref:
        e = (got[k].double() - ref[k]).abs()
        bad = ~(e <= tol[k])
        assert not bad.any(), (k, int(bad.sum()), e[bad].max().item(), (e / tol[k].clamp(min=1e-300)).max().item())


@pytest.mark.parametrize("M,vocab,d,rank,ignored", [
    (1, 1, 8, 0, 0.0),
    (1, 257, 64, 16, 0.0),
    (21, 1024, 64, 16, 0.0),
    (130, 1000, 72, 8, 0.3),
    (255, 511, 200, 0, 0.5),
    (257, 2049, 136, 256, 0.1),
    (600, 777, 520, 40, 0.4),
    (513, 4096, 256, 64, 0.0),
    (64, 20000, 320, 248, 0.1),
])
def test_against_the_formulas(M, vocab, d, rank, ignored):
    x = make(M, vocab, d, rank, ignored, seed=M + vocab)
    got = run(x)
    ref, tol = reference(x)
    assert got["status"] == 0
    check(got, ref, tol)


@pytest.mark.parametrize("M,vocab,d,rank,ignored", [
    (3000, 70000, 64, 16, 0.2),      # several pieces of the vocabulary
    (1001, 50003, 200, 0, 0.4),      # tiles of 192 and 224 columns: odd numbers of blocks
    (97, 60001, 328, 40, 0.0),
    (403, 40009, 72, 200, 0.0),      # dA tiles of 256 and 160 columns, split
    (2100, 20011, 328, 8, 0.1),      # dB tiles of 512 columns
])
def test_many_tiles_for_each_pair(M, vocab, d, rank, ignored):
    """Every pair of CTAs goes over many tiles, so that what a tile leaves
    behind (boxes still being stored, accumulators, ring stages) meets the
    next one.  Twice: the bits agree too."""
    import torch
    x = make(M, vocab, d, rank, ignored, seed=3)
    got, again = run(x), run(x)
    ref, tol = _reference_cuda({k: v.cuda() if v is not None else None for k, v in x.items()})
    check(got, ref, tol)
    for k in ref:
        assert torch.equal(got[k], again[k]), k


def _reference_cuda(c):
    """reference() with its large products on the GPU, in 64 bits."""
    import torch
    f = torch.float64
    ok = c["target"] >= 0
    t = c["target"].long().clamp(min=0)
    A, B = c["h"].to(f), c["W"].to(f)
    if c["U"] is not None:
        pv = c["prev"].long()
        A, B = torch.cat([A, c["U"][pv].to(f)], 1), torch.cat([B, c["V"].to(f)], 1)
    A = torch.where(ok[:, None], A, torch.zeros((), dtype=f, device="cuda"))
    z = A @ B.T
    lse = torch.logsumexp(z, 1)
    rows = torch.arange(len(t), device="cuda")
    zt = z[rows, t]
    zmax = z.abs().amax(1)
    dz = (A.shape[1] / 16 + 5) * 2.0 ** -23 * (A.abs() @ B.abs().T).amax(1)
    dl = dz + 2.0 ** -20 * (1 + zmax)
    G = (z - lse[:, None]).exp_()
    G[rows, t] -= 1.0
    G *= torch.where(ok, c["dloss"].to(f), 0.0)[:, None]
    d = c["h"].shape[1]
    dA, dB, mA, mB = G @ B, G.T @ A, G.abs() @ B.abs(), G.abs().T @ A.abs()
    ref = {"loss": torch.where(ok, lse - zt, 0.0), "lse": torch.where(ok, lse, 0.0),
           "dh": dA[:, :d], "dW": dB[:, :d]}
    mags = {"dh": mA[:, :d], "dW": mB[:, :d]}
    if c["U"] is not None:
        zero = torch.zeros(c["U"].shape, dtype=f, device="cuda")
        ref["dV"], mags["dV"] = dB[:, d:], mB[:, d:]
        ref["dU"], mags["dU"] = zero.index_add(0, pv, dA[:, d:]), zero.index_add(0, pv, mA[:, d:])
    rel = 2.0 ** -8 + (dz + dl).amax() + max(B.shape[0], A.shape[0]) / 16 * 2.0 ** -23
    tol = {"loss": dz + dl, "lse": dl}
    for k, m in mags.items():
        tol[k] = 2.0 ** -8 * ref[k].abs() + rel * m
    return {k: v.cpu() for k, v in ref.items()}, {k: v.cpu() for k, v in tol.items()}


# ------------------------------------------------- what goes wrong at edges
def _mixed(seed=11):
    x = make(300, 700, 72, 24, 0.3, seed=seed)
    return x


def test_ignored_rows_may_hold_anything():
    """NaN, infinities and tokens out of range in rows without a target reach
    no output."""
    import torch
    x = _mixed()
    ref, tol = reference(x)
    bad = (x["target"] < 0).nonzero()[:, 0]
    x["h"][bad[0::3]] = float("nan")
    x["h"][bad[1::3]] = float("inf")
    x["prev"][bad[0::2]] = 1 << 30
    x["target"][bad[0::2]] = -(1 << 31)
    x["dloss"][bad] = float("nan")
    got = run(x)
    assert got["status"] == 0
    check(got, ref, tol)
    for k in ("loss", "lse", "dh"):
        assert torch.all(got[k][bad] == 0)


@pytest.mark.parametrize("M", [1, 300])
def test_no_row_has_a_target(M):
    import torch
    x = make(M, 333, 64, 16, seed=5)
    x["target"][:] = -1
    x["h"][:] = float("nan")
    got = run(x)
    for k in ("loss", "lse", "dh", "dW", "dU", "dV"):
        assert torch.all(got[k] == 0), k


def test_tokens_out_of_range_are_flagged():
    from speculative_decoding_draft_dspark_gb300 import dspark as D
    x = _mixed(12)
    ok = (x["target"] >= 0).nonzero()[:, 0]
    x["prev"][ok[0]] = -5
    x["prev"][ok[1]] = 700
    ref, tol = reference(x)
    got = run(x)
    assert got["status"] == D.DEV_TOKEN_OOR
    check(got, ref, tol)
    x["prev"][ok[:2]] = 3
    x["target"][ok[2]] = 700
    x["dloss"][ok[2]] = 0.0
    ref, tol = reference(x)
    got = run(x)
    assert got["status"] == D.DEV_TOKEN_OOR
    check(got, ref, tol)
    assert got["loss"][ok[2]] == 0


def test_rows_apart_and_another_stream():
    import torch
    x = _mixed(13)
    h = torch.full((300, 104), 5.0, dtype=torch.bfloat16, device="cuda")
    dh = torch.full((300, 80), 3.0, dtype=torch.bfloat16, device="cuda")
    h[:, 16:88] = x["h"].cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run(x, h=h[:, 16:88], dh=dh[:, :72])
    ref, tol = reference(x)
    check(got, ref, tol)
    assert torch.all(dh[:, 72:] == 3.0)


def test_rows_weigh_differently():
    import torch
    x = _mixed(14)
    g = torch.Generator().manual_seed(1)
    x["dloss"] = torch.randn(300, generator=g) * torch.exp2(torch.randint(-20, 4, (300,), generator=g).float())
    x["dloss"][::7] = 0.0
    ref, tol = reference(x)
    check(run(x), ref, tol)
    x["dloss"][:] = 0.0
    got = run(x)
    for k in ("dh", "dW", "dU", "dV"):
        assert torch.all(got[k] == 0), k


@pytest.mark.parametrize("tokens", [1, 3])
def test_rows_share_a_token_and_runs_agree(tokens):
    """dU sums the rows of a token; the same inputs give the same bits."""
    import torch
    x = make(900, 500, 64, 256, 0.1, seed=15)
    x["prev"] = x["prev"] % tokens * 7
    ref, tol = reference(x)
    a, b = run(x), run(x)
    check(a, ref, tol)
    for k in ref:
        assert torch.equal(a[k], b[k]), k


def test_large_and_infinite_scores():
    """Scores of thousands neither overflow nor lose the loss; an infinite or
    NaN score stays in its own row."""
    import torch
    x = make(40, 600, 64, 0, seed=16, sd=600.0)
    ref, tol = reference(x)
    assert ref["lse"].abs().max() > 2000
    got = run(x)
    check(got, ref, tol, ["loss", "lse"])
    x["h"][3, 0] = 1e38
    x["W"][:, 0] = x["W"][:, 0].abs() + 10.0     # row 3: every score +infinity
    x["h"][5, 1] = float("nan")
    x["target"][7] = -1
    x["h"][7] = float("nan")
    ref, tol = reference(x)
    got = run(x)
    assert torch.isinf(got["lse"][3]) and got["lse"][3] > 0 and torch.isnan(got["loss"][3])
    assert torch.isnan(got["lse"][5]) and torch.isnan(got["loss"][5])
    rest = torch.ones(40, dtype=torch.bool)
    rest[[3, 5]] = False
    for k in ("loss", "lse"):
        assert torch.all((got[k].double() - ref[k])[rest].abs() <= tol[k][rest])
    for k in ("dh",):
        keep = rest.clone()
        assert torch.isfinite(got[k][keep]).all() and torch.isnan(got[k][5]).all()


def test_gradient_against_differences():
    """Central differences of the kernel's own loss along random sign patterns
    of step 2^-6.  The factors are multiples of 2^-5 below 2, so that both sides
    are exact in bf16.  Error: the third derivative (bounded by twice the cube
    of the change of a score, |dz| <= step sum |other factor|) times step^2 / 6,
    the loss's own error over the step, and the gradient's bound."""
    import torch
    from speculative_decoding_draft_dspark_gb300 import head as H
    M, vocab, d, rank, step = 6, 90, 32, 16, 2.0 ** -6
    g = torch.Generator().manual_seed(21)
    grid = lambda *s: (torch.randint(-8, 9, s, generator=g).float() / 32).bfloat16()  # noqa: E731
    x = {"h": grid(M, d), "W": grid(vocab, d), "U": grid(vocab, rank), "V": grid(vocab, rank),
         "prev": torch.randint(0, vocab, (M,), generator=g, dtype=torch.int32),
         "target": torch.randint(0, vocab, (M,), generator=g, dtype=torch.int32)}
    x["target"][2] = -1
    x["dloss"] = torch.randn(M, generator=g)
    got = run(x)
    ref, tol = reference(x)
    weight = x["dloss"].double()

    def objective(y):
        o = run(y, grad=False)
        return (o["loss"].double() * weight).sum().item()

    for name, grad in (("h", "dh"), ("W", "dW"), ("U", "dU"), ("V", "dV")):
        for _ in range(3):
            sign = torch.randint(0, 2, x[name].shape, generator=g).float() * 2 - 1
            hi, lo = dict(x), dict(x)
            hi[name] = (x[name].float() + step * sign).bfloat16()
            lo[name] = (x[name].float() - step * sign).bfloat16()
            assert torch.equal(hi[name].float() - lo[name].float(), 2 * step * sign)
            slope = (objective(hi) - objective(lo)) / (2 * step)
            other = {"h": "W", "W": "h", "U": "V", "V": "U"}[name]
            dz = x[other].double().abs().sum(1).max().item()       # change of a score by a unit step
            err = (2 * (2 * dz) ** 3 * step ** 2 / 6 + tol["loss"].max().item() / step) * weight.abs().sum().item()
            err += (tol[grad].double()).sum().item()
            have = (got[grad].double() * sign.double()).sum().item()
            assert abs(slope - have) <= err, (name, slope, have, err)
            assert err < 0.5 * abs(ref[grad]).sum().item()          # the bound says something


def test_captured_in_a_graph():
    """Loss and gradient replayed from a CUDA graph follow the inputs."""
    import torch
    from speculative_decoding_draft_dspark_gb300 import head as H
    a, b = _mixed(17), _mixed(18)
    c = {k: v.cuda() for k, v in a.items()}
    M, vocab, d, rank = 300, 700, 72, 24
    new = lambda t: torch.empty_like(t)  # noqa: E731
    o = {"loss": torch.empty(M, device="cuda"), "lse": torch.empty(M, device="cuda"), "dh": new(c["h"]),
         "dW": new(c["W"]), "dU": new(c["U"]), "dV": new(c["V"])}
    ws = H.new_workspace(H.dspark_head_workspace_size(M, vocab, d, rank, True))

    def step():
        H.dspark_head_loss(c["h"], c["W"], c["U"], c["V"], c["prev"], c["target"], o["loss"], o["lse"], ws)
        H.dspark_head_loss_grad(c["h"], c["W"], c["U"], c["V"], c["prev"], c["target"], o["lse"], c["dloss"],
                                o["dh"], o["dW"], o["dU"], o["dV"], ws)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x in (b, a):
        for k in c:
            c[k].copy_(x[k])
        graph.replay()
        torch.cuda.synchronize()
        ref, tol = reference(x)
        check({k: v.cpu() for k, v in o.items()}, ref, tol)


@pytest.mark.parametrize("M,vocab,d,rank", [(2, 33000, 72, 24), (97, 21003, 136, 0), (7, 9000, 1032, 56)])
def test_few_rows_in_many_splits(M, vocab, d, rank):
    """Few rows: the reduction over the vocabulary is split up to 32 times, and a
    block of 64 columns of dW and dV may lie on either side of d's end."""
    x = make(M, vocab, d, rank, seed=M)
    got = run(x)
    ref, tol = reference(x)
    assert got["status"] == 0
    check(got, ref, tol)


@pytest.mark.parametrize("d,scale", [(256, 16.0), (2304, 4.0), (2304, -16.0), (4096, 16.0)])
def test_scores_are_not_too_small(d, scale):
    """One vocabulary entry: lse is the score itself and the loss 0.  An adder
    that truncates takes about 2^-26 of a score with each 16 products; a quarter
    of that is allowed of the mean of 4096 rows' scores (a score's own share means
    nothing where it is near 0).  The loss: six roundings of
    2^-24 of the score (its product with log2 e and back, the two constants, the
    scaling, lse) and 2^-21 for the exponential and the logarithm."""
    import torch
    g = torch.Generator().manual_seed(d)
    W = (torch.randn(1, d, generator=g) * 2.0 / d ** 0.5).bfloat16()
    w = W.float()
    h = (torch.randn(4096, d, generator=g) + scale * w / w.square().sum()).bfloat16()
    x = {"h": h, "W": W, "U": None, "V": None, "prev": None,
         "target": torch.zeros(4096, dtype=torch.int32), "dloss": torch.ones(4096)}
    got = run(x, grad=False)
    z = h.double() @ W.double()[0]
    lost = ((z - got["lse"].double()).sum() / z.sum()).item()
    assert abs(lost) <= 0.25 * d / 16 * 2.0 ** -26, lost
    assert (got["loss"].double().abs() <= 6 * 2.0 ** -24 * z.abs() + 2.0 ** -21).all()


@pytest.mark.parametrize("weight", [float("inf"), float("nan")])
def test_a_weight_that_is_not_finite_stays_in_its_row(weight):
    import torch
    x = make(45, 700, 72, 24, seed=11)
    x["dloss"] = torch.rand(45, generator=torch.Generator().manual_seed(1)) - 0.3
    ref, tol = reference({**x, "dloss": torch.where(torch.arange(45) == 7, 0.0, x["dloss"])})
    x["dloss"][7] = weight
    got = run(x)
    rest = torch.arange(45) != 7
    check({"dh": got["dh"][rest]}, {"dh": ref["dh"][rest]}, {"dh": tol["dh"][rest]})
    assert not torch.isfinite(got["dh"][7]).any()


def test_masks_of_the_lowest_value():
    """bf16's lowest value as a mask, through a column of V: entries that it masks
    weigh nothing, and where it masks every entry their scores are equal and
    finite, so the loss is log vocab.  (A row's score is the mask's value alone
    there, h being 0.)  The mask adds nothing to what remains, so the bounds are
    those of the problem without it."""
    import math
    import torch
    lowest = torch.finfo(torch.bfloat16).min
    M, vocab, d, rank = 40, 600, 64, 16
    x = make(M, vocab, d, rank, seed=19)
    x["U"][:], x["V"][:] = 0.0, 0.0
    x["U"][1, 0] = x["U"][2, 1] = 1.0
    x["V"][:, 0], x["V"][::2, 1] = lowest, lowest
    everything, half, nothing = slice(0, 10), slice(10, 30), slice(30, 40)
    x["prev"][everything], x["prev"][half], x["prev"][nothing] = 1, 2, 3
    x["h"][everything] = 0.0
    x["target"][half] |= 1
    x["dloss"][everything] = 0.0
    got = run(x)
    assert got["status"] == 0
    assert ((got["loss"][everything] - math.log(vocab)).abs() <= 2.0 ** -20 * math.log(vocab)).all()
    assert ((got["lse"][everything] / lowest - 1).abs() <= 2.0 ** -22).all()
    for rows, entries in ((half, slice(1, None, 2)), (nothing, slice(None))):
        part = {k: x[k][rows] for k in ("h", "target", "dloss")}
        part["target"] = part["target"] // (2 if rows is half else 1)
        ref, tol = reference({**part, "W": x["W"][entries], "U": None, "V": None, "prev": None})
        check({k: got[k][rows] for k in ("loss", "lse", "dh")}, ref, tol, ["loss", "lse", "dh"])
    for k in ("dW", "dU", "dV"):
        assert torch.isfinite(got[k]).all(), k


@pytest.mark.parametrize("d,rank", [(256, 0), (2048, 256), (4096, 256), (65536, 0), (65536, 256)])
@pytest.mark.parametrize("where", ["one", "first", "last", "all"])
def test_exact_scores_stay_exact(d, rank, where):
    """One vocabulary entry, so that lse is the score and the loss and its gradient
    are 0.  The factors are integers, and every product and sum of a row's is an
    integer below 2^24, which fp32 and an adder that truncates both hold: the
    score has no error at all, in one column of h, at the reduction's beginning,
    at its end (the factors' part) or all over it."""
    import torch
    M, g = 300, torch.Generator().manual_seed(d + rank)
    n = lambda *s: torch.randint(-8, 9, s, generator=g).float()  # noqa: E731
    h, W, U, V = n(M, d), n(1, d), n(1, rank), n(1, rank)
    if where == "one":
        keep = torch.zeros(d)
        keep[d // 3] = 1.0
        W[0, d // 3] = 5.0
        h[:, d // 3] += 16.0
    else:
        keep = torch.zeros(d)
        keep[:40] = where in ("first", "all")
        keep[-40:] = where in ("last", "all") and rank == 0 or where == "all"
        keep[40:-40] = where == "all"
    h *= keep
    if where in ("one", "first"):
        U[:] = 0.0
    x = {k: v.bfloat16() for k, v in (("h", h), ("W", W), ("U", U), ("V", V))}
    if rank == 0:
        x["U"] = x["V"] = None
    x.update(prev=torch.zeros(M, dtype=torch.int32) if rank else None,
             target=torch.zeros(M, dtype=torch.int32), dloss=torch.ones(M))
    got = run(x)
    z = (h.double() @ W.double().T)[:, 0]
    if rank:
        z += (U.double() @ V.double().T)[0, 0]
    assert 0 < z.abs().max() < 2 ** 24
    assert torch.equal(got["lse"].double(), z)
    for k in ("loss", "dh", "dW") + (("dU", "dV") if rank else ()):
        assert torch.all(got[k] == 0), k


@pytest.mark.parametrize("counted", [15, 16, 17, 33, 300])
def test_an_infinite_mask_stays_in_its_entries(counted):
    """V holds -infinity where U[prev] holds 1: masked entries score -infinity and
    weigh nothing, so their dW and dV are 0, also where the counted rows do not fill
    up a 16.  (dU is not defined there: the formula multiplies 0 by infinity.)"""
    import torch
    vocab, d, rank = 500, 64, 16
    x = make(counted, vocab, d, rank, seed=23)
    masked = torch.arange(vocab) % 3 == 1
    x["U"][:, 0] = 1.0
    x["V"][:, 0] = torch.where(masked, -float("inf"), 0.0)
    x["target"] = x["target"] // 3 * 3 % vocab
    assert not masked[x["target"].long()].any()
    got = run(x)
    keep = (~masked).nonzero()[:, 0]
    place = torch.full((vocab,), -1)
    place[keep] = torch.arange(len(keep))
    A = torch.cat([x["h"], x["U"][x["prev"].long()]], 1)
    B = torch.cat([x["W"], x["V"]], 1)[keep]
    ref, tol = reference({"h": A, "W": B, "U": None, "V": None, "prev": None, "dloss": x["dloss"],
                          "target": place[x["target"].long()].int()})
    check(got, ref, tol, ["loss", "lse"])
    check({"dh": got["dh"]}, {"dh": ref["dh"][:, :d]}, {"dh": tol["dh"][:, :d]})
    check({"dW": got["dW"][keep]}, {"dW": ref["dW"][:, :d]}, {"dW": tol["dW"][:, :d]})
    check({"dV": got["dV"][keep]}, {"dV": ref["dW"][:, d:]}, {"dV": tol["dW"][:, d:]})
    for k in ("dW", "dV"):
        assert torch.all(got[k][masked] == 0), k


def test_one_row_of_a_wider_buffer():
    """One row, of h and of dh, in a buffer whose pitch is not a multiple of 8."""
    import torch
    x = make(1, 300, 64, 16, seed=29)
    h = torch.full((1, 1003), 5.0, dtype=torch.bfloat16, device="cuda")
    dh = torch.full((1, 1003), 3.0, dtype=torch.bfloat16, device="cuda")
    h[:, :64] = x["h"].cuda()
    got = run(x, h=h[:, :64], dh=dh[:, :64])
    ref, tol = reference(x)
    check(got, ref, tol)
    assert torch.all(dh[:, 64:] == 3.0)
