"""Residual norm, its gradient and dropout on the GPU against the formulas in
64 bits (numpy), Philox in Python integers included.

Error bounds (derived, per element; u = 2^-24, ub = 2^-8 for a bf16 output or
u for fp32):
* a row's sum of d squares, added pairwise over lanes after at most 32 in
  order: relative (32 + 5 + 32 + 2) u; rstd half of that plus 2 u.  In all
  rstd 2^-18 relative, with room.
* r: one scaling and one addition: 2 u (|residual| + |dropout(x)|) + ub |r|.
* y: (2^-18 + 4 u) |y| + ub |y|, plus r's error times rstd gain.
* scale: as y's largest, 2^-17 relative; q: half a unit of e4m3 at |q| (2^-4
  |q|, at least 2^-10), and 2^-16 |q|.
* gradient: rstd (2^-18 (|a| + |xh| mean |a xh|)) + ub |dr'|; dgain: 2^-18 of
  the sum of magnitudes (up to M / 608 in order, then 608) + ub |dgain|.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
MASK = 0xFFFFFFFF


def philox(c, k):
    """The four words of Philox4x32-10, in Python integers."""
    c, k = list(c), list(k)
    for _ in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & MASK, (p0 >> 32) ^ c[3] ^ k[1], p0 & MASK]
        k = [(k[0] + 0x9E3779B9) & MASK, (k[1] + 0xBB67AE85) & MASK]
    return c


def kept(M, d, p, seed, offset):
    """[M, d] mask and the scale of what is kept."""
    if p == 0.0:
        return np.ones((M, d), bool), 1.0
    T = int(np.floor((1.0 - p) * 65536.0 + 0.5))
    m = np.zeros((M, -(-d // 8) * 8), bool)
    for i in range(M):
        for g in range(m.shape[1] // 8):
            w = philox((g, i, 1 << 31, offset), (seed & MASK, seed >> 32))
            for e in range(8):
                m[i, 8 * g + e] = ((w[e // 2] >> (16 * (e % 2))) & 0xFFFF) < T
    return m[:, :d], 65536.0 / max(T, 1)


def tensors(M, d, dtype, n, seed, pad=0):
    """n [M, d] tensors (rows d + pad apart) on the GPU, of which the values
    are exact in dtype."""
    import torch
    g = torch.Generator().manual_seed(seed)
    out = []
    for k in range(n):
        t = torch.empty(M, d + pad, dtype=dtype, device="cuda")[:, :d]
        t.copy_((torch.randn(M, d, generator=g) * (1.0 + k)).to(dtype))
        out.append(t)
    return out


def f8(t):
    return t.double().cpu().numpy()


def dtypes(name):
    import torch
    return {"bf16": (torch.bfloat16, 2.0 ** -8), "f32": (torch.float32, U)}[name]


SHAPES = [(1, 8), (1, 2048), (3, 64), (5, 1), (7, 127), (4, 129), (9, 1000), (33, 1003),
          (2, 2055), (6, 4104), (2, 8192), (3, 20000), (1, 32768), (700, 264)]


@pytest.mark.parametrize("M,d", SHAPES)
@pytest.mark.parametrize("name,out,p,pad,res", [
    ("bf16", "same", 0.0, 0, True), ("bf16", "row8", 0.0, 8, True), ("bf16", "group8", 0.0, 3, False),
    ("f32", "same", 0.0, 4, False), ("f32", "group8", 0.0, 0, True), ("f32", "row8", 0.0, 1, True),
])
def test_norm(M, d, name, out, p, pad, res):
    run_norm(M, d, name, out, p, pad, res)


@pytest.mark.parametrize("M,d,name,out,p,pad", [
    (5, 264, "bf16", "same", 0.1, 0), (3, 131, "bf16", "row8", 0.5, 0),
    (4, 300, "f32", "same", 0.25, 4), (2, 1001, "f32", "group8", 0.9, 0),
    (3, 64, "bf16", "same", 1.0, 0), (3, 65, "f32", "same", 1.0, 0),
])
def test_norm_with_dropout(M, d, name, out, p, pad):
    run_norm(M, d, name, out, p, pad, True)


def run_norm(M, d, name, out, p, pad, res):
    import torch
    from speculative_decoding_draft_dspark_gb300 import head as H
    dtype, ub = dtypes(name)
    x, residual, r, y = tensors(M, d, dtype, 4, M * d, pad)
    gain = (torch.rand(d, generator=torch.Generator().manual_seed(d)) + 0.5).to(dtype).cuda()
    if out != "same":
        y = torch.empty(M, d + pad, dtype=torch.uint8, device="cuda")[:, :d].view(torch.float8_e4m3fn)
    group = 128 if out == "group8" else 0
    ng = -(-d // 128) if group else 1
    scale, rstd = torch.zeros(M, ng, device="cuda"), torch.zeros(M, device="cuda")
    seed, offset, eps = 0x123456789ABCDEF, 41, 1e-5
    H.dspark_residual_norm(x, residual if res else None, gain, r, y, scale, rstd, eps=eps, group=group,
                           p=p, seed=seed, offset=offset)
    torch.cuda.synchronize()
    m, s = kept(M, d, p, seed, offset)
    b = f8(residual) if res else np.zeros((M, d))
    dx = np.where(m, f8(x) * s, 0.0)
    r64 = b + dx
    rerr = 2 * U * (np.abs(b) + np.abs(dx))
    rstd64 = 1.0 / np.sqrt((r64 ** 2).mean(1) + eps)
    g = f8(gain)
    y64 = r64 * rstd64[:, None] * g
    yerr = (2.0 ** -18 + 4 * U) * np.abs(y64) + rerr * rstd64[:, None] * np.abs(g)
    assert np.all(np.abs(f8(r) - r64) <= rerr + ub * np.abs(r64))
    assert np.all(np.abs(f8(rstd) - rstd64) <= 2.0 ** -18 * rstd64)
    if out == "same":
        assert np.all(np.abs(f8(y) - y64) <= yerr + ub * np.abs(y64))
        return
    q = y.float().double().cpu().numpy()
    got = f8(scale)
    for j in range(ng):
        cols = slice(128 * j, min(d, 128 * (j + 1))) if group else slice(0, d)
        top = np.abs(y64[:, cols]).max(1)
        want = np.where(top == 0, 1.0, top / 448.0)
        assert np.all(np.abs(got[:, j] - want) <= 2.0 ** -17 * want + (yerr[:, cols].max(1) / 448.0))
        q64 = y64[:, cols] / want[:, None]
        qerr = np.maximum(2.0 ** -4 * np.abs(q64), 2.0 ** -10) + 2.0 ** -16 * np.abs(q64) + \
            yerr[:, cols] / want[:, None]
        assert np.all(np.abs(q[:, cols] - q64) <= qerr)
        assert np.all(np.abs(q[:, cols]).max(1)[top > 0] == 448.0)


@pytest.mark.parametrize("M,d,name,p,pad,dr,dgain", [
    (1, 8, "bf16", 0.0, 0, True, True), (1, 2048, "f32", 0.0, 0, False, True),
    (5, 1, "f32", 0.0, 0, True, True), (37, 127, "bf16", 0.0, 1, True, True),
    (700, 264, "bf16", 0.0, 8, True, True), (3000, 40, "f32", 0.0, 0, True, True),
    (1500, 1000, "bf16", 0.0, 0, True, True), (4, 32768, "f32", 0.0, 0, True, True),
    (3, 20001, "bf16", 0.0, 0, True, True), (9, 264, "bf16", 0.3, 0, True, True),
    (9, 267, "f32", 0.3, 2, True, True), (6, 520, "f32", 0.5, 4, False, False),
    (2, 4104, "bf16", 0.0, 0, True, False),
])
def test_norm_grad(M, d, name, p, pad, dr, dgain):
    import torch
    from speculative_decoding_draft_dspark_gb300 import head as H
    dtype, ub = dtypes(name)
    dy, dr_in, r, dx, ds = tensors(M, d, dtype, 5, M + d, pad)
    gain = (torch.rand(d, generator=torch.Generator().manual_seed(d)) + 0.5).to(dtype).cuda()
    rstd = torch.rsqrt(r.float().square().mean(1) + 1e-6)
    dg = torch.full((d,), 7.0, dtype=dtype, device="cuda")
    ws = H.new_workspace(H.dspark_norm_workspace_size(M, d))
    seed, offset = 987654321987, 7
    H.dspark_residual_norm_grad(dy, dr_in if dr else None, r, gain, rstd, dx, ds, dg if dgain else None,
                                ws, p=p, seed=seed, offset=offset)
    torch.cuda.synchronize()
    a, xh, rs = f8(dy) * f8(gain), f8(r) * f8(rstd)[:, None], f8(rstd)[:, None]
    base = f8(dr_in) if dr else np.zeros((M, d))
    c = (a * xh).mean(1, keepdims=True)
    ref = base + rs * (a - xh * c)
    tol = rs * 2.0 ** -18 * (np.abs(a) + np.abs(xh) * np.abs(a * xh).mean(1, keepdims=True)) + \
        ub * np.abs(ref) + 2 * U * np.abs(base)
    assert np.all(np.abs(f8(ds) - ref) <= tol)
    m, s = kept(M, d, p, seed, offset)
    assert np.all(np.abs(f8(dx) - np.where(m, ref * s, 0.0)) <= np.where(m, (tol + U * np.abs(ref)) * s, 0.0))
    if dgain:
        want = (f8(dy) * xh).sum(0)
        assert np.all(np.abs(f8(dg) - want) <= 2.0 ** -18 * np.abs(f8(dy) * xh).sum(0) + ub * np.abs(want))
    else:
        assert np.all(f8(dg) == 7.0)


@pytest.mark.parametrize("M,d,name,p,pad,res", [
    (1, 8, "f32", 0.5, 0, False), (3, 1003, "f32", 0.25, 0, True), (5, 256, "bf16", 0.1, 8, True),
    (4, 77, "bf16", 0.75, 1, False), (19, 520, "bf16", 1.0, 0, True), (19, 33, "f32", 0.0, 0, True),
])
def test_dropout(M, d, name, p, pad, res):
    import torch
    from speculative_decoding_draft_dspark_gb300 import head as H
    dtype, ub = dtypes(name)
    x, residual, y = tensors(M, d, dtype, 3, d, pad)
    seed, offset = (1 << 63) + 5, MASK
    H.dspark_dropout(x, residual if res else None, y, p=p, seed=seed, offset=offset)
    torch.cuda.synchronize()
    m, s = kept(M, d, p, seed, offset)
    b = f8(residual) if res else np.zeros((M, d))
    dx = np.where(m, f8(x) * s, 0.0)
    assert np.all(np.abs(f8(y) - (b + dx)) <= 2 * U * (np.abs(b) + np.abs(dx)) + ub * np.abs(b + dx))


# ------------------------------------------------- what goes wrong at edges
@pytest.mark.parametrize("d", [264, 1003, 9000])
def test_in_place(d):
    """r may be the residual or x, dx dy and dresidual dr."""
    import torch
    from speculative_decoding_draft_dspark_gb300 import head as H
    M = 9
    x, res, r, y, dy, dr = tensors(M, d, torch.bfloat16, 6, d)
    gain = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    kw = dict(p=0.3, seed=3, offset=4)
    rstd = torch.zeros(M, device="cuda")
    H.dspark_residual_norm(x, res, gain, r, y, None, rstd, eps=1e-5, **kw)
    for which in ("residual", "x"):
        x2, res2, y2 = x.clone(), res.clone(), torch.empty_like(y)
        r2 = res2 if which == "residual" else x2
        H.dspark_residual_norm(x2, res2, gain, r2, y2, None, None, eps=1e-5, **kw)
        assert torch.equal(r2, r) and torch.equal(y2, y)
    ws = H.new_workspace(H.dspark_norm_workspace_size(M, d))
    dx, ds, dg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(gain)
    H.dspark_residual_norm_grad(dy, dr, r, gain, rstd, dx, ds, dg, ws, **kw)
    a, b, g = dy.clone(), dr.clone(), torch.empty_like(gain)
    H.dspark_residual_norm_grad(a, b, r, gain, rstd, a, b, g, ws, **kw)
    assert torch.equal(a, dx) and torch.equal(b, ds) and torch.equal(g, dg)
    z = x.clone()
    H.dspark_dropout(x, res, y, **kw)
    H.dspark_dropout(z, res, z, **kw)
    assert torch.equal(z, y)


@pytest.mark.parametrize("d", [256, 1003, 8200])
@pytest.mark.parametrize("name", ["bf16", "f32"])
def test_nan_and_infinity_stay_where_they_are(name, d):
    """In its own row; nowhere where it is dropped."""
    import torch
    from speculative_decoding_draft_dspark_gb300 import head as H
    dtype, _ = dtypes(name)
    M, p, seed, offset = 6, 0.5, 77, 1
    m, _ = kept(M, d, p, seed, offset)
    x, res, r, y = tensors(M, d, dtype, 4, d)
    gain = torch.ones(d, dtype=dtype, device="cuda")
    lost, held = int(np.argmin(m[1])), int(np.argmax(m[4]))
    x[1, lost] = float("nan")
    x[2, int(np.argmin(m[2]))] = float("inf")
    x[4, held] = float("nan")
    for out in ("same", "row8", "group8"):
        q = y if out == "same" else torch.empty(M, d, dtype=torch.float8_e4m3fn, device="cuda")
        n = 1 if out == "row8" else -(-d // 128)
        scale = torch.zeros(M, n, device="cuda")
        H.dspark_residual_norm(x, res, gain, r, q, scale, None, eps=1e-5, group=128 if out == "group8" else 0,
                               p=p, seed=seed, offset=offset)
        bad = torch.isnan(q.float()).any(1).cpu().tolist()
        assert bad == [False, False, False, False, True, False], out
        assert torch.isnan(r.float()).sum() == 1 and torch.isinf(r.float()).sum() == 0
    H.dspark_dropout(x, None, y, p=p, seed=seed, offset=offset)
    f = y.float().cpu()
    assert torch.isnan(f).sum() == 1 and torch.isnan(f[4, held])
    assert torch.all(f[torch.from_numpy(~m)] == 0)


@pytest.mark.parametrize("out", ["same", "row8", "group8"])
def test_zero_rows_and_tiny_rows(out):
    """A row of zeros gives zeros and scales of 1; a row whose largest value is
    near fp32's smallest normals still uses the whole 8-bit range."""
    import torch
    from speculative_decoding_draft_dspark_gb300 import head as H
    M, d = 3, 300
    x = torch.zeros(M, d, device="cuda")
    x[1] = torch.linspace(-1, 1, d, device="cuda")
    gain = torch.full((d,), 1e-37, device="cuda")
    gain[:128] = 1.0 if out == "same" else 1e-37
    y = torch.empty(M, d, device="cuda") if out == "same" else \
        torch.empty(M, d, dtype=torch.float8_e4m3fn, device="cuda")
    n = 3 if out == "group8" else 1
    scale = torch.zeros(M, n, device="cuda")
    H.dspark_residual_norm(x, None, gain, None, y, scale, None, eps=1e-6, group=128 if out == "group8" else 0)
    assert torch.all(y.float()[[0, 2]] == 0) and torch.isfinite(y.float()).all()
    if out != "same":
        assert torch.all(scale[[0, 2]] == 1.0)
        assert y.float()[1].abs().max() == 448.0


def test_optional_outputs_and_streams():
    import torch
    from speculative_decoding_draft_dspark_gb300 import head as H
    M, d = 50, 520
    x, res, r, y, dy = tensors(M, d, torch.float32, 5, 9)
    gain = torch.rand(d, device="cuda") + 0.5
    rstd = torch.zeros(M, device="cuda")
    H.dspark_residual_norm(x, res, gain, r, y, None, rstd, eps=1e-5)
    y2 = torch.empty_like(y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        H.dspark_residual_norm(x, res, gain, None, y2, None, None, eps=1e-5)
    s.synchronize()
    assert torch.equal(y, y2)
    ws = H.new_workspace(H.dspark_norm_workspace_size(M, d))
    full = [torch.empty_like(x), torch.empty_like(x), torch.empty_like(gain)]
    H.dspark_residual_norm_grad(dy, None, r, gain, rstd, *full, ws)
    for i in range(3):
        one = [None, None, None]
        one[i] = torch.empty_like(full[i])
        H.dspark_residual_norm_grad(dy, None, r, gain, rstd, *one, ws, stream=s)
        s.synchronize()
        assert torch.equal(one[i], full[i])


def test_norm_gradient_against_differences():
    """Central differences in 32 bits of sum(w y + v r) along random directions.
    Step 2^-7 of values of order 1: truncation step^2 times a third derivative
    of at most 30 sum |w gain| / d^(1/2), rounding 2^-20 of the sum's magnitude
    over the step."""
    import torch
    from speculative_decoding_draft_dspark_gb300 import head as H
    M, d, step = 4, 200, 2.0 ** -7
    g = torch.Generator().manual_seed(2)
    n = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, res, gain, w, v = n(M, d), n(M, d), n(d), n(M, d), n(M, d)
    kw = dict(p=0.2, seed=8, offset=2)
    rstd, r, y = torch.zeros(M, device="cuda"), torch.empty_like(x), torch.empty_like(x)

    def objective(x, res, gain):
        H.dspark_residual_norm(x, res, gain, r, y, None, rstd, eps=1e-5, **kw)
        return ((w.double() * y.double()).sum() + (v.double() * r.double()).sum()).item()

    size = objective(x, res, gain)
    size = ((w * y).abs().sum() + (v * r).abs().sum()).item()
    dx, ds, dg = torch.empty_like(x), torch.empty_like(x), torch.empty_like(gain)
    ws = H.new_workspace(H.dspark_norm_workspace_size(M, d))
    H.dspark_residual_norm_grad(w, v, r, gain, rstd, dx, ds, dg, ws, **kw)
    tol = 30 * step ** 2 * (w * gain).abs().sum().item() / d ** 0.5 + 2.0 ** -20 * size / step
    for name, grad in (("x", dx), ("residual", ds), ("gain", dg)):
        for _ in range(3):
            u = n(*grad.shape)
            u = u / u.norm()
            at = {"x": x, "residual": res, "gain": gain}
            hi, lo = dict(at), dict(at)
            hi[name], lo[name] = at[name] + step * u, at[name] - step * u
            slope = (objective(*hi.values()) - objective(*lo.values())) / (2 * step)
            have = (grad.double() * u.double()).sum().item()
            assert abs(slope - have) <= tol, (name, slope, have, tol)


def test_rows_are_summed_in_a_fixed_order():
    import torch
    from speculative_decoding_draft_dspark_gb300 import head as H
    for M, d in ((4000, 1000), (500, 2048), (300, 1001), (40, 20000)):
        dy, dr, r = tensors(M, d, torch.bfloat16, 3, M)
        gain = torch.ones(d, dtype=torch.bfloat16, device="cuda")
        rstd = torch.rsqrt(r.float().square().mean(1) + 1e-6)
        ws = H.new_workspace(H.dspark_norm_workspace_size(M, d))
        out = []
        for _ in range(3):
            o = [torch.empty_like(r), torch.empty_like(r), torch.empty_like(gain)]
            H.dspark_residual_norm_grad(dy, dr, r, gain, rstd, *o, ws)
            out.append(o)
        for o in out[1:]:
            assert all(torch.equal(a, b) for a, b in zip(o, out[0]))


def test_captured_in_a_graph():
    import torch
    from speculative_decoding_draft_dspark_gb300 import head as H
    M, d = 30, 264
    x, res, r, y = tensors(M, d, torch.bfloat16, 4, 1)
    gain = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    rstd, dg = torch.zeros(M, device="cuda"), torch.empty_like(gain)
    dx, ds = torch.empty_like(x), torch.empty_like(x)
    ws = H.new_workspace(H.dspark_norm_workspace_size(M, d))
    kw = dict(p=0.1, seed=5, offset=6)

    def step():
        H.dspark_residual_norm(x, res, gain, r, y, None, rstd, eps=1e-5, **kw)
        H.dspark_residual_norm_grad(y, res, r, gain, rstd, dx, ds, dg, ws, **kw)
        H.dspark_dropout(dx, ds, r, **kw)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(res * 0.5 + 1)
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (r, y, rstd, dx, ds, dg)]
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (r, y, rstd, dx, ds, dg)))


@pytest.mark.parametrize("M,d,pad,first", [(3, 77, 0, 1), (4, 256, 1, 0), (3, 257, 2, 2), (2, 512, 0, 1),
                                           (5, 1003, 3, 0), (2, 2049, 0, 3), (2, 8195, 1, 1)])
def test_rows_at_any_address(M, d, pad, first, monkeypatch):
    """bf16 rows that begin in the middle of a word, each tensor's elsewhere;
    nothing beside a row is written."""
    import sys
    import torch
    kept_flat = []

    def placed(M, d, dtype, n, seed, pad=0):
        g = torch.Generator().manual_seed(seed)
        out = []
        for k in range(n):
            at, step = (first + k) % 4, d + pad
            flat = torch.full((at + M * step + 8,), -7.0, dtype=dtype, device="cuda")
            t = flat.as_strided((M, d), (step, 1), at)
            t.copy_((torch.randn(M, d, generator=g) * (1.0 + k)).to(dtype))
            kept_flat.append((flat, at, step, d))
            out.append(t)
        return out

    monkeypatch.setattr(sys.modules[__name__], "tensors", placed)
    run_norm(M, d, "bf16", "same", 0.3, pad, True)
    run_norm(M, d, "bf16", "row8", 0.0, pad, True)
    run_norm(M, d, "bf16", "group8", 0.3, pad, False)
    test_norm_grad(M, d, "bf16", 0.3, pad, True, True)
    test_dropout(M, d, "bf16", 0.3, pad, True)
    for flat, at, step, d in kept_flat:
        beside = torch.ones_like(flat, dtype=torch.bool)
        beside.as_strided((M, d), (step, 1), at)[:] = False
        assert (flat[beside] == -7.0).all()


@pytest.mark.parametrize("d", [1024, 1003])
@pytest.mark.parametrize("out", ["row8", "group8"])
def test_bytes_are_the_quotients_rounded_to_nearest(out, d):
    """The same call with y in 32 bits gives the kernel's own y: scale is max |y| /
    448 and the bytes y / scale, both as fp32 divides, and rounded to nearest even.
    Enough elements that some lie within an ulp of a tie."""
    import torch
    from speculative_decoding_draft_dspark_gb300 import head as H
    M, group = 4096, 128 if out == "group8" else 0
    x, res, y = tensors(M, d, torch.float32, 3, 77)
    gain = torch.rand(d, generator=torch.Generator().manual_seed(d)).cuda() + 0.5
    H.dspark_residual_norm(x, res, gain, None, y, None, None, eps=1e-6)
    n = -(-d // 128) if group else 1
    scale = torch.zeros(M, n, device="cuda")
    q = torch.empty(M, d, dtype=torch.float8_e4m3fn, device="cuda")
    H.dspark_residual_norm(x, res, gain, None, q, scale, None, eps=1e-6, group=group)
    width = group or d
    parts = torch.nn.functional.pad(y.cpu(), (0, n * width - d)).reshape(M, n, width)
    want = parts.abs().amax(2) / 448.0
    assert torch.equal(scale.cpu(), want)
    byte = (parts / want[:, :, None]).reshape(M, n * width)[:, :d].to(torch.float8_e4m3fn)
    assert torch.equal(q.cpu().view(torch.uint8), byte.contiguous().view(torch.uint8))


@pytest.mark.parametrize("out", ["row8", "group8"])
@pytest.mark.parametrize("d", [256, 300])
def test_scale_that_underflows_is_one(out, d):
    """Values below 448 x 2^-150: max |y| / 448 is 0 in fp32, the scale 1 and every
    byte 0, of the zeros among them too."""
    import torch
    from speculative_decoding_draft_dspark_gb300 import head as H
    M = 4
    x = torch.ones(M, d, device="cuda")
    x[:, ::3] = 0.0
    gain = torch.full((d,), 2.0 ** -143, device="cuda")       # y below 2^-142
    scale = torch.zeros(M, -(-d // 128) if out == "group8" else 1, device="cuda")
    q = torch.ones(M, d, device="cuda").to(torch.float8_e4m3fn)
    H.dspark_residual_norm(x, None, gain, None, q, scale, None, eps=1e-6, group=128 if out == "group8" else 0)
    assert torch.all(scale == 1.0) and torch.all(q.float() == 0.0)


# -------------------------------------------------- every layout of a row
def kept_by_arrays(M, d, p, seed, offset):
    """kept() with the words of all elements at once."""
    if p == 0.0:
        return np.ones((M, d), bool), 1.0
    T = int(np.floor((1.0 - p) * 65536.0 + 0.5))
    n = -(-d // 8)
    low, half = np.uint64(MASK), np.uint64(32)
    c = [np.broadcast_to(np.arange(n, dtype=np.uint64)[None, :], (M, n)),
         np.broadcast_to(np.arange(M, dtype=np.uint64)[:, None], (M, n)),
         np.full((M, n), 1 << 31, np.uint64), np.full((M, n), offset, np.uint64)]
    k = [seed & MASK, seed >> 32]
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> half) ^ c[1] ^ np.uint64(k[0]), p1 & low, (p0 >> half) ^ c[3] ^ np.uint64(k[1]), p0 & low]
        k = [(k[0] + 0x9E3779B9) & MASK, (k[1] + 0xBB67AE85) & MASK]
    lanes = np.stack([h for w in c for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], -1)
    return lanes.reshape(M, 8 * n)[:, :d] < T, 65536.0 / max(T, 1)


def guarded(monkeypatch, first):
    """Makes tensors() place each tensor `first` elements (0 or 2) into a buffer of
    its own, and returns a check that nothing beside the rows was written."""
    import sys
    import torch
    buffers = []

    def placed(M, d, dtype, n, seed, pad=0):
        g = torch.Generator().manual_seed(seed)
        out = []
        for k in range(n):
            at, step = first, d + pad
            flat = torch.full((at + M * step + 8,), -7.0, dtype=dtype, device="cuda")
            t = flat.as_strided((M, d), (step, 1), at)
            t.copy_((torch.randn(M, d, generator=g) * (1.0 + k)).to(dtype))
            buffers.append((flat, at, step, M, d))
            out.append(t)
        return out

    def untouched():
        for flat, at, step, M, d in buffers:
            beside = torch.ones_like(flat, dtype=torch.bool)
            beside.as_strided((M, d), (step, 1), at)[:] = False
            assert (flat[beside] == -7.0).all()

    here = sys.modules[__name__]
    monkeypatch.setattr(here, "tensors", placed)
    monkeypatch.setattr(here, "kept", kept_by_arrays)
    return untouched


def test_both_ways_to_draw_the_words_agree():
    a, b = kept(5, 77, 0.3, 0x123456789ABCDEF, 41), kept_by_arrays(5, 77, 0.3, 0x123456789ABCDEF, 41)
    assert np.array_equal(a[0], b[0]) and a[1] == b[1]


@pytest.mark.parametrize("M,d,pad,first", [
    (1, 2, 0, 0), (5, 2, 2, 2), (3, 6, 0, 0), (7, 126, 0, 2), (4, 130, 2, 0), (9, 300, 0, 0),
    (5, 1002, 2, 0), (3, 2044, 0, 2), (2, 8190, 0, 0), (2, 8194, 0, 0), (3, 20002, 2, 2),
    (6, 64, 2, 0), (5, 264, 0, 2), (4, 2048, 2, 0), (2, 9000, 2, 0),
])
def test_bf16_rows_at_four_bytes(M, d, pad, first, monkeypatch):
    """Even widths that are no multiple of 8, and rows that begin at 4 bytes but
    not at 16: norm in 16 and 8 bits, its gradient and dropout, with and without a
    mask, and nothing beside a row is written."""
    untouched = guarded(monkeypatch, first)
    for out in ("same", "row8", "group8"):
        for p in (0.0, 0.3):
            run_norm(M, d, "bf16", out, p, pad, out != "group8")
    for p, dr in ((0.0, False), (0.3, True)):
        test_norm_grad(M, d, "bf16", p, pad, dr, True)
        test_dropout(M, d, "bf16", p, pad, dr)
    untouched()


@pytest.mark.parametrize("d,pad", [(300, 0), (264, 2), (9002, 0)])
def test_bf16_rows_at_four_bytes_in_place(d, pad):
    """As test_in_place; every other buffer is a clone at the same strides."""
    import torch
    from speculative_decoding_draft_dspark_gb300 import head as H
    M, kw = 9, dict(p=0.3, seed=3, offset=4)

    def clone(t):
        c = torch.empty(M, d + pad, dtype=t.dtype, device="cuda")[:, :d]
        return c.copy_(t)

    x, res, r, y, dy, dr, dx, ds = tensors(M, d, torch.bfloat16, 8, d, pad)
    gain = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    rstd = torch.zeros(M, device="cuda")
    H.dspark_residual_norm(x, res, gain, r, y, None, rstd, eps=1e-5, **kw)
    for which in ("residual", "x"):
        x2, res2, y2 = clone(x), clone(res), clone(y)
        r2 = res2 if which == "residual" else x2
        H.dspark_residual_norm(x2, res2, gain, r2, y2, None, None, eps=1e-5, **kw)
        assert torch.equal(r2, r) and torch.equal(y2, y)
    ws = H.new_workspace(H.dspark_norm_workspace_size(M, d))
    dg, g = torch.empty_like(gain), torch.empty_like(gain)
    H.dspark_residual_norm_grad(dy, dr, r, gain, rstd, dx, ds, dg, ws, **kw)
    a, b = clone(dy), clone(dr)
    H.dspark_residual_norm_grad(a, b, r, gain, rstd, a, b, g, ws, **kw)
    assert torch.equal(a, dx) and torch.equal(b, ds) and torch.equal(g, dg)
    z = clone(x)
    H.dspark_dropout(x, res, y, **kw)
    H.dspark_dropout(z, res, z, **kw)
    assert torch.equal(z, y)


@pytest.mark.parametrize("M,d,name,p,pad", [
    (9500, 256, "bf16", 0.0, 0), (9500, 264, "bf16", 0.2, 0),      # copied ahead: 15, 8, 4 and 1 rows a CTA
    (5001, 1000, "bf16", 0.1, 8), (3000, 2048, "bf16", 0.0, 0), (701, 8192, "bf16", 0.1, 0),
    (8001, 264, "f32", 0.1, 0), (8001, 265, "f32", 0.0, 0), (1000, 4104, "f32", 0.0, 0),
    (8001, 300, "bf16", 0.1, 0), (8001, 301, "bf16", 0.1, 0), (4001, 1002, "bf16", 0.0, 2),
    (1001, 9000, "f32", 0.0, 0), (1001, 9000, "bf16", 0.1, 0), (1001, 9002, "bf16", 0.0, 0),
])
def test_gradient_of_many_rounds(M, d, name, p, pad, monkeypatch):
    """More rows than the CTAs take in three rounds, whichever kernel goes over
    them: the ring of copies ahead (three stages) and the two sets of sums come
    round again, and the last round is not full."""
    untouched = guarded(monkeypatch, 0)
    test_norm_grad(M, d, name, p, pad, True, True)
    untouched()
