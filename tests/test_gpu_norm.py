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
