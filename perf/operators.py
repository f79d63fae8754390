"""The operators that train a drafter's head and make its hidden states, as
cases to be timed and compared.

* ``loss``, ``step``  softmax cross entropy of the Markov head's scores
  z = h W^T + U[prev] V^T over the vocabulary, and the same with the gradients
  of h, W, U and V (``step`` is one loss and one gradient call);
* ``norm``, ``norm_grad``  r = residual + dropout(x), y = r / rms(r) * gain,
  with y in the type of x or in 8 bits with scales, and its gradient;
* ``dropout``  residual + dropout(x) by itself.

``own`` chooses between the plain form (elementary torch operations in 32
bits) and the library's entry points.
"""
import math

import torch

own = False

EPS = 1e-6
GROUP = 128          # columns that share a scale where scales are by groups
F8_MAX = 448.0       # largest e4m3 number
F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MOST = 7168 * 262144 * (2048 + 256)    # the largest listed product


def listed():
    return [
        # loss of one decoded block of 3 requests x 7 positions: latency
        {"name": "loss_tiny", "op": "loss", "rows": 21, "vocab": 1024, "d": 64, "rank": 16, "ignored": 0.0},
        # evaluating 8 blocks of 7 at full vocabulary: one pass over W and V
        {"name": "loss_8x7", "op": "loss", "rows": 56, "vocab": 262144, "d": 2048, "rank": 256, "ignored": 0.0},
        # evaluating the benchmark's batch, a tenth of the rows without target
        {"name": "loss_256x7", "op": "loss", "rows": 1792, "vocab": 262144, "d": 2048, "rank": 256, "ignored": 0.1},
        # a small training micro-batch at the smaller vocabulary
        {"name": "step_64x7", "op": "step", "rows": 448, "vocab": 129280, "d": 2048, "rank": 256, "ignored": 0.1},
        # a plain output projection (no Markov factor), odd sizes, many prompt rows
        {"name": "step_ragged", "op": "step", "rows": 1001, "vocab": 50003, "d": 1000, "rank": 0, "ignored": 0.4},
        # a full training micro-batch
        {"name": "step_1024x7", "op": "step", "rows": 7168, "vocab": 262144, "d": 2048, "rank": 256, "ignored": 0.1},
        # serving: the hidden states of 8 blocks of 7 in 8 bits, one scale a row
        {"name": "norm_8x7_row8", "op": "norm", "rows": 56, "d": 2048, "type": "bf16", "out": "row8", "p": 0.0},
        # serving, the largest batch: 8 bits with a scale for 128 columns
        {"name": "norm_1024x15_group8", "op": "norm", "rows": 15360, "d": 2048, "type": "bf16", "out": "group8", "p": 0.0},
        # training: the gradient with dropout on the branch
        {"name": "norm_grad_1024x15", "op": "norm_grad", "rows": 15360, "d": 2048, "type": "bf16", "p": 0.1},
        # an odd width in 32 bits
        {"name": "norm_grad_odd", "op": "norm_grad", "rows": 777, "d": 5001, "type": "f32", "p": 0.0},
        # training: dropout on a branch before it joins the residual stream
        {"name": "dropout_1024x15", "op": "dropout", "rows": 15360, "d": 2048, "type": "bf16", "p": 0.1},
        # an odd width in 32 bits
        {"name": "dropout_odd", "op": "dropout", "rows": 777, "d": 1003, "type": "f32", "p": 0.25},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["loss", "step", "step", "norm", "norm_grad", "dropout"])
    if op in ("loss", "step"):
        while True:
            c = {"op": op, "rows": _log_int(rng, 1, 8192), "vocab": _log_int(rng, 256, 262144),
                 "d": 8 * _log_int(rng, 8, 512), "rank": rng.choice([0, 16, 8 * rng.randint(1, 32), 256]),
                 "ignored": rng.choice([0.0, 0.1, 0.5])}
            if c["rows"] * c["vocab"] * (c["d"] + c["rank"]) <= MOST:
                return c
    c = {"op": op, "rows": _log_int(rng, 1, 16384), "d": _log_int(rng, 64, 8192),
         "type": rng.choice(["bf16", "bf16", "f32"]), "p": rng.choice([0.0, 0.1, 0.3])}
    if op == "norm":
        c["out"] = rng.choice(["same", "row8", "group8"])
    if op == "dropout":
        c["p"] = rng.choice([0.1, 0.25, 0.5])
    return c


def _valid_rows(case):
    return case["rows"] - int(case["rows"] * case["ignored"])


def work(case):
    M, d = case["rows"], case["d"]
    if case["op"] in ("loss", "step"):
        n, v, r = _valid_rows(case), case["vocab"], case["rank"]
        D = d + r
        read = 2 * (n * D + v * D) + 8 * M
        if case["op"] == "loss":
            return {"bytes": read + 8 * M, "flops": 2 * n * v * D}
        return {"bytes": read + 12 * M + 2 * (M * d + v * (D + r)), "flops": 6 * n * v * D}
    e = 2 if case["type"] == "bf16" else 4
    if case["op"] == "norm":
        out = {"same": e * M * d, "row8": M * d + 4 * M, "group8": M * d + 4 * M * -(-d // GROUP)}[case["out"]]
        return {"bytes": 3 * e * M * d + out + 4 * M + e * d, "flops": 8 * M * d}
    if case["op"] == "norm_grad":
        return {"bytes": 5 * e * M * d + 4 * M + 2 * e * d, "flops": 12 * M * d}
    return {"bytes": 3 * e * M * d, "flops": 2 * M * d}


def _inputs(case, seed):
    """The inputs as a training or serving program has them, on the GPU."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(sd, *shape, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * sd).to(dtype)

    M, d = case["rows"], case["d"]
    s = {}
    if case["op"] in ("loss", "step"):
        v, r = case["vocab"], case["rank"]
        s["h"] = normal(1.0, M, d)
        s["W"] = normal(2.0 / math.sqrt(d), v, d)
        s["U"] = normal(0.02, v, r) if r else None
        s["V"] = normal(0.02, v, r) if r else None
        s["prev"] = torch.randint(0, v, (M,), generator=g, device="cuda", dtype=torch.int32) if r else None
        s["target"] = torch.randint(0, v, (M,), generator=g, device="cuda", dtype=torch.int32)
        n = _valid_rows(case)
        s["target"][torch.randperm(M, generator=g, device="cuda")[n:]] = -1
        if case["op"] == "step":
            s["dloss"] = torch.full((M,), 1.0 / max(n, 1), device="cuda")
        return s
    t = TYPES[case["type"]]
    s["seed"], s["offset"] = int(seed) * 2654435761 % (1 << 63), int(seed) % 1000
    s["x"] = normal(1.0, M, d, dtype=t)
    s["residual"] = normal(3.0, M, d, dtype=t)
    if case["op"] != "dropout":
        s["gain"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(t)
    if case["op"] == "norm_grad":
        s["dy"], s["dr"], s["r"] = s.pop("x"), normal(1.0, M, d, dtype=t), s.pop("residual")
        s["rstd"] = torch.rsqrt(s["r"].float().square().mean(1) + EPS)
    return s


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    M, d = case["rows"], case["d"]

    def new(dtype, *shape):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    # the buffers that a program keeps for the results
    if case["op"] in ("loss", "step"):
        v, r = case["vocab"], case["rank"]
        out = {"loss": new(torch.float32, M), "lse": new(torch.float32, M)}
        if case["op"] == "step":
            out["dh"], out["dW"] = torch.empty_like(s["h"]), torch.empty_like(s["W"])
            if r:
                out["dU"], out["dV"] = torch.empty_like(s["U"]), torch.empty_like(s["V"])
    elif case["op"] == "norm":
        out = {"r": torch.empty_like(s["x"]), "rstd": new(torch.float32, M)}
        if case["out"] == "same":
            out["y"] = torch.empty_like(s["x"])
        else:
            out["y"] = new(F8, M, d)
            out["scale"] = new(torch.float32, M, 1 if case["out"] == "row8" else -(-d // GROUP))
    elif case["op"] == "norm_grad":
        out = {"dx": torch.empty_like(s["r"]), "dresidual": torch.empty_like(s["r"]), "dgain": torch.empty_like(s["gain"])}
    else:
        out = {"y": torch.empty_like(s["x"])}
    s["out"] = out
    if own:
        from speculative_decoding_draft_dspark_gb300 import head as H
        if case["op"] in ("loss", "step"):
            s["ws"] = H.new_workspace(H.dspark_head_workspace_size(M, v, d, r, case["op"] == "step"))
        elif case["op"] == "norm_grad":
            s["ws"] = H.new_workspace(H.dspark_norm_workspace_size(M, d))
    return s


def _run_own(s):
    from speculative_decoding_draft_dspark_gb300 import head as H
    case, out = s["case"], s["out"]
    if case["op"] in ("loss", "step"):
        H.dspark_head_loss(s["h"], s["W"], s["U"], s["V"], s["prev"], s["target"], out["loss"], out["lse"], s["ws"])
        if case["op"] == "step":
            H.dspark_head_loss_grad(s["h"], s["W"], s["U"], s["V"], s["prev"], s["target"], out["lse"], s["dloss"],
                                    out["dh"], out["dW"], out.get("dU"), out.get("dV"), s["ws"])
    elif case["op"] == "norm":
        H.dspark_residual_norm(s["x"], s["residual"], s["gain"], out["r"], out["y"], out.get("scale"), out["rstd"],
                               eps=EPS, group=GROUP if case["out"] == "group8" else 0,
                               p=case["p"], seed=s["seed"], offset=s["offset"])
    elif case["op"] == "norm_grad":
        H.dspark_residual_norm_grad(s["dy"], s["dr"], s["r"], s["gain"], s["rstd"], out["dx"], out["dresidual"],
                                    out["dgain"], s["ws"], p=case["p"], seed=s["seed"], offset=s["offset"])
    else:
        H.dspark_dropout(s["x"], s["residual"], out["y"], p=case["p"], seed=s["seed"], offset=s["offset"])
    return out


# ------------------------------------------------------------- plain form
def _plain_z(s):
    valid = s["target"] >= 0
    A, B = s["h"].float(), s["W"].float()
    if s["U"] is not None:
        A = torch.cat([A, s["U"][s["prev"].long()].float()], 1)
        B = torch.cat([B, s["V"].float()], 1)
    A = torch.where(valid[:, None], A, 0.0)
    return valid, A, B, A @ B.T


def _plain_loss(s):
    valid, A, B, z = _plain_z(s)
    rows = torch.arange(len(valid), device=z.device)
    t = s["target"].clamp(min=0).long()
    zt = z[rows, t]
    m = z.max(1, keepdim=True).values
    e = (z - m).exp()
    total = e.sum(1, keepdim=True)
    lse = (m + total.log())[:, 0]
    out = {"loss": torch.where(valid, lse - zt, 0.0), "lse": torch.where(valid, lse, 0.0)}
    if s["case"]["op"] == "step":
        G = e / total
        G[rows, t] -= 1.0
        G *= torch.where(valid, s["dloss"], 0.0)[:, None]
        dA, dB = G @ B, G.T @ A
        d = s["case"]["d"]
        out["dh"], out["dW"] = dA[:, :d].to(s["h"].dtype), dB[:, :d].to(s["W"].dtype)
        if s["U"] is not None:
            dU = torch.zeros(s["U"].shape, device=z.device).index_add_(0, s["prev"].long(), dA[:, d:])
            out["dU"], out["dV"] = dU.to(s["U"].dtype), dB[:, d:].to(s["V"].dtype)
    return out


def _philox_words(c0, c1, c2, c3, k0, k1):
    """Four int64 tensors with the 32-bit words of Philox4x32-10."""
    mask = 0xFFFFFFFF
    c = [c0, c1, c2, c3]
    for i in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57    # their low 64 bits
        c = [((b >> 32) & mask) ^ c[1] ^ ((k0 + i * 0x9E3779B9) & mask), b & mask,
             ((a >> 32) & mask) ^ c[3] ^ ((k1 + i * 0xBB67AE85) & mask), a & mask]
    return c


def _plain_dropout(x, s):
    p = s["case"]["p"]
    if p == 0.0:
        return x
    keep = int(math.floor((1.0 - p) * 65536.0 + 0.5))
    M, d = x.shape
    n = -(-d // 8)
    col = torch.arange(n, device=x.device, dtype=torch.int64)[None, :].expand(M, n)
    row = torch.arange(M, device=x.device, dtype=torch.int64)[:, None].expand(M, n)
    c2, c3 = torch.full_like(col, 0x80000000), torch.full_like(col, s["offset"])
    w = _philox_words(col, row, c2, c3, s["seed"] & 0xFFFFFFFF, s["seed"] >> 32)
    lanes = torch.stack([v for word in w for v in (word & 0xFFFF, word >> 16)], -1).reshape(M, 8 * n)[:, :d]
    return torch.where(lanes < keep, x * (65536.0 / max(keep, 1)), 0.0)


def _run_plain(s):
    case = s["case"]
    if case["op"] in ("loss", "step"):
        return _plain_loss(s)
    if case["op"] == "dropout":
        return {"y": (s["residual"].float() + _plain_dropout(s["x"].float(), s)).to(s["x"].dtype)}
    if case["op"] == "norm":
        t = s["x"].dtype
        r = s["residual"].float() + _plain_dropout(s["x"].float(), s)
        rstd = torch.rsqrt((r * r).mean(1) + EPS)
        y = r * rstd[:, None] * s["gain"].float()
        out = {"r": r.to(t), "rstd": rstd}
        if case["out"] == "same":
            out["y"] = y.to(t)
            return out
        M, d = y.shape
        width = d if case["out"] == "row8" else GROUP
        n = -(-d // width)
        parts = torch.cat([y, y.new_zeros(M, n * width - d)], 1).reshape(M, n, width)
        scale = parts.abs().amax(2) / F8_MAX
        scale = torch.where(scale == 0.0, 1.0, scale)
        out["y"] = (parts / scale[:, :, None]).reshape(M, n * width)[:, :d].contiguous().to(F8)
        out["scale"] = scale
        return out
    dy, r, rstd = s["dy"].float(), s["r"].float(), s["rstd"][:, None]
    xh, a = r * rstd, dy * s["gain"].float()
    dr = s["dr"].float() + rstd * (a - xh * (a * xh).mean(1, keepdim=True))
    return {"dx": _plain_dropout(dr, s).to(s["r"].dtype), "dresidual": dr.to(s["r"].dtype),
            "dgain": (dy * xh).sum(0).to(s["gain"].dtype)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------- 64-bit values
def _exact_keep(case, s, M, d):
    """Which elements dropout keeps, from Philox4x32-10 in Python's own wide
    integers on numpy arrays."""
    import numpy as np
    keep = int(math.floor((1.0 - case["p"]) * 65536.0 + 0.5))
    cols = np.arange(-(-d // 8), dtype=np.uint64)
    mask = np.uint64(0xFFFFFFFF)
    s32 = np.uint64(32)
    got = np.empty((M, 8 * len(cols)), dtype=bool)
    for lo in range(0, M, 1024):
        rows = np.arange(lo, min(M, lo + 1024), dtype=np.uint64)
        x0, x1 = np.meshgrid(cols, rows)
        x2, x3 = np.full_like(x0, 0x80000000), np.full_like(x0, s["offset"])
        k0, k1 = s["seed"] & 0xFFFFFFFF, s["seed"] >> 32
        for _ in range(10):
            p0, p1 = x0 * np.uint64(0xD2511F53), x2 * np.uint64(0xCD9E8D57)
            x0, x1, x2, x3 = (p1 >> s32) ^ x1 ^ np.uint64(k0), p1 & mask, (p0 >> s32) ^ x3 ^ np.uint64(k1), p0 & mask
            k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
        for j, w in enumerate((x0, x1, x2, x3)):
            got[lo:lo + len(rows), 2 * j::8] = (w & np.uint64(0xFFFF)) < keep
            got[lo:lo + len(rows), 2 * j + 1::8] = (w >> np.uint64(16)) < keep
    return torch.from_numpy(np.ascontiguousarray(got[:, :d])).cuda(), 65536.0 / max(keep, 1)


def exact(case, seed):
    s = _inputs(case, seed)
    f8 = torch.float64
    M, d = case["rows"], case["d"]
    if case["op"] in ("loss", "step"):
        v, r = case["vocab"], case["rank"]
        if (2 if case["op"] == "loss" else 8) * M * v * (d + r) > 8e12:
            return None
        idx = (s["target"] >= 0).nonzero()[:, 0]
        t = s["target"][idx].long()
        h = s["h"][idx].to(f8)
        e = s["U"][s["prev"][idx].long()].to(f8) if r else None
        step = max(256, (1 << 28) // max(len(idx), 1))
        pieces = [(lo, min(v, lo + step)) for lo in range(0, v, step)]

        def scores(lo, hi):
            z = h @ s["W"][lo:hi].to(f8).T
            return z + e @ s["V"][lo:hi].to(f8).T if r else z

        lse = torch.full((len(idx),), -math.inf, dtype=f8, device="cuda")
        for lo, hi in pieces:
            lse = torch.logaddexp(lse, torch.logsumexp(scores(lo, hi), 1))
        zt = (h * s["W"][t].to(f8)).sum(1) + ((e * s["V"][t].to(f8)).sum(1) if r else 0.0)

        def whole(x):
            full = torch.zeros((M,) + tuple(x.shape[1:]), dtype=f8, device="cuda")
            full[idx] = x
            return full

        out = {"loss": whole(lse - zt), "lse": whole(lse)}
        if case["op"] == "step":
            dh = torch.zeros(len(idx), d, dtype=f8, device="cuda")
            de = torch.zeros(len(idx), r, dtype=f8, device="cuda")
            dW, dV = [], []
            w = s["dloss"][idx].to(f8)[:, None]
            for lo, hi in pieces:
                p = (scores(lo, hi) - lse[:, None]).exp()
                here = ((t >= lo) & (t < hi)).nonzero()[:, 0]
                p[here, t[here] - lo] -= 1.0
                p *= w
                dh += p @ s["W"][lo:hi].to(f8)
                dW.append(p.T @ h)
                if r:
                    de += p @ s["V"][lo:hi].to(f8)
                    dV.append(p.T @ e)
            out["dh"], out["dW"] = whole(dh), torch.cat(dW)
            if r:
                out["dU"] = torch.zeros(v, r, dtype=f8, device="cuda").index_add_(0, s["prev"][idx].long(), de)
                out["dV"] = torch.cat(dV)
        return out
    if case["p"]:
        kept, scale = _exact_keep(case, s, M, d)

        def drop(x):
            return torch.where(kept, x * scale, torch.zeros_like(x))
    else:
        def drop(x):
            return x
    if case["op"] == "dropout":
        return {"y": s["residual"].to(f8) + drop(s["x"].to(f8))}
    gain = s["gain"].to(f8)
    if case["op"] == "norm":
        r = s["residual"].to(f8) + drop(s["x"].to(f8))
        rstd = 1.0 / torch.sqrt(r.square().sum(1) / d + EPS)
        y = r * gain * rstd[:, None]
        out = {"r": r, "rstd": rstd, "y": y}
        if case["out"] != "same":
            n = 1 if case["out"] == "row8" else -(-d // GROUP)
            of = torch.arange(d, device="cuda") // (d if n == 1 else GROUP)
            top = torch.zeros(M, n, dtype=f8, device="cuda").scatter_reduce(1, of.expand(M, d), y.abs(), "amax")
            out["scale"] = torch.where(top > 0, top / F8_MAX, torch.ones_like(top))
            out["y"] = y / out["scale"][:, of]
        return out
    dy, r, rstd = s["dy"].to(f8), s["r"].to(f8), s["rstd"].to(f8)[:, None]
    dot = (dy * gain * r).sum(1, keepdim=True) / d
    dr = s["dr"].to(f8) + dy * gain * rstd - r * rstd ** 3 * dot
    return {"dx": drop(dr), "dresidual": dr, "dgain": (dy * r * rstd).sum(0)}
