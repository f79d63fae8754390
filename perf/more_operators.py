"""The operators around the target's pass over the verify list, as cases to be
timed and compared.

* ``rows``    from the scheduler's draft lengths to the rows of the target's
  step: offsets, positions, input tokens, cache slots and the pages that the
  step's tokens need, taken from the free list;
* ``append``  rotary positions on the queries and keys, keys and values written
  to the paged cache; ``rotary``  the rotation by itself, or its gradient;
* ``attend``  attention of each request's rows (one token, a chain of drafts, a
  tree of drafts, a chunk of the prompt) over its pages of the cache;
* ``adjust``  penalties for repeated tokens, biases and grammar masks on the
  target's logits, before they are verified.

``own`` chooses between the plain form (elementary torch operations in 32
bits) and the library's entry points.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BASE = 10000.0
ORIGINAL = 4096      # positions that a scaled model was trained for


def listed():
    return [
        # the rows of a step of 8 requests with up to 7 drafts each: latency
        {"name": "rows_8x7", "op": "rows", "requests": 8, "drafts": 7, "prompts": 0, "chunk": 0, "tree": False,
         "ctx": 1000, "page": 16},
        # the largest batch, a tenth of the requests with 32 tokens of their prompt
        {"name": "rows_1024x15", "op": "rows", "requests": 1024, "drafts": 15, "prompts": 102, "chunk": 32,
         "tree": True, "ctx": 8192, "page": 16},
        # a layer's queries and keys while 8 requests verify 7 drafts: latency
        {"name": "append_8x8", "op": "append", "rows": 64, "heads": 32, "kv": 8, "d": 128, "rot": 128,
         "interleaved": False, "scaling": "none", "page": 16, "type": "bf16", "reach": 8192},
        # chunks of prompts, positions scaled for a long context
        {"name": "append_prompt", "op": "append", "rows": 8192, "heads": 32, "kv": 8, "d": 128, "rot": 128,
         "interleaved": False, "scaling": "parts", "page": 64, "type": "bf16", "reach": 131072},
        # training: the gradient of the rotation, part of an odd head, neighbours in pairs, 32 bits
        {"name": "rotary_grad_odd", "op": "rotary", "rows": 1001, "heads": 10, "kv": 5, "d": 75, "rot": 50,
         "interleaved": True, "scaling": "linear", "inverse": True, "type": "f32", "reach": 32768},
        # one request, one token, a long context: latency
        {"name": "attend_1x1", "op": "attend", "requests": 1, "rows": 1, "tree": False, "ctx": 8192, "ctx_least": 8192,
         "heads": 32, "kv": 8, "d": 128, "page": 16},
        # verifying 7 drafts of each of 64 requests
        {"name": "attend_64x8", "op": "attend", "requests": 64, "rows": 8, "tree": False, "ctx": 8192, "ctx_least": 0,
         "heads": 32, "kv": 8, "d": 128, "page": 16},
        # trees of 24 drafts, many requests with short contexts, narrow heads
        {"name": "attend_tree", "op": "attend", "requests": 256, "rows": 25, "tree": True, "ctx": 2001, "ctx_least": 1,
         "heads": 24, "kv": 4, "d": 64, "page": 32},
        # chunks of 512 tokens of 16 prompts: bound by arithmetic
        {"name": "attend_prompt", "op": "attend", "requests": 16, "rows": 512, "tree": False, "ctx": 7680,
         "ctx_least": 0, "heads": 32, "kv": 8, "d": 128, "page": 64},
        # penalties and biases for 8 requests with 7 drafts, in place: latency
        {"name": "adjust_8x8", "op": "adjust", "requests": 8, "rows": 8, "tree": False, "vocab": 262144,
         "history": 2048, "bias": 16, "masked": 0.0, "in_place": True, "type": "bf16"},
        # the benchmark's batch, half of the rows held to a grammar, in place
        {"name": "adjust_256x8", "op": "adjust", "requests": 256, "rows": 8, "tree": False, "vocab": 262144,
         "history": 4096, "bias": 64, "masked": 0.5, "in_place": True, "type": "bf16"},
        # trees, an odd vocabulary in 32 bits, the raw logits kept
        {"name": "adjust_tree_odd", "op": "adjust", "requests": 33, "rows": 17, "tree": True, "vocab": 50003,
         "history": 1000, "bias": 5, "masked": 1.0, "in_place": False, "type": "f32"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rows", "append", "rotary", "attend", "attend", "attend", "adjust", "adjust"])
    if op == "rows":
        n = _log_int(rng, 1, 1024)
        return {"op": op, "requests": n, "drafts": rng.randint(1, 15), "prompts": rng.choice([0, n // 10, n // 3]),
                "chunk": _log_int(rng, 1, 512) if n < 100 else 32, "tree": rng.random() < 0.5,
                "ctx": _log_int(rng, 1, 8192), "page": rng.choice([16, 32, 64, 128])}
    if op in ("append", "rotary"):
        kv = rng.choice([1, 2, 4, 5, 8])
        d = rng.choice([64, 96, 128, 128, 8 * rng.randint(4, 16)])
        c = {"op": op, "rows": _log_int(rng, 1, 8192), "heads": kv * rng.randint(1, 4), "kv": kv, "d": d,
             "rot": rng.choice([d, d, d // 2 // 2 * 2]), "interleaved": rng.random() < 0.4,
             "scaling": rng.choice(["none", "linear", "parts"]), "type": rng.choice(["bf16", "bf16", "f32"]),
             "reach": _log_int(rng, 1000, 1000000)}
        if op == "append":
            c["page"] = rng.choice([16, 32, 64, 128])
        else:
            c["inverse"] = rng.random() < 0.5
        return c
    if op == "attend":
        while True:
            kv = rng.choice([1, 2, 4, 8])
            form = rng.choice(["one", "chain", "tree", "chunk"])
            c = {"op": op, "requests": _log_int(rng, 1, 256), "tree": form == "tree",
                 "rows": {"one": 1, "chain": rng.randint(2, 16), "tree": rng.randint(2, 64),
                          "chunk": _log_int(rng, 17, 1000)}[form],
                 "ctx": _log_int(rng, 1, 8192), "heads": kv * rng.choice([1, 2, 3, 4, 6, 8, 16]), "kv": kv,
                 "d": rng.choice([64, 80, 128, 128, 256]), "page": rng.choice([16, 32, 64, 128])}
            c["ctx_least"] = rng.choice([0, 0, 1, c["ctx"] // 2, c["ctx"]])
            seen = c["requests"] * (c["ctx"] + c["rows"])
            if seen * c["rows"] * c["heads"] * c["d"] <= 16 * 8192 * 512 * 32 * 128 \
                    and seen * c["rows"] * c["heads"] <= 16 * 8192 * 512 * 32 \
                    and seen * kv * c["d"] <= 64 * 8200 * 8 * 128:
                return c
    while True:
        c = {"op": op, "requests": _log_int(rng, 1, 256), "rows": rng.randint(1, 16), "tree": rng.random() < 0.4,
             "vocab": rng.choice([_log_int(rng, 256, 262144), 32 * _log_int(rng, 8, 8192)]),
             "history": _log_int(rng, 1, 4096),
             "bias": rng.choice([0, rng.randint(1, 64)]), "masked": rng.choice([0.0, 0.5, 1.0]),
             "in_place": rng.random() < 0.6, "type": rng.choice(["bf16", "bf16", "f32"])}
        if c["requests"] * c["rows"] * c["vocab"] <= 256 * 8 * 262144 // 2:
            return c


# ------------------------------------------------- what a case's seed permutes
def _spread(lo, hi, n):
    """n whole numbers evenly from lo to hi."""
    return [lo + (hi - lo) * i // max(n - 1, 1) if n > 1 else hi for i in range(n)]


def _row_counts(c):
    """Draft lengths of the requests that sample, prompt chunks of the others."""
    sampling = c["requests"] - c["prompts"]
    return [i % (c["drafts"] + 1) for i in range(sampling)], [1 + (c["chunk"] - 1) * i // max(c["prompts"] - 1, 1)
                                                             for i in range(c["prompts"])]


def _pages_of(tokens, page):
    return -(-tokens // page)


def work(case):
    c, op = case, case["op"]
    e = 2 if c.get("type", "bf16") == "bf16" else 4
    if op == "rows":
        drafts, chunks = _row_counts(c)
        n, rows = c["requests"], sum(drafts) + len(drafts) + sum(chunks)
        new = _pages_of(rows, c["page"])
        tree = 8 * rows if c["tree"] else 0
        return {"bytes": 21 * n + 8 * n + 20 * rows + 4 * (sum(drafts) + len(drafts)) + 8 * rows + tree + 8 * new,
                "flops": 0}
    if op in ("append", "rotary"):
        rows, q, k = c["rows"], c["heads"] * c["d"], c["kv"] * c["d"]
        moved = 2 * (q + 2 * k) if op == "append" else 2 * (q + k)
        return {"bytes": rows * (e * moved + (8 if op == "append" else 4)) + 8 * (c["rot"] // 2),
                "flops": 3 * rows * (c["heads"] + c["kv"]) * c["rot"]}
    if op == "attend":
        n, L, H = c["requests"], c["rows"], c["heads"]
        ctx = sum(_spread(c["ctx_least"], c["ctx"], n))
        cached = 2 * 2 * (ctx + n * L) * c["kv"] * c["d"]
        seen = L * ctx + n * L * (L + 1) // 2
        return {"bytes": cached + n * L * H * (4 * c["d"] + 4) + 4 * (ctx + n * L) // c["page"] + 12 * n
                + (8 * n * L if c["tree"] else 0), "flops": 4 * seen * H * c["d"]}
    rows, v = c["requests"] * c["rows"], c["vocab"]
    hist = sum(_spread(1, c["history"], c["requests"]))
    small = 4 * hist + c["requests"] * (24 + 4 * c["rows"] + 8 * c["bias"])
    masked = int(rows * c["masked"])
    if c["in_place"]:
        # what changes: the tokens seen (a row at most), the biases, and what a mask forbids
        touched = rows * (min(400, hist // c["requests"]) + c["bias"])
        return {"bytes": small + 2 * e * touched + masked * (v // 8 + e * v * 3 // 4), "flops": 6 * touched}
    return {"bytes": small + 2 * e * rows * v + masked * v // 8, "flops": 6 * rows * v}


def _tree_masks(requests, width, g):
    """Masks of random trees, [requests, width] int64: bit i of row j says that j
    descends from i (or is it); each row's parent comes before it."""
    parent = (torch.rand(requests, width, generator=g, device="cuda") * torch.arange(width, device="cuda")).long()
    mask = torch.zeros(requests, width, dtype=torch.int64, device="cuda")
    mask[:, 0] = 1
    for j in range(1, width):
        mask[:, j] = mask.gather(1, parent[:, j:j + 1])[:, 0] | (1 << j if j < 63 else -(1 << 63))
    return mask


def _inputs(case, seed):
    """The inputs as a serving or training program has them, on the GPU."""
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(sd, *shape, dtype=torch.bfloat16):
        x = torch.empty(*shape, dtype=dtype, device="cuda")
        return x.normal_(0.0, sd, generator=g)

    def perm(n):
        return torch.randperm(n, generator=g, device="cuda")

    def i32(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    def tokens(*shape, vocab):
        return torch.randint(0, vocab, shape, generator=g, device="cuda", dtype=torch.int32)

    s = {}
    if c["op"] == "rows":
        n, K, P = c["requests"], c["drafts"], c["page"]
        drafts, chunks = _row_counts(c)
        order = perm(n)
        s["draft_len"] = i32(drafts + [0] * len(chunks))[order]
        s["chunk_len"] = i32([0] * len(drafts) + chunks)[order]
        s["mask"] = torch.tensor([1] * len(drafts) + [0] * len(chunks), dtype=torch.uint8, device="cuda")[order]
        s["ctx_len"] = i32(_spread(0, c["ctx"], n))[perm(n)]
        s["tree"] = _tree_masks(n, K + 1, g) if c["tree"] else None
        if c["tree"]:
            s["tree"] *= s["mask"].long()[:, None]      # prompts are chains
        s["tokens"] = tokens(n, c["ctx"] + max(chunks, default=0) + 1, vocab=262144)
        s["draft_tokens"] = tokens(n, K, vocab=262144)
        owned = (s["ctx_len"] + P - 1) // P
        width = _pages_of(c["ctx"] + max(K + 1, max(chunks, default=0)), P)
        pages = n * width + 8
        ids = perm(pages).int()
        s["block_table"] = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
        have = torch.arange(width, device="cuda")[None, :] < owned[:, None]
        s["block_table"] = torch.where(have, ids[8:].reshape(n, width), s["block_table"])
        s["page_count"] = owned.int()
        free = torch.cat([ids[:8], ids[8:][~have.reshape(-1)]])
        s["free_pages"], s["free_count"], s["pages"] = free, i32([free.numel()]), pages
        s["total"] = sum(drafts) + len(drafts) + sum(chunks)
        return s
    if c["op"] in ("append", "rotary"):
        R, H, k, d = c["rows"], c["heads"], c["kv"], c["d"]
        t = TYPES[c["type"]]
        qkv = normal(1.0, R, (H + 2 * k) * d, dtype=t)          # a layer's fused projection
        s["q"] = qkv[:, :H * d].view(R, H, d)
        s["k"] = qkv[:, H * d:(H + k) * d].view(R, k, d)
        s["v"] = qkv[:, (H + k) * d:].view(R, k, d)
        s["position"] = torch.randint(0, c["reach"], (R,), generator=g, device="cuda", dtype=torch.int32)
        if c["op"] == "append":
            pages = _pages_of(R, c["page"]) * 2
            s["k_cache"], s["v_cache"] = (normal(1.0, pages, c["page"], k, d, dtype=t) for _ in range(2))
            s["slot"] = perm(pages * c["page"])[:R].int()
        return s
    if c["op"] == "attend":
        n, L, P = c["requests"], c["rows"], c["page"]
        ctx = _spread(c["ctx_least"], c["ctx"], n)
        s["ctx_len"] = i32(ctx)[perm(n)]
        s["cu_rows"] = i32([i * L for i in range(n + 1)])
        s["q"] = normal(1.0, n * L, c["heads"], c["d"])
        width = _pages_of(c["ctx"] + L, P)
        pages = sum(_pages_of(x + L, P) for x in ctx)
        s["k_cache"], s["v_cache"] = (normal(1.0, pages, P, c["kv"], c["d"]) for _ in range(2))
        ends = (s["ctx_len"] + L + P - 1) // P
        have = torch.arange(width, device="cuda")[None, :] < ends[:, None]
        at = (have.reshape(-1).cumsum(0) - 1).clamp(min=0)
        s["block_table"] = torch.where(have, perm(pages).int()[at].reshape(n, width), -1).int()
        s["tree"] = _tree_masks(n, L, g) if c["tree"] else None
        return s
    n, L, v = c["requests"], c["rows"], c["vocab"]
    t = TYPES[c["type"]]
    s["logits"] = normal(2.0, n * L, v, dtype=t)
    s["cu_rows"] = i32([i * L for i in range(n + 1)])
    hist = i32(_spread(1, c["history"], n))[perm(n)]
    # a text repeats itself: tokens from a few hundred
    few = tokens(n, 400, vocab=v)
    s["tokens"] = few.gather(1, torch.randint(0, 400, (n, c["history"]), generator=g, device="cuda"))
    s["hist_len"], s["prompt_len"] = hist, hist // 3
    s["draft_tokens"] = few[:, :max(L - 1, 1)].contiguous()
    s["tree"] = _tree_masks(n, L, g) if c["tree"] else None
    s["repetition"] = 1.0 + torch.rand(n, generator=g, device="cuda") * 0.5
    s["frequency"] = torch.rand(n, generator=g, device="cuda")
    s["presence"] = torch.rand(n, generator=g, device="cuda")
    if c["bias"]:
        # tokens of the text, and others
        b = torch.cat([few[:, :c["bias"] // 2], tokens(n, c["bias"] - c["bias"] // 2, vocab=v)], 1)
        s["bias_token"] = b.contiguous()
        s["bias_value"] = normal(3.0, n, c["bias"], dtype=torch.float32)
        s["bias_count"] = torch.full((n,), c["bias"], dtype=torch.int32, device="cuda")
    if c["masked"]:
        m = max(1, int(n * L * c["masked"]))
        # three quarters forbidden, mostly in runs as a grammar leaves them
        words = -(-v // 32)
        keep = torch.randint(-1 << 31, 1 << 31, (m, words), generator=g, device="cuda", dtype=torch.int64).int()
        keep &= -(torch.rand(m, words, generator=g, device="cuda") < 0.5).int()
        s["mask"] = keep
        s["mask_index"] = torch.full((n * L,), -1, dtype=torch.int32, device="cuda")
        s["mask_index"][perm(n * L)[:m]] = torch.arange(m, dtype=torch.int32, device="cuda")
    return s


def _inv_freq(c):
    """Angles a position, [rot / 2] fp64: base^(-2i / rot), scaled."""
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda")
    f = BASE ** (-2.0 * i / c["rot"])
    if c["scaling"] == "linear":
        return f / 8.0
    if c["scaling"] == "parts":
        # frequencies that turn over 32 times within the original length stay,
        # those that turn less than once are stretched, a ramp over i between
        low, high = (c["rot"] * math.log(ORIGINAL / (b * 2.0 * math.pi)) / (2.0 * math.log(BASE)) for b in (32.0, 1.0))
        low, high = max(math.floor(low), 0), min(math.ceil(high), c["rot"] // 2 - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
        return f * (1.0 - ramp) + f / 32.0 * ramp
    return f


def _amplitude(c):
    return 0.1 * math.log(32.0) + 1.0 if c["scaling"] == "parts" else 1.0


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    c = case

    def new(dtype, *shape, fill=None):
        if fill is None:
            return torch.empty(*shape, dtype=dtype, device="cuda")
        return torch.full(shape, fill, dtype=dtype, device="cuda")

    # the buffers that a program keeps for the results
    if c["op"] == "rows":
        n, most, i32 = c["requests"], s["total"] + 8, torch.int32
        s["out"] = {"cu_rows": new(i32, n + 1), "cu_out": new(i32, n + 1), "page_count": new(i32, n),
                    "free_count": new(i32, 1)}
        for k in ("row_request", "position", "slot", "row_token", "out_row"):
            s["out"][k] = new(i32, most, fill=-9)
        s["out"]["block_table"] = s["block_table"]
    elif c["op"] == "rotary":
        s["out"] = {"q": torch.empty_like(s["q"]).contiguous(), "k": torch.empty_like(s["k"]).contiguous()}
    elif c["op"] == "append":
        s["out"] = {"q": torch.empty_like(s["q"]).contiguous(), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    elif c["op"] == "attend":
        s["out"] = {"out": torch.empty_like(s["q"]), "lse": new(torch.float32, *s["q"].shape[:2])}
    else:
        s["out"] = {"logits": s["logits"] if c["in_place"] else torch.empty_like(s["logits"])}
    if c["op"] in ("append", "rotary"):
        s["inv_freq"] = _inv_freq(c)
    if own:
        from speculative_decoding_draft_dspark_gb300 import target as T
        if c["op"] in ("append", "rotary"):
            how = {"none": {}, "linear": {"scaling": T.ROPE_LINEAR, "factor": 8.0},
                   "parts": {"scaling": T.ROPE_BY_PARTS, "factor": 32.0, "original": ORIGINAL, "low": 1.0,
                             "high": 32.0}}[c["scaling"]]
            s["turns"] = T.dspark_rotary_table(c["rot"], BASE, **how).cuda()
        elif c["op"] == "attend":
            s["ws"] = T.new_workspace(T.dspark_attention_workspace_size(c["requests"], c["rows"], c["heads"], c["kv"],
                                                                        c["d"]))
        else:
            s["ws"] = T.new_workspace(256)
    return s


def _run_own(s):
    from speculative_decoding_draft_dspark_gb300 import target as T
    c, out = s["case"], s["out"]
    if c["op"] == "rows":
        T.dspark_step_rows(s["draft_len"], s["mask"], s["chunk_len"], s["ctx_len"], s["tree"], s["tokens"],
                           s["draft_tokens"], s["page_count"], s["free_pages"], s["free_count"], out["block_table"],
                           out["page_count"], out["free_count"], out["cu_rows"], out["cu_out"], out["row_request"],
                           out["position"], out["slot"], out["row_token"], out["out_row"], s["ws"],
                           page_size=c["page"], num_pages=s["pages"])
    elif c["op"] == "rotary":
        T.dspark_rotary(s["q"], s["k"], s["position"], s["turns"], out["q"], out["k"], interleaved=c["interleaved"],
                        inverse=c["inverse"], amplitude=_amplitude(c))
    elif c["op"] == "append":
        T.dspark_rotary_append(s["q"], s["k"], s["v"], s["position"], s["slot"], s["turns"], out["q"], out["k_cache"],
                               out["v_cache"], interleaved=c["interleaved"], amplitude=_amplitude(c))
    elif c["op"] == "attend":
        T.dspark_tree_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["ctx_len"], s["cu_rows"],
                                s["tree"], out["out"], out["lse"], s["ws"], max_len=c["rows"],
                                scale=1.0 / math.sqrt(c["d"]))
    else:
        T.dspark_adjust_logits(s["logits"], s["cu_rows"], s["tokens"], s["hist_len"], s["prompt_len"],
                               s["draft_tokens"], s["tree"], out["logits"], s["ws"], repetition=s["repetition"],
                               frequency=s["frequency"], presence=s["presence"], bias_token=s.get("bias_token"),
                               bias_value=s.get("bias_value"), bias_count=s.get("bias_count"), mask=s.get("mask"),
                               mask_index=s.get("mask_index"))
    return out


# ------------------------------------------------------------- plain form
def _bits(words):
    """Bits of whole numbers, lowest first, on a new last dimension."""
    n = 8 * words.element_size()
    return (words[..., None] >> torch.arange(n, device=words.device, dtype=words.dtype)) & 1


def _plain_rows(s):
    c, P = s["case"], s["case"]["page"]
    n, K, total = c["requests"], c["drafts"], s["total"]
    samples = s["mask"] != 0
    count = torch.where(samples, s["draft_len"] + 1, s["chunk_len"]).long()
    ctx = s["ctx_len"].long()
    out = {k: torch.full_like(v, -9) for k, v in s["out"].items() if k not in ("block_table", "page_count")}
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    cu, cu_out = (torch.cat([zero, x.cumsum(0)]) for x in (count, torch.where(samples, count, 0)))
    out["cu_rows"], out["cu_out"] = cu.int(), cu_out.int()
    # pages: the first pops the end of the free list
    owned = s["page_count"].long()
    need = ((ctx + count + P - 1) // P - owned).clamp(min=0)
    first = need.cumsum(0) - need
    fresh = torch.arange(s["block_table"].shape[1], device="cuda")[None, :] - owned[:, None]
    pick = s["free_count"].long() - 1 - first[:, None] - fresh.clamp(min=0)
    table = torch.where((fresh >= 0) & (fresh < need[:, None]), s["free_pages"][pick.clamp(min=0)], s["block_table"])
    s["block_table"].copy_(table)
    out["block_table"], out["page_count"] = s["block_table"], (owned + need).int()
    out["free_count"] = (s["free_count"] - need.sum()).int()
    # rows
    r = torch.repeat_interleave(torch.arange(n, device="cuda"), count, output_size=total)
    j = torch.arange(total, device="cuda") - cu[r]
    depth = j
    if s["tree"] is not None:
        at = j.clamp(max=K)
        bits = _bits(s["tree"][r, at])
        within = torch.arange(64, device="cuda") < count[r][:, None]
        ancestors = (bits * within).sum(1) - bits.gather(1, at[:, None])[:, 0]
        depth = torch.where((s["tree"][r, 0] & 1 == 1) & (count[r] <= K + 1), ancestors, j)
    index = ctx[r] + j
    drafted = samples[r] & (j > 0)
    token = torch.where(drafted, s["draft_tokens"][r, (j - 1).clamp(0, K - 1)],
                        s["tokens"][r, index.clamp(max=s["tokens"].shape[1] - 1)])
    out["row_request"][:total] = r.int()
    out["position"][:total] = (ctx[r] + depth).int()
    out["slot"][:total] = (table[r, index // P] * P + index % P).int()
    out["row_token"][:total] = token
    out["out_row"][torch.where(samples[r], cu_out[r] + j, out["out_row"].numel() - 1)] = \
        torch.where(samples[r], torch.arange(total, device="cuda"), -9).int()
    return out


def _rotate(x, cos, sin, rot, interleaved):
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = torch.empty_like(x)
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    y[..., rot:] = x[..., rot:]
    return y


def _plain_rotary(s):
    c, t = s["case"], s["q"].dtype
    angle = s["position"].double()[:, None, None] * s["inv_freq"]
    cos, sin = ((f(angle) * _amplitude(c)).float() for f in (torch.cos, torch.sin))
    if c.get("inverse"):
        sin = -sin
    q, k = (_rotate(x.float(), cos, sin, c["rot"], c["interleaved"]).to(t) for x in (s["q"], s["k"]))
    if c["op"] == "rotary":
        return {"q": q, "k": k}
    slot = s["slot"].long()
    page, at = slot // c["page"], slot % c["page"]
    s["k_cache"][page, at], s["v_cache"][page, at] = k, s["v"]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    c = s["case"]
    n, L, H, kv, d, P = (c[k] for k in ("requests", "rows", "heads", "kv", "d", "page"))
    S = c["ctx"] + L
    t = torch.arange(S, device="cuda")
    page = s["block_table"].long().clamp(min=0)[:, t // P]
    K, V = (x[page, t % P].permute(0, 2, 1, 3).float() for x in (s["k_cache"], s["v_cache"]))    # [n, kv, S, d]
    q = s["q"].view(n, L, kv, H // kv, d).permute(0, 2, 1, 3, 4).reshape(n, kv, L * (H // kv), d).float()
    score = (q @ K.transpose(2, 3) * (1.0 / math.sqrt(d))).view(n, kv, L, H // kv, S)
    i = t - s["ctx_len"].long()[:, None]                                                         # [n, S], in the step
    j = torch.arange(L, device="cuda")[:, None]
    if s["tree"] is None:
        seen = i[:, None, :] <= j
    else:
        bit = (s["tree"][:, :, None] >> i[:, None, :].clamp(0, 63)) & 1
        seen = (i[:, None, :] < 0) | ((bit == 1) & (i[:, None, :] < L))
    score = torch.where(seen[:, None, :, None, :], score, -math.inf)
    top = score.max(4, keepdim=True).values
    p = (score - top).exp()
    total = p.sum(4, keepdim=True)
    V = torch.where((i < L)[:, None, :, None], V, 0.0)
    y = (p / total).view(n, kv, L * (H // kv), S) @ V
    y = y.view(n, kv, L, H // kv, d).permute(0, 2, 1, 3, 4).reshape(n * L, H, d)
    lse = (top + total.log()).view(n, kv, L, H // kv).permute(0, 2, 1, 3).reshape(n * L, H)
    return {"out": y.to(s["q"].dtype), "lse": lse}


def _plain_adjust(s):
    c = s["case"]
    n, L, v = c["requests"], c["rows"], c["vocab"]
    x = s["logits"].float().view(n, L, v)
    at = torch.arange(s["tokens"].shape[1], device="cuda")[None, :]
    token = s["tokens"].long()
    count = torch.zeros(n, v, device="cuda")
    said = ((at >= s["prompt_len"][:, None]) & (at < s["hist_len"][:, None])).float()
    prompt = torch.zeros_like(count).scatter_add_(1, token, (at < s["prompt_len"][:, None]).float()) > 0
    count = count.scatter_add_(1, token, said)[:, None, :].repeat(1, L, 1)
    if L > 1:
        # the drafts on a row's path: all before it, or its ancestors and itself
        path = torch.ones(L, L, device="cuda").tril().expand(n, L, L) if s["tree"] is None \
            else _bits(s["tree"])[:, :, :L].float()
        count.scatter_add_(2, s["draft_tokens"].long()[:, None, :].expand(n, L, L - 1), path[:, :, 1:].contiguous())
    seen = (count > 0) | prompt[:, None, :]
    rep = s["repetition"][:, None, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None, None] * count
    x = torch.where(count > 0, x - s["presence"][:, None, None], x)
    if c["bias"]:
        bias = torch.zeros(n, v, device="cuda").scatter_add_(1, s["bias_token"].long(), s["bias_value"])
        x = x + bias[:, None, :]
    x = x.view(n * L, v)
    if c["masked"]:
        index = s["mask_index"].long()
        keep = _bits(s["mask"]).view(len(s["mask"]), -1)[:, :v] != 0
        x = torch.where(keep[index.clamp(min=0)] | (index < 0)[:, None], x, -math.inf)
    y = x.to(s["logits"].dtype)
    if c["in_place"]:
        y = s["logits"].copy_(y)
    return {"logits": y}


def _run_plain(s):
    return {"rows": _plain_rows, "append": _plain_rotary, "rotary": _plain_rotary, "attend": _plain_attend,
            "adjust": _plain_adjust}[s["case"]["op"]](s)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------- 64-bit values
def _exact_turned(x, angle, amplitude, c):
    """Each pair of x as a complex number times amplitude e^(i angle)."""
    x, rot = x.double(), c["rot"]
    pair = x[..., :rot].unflatten(-1, (rot // 2, 2)) if c["interleaved"] \
        else x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    z = torch.view_as_complex(pair.contiguous()) * torch.polar(torch.full_like(angle, amplitude), angle)[:, None, :]
    z = torch.view_as_real(z)
    z = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, x[..., rot:]], -1)


def _exact_frequency(c, i):
    """Angle a position of pair i, as a Python number."""
    f = math.exp(-2.0 * i / c["rot"] * math.log(BASE))
    if c["scaling"] == "linear":
        return f / 8.0
    if c["scaling"] == "parts":
        edge = [c["rot"] / 2.0 * math.log(ORIGINAL / (2.0 * math.pi * b)) / math.log(BASE) for b in (32.0, 1.0)]
        low, high = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), c["rot"] // 2 - 1)
        w = min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
        return f + w * (f / 32.0 - f)
    return f


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    f8 = torch.float64
    if c["op"] == "rows":
        return None                    # whole numbers
    if c["op"] in ("append", "rotary"):
        freq = torch.tensor([_exact_frequency(c, i) for i in range(c["rot"] // 2)], dtype=f8, device="cuda")
        angle = s["position"].to(f8)[:, None] * freq * (-1.0 if c.get("inverse") else 1.0)
        q, k = (_exact_turned(s[x], angle, _amplitude(c), c) for x in "qk")
        if c["op"] == "rotary":
            return {"q": q, "k": k}
        flat = {}
        for name, x in (("k_cache", k), ("v_cache", s["v"].to(f8))):
            flat[name] = s[name].to(f8).flatten(0, 1).index_copy(0, s["slot"].long(), x).view(s[name].shape)
        return {"q": q, **flat}
    if c["op"] == "attend":
        n, L, H, kv, d, P = (c[k] for k in ("requests", "rows", "heads", "kv", "d", "page"))
        if 4 * d * H * L * n * (c["ctx"] + L) > 4e12:
            return None
        y, lse = torch.zeros(n * L, H, d, dtype=f8, device="cuda"), torch.zeros(n * L, H, dtype=f8, device="cuda")
        for r, ctx in enumerate(s["ctx_len"].tolist()):
            pages = s["block_table"][r, :_pages_of(ctx + L, P)].long()
            K, V = (x[pages].flatten(0, 1)[:ctx + L].to(f8) for x in (s["k_cache"], s["v_cache"]))
            allowed = torch.ones(L, ctx + L, dtype=torch.bool, device="cuda")
            if s["tree"] is None:
                allowed[:, ctx:] = torch.ones(L, L, device="cuda").tril() > 0
            else:
                allowed[:, ctx:] = torch.tensor([[m >> i & 1 for i in range(L)] for m in s["tree"][r].tolist()],
                                                device="cuda") > 0
            for h in range(kv):
                rows, heads = slice(r * L, r * L + L), slice(h * (H // kv), (h + 1) * (H // kv))
                z = torch.einsum("lgd,sd->gls", s["q"][rows, heads].to(f8), K[:, h]) / math.sqrt(d)
                z = z.masked_fill(~allowed, -math.inf)
                lse[rows, heads] = z.logsumexp(2).T
                y[rows, heads] = torch.einsum("gls,sd->lgd", torch.softmax(z, 2), V[:, h])
        return {"out": y, "lse": lse}
    n, L, v = c["requests"], c["rows"], c["vocab"]
    y = s["logits"].to(f8)
    for r in range(n):
        hist, prompt = int(s["hist_len"][r]), int(s["prompt_len"][r])
        before = torch.bincount(s["tokens"][r, :prompt].long(), minlength=v)
        said = torch.bincount(s["tokens"][r, prompt:hist].long(), minlength=v)
        masks = s["tree"][r].tolist() if s["tree"] is not None else [(2 << j) - 1 for j in range(L)]
        for j in range(L):
            path = [i - 1 for i in range(1, L) if masks[j] >> i & 1]
            now = said + torch.bincount(s["draft_tokens"][r, path].long(), minlength=v) if path else said
            row, used = y[r * L + j], (now + before) > 0
            row = torch.where(used & (row > 0), row / s["repetition"][r].to(f8),
                              torch.where(used, row * s["repetition"][r].to(f8), row))
            row = row - now * s["frequency"][r].to(f8) - (now > 0) * s["presence"][r].to(f8)
            if c["bias"]:
                row = row.index_add(0, s["bias_token"][r].long(), s["bias_value"][r].to(f8))
            if c["masked"] and int(s["mask_index"][r * L + j]) >= 0:
                words = s["mask"][int(s["mask_index"][r * L + j])].long() & 0xFFFFFFFF
                allowed = (words[:, None] // (1 << torch.arange(32, device="cuda"))) % 2
                row = row.masked_fill(allowed.flatten()[:v] == 0, -math.inf)
            y[r * L + j] = row
    return {"logits": y}
