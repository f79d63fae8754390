"""Plain 64-bit forms of the target step's operators, on the CPU, and the
inputs that their tests draw."""
import math

import torch

F64 = torch.float64


def is_tree(masks, count):
    return masks is not None and 0 < count <= len(masks) and bool(masks[0] & 1)


def attended(masks, count, j):
    """Rows of its request that row j attends."""
    if is_tree(masks, count):
        return [i for i in range(count) if int(masks[j]) >> i & 1]
    return list(range(j + 1))


def tree_masks(g, N, width):
    """Random trees as [N, width] int64 masks: parents come first."""
    out = torch.zeros(N, width, dtype=torch.int64)
    for n in range(N):
        m = [1]
        for j in range(1, width):
            up = int(torch.randint(0, j, (1,), generator=g))
            m.append(m[up] | (1 << j))
        out[n] = torch.tensor([x - (1 << 64) if x >> 63 else x for x in m])
    return out


# ------------------------------------------------------------------- rows
def rows(draft_len, mask, chunk_len, ctx_len, tree, tokens, draft_tokens, page_count, free, page, max_pages,
         num_pages, max_rows, table):
    """Everything dspark_step_rows writes, as lists; table is changed in place."""
    N, K = len(draft_len), len(draft_tokens[0])
    out = {k: [] for k in ("row_request", "position", "slot", "row_token", "out_row")}
    cu, cu_out, owned_out, free = [0], [0], [], list(free)
    total = 0
    for n in range(N):
        samples = mask is None or mask[n]
        count = min(max(draft_len[n], 0), K) + 1 if samples else max(chunk_len[n] if chunk_len else 0, 0)
        count = min(count, max_rows - total)
        ctx, owned = max(ctx_len[n], 0), min(max(page_count[n], 0), max_pages)
        want = min(-(-(ctx + count) // page), max_pages) if count else 0
        took = 0
        for k in range(owned, want):
            took += bool(free)
            table[n][k] = free.pop() if free else -1
        owned_out.append(owned + took)
        masks = None if tree is None else tree[n]
        for j in range(count):
            index = ctx + j
            depth = len([i for i in attended(masks, count, j) if i != j]) if is_tree(masks, count) else j
            k = index // page
            id = table[n][k] if k < max_pages else -1
            out["row_request"].append(n)
            out["position"].append(ctx + depth)
            out["slot"].append(id * page + index % page if 0 <= id < num_pages else -1)
            drafted = samples and j > 0
            out["row_token"].append(draft_tokens[n][j - 1] if drafted else
                                    (tokens[n][index] if index < len(tokens[n]) else 0))
            if samples:
                out["out_row"].append(total + j)
        total += count
        cu.append(total)
        cu_out.append(len(out["out_row"]))
    return {**out, "cu_rows": cu, "cu_out": cu_out, "page_count": owned_out, "free_count": len(free)}


# ----------------------------------------------------------------- rotary
def rotate(x, position, freq, rot, interleaved, amplitude=1.0, inverse=False):
    x = x.to(F64)
    t = position.to(F64)[:, None] * freq.to(F64)[None, :] * (-1.0 if inverse else 1.0)
    c, s = (torch.cos(t) * amplitude)[:, None], (torch.sin(t) * amplitude)[:, None]
    y = x.clone()
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


# -------------------------------------------------------------- attention
def attention(q, k_cache, v_cache, table, ctx_len, cu, tree, scale):
    """(out, lse, size): size is sum p |v|, what a rounding of p weighs."""
    R, H, d = q.shape
    pages, page, kv, _ = k_cache.shape
    out = torch.zeros(R, H, d, dtype=F64)
    size = torch.zeros(R, H, d, dtype=F64)
    lse = torch.full((R, H), -math.inf, dtype=F64)
    for n in range(len(ctx_len)):
        first, count, ctx = cu[n], cu[n + 1] - cu[n], max(int(ctx_len[n]), 0)
        if count <= 0:
            continue
        index = torch.arange(min(ctx + count, table.shape[1] * page))
        ids = table[n, index // page].long()
        there = (ids >= 0) & (ids < pages)
        K = k_cache[ids.clamp(0, pages - 1), index % page].to(F64)
        V = v_cache[ids.clamp(0, pages - 1), index % page].to(F64)
        for j in range(count):
            seen = there & (index < ctx)
            for i in attended(None if tree is None else [int(x) for x in tree[n]], count, j):
                if ctx + i < len(index):
                    seen[ctx + i] = there[ctx + i]
            at = seen.nonzero()[:, 0]
            if len(at) == 0:
                continue
            for h in range(H):
                kh = h // (H // kv)
                s = (K[at, kh] @ q[first + j, h].to(F64)) * scale
                lse[first + j, h] = torch.logsumexp(s, 0)
                p = torch.softmax(s, 0)
                out[first + j, h] = p @ V[at, kh]
                size[first + j, h] = p @ V[at, kh].abs()
    return out, lse, size


# ----------------------------------------------------------------- logits
def adjust(logits, cu, tokens, hist_len, prompt_len, draft_tokens, tree, repetition=None, frequency=None,
           presence=None, bias_token=None, bias_value=None, bias_count=None, mask=None, mask_index=None):
    """(values, size): size bounds what each rounding of the operations is relative to."""
    y = logits.to(F64).clone()
    size = y.abs()
    R, vocab = y.shape
    for n in range(len(hist_len)):
        count = cu[n + 1] - cu[n]
        hist = tokens[n, :hist_len[n]].tolist()
        prompt = int(prompt_len[n]) if prompt_len is not None else 0
        for j in range(count):
            r = cu[n] + j
            masks = None if tree is None else [int(x) for x in tree[n]]
            path = [int(draft_tokens[n, i - 1]) for i in attended(masks, count, j)
                    if i >= 1 and draft_tokens is not None and i - 1 < draft_tokens.shape[1]]
            said = {}
            for t in hist[prompt:] + path:
                said[t] = said.get(t, 0) + 1
            for t in sorted(set(hist) | set(path)):
                if not 0 <= t < vocab:
                    continue
                x, c = y[r, t], said.get(t, 0)
                if repetition is not None:
                    x = x / repetition[n].to(F64) if x > 0 else x * repetition[n].to(F64)
                size[r, t] = max(size[r, t], abs(x))
                if frequency is not None:
                    x = x - frequency[n].to(F64) * c
                    size[r, t] += abs(frequency[n].to(F64)) * c
                if presence is not None and c:
                    x = x - presence[n].to(F64)
                    size[r, t] += abs(presence[n].to(F64))
                y[r, t] = x
            if bias_token is not None:
                for i in range(int(bias_count[n])):
                    t = int(bias_token[n, i])
                    if 0 <= t < vocab:
                        y[r, t] += bias_value[n, i].to(F64)
                        size[r, t] += abs(bias_value[n, i].to(F64))
            m = -1 if mask is None else (r if mask_index is None else int(mask_index[r]))
            if 0 <= m < (0 if mask is None else len(mask)):
                words = mask[m].long() & 0xFFFFFFFF
                bits = (words[:, None] >> torch.arange(32)) & 1
                y[r, bits.flatten()[:vocab] == 0] = -math.inf
    return y, size
