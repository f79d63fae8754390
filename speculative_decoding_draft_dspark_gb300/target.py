"""ctypes binding of include/dspark_target.h (argument marshalling only): the
target's pass over the verify list, from the scheduler's draft lengths to the
logits that dspark_greedy_verify reads.

As in ``dspark``: every function has the name of the C entry point it calls
and passes ``torch`` tensors as raw device pointers with the current CUDA
stream; there is no CPU or PyTorch fallback.  Shapes, types and layouts that
the C call cannot see from a pointer are checked here (``ValueError``).
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

from . import dspark as _d
from .dspark import _F, _I32, _I64, _P, _SZ, new_workspace
from .head import _done, _dtype, _flat, _place, _refuse, _rows, _space, _stream

HEADER = os.path.join(os.path.dirname(_d.HERE), "include", "dspark_target.h")

DEV_PAGES_SHORT = 64
DEV_ROWS_SHORT = 128
DEV_LEN_OOR = 256
DEV_PAGE_OOR = 512
ROPE_PLAIN = 0
ROPE_LINEAR = 1
ROPE_BY_PARTS = 2
ROPE_BY_TURNS = 3

_D = ctypes.c_double
_HEADS = [_P, _I64, _I64]

_SIGS = {
    "dspark_step_rows": (_I32, [_P, _P, _P, _P, _P, _I32, _P, _I64, _I32, _P, _I32, _I32, _P, _P,
                                _I32, _P, _I32, _I32, _P, _I64, _I32, _P, _P, _P, _P, _I32, _P,
                                _P, _P, _P, _P, _P, _SZ, _P]),
    "dspark_rotary_table": (_I32, [_I32, _D, _I32, _D, _D, _D, _D, _P]),
    "dspark_rotary": (_I32, [*_HEADS, _I32, *_HEADS, _I32, _I32, _I32, _I32, _P, _P, _P, _I32,
                             _I32, _I32, _F, *_HEADS, *_HEADS, _P]),
    "dspark_rotary_append": (_I32, [*_HEADS, _I32, *_HEADS, *_HEADS, _I32, _I32, _I32, _I32, _P,
                                    _P, _P, _P, _I32, _I32, _F, *_HEADS, _P, _P, _I64, _I64, _I64,
                                    _I32, _I32, _P]),
    "dspark_attention_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32]),
    "dspark_tree_attention": (_I32, [*_HEADS, _P, _P, _I64, _I64, _I64, _I32, _I32, _P, _I64,
                                     _I32, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                                     _F, *_HEADS, _P, _P, _SZ, _P]),
    "dspark_adjust_logits": (_I32, [_P, _I64, _I32, _I32, _I32, _P, _I32, _P, _I64, _I32, _P, _P,
                                    _P, _I32, _P, _I32, _P, _P, _P, _P, _P, _P, _I32, _P, _I64,
                                    _I32, _P, _P, _I64, _P, _SZ, _P]),
}

__all__ = sorted(_SIGS) + ["new_workspace"]

_lib = None
_I32_MAX = (1 << 31) - 1


def header_functions() -> list[str]:
    """Names of the entry points declared in include/dspark_target.h."""
    with open(HEADER) as f:
        txt = f.read()
    return sorted(set(re.findall(r"DSPARK_API\s+[\w\s\*]+?\b(dspark_\w+)\s*\(", txt)))


def load() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = _d.load()
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _sizes(name, t, dims):
    """Shape of a tensor of so many dimensions, each below 2^31."""
    if t is None or t.dim() != dims:
        raise ValueError(f"{name} must be {dims}-D")
    shape = t.shape
    if max(shape) > _I32_MAX:
        raise ValueError(f"{name}'s dimensions must be below 2^31, got {tuple(shape)}")
    return shape


def _int(name, value, low=0):
    """A whole number that C takes in 32 bits; more would be cut off on the way."""
    if not low <= value <= _I32_MAX:
        raise ValueError(f"{name} must be in [{low}, 2^31), got {value}")
    return value


def _maybe(name, t, shape, dtype, dev):
    return None if t is None else _flat(name, t, shape, dtype, dev)


def _heads(name, t, shape, dtype, dev):
    """(pointer, row stride, head stride) of a [rows, heads, d] tensor whose
    columns are contiguous."""
    if t is None or t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _refuse(name, t, shape, dtype, dev)
    rows, heads, d = shape
    row, head, one = t.stride()
    if one != 1 and d > 1:
        raise ValueError(f"{name} must be contiguous along its columns")
    # the stride of a dimension with one entry means nothing
    if heads <= 1:
        head = d
    if rows <= 1:
        row = max(1, heads) * max(head, d)
    return t.data_ptr(), row, head


def _caches(k_cache, v_cache, heads, d, dtype, dev):
    """(pointers, strides, page size, pages) of a cache's keys and values."""
    shape = _sizes("k_cache", k_cache, 4)
    if (k_cache.dtype is not dtype or shape[2] != heads or shape[3] != d
            or k_cache.get_device() != dev):
        _refuse("k_cache", k_cache, torch.Size((shape[0], shape[1], heads, d)), dtype, dev)
    if (v_cache is None or v_cache.dtype is not dtype or v_cache.shape != shape
            or v_cache.get_device() != dev):
        _refuse("v_cache", v_cache, shape, dtype, dev)
    strides = page, token, head, one = k_cache.stride()
    if one != 1 and d > 1:
        raise ValueError("k_cache must be contiguous along its columns")
    pages, size = shape[0], shape[1]
    if v_cache.stride() != strides and any(
            a != b for a, b, n in zip(strides, v_cache.stride(), shape) if n > 1):
        raise ValueError("k_cache and v_cache must have the same strides")
    # as above, in an order that nests
    if heads <= 1:
        head = d
    if size <= 1:
        token = heads * head
    if pages <= 1:
        page = max(size * token, heads * head)
    return (k_cache.data_ptr(), v_cache.data_ptr()), (page, token, head), size, pages


def _tree(tree, N, dev):
    """(pointer, width) of the rows' masks."""
    if tree is None:
        return None, 0
    width = _sizes("tree", tree, 2)[1]
    return _flat("tree", tree, (N, width), torch.int64, dev), width


def _count(n_rows, dev):
    return None if n_rows is None else _flat("n_rows", n_rows, (1,), torch.int32, dev)


# ------------------------------------------------------------------- rows
def dspark_step_rows(draft_len, sampling_mask, chunk_len, ctx_len, tree, tokens, draft_tokens,
                     page_count, free_pages, free_count, block_table, page_count_out,
                     free_count_out, cu_rows, cu_out, row_request, position, slot, row_token,
                     out_row, workspace, *, page_size, num_pages, stream=None,
                     raise_on_error=True) -> int:
    """Rows, pages and slots of a target step.  draft_len/ctx_len/page_count [N]
    int32, sampling_mask [N] uint8 or None, chunk_len [N] int32 or None, tree [N,
    width] int64 masks or None, tokens [N, width] int32 (rows may be apart) or None
    with row_token None, draft_tokens [N, K], free_pages [any], free_count [1];
    block_table [N, max_pages] (rows may be apart; in and out); out: page_count_out
    [N], free_count_out [1], cu_rows/cu_out [N + 1], row_request, position, slot,
    row_token and out_row [max_rows]."""
    i32 = torch.int32
    N, K = _sizes("draft_tokens", draft_tokens, 2)
    dev = _place("draft_tokens", draft_tokens)
    if sampling_mask is not None and sampling_mask.dtype is torch.bool:
        sampling_mask = sampling_mask.view(torch.uint8)
    ptree, width = _tree(tree, N, dev)
    if (tokens is None) != (row_token is None):
        raise ValueError("tokens and row_token are required together (or neither)")
    tokens_width = 0 if tokens is None else _sizes("tokens", tokens, 2)[1]
    ptokens, stokens = _rows("tokens", tokens, (N, tokens_width), i32, dev)
    max_rows, = _sizes("slot", slot, 1)
    max_pages = _sizes("block_table", block_table, 2)[1]
    ptable, stable = _rows("block_table", block_table, (N, max_pages), i32, dev)
    free_max, = _sizes("free_pages", free_pages, 1)
    code = (_lib or load()).dspark_step_rows(
        _flat("draft_len", draft_len, (N,), i32, dev),
        _maybe("sampling_mask", sampling_mask, (N,), torch.uint8, dev),
        _maybe("chunk_len", chunk_len, (N,), i32, dev), _flat("ctx_len", ctx_len, (N,), i32, dev),
        ptree, width, ptokens, stokens, tokens_width,
        _flat("draft_tokens", draft_tokens, (N, K), i32, dev), N, K,
        _flat("page_count", page_count, (N,), i32, dev),
        _flat("free_pages", free_pages, (free_max,), i32, dev), free_max,
        _flat("free_count", free_count, (1,), i32, dev), _int("page_size", page_size),
        _int("num_pages", num_pages), ptable, stable, max_pages,
        _flat("page_count_out", page_count_out, (N,), i32, dev),
        _flat("free_count_out", free_count_out, (1,), i32, dev),
        _flat("cu_rows", cu_rows, (N + 1,), i32, dev), _flat("cu_out", cu_out, (N + 1,), i32, dev),
        max_rows, _flat("row_request", row_request, (max_rows,), i32, dev),
        _flat("position", position, (max_rows,), i32, dev),
        _flat("slot", slot, (max_rows,), i32, dev),
        _maybe("row_token", row_token, (max_rows,), i32, dev),
        _flat("out_row", out_row, (max_rows,), i32, dev), *_space(workspace, dev), _stream(stream))
    return _done("dspark_step_rows", code, raise_on_error)


# ----------------------------------------------------------------- rotary
def dspark_rotary_table(rot, base, *, scaling=ROPE_PLAIN, factor=1.0, original=0.0, low=0.0,
                        high=0.0):
    """Turns a position of each pair, [rot / 2] int64 on the CPU (the bits of C's
    uint64), from base and a long context's scaling as in
    include/dspark_target.h."""
    turns = torch.empty(max(0, _int("rot", rot) // 2), dtype=torch.int64)
    code = (_lib or load()).dspark_rotary_table(rot, base, _int("scaling", scaling), factor,
                                                original, low, high, turns.data_ptr())
    _done("dspark_rotary_table", code, True)
    return turns


def _turns(turns, dev):
    half, = _sizes("turns", turns, 1)
    return _flat("turns", turns, (half,), torch.int64, dev), 2 * half


def dspark_rotary(q, k, position, turns, q_out, k_out, *, n_rows=None, interleaved=False,
                  inverse=False, amplitude=1.0, stream=None, raise_on_error=True) -> int:
    """Rotates q [R, Hq, d] into q_out and k [R, Hk, d] into k_out (bf16 or fp32;
    rows and heads may be apart; either pair may be None; in place where the output
    is the input).  position [R] int32, turns from dspark_rotary_table on the GPU,
    n_rows [1] int32 or None; inverse: the gradient."""
    one = q if q is not None else k
    name = "q" if q is not None else "k"
    R, _, d = _sizes(name, one, 3)
    dev = _place(name, one)
    dt, t = _dtype(name, one), one.dtype
    sides = []
    for a, b, na, nb in ((q, q_out, "q", "q_out"), (k, k_out, "k", "k_out")):
        if (a is None) != (b is None):
            raise ValueError(f"{na} and {nb} are required together (or neither)")
        if a is None:
            sides.append(((None, 0, 0), 0, (None, 0, 0)))
            continue
        shape = _sizes(na, a, 3)
        if shape[0] != R or shape[2] != d:
            raise ValueError(f"{na} must be {(R, shape[1], d)}, got {tuple(shape)}")
        sides.append((_heads(na, a, shape, t, dev), shape[1], _heads(nb, b, shape, t, dev)))
    (pq, Hq, pqo), (pk, Hk, pko) = sides
    pt, rot = _turns(turns, dev)
    code = (_lib or load()).dspark_rotary(
        *pq, Hq, *pk, Hk, dt, R, d, _flat("position", position, (R,), torch.int32, dev),
        _count(n_rows, dev), pt, rot, int(bool(interleaved)), int(bool(inverse)), amplitude, *pqo,
        *pko, _stream(stream))
    return _done("dspark_rotary", code, raise_on_error)


def dspark_rotary_append(q, k, v, position, slot, turns, q_out, k_cache, v_cache, *, n_rows=None,
                         interleaved=False, amplitude=1.0, stream=None,
                         raise_on_error=True) -> int:
    """Rotates q [R, Hq, d] into q_out, and k [R, Hk, d] into slot [R] of k_cache
    [pages, page_size, Hk, d]; copies v into v_cache alike.  The caches have the
    same strides, in any order."""
    R, Hq, d = _sizes("q", q, 3)
    Hk = _sizes("k", k, 3)[1]
    dev = _place("q", q)
    dt, t = _dtype("q", q), q.dtype
    shape, kv = q.shape, k.shape
    if kv[0] != R or kv[2] != d:
        raise ValueError(f"k must be {(R, Hk, d)}, got {tuple(kv)}")
    caches, strides, page_size, pages = _caches(k_cache, v_cache, Hk, d, t, dev)
    pt, rot = _turns(turns, dev)
    code = (_lib or load()).dspark_rotary_append(
        *_heads("q", q, shape, t, dev), Hq, *_heads("k", k, kv, t, dev),
        *_heads("v", v, kv, t, dev), Hk, dt, R, d,
        _flat("position", position, (R,), torch.int32, dev),
        _flat("slot", slot, (R,), torch.int32, dev), _count(n_rows, dev), pt, rot,
        int(bool(interleaved)), amplitude, *_heads("q_out", q_out, shape, t, dev), *caches,
        *strides, page_size, pages, _stream(stream))
    return _done("dspark_rotary_append", code, raise_on_error)


# -------------------------------------------------------------- attention
def dspark_attention_workspace_size(N: int, max_len: int, Hq: int, Hk: int, d: int) -> int:
    if max(N, max_len, Hq, Hk, d) > _I32_MAX:
        return 0                                   # as for all that is not supported
    return int(load().dspark_attention_workspace_size(N, max_len, Hq, Hk, d))


def dspark_tree_attention(q, k_cache, v_cache, block_table, ctx_len, cu_rows, tree, out, lse,
                          workspace, *, max_len, scale, stream=None, raise_on_error=True) -> int:
    """Attention of q [R, Hq, d] over the caches [pages, page_size, Hk, d] (bf16),
    each request's rows over its pages: block_table [N, max_pages] int32 (rows may
    be apart), ctx_len [N], cu_rows [N + 1], tree [N, width] int64 masks or None
    (chains); out like q, lse [R, Hq] fp32 or None; no request has more than max_len
    rows."""
    bf16, i32 = torch.bfloat16, torch.int32
    shape = R, Hq, d = _sizes("q", q, 3)
    dev = _place("q", q)
    Hk = _sizes("k_cache", k_cache, 4)[2]
    caches, strides, page_size, pages = _caches(k_cache, v_cache, Hk, d, bf16, dev)
    N, max_pages = _sizes("block_table", block_table, 2)
    ptable, stable = _rows("block_table", block_table, (N, max_pages), i32, dev)
    ptree, width = _tree(tree, N, dev)
    code = (_lib or load()).dspark_tree_attention(
        *_heads("q", q, shape, bf16, dev), *caches, *strides, page_size, pages, ptable, stable,
        max_pages, _flat("ctx_len", ctx_len, (N,), i32, dev),
        _flat("cu_rows", cu_rows, (N + 1,), i32, dev), ptree, width, N, R,
        _int("max_len", max_len), Hq, Hk, d, scale, *_heads("out", out, shape, bf16, dev),
        _maybe("lse", lse, (R, Hq), torch.float32, dev), *_space(workspace, dev), _stream(stream))
    return _done("dspark_tree_attention", code, raise_on_error)


# ----------------------------------------------------------------- logits
def dspark_adjust_logits(logits, cu_rows, tokens, hist_len, prompt_len, draft_tokens, tree, out,
                         workspace, *, repetition=None, frequency=None, presence=None,
                         bias_token=None, bias_value=None, bias_count=None, mask=None,
                         mask_index=None, stream=None, raise_on_error=True) -> int:
    """Penalties, biases and masks on logits [R, vocab] (bf16 or fp32; rows may be
    apart) into out (logits itself: in place).  cu_rows [N + 1], tokens [N, width]
    int32 (rows may be apart: of a long buffer, pass the columns that hist_len may
    reach), hist_len [N], prompt_len [N] or None, draft_tokens
    [N, K] or None, tree [N, width] int64 masks or None; repetition, frequency and
    presence [N] fp32 or None; bias_token [N, most] int32, bias_value fp32 and
    bias_count [N], or None; mask [rows, words] int32 (rows may be apart), 1 =
    allowed, and mask_index [R] int32 (negative: not masked), or None."""
    i32, f32 = torch.int32, torch.float32
    shape = R, vocab = _sizes("logits", logits, 2)
    dev = _place("logits", logits)
    dt, t = _dtype("logits", logits), logits.dtype
    N, width = _sizes("tokens", tokens, 2)
    pl, sl = _rows("logits", logits, shape, t, dev)
    if out is None:
        raise ValueError("out is required")
    po, so = _rows("out", out, shape, t, dev)
    ptokens, stokens = _rows("tokens", tokens, (N, width), i32, dev)
    K, pdraft = 0, None
    if draft_tokens is not None:
        K = _sizes("draft_tokens", draft_tokens, 2)[1]
        pdraft = _flat("draft_tokens", draft_tokens, (N, K), i32, dev)
    ptree, tree_width = _tree(tree, N, dev)
    if not (bias_token is None) == (bias_value is None) == (bias_count is None):
        raise ValueError("bias_token, bias_value and bias_count are required together (or none)")
    most = 0 if bias_token is None else _sizes("bias_token", bias_token, 2)[1]
    mask_rows, pmask, smask = 0, None, 0
    if mask is not None:
        mask_rows, words = _sizes("mask", mask, 2)
        pmask, smask = _rows("mask", mask, (mask_rows, words), i32, dev)
        if words < (vocab + 31) // 32:
            raise ValueError(f"mask must have {(vocab + 31) // 32} words a row, got {words}")
        if mask_index is None and mask_rows < R:
            raise ValueError(f"mask must have a row for each of the {R} rows, got {mask_rows}")
    elif mask_index is not None:
        raise ValueError("mask_index needs a mask")
    code = (_lib or load()).dspark_adjust_logits(
        pl, sl, dt, R, vocab, _flat("cu_rows", cu_rows, (N + 1,), i32, dev), N, ptokens, stokens,
        width, _flat("hist_len", hist_len, (N,), i32, dev),
        _maybe("prompt_len", prompt_len, (N,), i32, dev), pdraft, K, ptree, tree_width,
        _maybe("repetition", repetition, (N,), f32, dev),
        _maybe("frequency", frequency, (N,), f32, dev),
        _maybe("presence", presence, (N,), f32, dev),
        _maybe("bias_token", bias_token, (N, most), i32, dev),
        _maybe("bias_value", bias_value, (N, most), f32, dev),
        _maybe("bias_count", bias_count, (N,), i32, dev), most, pmask, smask, mask_rows,
        _maybe("mask_index", mask_index, (R,), i32, dev), po, so, *_space(workspace, dev),
        _stream(stream))
    return _done("dspark_adjust_logits", code, raise_on_error)
