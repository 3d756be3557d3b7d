"""What a serving step needs around the calls of decode.py (include/libred_serve.h):
where the next tokens go in the paged cache, attention over the pages that a
cheap score selects, and sampling from filtered probabilities.

The conventions are those of decode.py: each function has the name of the C
entry point it calls, tensors are taken with the strides they have as long as
their last dimension is contiguous, and with a stream given, outputs are
allocated there. Nothing here is differentiable.
"""
import ctypes

import torch

from .decode import (_CACHES, _FLOAT32, _FLOATS, _HALVES, _INT32, _INT64, TYPES, PagedCache, _any, _call, _attend, _on, _pack_cache,
                     _packer, _rows, _whole)

_P = ctypes.c_void_p
_Z = ctypes.c_size_t
_I = ctypes.c_int
_L = ctypes.c_int64


# The structs of libred_serve.h.
class PlanSlotsArgs(ctypes.Structure):
    _fields_ = [("batch", _Z), ("tokens", _Z), ("places", _Z), ("pages", _Z), ("lens", _P), ("counts", _P), ("done", _P),
                ("table", _P), ("table_cols", _Z), ("table_stride", _L), ("held", _P), ("free_pages", _P), ("free_count", _P),
                ("slots", _P), ("pos", _P), ("starts", _P), ("granted", _P)]


class PageBoundsArgs(ctypes.Structure):
    _fields_ = [("type", _I), ("batch", _Z), ("most", _Z), ("cache", PagedCache), ("table", _P), ("table_cols", _Z),
                ("table_stride", _L), ("lens", _P), ("first", _P), ("lo", _P), ("hi", _P),
                ("bound_page_stride", _L), ("bound_head_stride", _L)]


class SelectPagesArgs(ctypes.Structure):
    _fields_ = [("type", _I), ("batch", _Z), ("nodes", _Z), ("q_heads", _Z), ("kv_heads", _Z), ("dim", _Z), ("pages", _Z),
                ("places", _Z), ("budget", _Z), ("first", _Z), ("last", _Z), ("max_len", _Z), ("q", _P),
                ("q_batch_stride", _L), ("q_node_stride", _L), ("q_head_stride", _L), ("lo", _P), ("hi", _P),
                ("bound_page_stride", _L), ("bound_head_stride", _L), ("table", _P), ("table_cols", _Z), ("table_stride", _L),
                ("lens", _P), ("node_count", _P), ("selected", _P), ("selected_lens", _P)]


class SampleArgs(ctypes.Structure):
    _fields_ = [("type", _I), ("probs_type", _I), ("batch", _Z), ("steps", _Z), ("vocab", _Z), ("logits", _P),
                ("batch_stride", _L), ("step_stride", _L), ("temperature", _P), ("top_k", _P), ("top_p", _P), ("min_p", _P),
                ("r", _P), ("tokens", _P), ("probs", _P), ("probs_batch_stride", _L), ("probs_step_stride", _L)]


_pack_plan, _pack_bounds = _packer(PlanSlotsArgs), _packer(PageBoundsArgs)
_pack_select, _pack_sample = _packer(SelectPagesArgs), _packer(SampleArgs)

SIGNATURES = {
    "red_plan_slots": (_I, [_P, _P]),
    "red_page_bounds": (_I, [_P, _P]),
    "red_select_pages": (_I, [_P, _P]),
    "red_sparse_attention": (_I, [_P, _L, _P]),
    "red_sample": (_I, [_P, _P]),
}


def _table(name, table, device, batch):
    """-> (address, columns, stride) of a table (batch, pages of a sequence)."""
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError(f"{name}: table must be ({batch}, pages of a sequence)")
    _rows(name, "table", table, _INT32, device, (batch, table.shape[1]))
    return table.data_ptr(), table.shape[1], table.stride(0)


def _count(name, what, n):
    if n < 0:
        raise ValueError(f"{name}: {what} must not be negative")
    return n


def red_plan_slots(lens, counts, table, held, free_pages, free_count, places, tokens, done=None, stream=None):
    """Pages and slots for counts[b] more tokens of every sequence, which holds
    lens[b] of them (batch; int32, as are all inputs). table (batch, pages of a
    sequence), held (batch: how many of them it has), free_pages (a stack, -1
    behind its height) and free_count (1: the height) are updated: rows with
    done[b] != 0 give their pages back first, then sequences get the pages they
    lack, in order, from the top of the stack; from the first that there are not
    enough for on, those that lack any get none. -> (slots (tokens) int64, -1
    where a sequence got no place or none has the token, pos (tokens) int64,
    starts (batch + 1) int32: the number of a sequence's first token, granted
    (batch) int32: counts, or 0 where there was no place)."""
    if stream is not None:
        return _on(stream, red_plan_slots, lens, counts, table, held, free_pages, free_count, places, tokens, done)
    name = "red_plan_slots"
    device = _any(name, "lens", lens, (_INT32,), 1, "(batch)")
    batch, at = lens.shape[0], lens.device
    tp, cols, t0 = _table(name, table, device, batch)
    if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1:
        raise ValueError(f"{name}: free_pages must have one dimension")
    pages = free_pages.shape[0]
    _count(name, "tokens", tokens)
    if places < 1:
        raise ValueError(f"{name}: places must be positive")
    slots, pos = (torch.empty(tokens, dtype=_INT64, device=at) for _ in range(2))
    starts, granted = torch.empty(batch + 1, dtype=_INT32, device=at), torch.empty(batch, dtype=_INT32, device=at)
    one = (batch,)
    _call(name, device, None, _pack_plan(
        batch, tokens, places, pages, _whole(name, "lens", lens, _INT32, device, one),
        _whole(name, "counts", counts, _INT32, device, one), 0 if done is None else _whole(name, "done", done, _INT32, device, one),
        tp, cols, t0, _whole(name, "held", held, _INT32, device, one), _whole(name, "free_pages", free_pages, _INT32, device, (pages,)),
        _whole(name, "free_count", free_count, _INT32, device, (1,)), slots.data_ptr(), pos.data_ptr(), starts.data_ptr(),
        granted.data_ptr()))
    return slots, pos, starts, granted


def _bounds(name, lo, hi, dtype, device, shape):
    """-> (address of lo, of hi, stride of pages, of heads)"""
    _rows(name, "lo", lo, dtype, device, shape)
    _rows(name, "hi", hi, dtype, device, shape)
    if lo.stride() != hi.stride():
        raise ValueError(f"{name}: lo and hi must have the same strides")
    return lo.data_ptr(), hi.data_ptr(), *lo.stride()[:2]


def red_page_bounds(k_pages, table, lens, lo, hi, first=None, most=None, k_scales=None, stream=None):
    """Write the least and the largest elements of the keys of whole pages of a
    paged cache (see red_cache_write) to lo and hi (pages, heads, dim; float16
    or bfloat16, the cache's type where that has 16 bits): of the pages of
    sequence b that hold tokens first[b] (int32; None: 0) to lens[b] - 1, at
    most `most` pages of a sequence (None: what the table holds)."""
    name = "red_page_bounds"
    device = _any(name, "k_pages", k_pages, _CACHES, 4, "(pages, heads, places, dim)")
    pages, heads, places, dim = k_pages.shape
    kind = TYPES[k_pages.dtype]
    dtype = lo.dtype if isinstance(lo, torch.Tensor) else None
    if dtype not in _HALVES or (kind < 3 and dtype is not k_pages.dtype):
        _any(name, "lo", lo, _HALVES if kind >= 3 else (k_pages.dtype,), 3, "(pages, heads, dim)")
    if (kind >= 3) != (k_scales is not None):
        raise ValueError(f"{name}: 8-bit caches take k_scales, 16-bit ones do not")
    ks, strides = 0, (0, 0, 0)
    if k_scales is not None:
        if not isinstance(k_scales, torch.Tensor) or k_scales.dtype is not _FLOAT32 or k_scales.get_device() != device or \
                k_scales.shape != k_pages.shape[:3]:
            raise ValueError(f"{name}: k_scales must be float32 {tuple(k_pages.shape[:3])} on cuda:{device}")
        ks, strides = k_scales.data_ptr(), k_scales.stride()
    batch = lens.shape[0] if isinstance(lens, torch.Tensor) and lens.dim() == 1 else -1
    lens_at = _whole(name, "lens", lens, _INT32, device, (batch,))
    tp, cols, t0 = _table(name, table, device, batch)
    at = _bounds(name, lo, hi, dtype, device, (pages, heads, dim))
    _call(name, device, stream, _pack_bounds(
        TYPES[dtype], batch, cols if most is None else _count(name, "most", most),
        k_pages.data_ptr(), 0, ks, 0, kind, pages, heads, places, dim, *k_pages.stride()[:3], *strides, tp, cols, t0, lens_at,
        0 if first is None else _whole(name, "first", first, _INT32, device, (batch,)), *at))


def red_select_pages(q, lo, hi, table, lens, places, budget, first=1, last=1, max_len=None, node_count=None, stream=None):
    """The pages worth reading for the queries q (batch, nodes, q heads, dim;
    float16 or bfloat16) of sequences of lens[b] tokens and their nodes, in
    pages of `places` tokens, for each kv head, by the bounds lo and hi of the
    pages' keys (pages, kv heads, dim; see red_page_bounds): the first `first`
    pages, the last ones from lens[b] // places - last on, and of the others
    those with the largest bounds of q . k, summed over the nodes and the query
    heads of a kv head, `budget` pages in all. node_count, max_len: as
    red_tree_attention takes them. -> (selected (batch, kv heads, budget) int32:
    page numbers in the order of the sequence, then -1, and lens (batch) int32:
    tokens of the selected pages before the nodes), which red_sparse_attention
    takes."""
    if stream is not None:
        return _on(stream, red_select_pages, q, lo, hi, table, lens, places, budget, first, last, max_len, node_count)
    name = "red_select_pages"
    device = _any(name, "q", q, _HALVES, 4, "(batch, nodes, q heads, dim)")
    batch, nodes, q_heads, dim = q.shape
    if not isinstance(lo, torch.Tensor) or lo.dim() != 3:
        raise ValueError(f"{name}: lo must be (pages, kv heads, {dim})")
    pages, heads, _ = lo.shape
    at = _bounds(name, lo, hi, q.dtype, device, (pages, heads, dim))
    tp, cols, t0 = _table(name, table, device, batch)
    for what, n in (("budget", budget), ("first", first), ("last", last), ("max_len", max_len or 0)):
        _count(name, what, n)
    if places < 1:
        raise ValueError(f"{name}: places must be positive")
    selected = torch.empty((batch, heads, budget), dtype=_INT32, device=q.device)
    selected_lens = torch.empty(batch, dtype=_INT32, device=q.device)
    _call(name, device, None, _pack_select(
        TYPES[q.dtype], batch, nodes, q_heads, heads, dim, pages, places, budget, first, last,
        cols * places if max_len is None else max_len, q.data_ptr(), *q.stride()[:3], *at, tp, cols, t0,
        _whole(name, "lens", lens, _INT32, device, (batch,)),
        0 if node_count is None else _whole(name, "node_count", node_count, _INT32, device, (batch,)),
        selected.data_ptr(), selected_lens.data_ptr()))
    return selected, selected_lens


def red_sparse_attention(q, k_pages, v_pages, table, lens, scale, max_len=None, tree_mask=None, node_count=None, k_scales=None,
                         v_scales=None, out=None, stream=None):
    """red_tree_attention with a table for each kv head: table (batch, kv heads,
    pages of a sequence; int32). With what red_select_pages returns it attends
    over the selected pages."""
    if stream is not None:
        return _on(stream, red_sparse_attention, q, k_pages, v_pages, table, lens, scale, max_len, tree_mask, node_count,
                   k_scales, v_scales, out)
    return _attend("red_sparse_attention", q, k_pages, v_pages, table, lens, scale, max_len, tree_mask, node_count, k_scales,
                   v_scales, out)


def red_sample(logits, r=None, temperature=None, top_k=None, top_p=None, min_p=None, probs=None, stream=None):
    """A token from every row of logits (batch, vocab) or (batch, steps, vocab;
    float32, float16 or bfloat16) by the random numbers r (batch) or (batch,
    steps; float32), from the probabilities of logits / temperature that top_k,
    top_p and min_p leave (each of them batch numbers, top_k int32, the others
    float32; None: not used). temperature 0 takes the first of the largest
    logits. probs: a float type, for the probabilities themselves as well (those
    that red_verify_drafts takes). -> (tokens int64 or None without r, probs or
    None)."""
    if stream is not None:
        return _on(stream, red_sample, logits, r, temperature, top_k, top_p, min_p, probs)
    name = "red_sample"
    dims = 2 if isinstance(logits, torch.Tensor) and logits.dim() == 2 else 3
    device = _any(name, "logits", logits, _FLOATS, dims, "(batch, vocab) or (batch, steps, vocab)")
    shape, strides = logits.shape, logits.stride()
    batch, vocab = shape[0], shape[-1]
    steps, step_stride = (1, 0) if dims == 2 else (shape[1], strides[1])
    if vocab < 1:
        raise ValueError(f"{name}: logits must have a vocabulary")
    one = (batch,)
    tp, kp, pp, mp = (0 if x is None else _whole(name, what, x, dtype, device, one) for what, x, dtype in (
        ("temperature", temperature, _FLOAT32), ("top_k", top_k, _INT32), ("top_p", top_p, _FLOAT32), ("min_p", min_p, _FLOAT32)))
    if probs is not None and probs not in _FLOATS:
        raise TypeError(f"{name}: probs must be torch.float32, torch.float16 or torch.bfloat16")
    tokens = given = None
    rp = 0
    if r is not None:
        rp = _whole(name, "r", r, _FLOAT32, device, shape[:-1])
        tokens = torch.empty(shape[:-1], dtype=_INT64, device=logits.device)
    p0 = p1 = 0
    if probs is not None:
        given = torch.empty(shape, dtype=probs, device=logits.device)
        p0, p1 = given.stride(0), 0 if dims == 2 else given.stride(1)
    _call(name, device, None, _pack_sample(
        TYPES[logits.dtype], 0 if probs is None else TYPES[probs], batch, steps, vocab, logits.data_ptr(), strides[0], step_stride,
        tp, kp, pp, mp, rp, 0 if tokens is None else tokens.data_ptr(), 0 if given is None else given.data_ptr(), p0, p1))
    return tokens, given
