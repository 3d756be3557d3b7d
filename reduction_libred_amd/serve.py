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


# The arguments are checked in one expression; where that does not hold, they are
# gone through one by one for what is wrong.
def _table(name, table, device, batch):
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError(f"{name}: table must be ({batch}, pages of a sequence)")
    _rows(name, "table", table, _INT32, device, (batch, table.shape[1]))


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
    _count("red_plan_slots", "tokens", tokens)
    try:
        one, (batch, cols), pages, device = lens.shape, table.shape, free_pages.shape, lens.get_device()
        fits = (lens.dtype is _INT32 and counts.dtype is _INT32 and table.dtype is _INT32 and held.dtype is _INT32 and
                free_pages.dtype is _INT32 and free_count.dtype is _INT32 and device >= 0 and counts.get_device() == device and
                table.get_device() == device and held.get_device() == device and free_pages.get_device() == device and
                free_count.get_device() == device and one == (batch,) and counts.shape == one and held.shape == one and
                len(pages) == 1 and free_count.shape == (1,) and lens.is_contiguous() and counts.is_contiguous() and
                held.is_contiguous() and free_pages.is_contiguous() and (table.stride(1) == 1 or cols <= 1) and places >= 1 and
                (done is None or (done.dtype is _INT32 and done.get_device() == device and done.shape == one and done.is_contiguous())))
    except (AttributeError, TypeError, ValueError):
        fits = False
    if not fits:
        _plan_check(lens, counts, table, held, free_pages, free_count, places, done)
    at = lens.device
    slots, pos = torch.empty(tokens, dtype=_INT64, device=at), torch.empty(tokens, dtype=_INT64, device=at)
    starts, granted = torch.empty(batch + 1, dtype=_INT32, device=at), torch.empty(batch, dtype=_INT32, device=at)
    _call("red_plan_slots", device, None, _pack_plan(
        batch, tokens, places, pages[0], lens.data_ptr(), counts.data_ptr(), 0 if done is None else done.data_ptr(), table.data_ptr(), cols,
        table.stride(0), held.data_ptr(), free_pages.data_ptr(), free_count.data_ptr(), slots.data_ptr(), pos.data_ptr(),
        starts.data_ptr(), granted.data_ptr()))
    return slots, pos, starts, granted


def _plan_check(lens, counts, table, held, free_pages, free_count, places, done):
    """Raise what is wrong with the arguments."""
    name = "red_plan_slots"
    device = _any(name, "lens", lens, (_INT32,), 1, "(batch)")
    batch = lens.shape[0]
    _table(name, table, device, batch)
    if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1:
        raise ValueError(f"{name}: free_pages must have one dimension")
    for what, x, shape in (("counts", counts, (batch,)), ("done", done, (batch,)), ("held", held, (batch,)),
                           ("free_pages", free_pages, free_pages.shape), ("free_count", free_count, (1,))):
        if what != "done" or x is not None:
            _whole(name, what, x, _INT32, device, shape)
    if places < 1:
        raise ValueError(f"{name}: places must be positive")
    raise ValueError(f"{name}: lens must be contiguous")


def _bounds(name, lo, hi, dtype, device, shape):
    _rows(name, "lo", lo, dtype, device, shape)
    _rows(name, "hi", hi, dtype, device, shape)
    if lo.stride() != hi.stride():
        raise ValueError(f"{name}: lo and hi must have the same strides")


def red_page_bounds(k_pages, table, lens, lo, hi, first=None, most=None, k_scales=None, stream=None):
    """Write the least and the largest elements of the keys of whole pages of a
    paged cache (see red_cache_write) to lo and hi (pages, heads, dim; float16
    or bfloat16, the cache's type where that has 16 bits): of the pages of
    sequence b that hold tokens first[b] (int32; None: 0) to lens[b] - 1, at
    most `most` pages of a sequence (None: what the table holds)."""
    try:
        (pages, heads, places, dim), (p0, p1, p2, inner), kind, dtype = k_pages.shape, k_pages.stride(), TYPES[k_pages.dtype], lo.dtype
        (batch, cols), shape, device, (b0, b1, b2) = table.shape, lo.shape, k_pages.get_device(), lo.stride()
        fits = (0 < kind and dtype in _HALVES and (kind >= 3 or dtype is k_pages.dtype) and hi.dtype is dtype and
                lens.dtype is _INT32 and table.dtype is _INT32 and device >= 0 and lo.get_device() == device and
                hi.get_device() == device and lens.get_device() == device and table.get_device() == device and
                shape == (pages, heads, dim) and hi.shape == shape and hi.stride() == (b0, b1, b2) and
                ((inner == 1 and b2 == 1) or dim <= 1) and lens.shape == (batch,) and lens.is_contiguous() and
                (table.stride(1) == 1 or cols <= 1) and (kind >= 3) == (k_scales is not None) and
                (first is None or (first.dtype is _INT32 and first.get_device() == device and first.shape == lens.shape and
                                   first.is_contiguous())) and
                (k_scales is None or (k_scales.dtype is _FLOAT32 and k_scales.get_device() == device and
                                      k_scales.shape == k_pages.shape[:3])))
    except (AttributeError, TypeError, ValueError, KeyError):
        fits = False
    if not fits:
        _bounds_check(k_pages, table, lens, lo, hi, first, k_scales)
    ks, (s0, s1, s2) = (0, (0, 0, 0)) if k_scales is None else (k_scales.data_ptr(), k_scales.stride())
    _call("red_page_bounds", device, stream, _pack_bounds(
        TYPES[dtype], batch, cols if most is None else _count("red_page_bounds", "most", most), k_pages.data_ptr(), 0, ks, 0, kind,
        pages, heads, places, dim, p0, p1, p2, s0, s1, s2, table.data_ptr(), cols, table.stride(0), lens.data_ptr(),
        0 if first is None else first.data_ptr(), lo.data_ptr(), hi.data_ptr(), b0, b1))


def _bounds_check(k_pages, table, lens, lo, hi, first, k_scales):
    """Raise what is wrong with the arguments."""
    name = "red_page_bounds"
    device = _any(name, "k_pages", k_pages, _CACHES, 4, "(pages, heads, places, dim)")
    pages, heads, _, dim = k_pages.shape
    scaled = TYPES[k_pages.dtype] >= 3
    _any(name, "lo", lo, _HALVES if scaled else (k_pages.dtype,), 3, "(pages, heads, dim)")
    if scaled != (k_scales is not None):
        raise ValueError(f"{name}: 8-bit caches take k_scales, 16-bit ones do not")
    if k_scales is not None and not (isinstance(k_scales, torch.Tensor) and k_scales.dtype is _FLOAT32 and
                                     k_scales.get_device() == device and k_scales.shape == k_pages.shape[:3]):
        raise ValueError(f"{name}: k_scales must be float32 {tuple(k_pages.shape[:3])} on cuda:{device}")
    _any(name, "lens", lens, (_INT32,), 1, "(batch)")
    batch = lens.shape[0]
    _whole(name, "lens", lens, _INT32, device, (batch,))
    _table(name, table, device, batch)
    _bounds(name, lo, hi, lo.dtype, device, (pages, heads, dim))
    if first is not None:
        _whole(name, "first", first, _INT32, device, (batch,))
    raise ValueError(f"{name}: the last dimension of k_pages must be contiguous")


def red_select_pages(q, lo, hi, table, lens, places, budget, first=1, last=1, max_len=None, node_count=None, stream=None):
    """The pages worth reading for the queries q (batch, nodes, q heads, dim;
    float16 or bfloat16) of sequences of lens[b] tokens and their nodes, in
    pages of `places` tokens, for each kv head, by the bounds lo and hi of the
    pages' keys (pages, kv heads, dim; see red_page_bounds): the first `first`
    pages, the last ones from lens[b] // places - last on, and of the others
    those with the largest bounds of q . k, summed over the nodes and the query
    heads of a kv head, `budget` pages in all. node_count, max_len: as
    red_tree_attention takes them; for a scale below 0, -q is given here.
    -> (selected (batch, kv heads, budget) int32: page numbers in the order of
    the sequence, then -1, and lens (batch) int32: tokens of the selected pages
    before the nodes), which red_sparse_attention takes."""
    if stream is not None:
        return _on(stream, red_select_pages, q, lo, hi, table, lens, places, budget, first, last, max_len, node_count)
    try:
        (batch, nodes, q_heads, dim), (q0, q1, q2, inner), dtype, device = q.shape, q.stride(), q.dtype, q.get_device()
        (pages, heads, wide), (b0, b1, b2), (rows, cols), one = lo.shape, lo.stride(), table.shape, lens.shape
        fits = (dtype in _HALVES and lo.dtype is dtype and hi.dtype is dtype and table.dtype is _INT32 and lens.dtype is _INT32 and
                device >= 0 and lo.get_device() == device and hi.get_device() == device and table.get_device() == device and
                lens.get_device() == device and wide == dim and hi.shape == lo.shape and hi.stride() == (b0, b1, b2) and
                ((inner == 1 and b2 == 1) or dim <= 1) and rows == batch and (table.stride(1) == 1 or cols <= 1) and
                one == (batch,) and lens.is_contiguous() and budget >= 0 and first >= 0 and last >= 0 and places >= 1 and
                (max_len is None or max_len >= 0) and
                (node_count is None or (node_count.dtype is _INT32 and node_count.get_device() == device and
                                        node_count.shape == one and node_count.is_contiguous())))
    except (AttributeError, TypeError, ValueError):
        fits = False
    if not fits:
        _select_check(q, lo, hi, table, lens, places, budget, first, last, max_len, node_count)
    selected = torch.empty((batch, heads, budget), dtype=_INT32, device=q.device)
    selected_lens = torch.empty(batch, dtype=_INT32, device=q.device)
    _call("red_select_pages", device, None, _pack_select(
        TYPES[dtype], batch, nodes, q_heads, heads, dim, pages, places, budget, first, last,
        cols * places if max_len is None else max_len, q.data_ptr(), q0, q1, q2, lo.data_ptr(), hi.data_ptr(), b0, b1, table.data_ptr(),
        cols, table.stride(0), lens.data_ptr(), 0 if node_count is None else node_count.data_ptr(), selected.data_ptr(),
        selected_lens.data_ptr()))
    return selected, selected_lens


def _select_check(q, lo, hi, table, lens, places, budget, first, last, max_len, node_count):
    """Raise what is wrong with the arguments."""
    name = "red_select_pages"
    device = _any(name, "q", q, _HALVES, 4, "(batch, nodes, q heads, dim)")
    batch, _, _, dim = q.shape
    if not isinstance(lo, torch.Tensor) or lo.dim() != 3:
        raise ValueError(f"{name}: lo must be (pages, kv heads, {dim})")
    _bounds(name, lo, hi, q.dtype, device, (*lo.shape[:2], dim))
    _table(name, table, device, batch)
    for what, n in (("budget", budget), ("first", first), ("last", last), ("max_len", max_len or 0)):
        _count(name, what, n)
    if places < 1:
        raise ValueError(f"{name}: places must be positive")
    _whole(name, "lens", lens, _INT32, device, (batch,))
    if node_count is not None:
        _whole(name, "node_count", node_count, _INT32, device, (batch,))
    raise ValueError(f"{name}: arguments do not fit each other")


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
    try:
        shape, strides, dtype, device = logits.shape, logits.stride(), logits.dtype, logits.get_device()
        if len(shape) == 2:
            (batch, vocab), steps, step_stride, rows = shape, 1, 0, shape[:1]
        else:
            (batch, steps, vocab), (_, step_stride, _), rows = shape, strides, shape[:2]
        one = (batch,)
        fits = (dtype in _FLOATS and device >= 0 and vocab >= 1 and (strides[-1] == 1 or vocab == 1) and
                (probs is None or probs in _FLOATS) and
                (r is None or (r.dtype is _FLOAT32 and r.get_device() == device and r.shape == rows and r.is_contiguous())) and
                (temperature is None or _setting(temperature, _FLOAT32, device, one)) and
                (top_k is None or _setting(top_k, _INT32, device, one)) and
                (top_p is None or _setting(top_p, _FLOAT32, device, one)) and
                (min_p is None or _setting(min_p, _FLOAT32, device, one)))
    except (AttributeError, TypeError, ValueError):
        fits = False
    if not fits:
        _sample_check(logits, r, temperature, top_k, top_p, min_p, probs)
    tokens = None if r is None else torch.empty(rows, dtype=_INT64, device=logits.device)
    given, p0, p1 = None, 0, 0
    if probs is not None:
        given = torch.empty(shape, dtype=probs, device=logits.device)
        p0, p1 = steps * vocab, vocab
    _call("red_sample", device, None, _pack_sample(
        TYPES[dtype], 0 if probs is None else TYPES[probs], batch, steps, vocab, logits.data_ptr(), strides[0], step_stride,
        0 if temperature is None else temperature.data_ptr(), 0 if top_k is None else top_k.data_ptr(),
        0 if top_p is None else top_p.data_ptr(), 0 if min_p is None else min_p.data_ptr(), 0 if r is None else r.data_ptr(),
        0 if tokens is None else tokens.data_ptr(), 0 if given is None else given.data_ptr(), p0, p1))
    return tokens, given


def _setting(x, dtype, device, shape):
    return x.dtype is dtype and x.get_device() == device and x.shape == shape and x.is_contiguous()


def _sample_check(logits, r, temperature, top_k, top_p, min_p, probs):
    """Raise what is wrong with the arguments."""
    name = "red_sample"
    dims = 2 if isinstance(logits, torch.Tensor) and logits.dim() == 2 else 3
    device = _any(name, "logits", logits, _FLOATS, dims, "(batch, vocab) or (batch, steps, vocab)")
    if logits.shape[-1] < 1:
        raise ValueError(f"{name}: logits must have a vocabulary")
    for what, x, dtype in (("temperature", temperature, _FLOAT32), ("top_k", top_k, _INT32), ("top_p", top_p, _FLOAT32), ("min_p", min_p, _FLOAT32)):
        if x is not None:
            _whole(name, what, x, dtype, device, logits.shape[:1])
    if probs is not None and probs not in _FLOATS:
        raise TypeError(f"{name}: probs must be torch.float32, torch.float16 or torch.bfloat16")
    _whole(name, "r", r, _FLOAT32, device, logits.shape[:-1])
    raise ValueError(f"{name}: arguments do not fit each other")
