"""The reductions of a decoding step of drafted tokens (include/libred_decode.h).

Like the rest of the binding, each function has the name of the C entry point
it calls and only marshals arguments. Tensors are taken with the strides they
have, as long as their last dimension is contiguous.
"""
import ctypes

import torch

from . import _check, _stream_handle, lib

_P = ctypes.c_void_p
_Z = ctypes.c_size_t
_I = ctypes.c_int
_L = ctypes.c_int64
_F = ctypes.c_float

TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.int8: 3, torch.float8_e4m3fn: 4}


class Heads(ctypes.Structure):
    _fields_ = [("data", _P), ("heads", _L), ("token_stride", _L), ("head_stride", _L)]


class QkNormRopeArgs(ctypes.Structure):
    _fields_ = [("type", _I), ("interleaved", _I), ("tokens", _Z), ("dim", _Z), ("rot", _Z), ("eps", _F),
                ("q", Heads), ("k", Heads), ("q_out", Heads), ("k_out", Heads),
                ("q_weight", _P), ("k_weight", _P), ("pos", _P), ("freq", _P)]


class PagedCache(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_scales", _P), ("v_scales", _P), ("type", _I),
                ("pages", _Z), ("heads", _Z), ("places", _Z), ("dim", _Z),
                ("page_stride", _L), ("head_stride", _L), ("place_stride", _L),
                ("scale_page_stride", _L), ("scale_head_stride", _L), ("scale_place_stride", _L)]


class TreeAttentionArgs(ctypes.Structure):
    _fields_ = [("type", _I), ("scale", _F), ("batch", _Z), ("nodes", _Z), ("q_heads", _Z), ("max_len", _Z),
                ("q", _P), ("out", _P), ("lse", _P),
                ("q_batch_stride", _L), ("q_node_stride", _L), ("q_head_stride", _L),
                ("out_batch_stride", _L), ("out_node_stride", _L), ("out_head_stride", _L),
                ("cache", PagedCache), ("table", _P), ("table_cols", _Z), ("table_stride", _L),
                ("lens", _P), ("tree_mask", _P), ("node_count", _P)]


class VerifyDraftsArgs(ctypes.Structure):
    _fields_ = [("type", _I), ("batch", _Z), ("drafts", _Z), ("vocab", _Z),
                ("p", _P), ("p_batch_stride", _L), ("p_step_stride", _L),
                ("q", _P), ("q_batch_stride", _L), ("q_step_stride", _L),
                ("drafted", _P), ("u", _P), ("r", _P), ("draft_count", _P), ("accepted", _P), ("tokens", _P)]


SIGNATURES = {
    "red_verify_drafts": (_I, [ctypes.POINTER(VerifyDraftsArgs), _P]),
    "red_tree_attention": (_I, [ctypes.POINTER(TreeAttentionArgs), _P]),
    "red_qk_norm_rope": (_I, [ctypes.POINTER(QkNormRopeArgs), _P]),
    "red_qk_norm_rope_backward": (_I, [ctypes.POINTER(QkNormRopeArgs), ctypes.POINTER(Heads), ctypes.POINTER(Heads),
                                       _P, _P, _P]),
    "red_cache_write": (_I, [ctypes.POINTER(PagedCache), _I, ctypes.POINTER(Heads), ctypes.POINTER(Heads), _P, _Z, _P]),
    "red_cache_read": (_I, [ctypes.POINTER(PagedCache), _I, ctypes.POINTER(Heads), ctypes.POINTER(Heads), _P, _Z, _P]),
}


def _tensor(name, what, x, dtype, device, shape=None):
    """Refuse what is not a tensor of this type (a type or a tuple of them),
    on this device (None: any ROCm device), of this shape, with a contiguous
    last dimension."""
    if not isinstance(x, torch.Tensor) or x.device.type != "cuda":
        raise TypeError(f"{name}: {what} must be a tensor on a ROCm device")
    if device is not None and x.device != device:
        raise ValueError(f"{name}: {what} must be on {device}")
    if x.dtype != dtype and not (isinstance(dtype, tuple) and x.dtype in dtype):
        raise TypeError(f"{name}: {what} must be {dtype}, got {x.dtype}")
    if shape is not None and x.shape != shape:
        raise ValueError(f"{name}: {what} must have shape {tuple(shape)}, got {tuple(x.shape)}")
    if x.dim() and x.shape[-1] > 1 and x.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension of {what} must be contiguous")
    return x


def _vector(name, what, x, dtype, device, n):
    _tensor(name, what, x, dtype, device, (n,))
    return x.data_ptr()


def _heads(x):
    return Heads(x.data_ptr(), x.shape[1], x.stride(0), x.stride(1))


_FLOATS = (torch.float32, torch.float16, torch.bfloat16)


def _qk_norm_args(name, q, k, pos, freq, q_weight, k_weight, eps, interleaved, q_out, k_out):
    _tensor(name, "q", q, _FLOATS, None)
    if q.dim() != 3 or not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError(f"{name}: q and k must be (tokens, heads, dim)")
    tokens, _, dim = q.shape
    _tensor(name, "k", k, q.dtype, q.device, (tokens, k.shape[1], dim))
    args = QkNormRopeArgs(TYPES[q.dtype], 1 if interleaved else 0, tokens, dim, 2 * freq.numel(), eps, _heads(q), _heads(k))
    args.pos = _vector(name, "pos", pos, torch.int64, q.device, tokens)
    args.freq = _vector(name, "freq", freq, torch.float32, q.device, freq.numel())
    if q_weight is not None:
        args.q_weight = _vector(name, "q_weight", q_weight, q.dtype, q.device, dim)
    if k_weight is not None:
        args.k_weight = _vector(name, "k_weight", k_weight, q.dtype, q.device, dim)
    q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device) if q_out is None else \
        _tensor(name, "q_out", q_out, q.dtype, q.device, q.shape)
    k_out = torch.empty(k.shape, dtype=q.dtype, device=q.device) if k_out is None else \
        _tensor(name, "k_out", k_out, q.dtype, q.device, k.shape)
    args.q_out, args.k_out = _heads(q_out), _heads(k_out)
    return args, q_out, k_out


def red_qk_norm_rope(q, k, pos, freq, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, q_out=None,
                     k_out=None, stream=None):
    """RMS norm of every head of q (tokens, q heads, dim) and k (tokens, k
    heads, dim), times the weights, and the rotary rotation of the first
    2 * len(freq) elements by pos[t] * freq[i], in one pass. Pairs are halves
    apart, or neighbours if `interleaved`. float32, float16 or bfloat16; pos
    int64, freq float32. q_out and k_out may be q and k. -> (q_out, k_out)."""
    name = "red_qk_norm_rope"
    args, q_out, k_out = _qk_norm_args(name, q, k, pos, freq, q_weight, k_weight, eps, interleaved, q_out, k_out)
    with torch.cuda.device(q.device):
        st = lib().red_qk_norm_rope(ctypes.byref(args), _stream_handle(stream, q.device))
    _check(name, st)
    return q_out, k_out


def red_qk_norm_rope_backward(dq, dk, q, k, pos, freq, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                              stream=None):
    """Gradients of red_qk_norm_rope: dq and dk are those of its outputs.
    -> (gradient of q, of k, of q_weight, of k_weight), the weights' in float32
    (also where the weight is None, that is ones)."""
    name = "red_qk_norm_rope_backward"
    args, q_grad, k_grad = _qk_norm_args(name, q, k, pos, freq, q_weight, k_weight, eps, interleaved, None, None)
    _tensor(name, "dq", dq, q.dtype, q.device, q.shape)
    _tensor(name, "dk", dk, q.dtype, q.device, k.shape)
    dqw, dkw = torch.empty((2, q.shape[2]), dtype=torch.float32, device=q.device).unbind(0)
    hq, hk = _heads(dq), _heads(dk)
    with torch.cuda.device(q.device):
        st = lib().red_qk_norm_rope_backward(ctypes.byref(args), ctypes.byref(hq), ctypes.byref(hk), dqw.data_ptr(),
                                             dkw.data_ptr(), _stream_handle(stream, q.device))
    _check(name, st)
    return q_grad, k_grad, dqw, dkw


_CACHES = (torch.float16, torch.bfloat16, torch.int8, torch.float8_e4m3fn)


def _cache(name, k_pages, v_pages, k_scales, v_scales):
    _tensor(name, "k_pages", k_pages, _CACHES, None)
    if k_pages.dim() != 4:
        raise ValueError(f"{name}: k_pages must be (pages, heads, places, dim)")
    _tensor(name, "v_pages", v_pages, k_pages.dtype, k_pages.device, k_pages.shape)
    strides = k_pages.stride()
    if v_pages.stride() != strides:
        raise ValueError(f"{name}: k_pages and v_pages must have the same strides")
    c = PagedCache(k_pages.data_ptr(), v_pages.data_ptr(), None, None, TYPES[k_pages.dtype], *k_pages.shape, *strides[:3])
    scaled = c.type >= 3
    if scaled != (k_scales is not None) or scaled != (v_scales is not None):
        raise ValueError(f"{name}: 8-bit caches take k_scales and v_scales, 16-bit ones do not")
    if scaled:
        for what, x in (("k_scales", k_scales), ("v_scales", v_scales)):
            if not isinstance(x, torch.Tensor) or x.dtype != torch.float32 or x.device != k_pages.device or \
                    x.shape != k_pages.shape[:3]:
                raise ValueError(f"{name}: {what} must be float32 {tuple(k_pages.shape[:3])} on {k_pages.device}")
        if k_scales.stride() != v_scales.stride():
            raise ValueError(f"{name}: k_scales and v_scales must have the same strides")
        c.k_scales, c.v_scales = k_scales.data_ptr(), v_scales.data_ptr()
        c.scale_page_stride, c.scale_head_stride, c.scale_place_stride = k_scales.stride()
    return c


def red_cache_write(k, v, slots, k_pages, v_pages, k_scales=None, v_scales=None, stream=None):
    """Write k and v (tokens, heads, dim; float16 or bfloat16) into the paged
    cache k_pages, v_pages (pages, heads, places, dim): token t goes to place
    slots[t] % places of page slots[t] // places (int64; slots outside the cache
    are skipped). int8 and float8_e4m3fn caches take one scale a row in
    k_scales, v_scales (pages, heads, places; float32)."""
    name = "red_cache_write"
    c = _cache(name, k_pages, v_pages, k_scales, v_scales)
    device = k_pages.device
    _tensor(name, "k", k, _FLOATS[1:], device)
    shape = (slots.shape[0], k_pages.shape[1], k_pages.shape[3])
    _tensor(name, "k", k, k.dtype, device, shape)
    _tensor(name, "v", v, k.dtype, device, shape)
    sl = _vector(name, "slots", slots, torch.int64, device, shape[0])
    hk, hv = _heads(k), _heads(v)
    with torch.cuda.device(device):
        st = lib().red_cache_write(ctypes.byref(c), TYPES[k.dtype], ctypes.byref(hk), ctypes.byref(hv), sl, shape[0],
                                   _stream_handle(stream, device))
    _check(name, st)


def red_cache_read(k_pages, v_pages, slots, dtype, k_scales=None, v_scales=None, k_out=None, v_out=None, stream=None):
    """Read tokens back from a paged cache (see red_cache_write) as float16 or
    bfloat16. A slot outside the cache reads as zeros. -> (k, v), each (tokens,
    heads, dim)."""
    name = "red_cache_read"
    c = _cache(name, k_pages, v_pages, k_scales, v_scales)
    device = k_pages.device
    if dtype not in _FLOATS[1:]:
        raise TypeError(f"{name}: dtype must be torch.float16 or torch.bfloat16")
    shape = (slots.shape[0], k_pages.shape[1], k_pages.shape[3])
    sl = _vector(name, "slots", slots, torch.int64, device, shape[0])
    k_out = torch.empty(shape, dtype=dtype, device=device) if k_out is None else \
        _tensor(name, "k_out", k_out, dtype, device, shape)
    v_out = torch.empty(shape, dtype=dtype, device=device) if v_out is None else \
        _tensor(name, "v_out", v_out, dtype, device, shape)
    hk, hv = _heads(k_out), _heads(v_out)
    with torch.cuda.device(device):
        st = lib().red_cache_read(ctypes.byref(c), TYPES[dtype], ctypes.byref(hk), ctypes.byref(hv), sl, shape[0],
                                  _stream_handle(stream, device))
    _check(name, st)
    return k_out, v_out


def red_tree_attention(q, k_pages, v_pages, table, lens, scale, max_len=None, tree_mask=None, node_count=None,
                       k_scales=None, v_scales=None, out=None, stream=None):
    """Attention of drafted tokens q (batch, nodes, q heads, dim; float16 or
    bfloat16; at most 64 nodes) over a paged cache (see red_cache_write).
    Sequence b has lens[b] tokens (int32) and then its nodes, whose keys and
    values are in the cache as well; token t lies in page table[b, t // places]
    (int32). Node i sees all tokens below lens[b] and the nodes whose bits are
    set in tree_mask[b, i] (int64; None: nodes 0 .. i); node_count (int32)
    says how many nodes there are (None: all). max_len: the most tokens, nodes
    included, of a sequence (None: what the table holds). -> (out like q, lse
    (batch, nodes, q heads) float32); rows that see nothing hold 0 and -inf."""
    name = "red_tree_attention"
    c = _cache(name, k_pages, v_pages, k_scales, v_scales)
    device = k_pages.device
    _tensor(name, "q", q, _FLOATS[1:], device)
    if q.dim() != 4 or q.shape[3] != c.dim:
        raise ValueError(f"{name}: q must be (batch, nodes, q heads, {c.dim})")
    batch, nodes, heads, dim = q.shape
    _tensor(name, "table", table, torch.int32, device)
    if table.dim() != 2 or table.shape[0] != batch:
        raise ValueError(f"{name}: table must be ({batch}, pages of a sequence)")
    out = torch.empty(q.shape, dtype=q.dtype, device=device) if out is None else \
        _tensor(name, "out", out, q.dtype, device, q.shape)
    lse = torch.empty((batch, nodes, heads), dtype=torch.float32, device=device)
    cols = table.shape[1]
    a = TreeAttentionArgs(TYPES[q.dtype], scale, batch, nodes, heads, cols * c.places if max_len is None else max_len,
                          q.data_ptr(), out.data_ptr(), lse.data_ptr(), *q.stride()[:3], *out.stride()[:3], c,
                          table.data_ptr(), cols, table.stride(0), _vector(name, "lens", lens, torch.int32, device, batch))
    if tree_mask is not None:
        _tensor(name, "tree_mask", tree_mask, torch.int64, device, (batch, nodes))
        if not tree_mask.is_contiguous():
            raise ValueError(f"{name}: tree_mask must be contiguous")
        a.tree_mask = tree_mask.data_ptr()
    if node_count is not None:
        a.node_count = _vector(name, "node_count", node_count, torch.int32, device, batch)
    with torch.cuda.device(device):
        st = lib().red_tree_attention(ctypes.byref(a), _stream_handle(stream, device))
    _check(name, st)
    return out, lse


def red_verify_drafts(p, q, drafted, u, r, draft_count=None, stream=None):
    """Which drafted tokens (batch, drafts; int64) the target's probabilities p
    (batch, drafts + 1, vocab) accept against the draft's q (batch, drafts,
    vocab; None: its tokens were certain), by the random numbers u (batch,
    drafts) and r (batch; both float32), and the token drawn after them.
    draft_count (int32): how many drafts a sequence has (None: all).
    -> (accepted (batch) int32, tokens (batch, drafts + 1) int64: the accepted
    ones, the drawn one, then -1)."""
    name = "red_verify_drafts"
    _tensor(name, "p", p, _FLOATS, None)
    device = p.device
    if p.dim() != 3 or p.shape[1] < 1:
        raise ValueError(f"{name}: p must be (batch, drafts + 1, vocab)")
    batch, drafts, vocab = p.shape[0], p.shape[1] - 1, p.shape[2]
    a = VerifyDraftsArgs(TYPES[p.dtype], batch, drafts, vocab, p.data_ptr(), *p.stride()[:2])
    if q is not None:
        _tensor(name, "q", q, p.dtype, device, (batch, drafts, vocab))
        a.q, a.q_batch_stride, a.q_step_stride = q.data_ptr(), *q.stride()[:2]
    for what, x, dtype in (("drafted", drafted, torch.int64), ("u", u, torch.float32)):
        _tensor(name, what, x, dtype, device, (batch, drafts))
        if not x.is_contiguous():
            raise ValueError(f"{name}: {what} must be contiguous")
        setattr(a, what, x.data_ptr())
    a.r = _vector(name, "r", r, torch.float32, device, batch)
    if draft_count is not None:
        a.draft_count = _vector(name, "draft_count", draft_count, torch.int32, device, batch)
    accepted = torch.empty(batch, dtype=torch.int32, device=device)
    tokens = torch.empty((batch, drafts + 1), dtype=torch.int64, device=device)
    a.accepted, a.tokens = accepted.data_ptr(), tokens.data_ptr()
    with torch.cuda.device(device):
        st = lib().red_verify_drafts(ctypes.byref(a), _stream_handle(stream, device))
    _check(name, st)
    return accepted, tokens
