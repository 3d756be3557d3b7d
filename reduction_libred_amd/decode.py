"""The reductions of a decoding step of drafted tokens (include/libred_decode.h).

Like the rest of the binding, each function has the name of the C entry point
it calls and only marshals arguments. Tensors are taken with the strides they
have, as long as their last dimension is contiguous. Where a call is given a
stream, its outputs are allocated there; ordering that stream behind the one
its inputs come from, and the outputs' readers behind it, is the caller's.
red_qk_norm_rope is differentiable; nothing else here is, and its results carry
no history.

A decoding step makes these calls with little work in each, so the way to the
C call is kept short: one look at a tensor where it is as it should be (what is
wrong is found out afterwards), and argument structs packed in one go.
"""
import ctypes
import struct
import warnings

import torch

from . import RedError, _stream_handle, lib

_P = ctypes.c_void_p
_Z = ctypes.c_size_t
_I = ctypes.c_int
_L = ctypes.c_int64
_F = ctypes.c_float

TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.int8: 3, torch.float8_e4m3fn: 4}


# The structs of libred_decode.h, each with a packer that takes their fields
# one after the other.
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


def _packer(cls):
    codes = {_P: "Q", _Z: "Q", _L: "q", _I: "i", _F: "f"}

    def fields(c):
        return "".join(codes[t] if t in codes else "0Q" + fields(t) + "0Q" for _, t in c._fields_)

    p = struct.Struct("@" + fields(cls) + "0Q")
    assert p.size == ctypes.sizeof(cls)
    return p.pack


_pack_heads, _pack_qk_norm, _pack_cache = _packer(Heads), _packer(QkNormRopeArgs), _packer(PagedCache)
_pack_attention, _pack_verify = _packer(TreeAttentionArgs), _packer(VerifyDraftsArgs)

SIGNATURES = {
    "red_qk_norm_rope": (_I, [_P, _P]),
    "red_qk_norm_rope_backward": (_I, [_P, _P, _P, _P, _P, _P]),
    "red_cache_write": (_I, [_P, _I, _P, _P, _P, _Z, _P]),
    "red_cache_read": (_I, [_P, _I, _P, _P, _P, _Z, _P]),
    "red_tree_attention": (_I, [_P, _P]),
    "red_verify_drafts": (_I, [_P, _P]),
}

_FLOATS = (torch.float32, torch.float16, torch.bfloat16)
_HALVES = _FLOATS[1:]
_CACHES = (torch.float16, torch.bfloat16, torch.int8, torch.float8_e4m3fn)
_INT32, _INT64, _FLOAT32 = torch.int32, torch.int64, torch.float32


def _refuse(name, what, x, dtype, device, shape, contiguous=False):
    """Raise what is wrong with x."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{name}: {what} must be a tensor on a ROCm device")
    if device is not None and x.get_device() != device:
        raise ValueError(f"{name}: {what} must be on cuda:{device}")
    if x.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name}: {what} must be {dtype}, got {x.dtype}")
    if x.shape != shape:
        raise ValueError(f"{name}: {what} must have shape {tuple(shape)}, got {tuple(x.shape)}")
    raise ValueError(f"{name}: {'' if contiguous else 'the last dimension of '}{what} must be contiguous")


def _any(name, what, x, dtypes, dims, layout):
    """The first tensor of a call, of one of these types and `dims`
    dimensions; -> its device."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype not in dtypes:
        _refuse(name, what, x, dtypes, None, None)
    if x.dim() != dims:
        raise ValueError(f"{name}: {what} must be {layout}")
    if x.stride(-1) != 1 and x.shape[-1] > 1:
        _refuse(name, what, x, dtypes, None, x.shape)
    return x.get_device()


def _rows(name, what, x, dtype, device, shape):
    """A tensor of this shape with a contiguous last dimension."""
    if not (isinstance(x, torch.Tensor) and x.dtype is dtype and x.get_device() == device and x.shape == shape and
            (x.stride(-1) == 1 or shape[-1] <= 1)):
        _refuse(name, what, x, dtype, device, shape)
    return x


def _whole(name, what, x, dtype, device, shape):
    """The address of a contiguous tensor of this shape."""
    if not (isinstance(x, torch.Tensor) and x.dtype is dtype and x.get_device() == device and x.shape == shape and
            x.is_contiguous()):
        _refuse(name, what, x, dtype, device, shape, True)
    return x.data_ptr()


_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_grad_enabled = torch.is_grad_enabled
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


_functions = {}


def _call(name, device, stream, *args):
    """lib().name(*args, stream) with `device` current."""
    if _current_device() != device:
        with torch.cuda.device(device):
            return _call(name, device, stream, *args)
    handle = _raw_stream(device) if stream is None and _raw_stream is not None else _stream_handle(stream, device)
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(lib(), name)
    st = f(*args, handle)
    if st:
        raise RedError(name, st, lib().red_last_hip_error())


def _on(stream, f, *args):
    """f(*args) with `stream` (a torch stream or a handle) the current one, so
    that what it allocates belongs to the stream that writes it."""
    if not isinstance(stream, torch.cuda.Stream):
        device = args[0].device if isinstance(args[0], torch.Tensor) and args[0].is_cuda else None
        stream = torch.cuda.ExternalStream(int(stream), device) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return f(*args)


def _qk_norm_check(name, q, k, pos, freq, q_weight, k_weight, q_out, k_out):
    """Raise what is wrong with the arguments, if anything is."""
    device = _any(name, "q", q, _FLOATS, 3, "(tokens, q heads, dim)")
    dtype, (tokens, _, dim) = q.dtype, q.shape
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError(f"{name}: k must be (tokens, k heads, dim)")
    _rows(name, "k", k, dtype, device, (tokens, k.shape[1], dim))
    for what, x, shape in (("q_out", q_out, q.shape), ("k_out", k_out, k.shape)):
        if x is not None:
            _rows(name, what, x, dtype, device, shape)
    _whole(name, "pos", pos, _INT64, device, (tokens,))
    _whole(name, "freq", freq, _FLOAT32, device, (freq.shape[0] if isinstance(freq, torch.Tensor) and freq.dim() == 1 else -1,))
    for what, x in (("q_weight", q_weight), ("k_weight", k_weight)):
        if x is not None:
            _whole(name, what, x, dtype, device, (dim,))


def _qk_norm(name, q, k, pos, freq, q_weight, k_weight, eps, interleaved, q_out, k_out):
    try:
        dtype, device, (tokens, heads, dim) = q.dtype, q.get_device(), q.shape
        k_tokens, kh, k_dim = k.shape
        half, = freq.shape
        fine = (device >= 0 and dtype in _FLOATS and k.dtype is dtype and k.get_device() == device and k_tokens == tokens and
                k_dim == dim and pos.dtype is _INT64 and pos.shape == (tokens,) and pos.get_device() == device and
                pos.is_contiguous() and freq.dtype is _FLOAT32 and freq.get_device() == device and freq.is_contiguous())
        q0, q1, q2 = q.stride()
        k0, k1, k2 = k.stride()
        fine = fine and (q2 == k2 == 1 or dim <= 1)
        for w in (q_weight, k_weight):
            if w is not None:
                fine = fine and w.dtype is dtype and w.shape == (dim,) and w.get_device() == device and w.is_contiguous()
    except (AttributeError, ValueError):
        fine = False
    if not fine or q_out is not None or k_out is not None:
        _qk_norm_check(name, q, k, pos, freq, q_weight, k_weight, q_out, k_out)
    if q_out is None:
        q_out = torch.empty_like(q)
    if k_out is None:
        k_out = torch.empty_like(k)
    a0, a1, a2 = q_out.stride()
    b0, b1, b2 = k_out.stride()
    if dim > 1:     # an output that was laid out like rows that overlap
        if a2 != 1:
            q_out = q.new_empty(q.shape)
            a0, a1, _ = q_out.stride()
        if b2 != 1:
            k_out = k.new_empty(k.shape)
            b0, b1, _ = k_out.stride()
    return device, q_out, k_out, _pack_qk_norm(
        TYPES[dtype], 1 if interleaved else 0, tokens, dim, 2 * half, eps, q.data_ptr(), heads, q0, q1, k.data_ptr(), kh, k0,
        k1, q_out.data_ptr(), heads, a0, a1, k_out.data_ptr(), kh, b0, b1,
        0 if q_weight is None else q_weight.data_ptr(), 0 if k_weight is None else k_weight.data_ptr(), pos.data_ptr(),
        freq.data_ptr())


def _heads(x):
    return _pack_heads(x.data_ptr(), x.shape[1], *x.stride()[:2])


def red_qk_norm_rope(q, k, pos, freq, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, q_out=None,
                     k_out=None, stream=None):
    """RMS norm of every head of q (tokens, q heads, dim) and k (tokens, k
    heads, dim), times the weights, and the rotary rotation of the first
    2 * len(freq) elements by pos[t] * freq[i], in one pass. Pairs are halves
    apart, or neighbours if `interleaved`. float32, float16 or bfloat16; pos
    int64, freq float32. q_out and k_out may be q and k. -> (q_out, k_out).
    Gradients go to q, k and the weights, unless q_out or k_out is given: what
    is written there carries no history, and a warning says so."""
    if stream is not None:
        return _on(stream, red_qk_norm_rope, q, k, pos, freq, q_weight, k_weight, eps, interleaved, q_out, k_out)
    name = "red_qk_norm_rope"
    try:
        history = _grad_enabled() and (q.requires_grad or k.requires_grad or q_weight is not None and q_weight.requires_grad or
                                       k_weight is not None and k_weight.requires_grad)
    except AttributeError:
        history = False     # no tensors: refused below
    if history:
        if q_out is None and k_out is None:
            return _QkNormRope.apply(q, k, q_weight, k_weight, pos, freq, eps, interleaved)
        warnings.warn(f"{name}: what is written to q_out and k_out carries no history", stacklevel=2)
    device, q_out, k_out, args = _qk_norm(name, q, k, pos, freq, q_weight, k_weight, eps, interleaved, q_out, k_out)
    _call(name, device, None, args)
    return q_out, k_out


def red_qk_norm_rope_backward(dq, dk, q, k, pos, freq, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                              stream=None):
    """Gradients of red_qk_norm_rope: dq and dk are those of its outputs.
    -> (gradient of q, of k, of q_weight, of k_weight), the weights' in float32
    (also where the weight is None, that is ones)."""
    if stream is not None:
        return _on(stream, red_qk_norm_rope_backward, dq, dk, q, k, pos, freq, q_weight, k_weight, eps, interleaved)
    return _qk_norm_backward(dq, dk, q, k, pos, freq, q_weight, k_weight, eps, interleaved, True, True)


def _qk_norm_backward(dq, dk, q, k, pos, freq, q_weight, k_weight, eps, interleaved, of_q_weight, of_k_weight):
    name = "red_qk_norm_rope_backward"
    device, q_grad, k_grad, args = _qk_norm(name, q, k, pos, freq, q_weight, k_weight, eps, interleaved, None, None)
    _rows(name, "dq", dq, q.dtype, device, q.shape)
    _rows(name, "dk", dk, q.dtype, device, k.shape)
    dqw = torch.empty(q.shape[2], dtype=_FLOAT32, device=q.device) if of_q_weight else None
    dkw = torch.empty(q.shape[2], dtype=_FLOAT32, device=q.device) if of_k_weight else None
    _call(name, device, None, args, _heads(dq), _heads(dk), dqw.data_ptr() if of_q_weight else None,
          dkw.data_ptr() if of_k_weight else None)
    return q_grad, k_grad, dqw, dkw


class _QkNormRope(torch.autograd.Function):
    """red_qk_norm_rope with red_qk_norm_rope_backward as its gradient."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, pos, freq, eps, interleaved):
        name = "red_qk_norm_rope"
        device, q_out, k_out, args = _qk_norm(name, q, k, pos, freq, q_weight, k_weight, eps, interleaved, None, None)
        _call(name, device, None, args)
        ctx.save_for_backward(q, k, q_weight, k_weight, pos, freq)
        ctx.eps, ctx.interleaved = eps, interleaved
        return q_out, k_out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq, dk):
        q, k, q_weight, k_weight, pos, freq = ctx.saved_tensors
        # A gradient may be broadcast (that of a sum), also along the rows.
        dq, dk = (x if x.stride(-1) == 1 or x.shape[-1] <= 1 else x.contiguous() for x in (dq, dk))
        of_q, of_k, of_qw, of_kw = ctx.needs_input_grad[:4]
        dq, dk, dqw, dkw = _qk_norm_backward(dq, dk, q, k, pos, freq, q_weight, k_weight, ctx.eps, ctx.interleaved, of_qw, of_kw)
        return (dq if of_q else None, dk if of_k else None, dqw.to(q.dtype) if of_qw else None,
                dkw.to(q.dtype) if of_kw else None, None, None, None, None)


def _cache_check(name, k_pages, v_pages, k_scales, v_scales):
    """Raise what is wrong with a cache, if anything is."""
    device = _any(name, "k_pages", k_pages, _CACHES, 4, "(pages, heads, places, dim)")
    dtype, shape = k_pages.dtype, k_pages.shape
    _rows(name, "v_pages", v_pages, dtype, device, shape)
    if v_pages.stride() != k_pages.stride():
        raise ValueError(f"{name}: k_pages and v_pages must have the same strides")
    scaled = TYPES[dtype] >= 3
    if scaled != (k_scales is not None) or scaled != (v_scales is not None):
        raise ValueError(f"{name}: 8-bit caches take k_scales and v_scales, 16-bit ones do not")
    if scaled:
        for what, x in (("k_scales", k_scales), ("v_scales", v_scales)):
            if not isinstance(x, torch.Tensor) or x.dtype is not _FLOAT32 or x.get_device() != device or x.shape != shape[:3]:
                raise ValueError(f"{name}: {what} must be float32 {tuple(shape[:3])} on cuda:{device}")
        if k_scales.stride() != v_scales.stride():
            raise ValueError(f"{name}: k_scales and v_scales must have the same strides")


_NO_SCALES = (0, 0, 0)


def _cache(name, k_pages, v_pages, k_scales, v_scales):
    """-> (device, the fields of a PagedCache)"""
    try:
        dtype, device, shape, strides = k_pages.dtype, k_pages.get_device(), k_pages.shape, k_pages.stride()
        kind = TYPES.get(dtype, 0)
        fine = (device >= 0 and kind > 0 and len(shape) == 4 and v_pages.dtype is dtype and v_pages.get_device() == device and
                v_pages.shape == shape and v_pages.stride() == strides and strides[3] == 1)
        ks = vs = 0
        scale_strides = _NO_SCALES
        if kind >= 3:
            scale_strides = k_scales.stride()
            ks, vs = k_scales.data_ptr(), v_scales.data_ptr()
            fine = (fine and k_scales.dtype is v_scales.dtype is _FLOAT32 and k_scales.get_device() == device and
                    v_scales.get_device() == device and k_scales.shape == v_scales.shape == shape[:3] and
                    v_scales.stride() == scale_strides)
        else:
            fine = fine and k_scales is v_scales is None
    except AttributeError:
        fine = False
    if not fine:
        _cache_check(name, k_pages, v_pages, k_scales, v_scales)
    return device, (k_pages.data_ptr(), v_pages.data_ptr(), ks, vs, kind, *shape, *strides[:3], *scale_strides)


def _slots(name, slots, k_pages, device):
    """-> (address of the slots, how many, the shape of their rows)"""
    n = slots.shape[0] if isinstance(slots, torch.Tensor) and slots.dim() == 1 else -1
    _, heads, _, dim = k_pages.shape
    return _whole(name, "slots", slots, _INT64, device, (n,)), n, (n, heads, dim)


def red_cache_write(k, v, slots, k_pages, v_pages, k_scales=None, v_scales=None, stream=None):
    """Write k and v (tokens, heads, dim; float16 or bfloat16) into the paged
    cache k_pages, v_pages (pages, heads, places, dim): token t goes to place
    slots[t] % places of page slots[t] // places (int64; slots outside the cache
    are skipped). int8 and float8_e4m3fn caches take one scale a row in
    k_scales, v_scales (pages, heads, places; float32)."""
    name = "red_cache_write"
    device, c = _cache(name, k_pages, v_pages, k_scales, v_scales)
    at, tokens, shape = _slots(name, slots, k_pages, device)
    dtype = k.dtype if isinstance(k, torch.Tensor) else None
    if dtype not in _HALVES:
        _any(name, "k", k, _HALVES, 3, "(tokens, heads, dim)")
    _rows(name, "k", k, dtype, device, shape)
    _rows(name, "v", v, dtype, device, shape)
    k0, k1, _ = k.stride()
    v0, v1, _ = v.stride()
    heads = shape[1]
    _call(name, device, stream, _pack_cache(*c), TYPES[dtype], _pack_heads(k.data_ptr(), heads, k0, k1),
          _pack_heads(v.data_ptr(), heads, v0, v1), at, tokens)


def red_cache_read(k_pages, v_pages, slots, dtype, k_scales=None, v_scales=None, k_out=None, v_out=None, stream=None):
    """Read tokens back from a paged cache (see red_cache_write) as float16 or
    bfloat16. A slot outside the cache reads as zeros. -> (k, v), each (tokens,
    heads, dim)."""
    if stream is not None:
        return _on(stream, red_cache_read, k_pages, v_pages, slots, dtype, k_scales, v_scales, k_out, v_out)
    name = "red_cache_read"
    device, c = _cache(name, k_pages, v_pages, k_scales, v_scales)
    if dtype not in _HALVES:
        raise TypeError(f"{name}: dtype must be torch.float16 or torch.bfloat16")
    at, tokens, shape = _slots(name, slots, k_pages, device)
    if k_out is None:
        k_out = torch.empty(shape, dtype=dtype, device=k_pages.device)
    else:
        _rows(name, "k_out", k_out, dtype, device, shape)
    if v_out is None:
        v_out = torch.empty(shape, dtype=dtype, device=k_pages.device)
    else:
        _rows(name, "v_out", v_out, dtype, device, shape)
    k0, k1, _ = k_out.stride()
    v0, v1, _ = v_out.stride()
    heads = shape[1]
    _call(name, device, stream, _pack_cache(*c), TYPES[dtype], _pack_heads(k_out.data_ptr(), heads, k0, k1),
          _pack_heads(v_out.data_ptr(), heads, v0, v1), at, tokens)
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
    if stream is not None:
        return _on(stream, red_tree_attention, q, k_pages, v_pages, table, lens, scale, max_len, tree_mask, node_count,
                   k_scales, v_scales, out)
    name = "red_tree_attention"
    device, c = _cache(name, k_pages, v_pages, k_scales, v_scales)
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or q.dtype not in _HALVES:
        _any(name, "q", q, _HALVES, 4, "(batch, nodes, q heads, dim)")
    dtype, shape = q.dtype, q.shape
    batch, nodes, heads, dim = shape
    _, _, places, width = k_pages.shape
    if dim != width:
        raise ValueError(f"{name}: q must be (batch, nodes, q heads, {width})")
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError(f"{name}: table must be ({batch}, pages of a sequence)")
    cols = table.shape[1]
    if max_len is not None and max_len < 0:
        raise ValueError(f"{name}: max_len must not be negative")
    q0, q1, q2, q3 = q.stride()
    if q.get_device() != device or (q3 != 1 and dim > 1):
        _rows(name, "q", q, dtype, device, shape)
    _rows(name, "table", table, _INT32, device, (batch, cols))
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else q.new_empty(shape)
    else:
        _rows(name, "out", out, dtype, device, shape)
    o0, o1, o2, _ = out.stride()
    lse = torch.empty((batch, nodes, heads), dtype=_FLOAT32, device=q.device)
    mask = 0 if tree_mask is None else _whole(name, "tree_mask", tree_mask, _INT64, device, (batch, nodes))
    count = 0 if node_count is None else _whole(name, "node_count", node_count, _INT32, device, (batch,))
    _call(name, device, stream, _pack_attention(
        TYPES[dtype], scale, batch, nodes, heads, cols * places if max_len is None else max_len, q.data_ptr(), out.data_ptr(),
        lse.data_ptr(), q0, q1, q2, o0, o1, o2, *c, table.data_ptr(), cols, table.stride(0),
        _whole(name, "lens", lens, _INT32, device, (batch,)), mask, count))
    return out, lse


def red_verify_drafts(p, q, drafted, u, r, draft_count=None, stream=None):
    """Which drafted tokens (batch, drafts; int64) the target's probabilities p
    (batch, drafts + 1, vocab) accept against the draft's q (batch, drafts,
    vocab; None: its tokens were certain), by the random numbers u (batch,
    drafts) and r (batch; both float32), and the token drawn after them.
    draft_count (int32): how many drafts a sequence has (None: all).
    -> (accepted (batch) int32, tokens (batch, drafts + 1) int64: the accepted
    ones, the drawn one, then -1)."""
    if stream is not None:
        return _on(stream, red_verify_drafts, p, q, drafted, u, r, draft_count)
    name = "red_verify_drafts"
    device = _any(name, "p", p, _FLOATS, 3, "(batch, drafts + 1, vocab)")
    dtype, (batch, steps, vocab), (p0, p1, _) = p.dtype, p.shape, p.stride()
    if steps < 1:
        raise ValueError(f"{name}: p must be (batch, drafts + 1, vocab)")
    drafts = steps - 1
    qp = q0 = q1 = 0
    if q is not None:
        qp, (q0, q1, _) = _rows(name, "q", q, dtype, device, (batch, drafts, vocab)).data_ptr(), q.stride()
    at, up = _whole(name, "drafted", drafted, _INT64, device, (batch, drafts)), _whole(name, "u", u, _FLOAT32, device, (batch, drafts))
    rp = _whole(name, "r", r, _FLOAT32, device, (batch,))
    count = 0 if draft_count is None else _whole(name, "draft_count", draft_count, _INT32, device, (batch,))
    accepted = torch.empty(batch, dtype=_INT32, device=p.device)
    tokens = torch.empty((batch, steps), dtype=_INT64, device=p.device)
    _call(name, device, stream, _pack_verify(TYPES[dtype], batch, drafts, vocab, p.data_ptr(), p0, p1, qp, q0, q1, at, up, rp,
                                             count, accepted.data_ptr(), tokens.data_ptr()))
    return accepted, tokens
