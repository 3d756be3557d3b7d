"""The decoding step's operators in float64 on the CPU, straight from their
formulas, with the sizes that error bounds are relative to."""
import math

import torch

F64 = torch.float64


def step(dtype):
    """Half a unit in the last place, relative: the error of one rounding."""
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the spacing of the subnormal numbers of `dtype`."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def pairs(rot, interleaved):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(y, pos, freq, interleaved, sign=1.0):
    """The rotation of y (tokens, heads, dim), and |y_a| + |y_b| of each pair
    (|y| where nothing turns)."""
    rot = 2 * freq.numel()
    a, b = pairs(rot, interleaved)
    angle = pos.to(F64)[:, None] * freq.to(F64)
    c, s = torch.cos(angle)[:, None], sign * torch.sin(angle)[:, None]
    out, size = y.clone(), y.abs()
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., a] * s + y[..., b] * c
    size[..., a] = size[..., b] = y[..., a].abs() + y[..., b].abs()
    return out, size


def qk_norm_rope(x, w, pos, freq, eps, interleaved):
    x = x.to(F64)
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return rotate(x * r * (w.to(F64) if w is not None else 1.0), pos, freq, interleaved)


def qk_norm_rope_backward(dy, x, w, pos, freq, eps, interleaved):
    """-> (dx, size of its terms, dw, sum of the magnitudes of its terms)"""
    x, dy = x.to(F64), dy.to(F64)
    w = w.to(F64) if w is not None else torch.ones(x.shape[-1], dtype=F64)
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    g, gsize = rotate(dy, pos, freq, interleaved, -1.0)
    h, hsize = g * w, gsize * w.abs()
    dx = r * (h - x * (r * r * (h * x).mean(-1, keepdim=True)))
    size = r * (hsize + x.abs() * (r * r * (hsize * x.abs()).mean(-1, keepdim=True)))
    return dx, size, (g * x * r).sum((0, 1)), (gsize * x.abs() * r).sum((0, 1))


def frequencies(rot):
    return torch.tensor([10000.0 ** (-2.0 * i / max(rot, 1)) for i in range(rot // 2)], dtype=torch.float32)


TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


def code_step(y, kind):
    """Spacing of the codes around y (already divided by the scale)."""
    if kind == torch.int8:
        return torch.ones_like(y)
    # three bits after the first, from 2^-6 on
    return torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)


def visible(lens, nodes, mask, count, total):
    """Which of `total` tokens every node of a sequence sees: (nodes, total)."""
    t = torch.arange(total)
    seen = torch.zeros(nodes, total, dtype=torch.bool)
    for i in range(min(count, nodes)):
        word = int(mask[i]) if mask is not None else (1 << (i + 1)) - 1
        for j in range(min(count, nodes)):
            if word >> j & 1 and lens + j < total:
                seen[i, lens + j] = True
        seen[i] |= t < lens
    return seen


def tree_attention(q, k, v, seen, scale):
    """One sequence and kv head: q (rows, dim), k and v (tokens, dim; values and
    their scales multiplied out), seen (rows, tokens) -> out, lse, and per row
    the softmax weights and the scores' sum of magnitudes (its largest)."""
    q, k = q.to(F64), k.to(F64)
    out = torch.zeros(q.shape[0], v.shape[1], dtype=F64)
    lse = torch.full((q.shape[0],), -math.inf, dtype=F64)
    weights, size = [], torch.zeros(q.shape[0], dtype=F64)
    for i in range(q.shape[0]):
        ks, vs = k[seen[i]], v[seen[i]].to(F64)
        s = (ks @ q[i]) * scale
        weights.append(torch.softmax(s, 0) if len(s) else s)
        if len(s):
            lse[i] = torch.logsumexp(s, 0)
            p = weights[-1][:, None]
            out[i] = torch.where(vs.isfinite(), p * vs, vs).sum(0)
            size[i] = ((ks.abs() @ q[i].abs()) * abs(scale)).max()
    return out, lse, weights, size


def verify(p, q, drafted, u, r, count):
    """One sequence: p (drafts + 1, vocab), q (drafts, vocab) or None."""
    n, vocab = 0, p.shape[1]
    while n < count:
        d = int(drafted[n])
        if not 0 <= d < vocab or not float(u[n]) * (float(q[n, d]) if q is not None else 1.0) < float(p[n, d]):
            break
        n += 1
    w = p[n].to(F64)
    if n < count:
        less = q[n].to(F64) if q is not None else torch.nn.functional.one_hot(drafted[n].clamp(0, vocab - 1), vocab).to(F64) * \
            float(0 <= int(drafted[n]) < vocab)
        rest = (w - less).clamp(min=0)
        w = rest if rest.sum() > 0 else w
    run = torch.cumsum(w, 0)
    positive = (w > 0).nonzero()[:, 0]
    if not len(positive) or run[-1].isnan():
        token = -1
    else:
        after = positive[run[positive] > float(r) * run[-1]]
        token = int(after[0] if len(after) else positive[-1])
    return n, [int(d) for d in drafted[:n]] + [token] + [-1] * (len(drafted) - n)


assert math.isclose(step(torch.bfloat16), 2.0 ** -8)
