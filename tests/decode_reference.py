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


assert math.isclose(step(torch.bfloat16), 2.0 ** -8)
