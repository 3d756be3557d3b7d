"""The decoding step's operators on the GPU, against float64 on the CPU.

Tolerances: one rounding to the output's type, plus the float32 arithmetic
before it, counted in roundings of 2^-24 against the size of the terms that
meet (the references return it)."""
import math
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected only with a GPU
    pytest.skip("no GPU visible", allow_module_level=True)

import decode_reference as R  # noqa: E402
import reduction_libred_amd as rl  # noqa: E402

DEV = torch.device("cuda:0")
F32, F16, BF16, I8, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.int8, torch.float8_e4m3fn
U = 2.0 ** -24
# Roundings of float32 between inputs and a norm's result: at most 8 + 6 in the
# sum of squares (halved by the root), 2 for the root, 3 products, 3 in the turn
# and 1 each in cosine and sine.
NORM_STEPS = 20
# The backward pass adds the mean of h x (8 + 6 + 4 products) and three more.
BACK_STEPS = 48


def say(*a):
    print("[decode-gpu]", *a, flush=True)
    sys.stdout.flush()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def close(what, got, want, size, dtype, steps):
    got, want = got.cpu().to(torch.float64), want
    allowed = R.step(dtype) * (want.abs() + steps * U * size) + steps * U * size + R.tiny(dtype)
    bad = ~((got - want).abs() <= allowed)
    if bad.any():
        i = int(torch.where(bad.flatten(), (got - want).abs().flatten() / allowed.flatten(), 0.0).nan_to_num(1e30).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, worst at {i}: {got.flatten()[i]} "
                             f"against {want.flatten()[i]}, allowed {allowed.flatten()[i]}")


def place(x, layout):
    """x on the GPU: 'own' storage, 'packed' (a part of wider rows), or
    'odd' (starting one element into its storage, rows one element apart)."""
    if layout == "own":
        return x.to(DEV)
    t, h, d = x.shape
    if layout == "packed":
        buf = torch.full((t, h + 3, d), float("nan"), dtype=x.dtype, device=DEV)
        v = buf[:, 2:2 + h]
    else:
        buf = torch.full((t * h * (d + 1) + 1,), float("nan"), dtype=x.dtype, device=DEV)
        v = buf[1:].view(t, h, d + 1)[..., :d]
    v.copy_(x)
    return v


NORMS = [  # tokens, q heads, k heads, dim, rot, interleaved, dtype, layout
    (1, 32, 8, 128, 128, False, BF16, "packed"), (12, 32, 8, 128, 128, False, F16, "own"), (300, 8, 2, 128, 128, True, BF16, "packed"),
    (5, 3, 1, 64, 64, False, F16, "own"), (7, 5, 5, 96, 36, True, F32, "own"), (9, 4, 4, 80, 40, False, BF16, "own"),
    (11, 2, 1, 100, 50, False, F16, "packed"), (11, 2, 1, 100, 50, False, F32, "own"), (3, 4, 2, 256, 64, False, F32, "packed"),
    (3, 4, 2, 256, 256, True, BF16, "own"), (4, 6, 2, 192, 98, False, BF16, "own"), (17, 1, 1, 72, 18, False, F16, "own"),
    (6, 2, 2, 32, 32, False, F32, "own"), (6, 9, 0, 128, 0, False, BF16, "own"), (2, 0, 3, 64, 2, False, F32, "own"),
    (5, 2, 1, 1, 0, False, F32, "own"), (5, 2, 1, 7, 6, False, F16, "own"), (4, 2, 1, 255, 254, True, BF16, "own"),
    (8, 3, 2, 128, 128, False, BF16, "odd"), (8, 3, 2, 128, 96, True, F16, "odd"), (8, 3, 2, 66, 30, False, F32, "odd"),
    (0, 4, 2, 64, 64, False, F16, "own"), (5000, 2, 1, 64, 64, False, BF16, "own"), (2, 300, 7, 128, 64, False, F16, "own"),
]


def norm_inputs(case, seed=1):
    t, hq, hk, d, rot, inter, dt, layout = case
    g = gen(seed)
    x = [torch.randn(t, h, d, generator=g).mul_(torch.exp(torch.randn(1, h, 1, generator=g))).to(dt) for h in (hq, hk)]
    w = [(1.0 + 0.3 * torch.randn(d, generator=g)).to(dt) for _ in range(2)]
    dy = [torch.randn(t, h, d, generator=g).to(dt) for h in (hq, hk)]
    pos = torch.randint(0, 1 << 20, (t,), generator=g)
    return x, w, dy, pos, R.frequencies(rot)


@pytest.mark.parametrize("case", NORMS, ids=str)
def test_qk_norm_rope(case):
    say(case)
    t, hq, hk, d, rot, inter, dt, layout = case
    x, w, dy, pos, freq = norm_inputs(case)
    q, k = (place(y, layout) for y in x)
    pos_d, freq_d = pos.to(DEV), freq.to(DEV)
    wd = [y.to(DEV) for y in w]
    out = rl.red_qk_norm_rope(q, k, pos_d, freq_d, wd[0], wd[1], eps=1e-6, interleaved=inter)
    for got, y, weight in zip(out, x, w):
        close("weights", got, *R.qk_norm_rope(y, weight, pos, freq, 1e-6, inter), dt, NORM_STEPS)
    out = rl.red_qk_norm_rope(q, k, pos_d, freq_d, eps=0.25, interleaved=inter, q_out=q, k_out=k)  # in place, no weights
    assert out[0].data_ptr() == q.data_ptr()
    for got, y in zip((q, k), x):
        close("in place", got, *R.qk_norm_rope(y, None, pos, freq, 0.25, inter), dt, NORM_STEPS)


@pytest.mark.parametrize("case", NORMS, ids=str)
def test_qk_norm_rope_backward(case):
    say(case)
    t, hq, hk, d, rot, inter, dt, layout = case
    x, w, dy, pos, freq = norm_inputs(case, 2)
    q, k = (place(y, layout) for y in x)
    dq, dk = (place(y, layout) for y in dy)
    got = rl.red_qk_norm_rope_backward(dq, dk, q, k, pos.to(DEV), freq.to(DEV), w[0].to(DEV), w[1].to(DEV), eps=1e-6,
                                       interleaved=inter)
    again = rl.red_qk_norm_rope_backward(dq, dk, q, k, pos.to(DEV), freq.to(DEV), w[0].to(DEV), w[1].to(DEV), eps=1e-6,
                                         interleaved=inter)
    for a, b in zip(got, again):
        assert torch.equal(a, b)
    for i in range(2):
        dx, size, dw, dsize = R.qk_norm_rope_backward(dy[i], x[i], w[i], pos, freq, 1e-6, inter)
        close("dx", got[i], dx, size, dt, BACK_STEPS)
        # at most 200 more additions on any path (a wave's rows), the rest in float64
        close("dw", got[2 + i], dw, dsize, F32, BACK_STEPS + 200)


def test_qk_norm_rope_backward_against_differences():
    case = (6, 3, 2, 48, 32, False, F32, "own")
    x, w, dy, pos, freq = norm_inputs(case, 3)
    got = rl.red_qk_norm_rope_backward(dy[0].to(DEV), dy[1].to(DEV), x[0].to(DEV), x[1].to(DEV), pos.to(DEV), freq.to(DEV),
                                       w[0].to(DEV), w[1].to(DEV))
    g = gen(4)
    h = 1e-5
    for i in range(2):
        for of in range(2):     # along x, along w
            ins = [x[i].double(), w[i].double()]
            v = torch.randn(ins[of].shape, generator=g, dtype=torch.float64)
            loss = []
            for s in (h, -h):
                moved = list(ins)
                moved[of] = ins[of] + s * v
                loss.append((R.qk_norm_rope(moved[0], moved[1], pos, freq, 1e-6, False)[0] * dy[i].double()).sum())
            want = (loss[0] - loss[1]) / (2 * h)
            grad = got[i if of == 0 else 2 + i].cpu().double()
            _, size, _, dsize = R.qk_norm_rope_backward(dy[i], x[i], w[i], pos, freq, 1e-6, False)
            allowed = (BACK_STEPS + 1) * U * ((size if of == 0 else dsize) * v.abs()).sum() + 1e-7 * want.abs() + 1e-6
            assert abs((grad * v).sum() - want) <= allowed, (i, of)


def test_qk_norm_rope_zero_rows_and_infinities():
    x = torch.zeros(4, 2, 64, dtype=F16)
    x[1, 0, 3] = float("inf")
    x[2, 1, 5] = float("nan")
    out, _ = rl.red_qk_norm_rope(x.to(DEV), x.to(DEV), torch.zeros(4, dtype=torch.int64, device=DEV), R.frequencies(64).to(DEV))
    out = out.cpu()
    assert torch.equal(out[0], torch.zeros(2, 64, dtype=F16)) and torch.equal(out[1, 1], torch.zeros(64, dtype=F16))
    assert out[1, 0, 3].isnan() and out[2, 1].isnan().all() and torch.equal(out[3], torch.zeros(2, 64, dtype=F16))


# ---------------------------------------------------------------------------
# The paged cache
# ---------------------------------------------------------------------------
CACHES = [  # tokens, heads, dim, places, pages, dtype, cache, layout of the tokens, layout of the cache
    (1, 8, 128, 16, 3, BF16, I8, "packed", "own"), (20, 8, 128, 16, 4, BF16, E4M3, "packed", "own"),
    (300, 2, 80, 24, 20, F16, I8, "own", "own"), (7, 3, 64, 1, 11, F16, E4M3, "own", "places first"),
    (33, 1, 256, 8, 9, BF16, I8, "own", "places first"), (65, 4, 112, 128, 1, F16, F16, "packed", "own"),
    (65, 4, 96, 32, 3, BF16, BF16, "own", "places first"), (40, 2, 192, 64, 2, BF16, E4M3, "own", "own"),
    (9, 2, 1, 4, 5, BF16, I8, "own", "own"), (9, 2, 7, 4, 5, F16, E4M3, "own", "own"), (9, 3, 100, 4, 5, F16, F16, "own", "own"),
    (9, 3, 255, 4, 5, BF16, I8, "own", "own"), (12, 2, 128, 8, 4, BF16, I8, "odd", "own"), (12, 2, 128, 8, 4, F16, F16, "own", "odd"),
    (12, 2, 64, 8, 4, F16, E4M3, "own", "odd"), (0, 2, 64, 8, 4, F16, I8, "own", "own"), (4000, 2, 64, 16, 300, BF16, I8, "own", "own"),
]


def empty_cache(pages, heads, places, dim, kind, layout, g):
    def one(shape, dt):
        raw = torch.randint(0, 100, (math.prod(shape) + 1,), generator=g, dtype=torch.int32)
        raw = raw.to(torch.int8).view(dt) if dt in (I8, E4M3) else raw.to(dt)
        raw = raw.to(DEV)
        return (raw[1:] if layout == "odd" and dt != F32 else raw[:-1]).view(shape)
    if layout == "places first":
        return [one((pages, places, heads, dim), kind).transpose(1, 2) for _ in range(2)], \
               [one((pages, places, heads), F32).transpose(1, 2) for _ in range(2)]
    return [one((pages, heads, places, dim), kind) for _ in range(2)], [one((pages, heads, places), F32) for _ in range(2)]


def bits(x):
    return x.view(torch.int8) if x.element_size() == 1 else x.view(torch.int16) if x.element_size() == 2 else x.view(torch.int32)


@pytest.mark.parametrize("case", CACHES, ids=str)
def test_cache_write_and_read(case):
    say(case)
    t, heads, dim, places, pages, dt, kind, layout, cache_layout = case
    g = gen(5)
    x = [torch.randn(t, heads, dim, generator=g).mul_(torch.exp(3 * torch.randn(t, heads, 1, generator=g))).to(dt) for _ in range(2)]
    if t >= 7 and dim > 1:
        x[0][0] = 0.0
        x[0][1, 0, 1] = float("inf")
        x[1][2, 0, 0] = float("nan")
        x[1][3, 0] *= float(torch.finfo(dt).tiny)          # far below 1, subnormals among them
        x[0][4, 0, 1:] = 0.0
    slots = torch.randperm(pages * places, generator=g)[:t]
    skipped = torch.zeros(t, dtype=torch.bool)
    if t >= 7:
        slots[5], slots[6] = -1, pages * places
        skipped[5] = skipped[6] = True
    pg, sc = empty_cache(pages, heads, places, dim, kind, cache_layout, g)
    before = [y.clone() for y in pg + sc]
    scaled = kind in R.TOP
    kw = dict(k_scales=sc[0], v_scales=sc[1]) if scaled else {}
    kv = [place(y, layout) for y in x]
    assert rl.red_cache_write(kv[0], kv[1], slots.to(DEV), pg[0], pg[1], **kw) is None
    back = rl.red_cache_read(pg[0], pg[1], slots.to(DEV), dt, **kw)
    page, at = (slots // places)[~skipped].to(DEV), (slots % places)[~skipped].to(DEV)
    keep = (~skipped).nonzero()[:, 0]
    for i in range(2):
        y = x[i][keep]
        got = bits(pg[i])[page, :, at]
        assert not bits(back[i])[skipped.to(DEV)].any()
        if not scaled:
            assert torch.equal(got.cpu(), bits(y)) and torch.equal(bits(back[i]).cpu()[keep], bits(y))
        else:
            top = y.float().abs().amax(-1)
            scale = sc[i][page, :, at].cpu()
            want = top / R.TOP[kind]
            assert torch.equal(scale.nan_to_num(-1.0, -2.0), want.nan_to_num(-1.0, -2.0))
            code = got.view(kind).cpu().float()
            fine = top.isfinite() & (top > 0)
            assert not code[~fine].any()
            unit = y[fine].double() / top[fine].double()[..., None] * R.TOP[kind]
            # half a step of the codes, and the roundings of M / top and of the product
            allowed = R.code_step(unit, kind) / 2 + 2.5 * U * unit.abs()
            assert ((code[fine].double() - unit).abs() <= allowed).all()
            # back: one product and one rounding
            again = (code * scale[..., None]).to(dt)
            both = torch.isnan(again) & torch.isnan(back[i].cpu()[keep])
            assert (both | (again == back[i].cpu()[keep])).all()
            assert back[i].cpu()[keep][~top.isfinite()].isnan().all()
    # nothing else changed
    for now, was in zip(pg + (sc if scaled else []), before):
        now, was = bits(now).clone(), bits(was)
        now[page, :, at] = was[page, :, at]
        assert torch.equal(now, was)


def test_python_refusals():
    q, k = torch.zeros(3, 4, 64, device=DEV), torch.zeros(3, 2, 64, device=DEV)
    pos, freq = torch.zeros(3, dtype=torch.int64, device=DEV), R.frequencies(64).to(DEV)
    f = rl.red_qk_norm_rope
    for args, kw, error in (((q.cpu(), k, pos, freq), {}, TypeError), ((q.double(), k, pos, freq), {}, TypeError),
                            ((q, k.half(), pos, freq), {}, TypeError), ((q, k[:2], pos, freq), {}, ValueError),
                            ((q, k, pos.int(), freq), {}, TypeError), ((q, k, pos[:2], freq), {}, ValueError),
                            ((q[0], k, pos, freq), {}, ValueError), ((q.transpose(1, 2), k, pos, freq), {}, ValueError),
                            ((q, k, pos, freq), dict(q_weight=torch.ones(63, device=DEV)), ValueError),
                            ((q, k, pos, torch.ones(33, device=DEV)), {}, rl.RedError),
                            ((q, k, pos, freq), dict(eps=-1.0), rl.RedError)):
        with pytest.raises(error):
            f(*args, **kw)
    pg = torch.zeros(2, 2, 4, 64, dtype=I8, device=DEV)
    sc = torch.zeros(2, 2, 4, device=DEV)
    kv, slots = torch.zeros(3, 2, 64, dtype=F16, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV)
    w = rl.red_cache_write
    for args, kw, error in (((kv, kv, slots, pg, pg), {}, ValueError), ((kv, kv, slots, pg, pg), dict(k_scales=sc), ValueError),
                            ((kv, kv, slots, pg.half(), pg.half()), dict(k_scales=sc, v_scales=sc), ValueError),
                            ((kv.float(), kv.float(), slots, pg, pg), dict(k_scales=sc, v_scales=sc), TypeError),
                            ((kv[:2], kv[:2], slots, pg, pg), dict(k_scales=sc, v_scales=sc), ValueError),
                            ((kv, kv, slots.int(), pg, pg), dict(k_scales=sc, v_scales=sc), TypeError),
                            ((kv.bfloat16(), kv.bfloat16(), slots, pg.half(), pg.half()), {}, rl.RedError)):
        with pytest.raises(error):
            w(*args, **kw)
    with pytest.raises(TypeError):
        rl.red_cache_read(pg, pg, slots, F32, k_scales=sc, v_scales=sc)
