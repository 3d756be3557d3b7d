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


@pytest.mark.parametrize("kind", [I8, E4M3, F16])
def test_cache_without_pages(kind):
    pg = torch.empty(0, 2, 4, 64, dtype=kind, device=DEV)
    sc = dict(k_scales=torch.empty(0, 2, 4, device=DEV), v_scales=torch.empty(0, 2, 4, device=DEV)) if kind in R.TOP else {}
    slots = torch.tensor([0, -1, 5], device=DEV)
    kv = torch.ones(3, 2, 64, dtype=F16, device=DEV)
    rl.red_cache_write(kv, kv, slots, pg, pg, **sc)
    for x in rl.red_cache_read(pg, pg, slots, F16, k_out=kv, **sc):
        assert x.shape == (3, 2, 64) and not x.any()
    table, lens = torch.zeros(1, 3, dtype=torch.int32, device=DEV), torch.tensor([7], dtype=torch.int32, device=DEV)
    out, lse = rl.red_tree_attention(torch.ones(1, 2, 2, 64, dtype=F16, device=DEV), pg, pg, table, lens, 1.0, **sc)
    assert not out.any() and (lse == -math.inf).all()


# ---------------------------------------------------------------------------
# Attention over the cache
# ---------------------------------------------------------------------------
ATTEND = [  # lens, nodes, q heads, kv heads, dim, places, tree, counts, dtype, cache, cache layout
    ([300], 1, 4, 1, 128, 16, False, None, F16, F16, "own"), ([1], 1, 2, 2, 64, 1, False, None, BF16, BF16, "own"),
    ([0, 5, 130], 4, 4, 2, 64, 24, True, [4, 0, 3], BF16, I8, "own"), ([127, 128, 129, 1000], 8, 8, 2, 128, 64, True, [8, 5, 8, 1], BF16, I8, "own"),
    ([500, 20], 64, 2, 1, 80, 8, True, [64, 33], F16, E4M3, "own"), ([77, 640], 63, 8, 1, 128, 32, True, None, BF16, BF16, "own"),
    ([64, 1, 2], 17, 6, 2, 96, 16, True, None, F16, I8, "places first"), ([900], 5, 3, 3, 256, 24, False, None, F16, F16, "own"),
    ([333], 40, 4, 1, 256, 128, True, None, BF16, E4M3, "own"), ([258, 31], 3, 8, 1, 192, 16, True, None, BF16, I8, "own"),
    ([200], 33, 2, 1, 192, 16, False, [20], F16, F16, "places first"), ([100, 0], 2, 16, 2, 16, 8, True, None, F16, I8, "own"),
    ([90], 9, 4, 1, 112, 1, True, None, BF16, E4M3, "own"), ([0], 64, 8, 1, 48, 128, True, None, BF16, BF16, "own"),
    ([0, 0], 1, 1, 1, 64, 16, False, [0, 1], F16, F16, "own"), ([2500, 3, 1700], 2, 4, 2, 64, 16, True, None, F16, E4M3, "own"),
    ([700, 1400] * 32, 1, 8, 8, 64, 32, False, None, BF16, I8, "own"), ([260, 1100] * 4, 64, 8, 4, 64, 64, True, None, F16, F16, "own"),
]


def attend_inputs(case, seed, scale_of_v=1.0):
    lens, nodes, hq, hk, dim, places, tree, counts, dt, kind, layout = case
    g = gen(seed)
    b = len(lens)
    per = -(-(max(lens) + nodes) // places) + 1
    pages = b * per + 2
    pg, sc = empty_cache(pages, hk, places, dim, kind, layout, g)
    for i in range(2):
        x = torch.randn(pages, hk, places, dim, generator=g)
        if kind == I8:
            pg[i].copy_((x * 36).clamp(-127, 127).round().to(I8))
        elif kind == E4M3:
            pg[i].view(I8).copy_((x * 120).clamp(-448, 448).to(E4M3).view(I8))
        else:
            pg[i].copy_(x.to(kind))
        sc[i].copy_((0.5 + torch.rand(pages, hk, places, generator=g)) / (36 if kind == I8 else 120) * (scale_of_v if i else 1.0))
    table = (torch.randperm(pages - 2, generator=g)[:b * per] + 1).to(torch.int32).view(b, per)
    q = (1.5 * torch.randn(b, nodes, hq, dim, generator=g)).to(dt)
    mask = None
    if tree:
        mask = torch.zeros(b, nodes, dtype=torch.int64)
        for i in range(b):
            for j in range(nodes):
                parent = int(torch.randint(-1, j, (1,), generator=g)) if j else -1
                word = ((int(mask[i, parent]) & (2 ** 64 - 1)) if parent >= 0 else 0) | 1 << j
                mask[i, j] = word - 2 ** 64 if word >= 2 ** 63 else word
    return pg, sc, table, q, mask


def check_attend(case, pg, sc, table, q, mask, scale, out, lse, pages_ok=None):
    lens, nodes, hq, hk, dim, places, tree, counts, dt, kind, layout = case
    group, scaled = hq // hk, kind in R.TOP
    hp = R.step(F16 if scaled else dt)
    code = [(p.view(I8).cpu().view(E4M3) if kind == E4M3 else p.cpu()).float() for p in pg]
    c = [s.cpu() if scaled else torch.ones(code[0].shape[:3]) for s in sc]
    out, lse = out.cpu().double(), lse.cpu().double()
    assert not out[~lse.isfinite() & (lse < 0)].any()
    for b, n in enumerate(lens):
        count = nodes if counts is None else counts[b]
        total = n + count
        seen = R.visible(n, nodes, mask[b] if tree else None, count, total).repeat_interleave(group, 0)
        t = torch.arange(total)
        page, at = table[b, t // places].long().cpu(), t % places
        ok = (page >= 0) & (page < code[0].shape[0])
        page = torch.where(ok, page, 0)
        for h in range(hk):
            k, v = (torch.where(ok[:, None], x[page, h, at], 0.0) for x in code)
            kc, vc = (torch.where(ok, x[page, h, at], 1.0) for x in c)
            rows = q[b, :, h * group:(h + 1) * group].reshape(nodes * group, dim)
            want, wlse, weights, size = R.tree_attention(rows, k.double() * kc.double()[:, None], v.double() * vc.double()[:, None], seen, scale)
            got = out[b, :, h * group:(h + 1) * group].reshape(nodes * group, dim)
            glse = lse[b, :, h * group:(h + 1) * group].reshape(-1)
            for i in range(nodes * group):
                if not seen[i].any():
                    assert glse[i] == -math.inf and not got[i].any(), (b, h, i)
                    continue
                p, vs, cs = weights[i][:, None], v[seen[i]].double(), vc[seen[i]].double()[:, None]
                es = (dim + 8) * U * size[i] + 16 * U * (1 + cs.log2().abs().max())
                terms = (p * cs * vs).nan_to_num(0.0, 0.0, 0.0)
                # rounded exponentials: 3.5 half steps of the root of the sum of
                # squares (6 standard deviations), and half the spacing of
                # subnormals where P is float16; then float32 sums
                sub = 2.0 ** -25 * (p * cs).max() * vs.nan_to_num(0.0, 0.0, 0.0).square().sum(0).sqrt() * 3.5
                allowed = (R.step(dt) * want[i].abs() + 3.5 * hp * terms.square().sum(0).sqrt() + sub +
                           ((len(p) + 32) * U + 2 * es) * terms.abs().sum(0) + R.tiny(dt))
                same = (got[i] == want[i]) | (got[i].isnan() & want[i].isnan())
                assert (same | ((got[i] - want[i]).abs() <= allowed)).all(), (b, h, i, (got[i] - want[i]).abs().max())
                assert abs(glse[i] - wlse[i]) <= es + (len(p) + 32) * U + 4 * U * wlse[i].abs(), (b, h, i, glse[i], wlse[i])


def attend(case, pg, sc, table, q, mask, scale, **kw):
    lens, counts, kind = case[0], case[7], case[9]
    if kind in R.TOP:
        kw.update(k_scales=sc[0], v_scales=sc[1])
    return rl.red_tree_attention(q.to(DEV) if q.device.type == "cpu" else q, pg[0], pg[1], table.to(DEV),
                                 torch.tensor(lens, dtype=torch.int32, device=DEV), scale,
                                 tree_mask=mask.to(DEV) if mask is not None else None,
                                 node_count=torch.tensor(counts, dtype=torch.int32, device=DEV) if counts is not None else None, **kw)


@pytest.mark.parametrize("case", ATTEND, ids=str)
def test_tree_attention(case):
    say(case)
    pg, sc, table, q, mask = attend_inputs(case, 11)
    scale = case[4] ** -0.5
    out, lse = attend(case, pg, sc, table, q, mask, scale, max_len=max(case[0]) + case[1])
    check_attend(case, pg, sc, table, q, mask, scale, out, lse)
    again = attend(case, pg, sc, table, q, mask, scale, max_len=max(case[0]) + case[1])
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("kind", [None, I8, E4M3], ids=str)
@pytest.mark.parametrize("dim", [48, 96, 112, 176])
@pytest.mark.parametrize("nodes, hq, hk", [(8, 4, 2), (17, 2, 2), (8, 4, 1), (33, 1, 1), (32, 4, 2), (13, 5, 1)])
def test_tree_attention_rows(nodes, hq, hk, dim, kind):
    """Numbers of rows (16, 17, 32, 33, 64, 65) and heads on both sides of the
    borders between the ways to share them among waves."""
    dt = F16 if (nodes + dim) % 2 else BF16
    case = ([70, 333], nodes, hq, hk, dim, 16, True, [nodes, max(nodes - 3, 1)], dt, kind or dt, "own")
    say(case)
    pg, sc, table, q, mask = attend_inputs(case, 17)
    out, lse = attend(case, pg, sc, table, q, mask, dim ** -0.5)
    check_attend(case, pg, sc, table, q, mask, dim ** -0.5, out, lse)


@pytest.mark.parametrize("kind", [None, I8, E4M3], ids=str)
@pytest.mark.parametrize("nodes, hq, hk, dim", [(4, 4, 2, 64), (3, 4, 1, 256), (9, 6, 2, 96), (8, 4, 1, 128), (33, 2, 2, 80),
                                                (24, 4, 1, 128), (33, 4, 2, 64), (33, 2, 1, 192), (8, 3, 1, 208)])
def test_tree_attention_shared_out(nodes, hq, hk, dim, kind):
    """Tiles of a few long sequences shared out over all blocks, with pieces to
    join, for every number of rows, head and cache type."""
    dt = BF16 if (nodes + dim // 16) % 2 else F16
    case = ([1500, 2100, 40], nodes, hq, hk, dim, 32, True, [nodes, nodes - 1, nodes], dt, kind or dt, "own")
    say(case)
    pg, sc, table, q, mask = attend_inputs(case, 18)
    out, lse = attend(case, pg, sc, table, q, mask, dim ** -0.5)
    check_attend(case, pg, sc, table, q, mask, dim ** -0.5, out, lse)


@pytest.mark.parametrize("case", [ATTEND[3], ATTEND[5], ATTEND[15]], ids=str)
@pytest.mark.parametrize("scale_of_v, scale", [(1e-20, 0.3), (1e15, -0.1), (1.0, 0.0)])
def test_tree_attention_scales(case, scale_of_v, scale):
    say(case, scale_of_v, scale)
    if case[3] is F16 and case[9] is E4M3 or case[8] is F16:
        scale_of_v = min(max(scale_of_v, 1e-3), 10.0)      # the output has to be in range
    pg, sc, table, q, mask = attend_inputs(case, 12, scale_of_v)
    out, lse = attend(case, pg, sc, table, q, mask, scale)
    check_attend(case, pg, sc, table, q, mask, scale, out, lse)


@pytest.mark.parametrize("case", [
    ([150, 40], 8, 4, 2, 64, 16, True, [8, 6], F16, F16, "own"), ([150, 40], 8, 4, 2, 64, 16, True, [8, 6], BF16, E4M3, "own"),
    ([150, 40], 64, 2, 1, 128, 16, True, [60, 50], BF16, BF16, "own"), ([150, 40], 8, 4, 2, 64, 16, True, [8, 6], F16, I8, "own")], ids=str)
def test_tree_attention_masked_places(case):
    """Infinities and NaN where no row, or not every row, sees them."""
    say(case)
    lens, nodes, counts, places, kind = case[0], case[1], case[7], case[5], case[9]
    pg, sc, table, q, mask = attend_inputs(case, 13)
    used = torch.zeros(pg[0].shape[0], places, dtype=torch.bool)
    for b, n in enumerate(lens):
        t = torch.arange(n + counts[b])
        used[table[b, t // places].long(), t % places] = True
    free = (~used).nonzero().to(DEV)
    bad = float("nan")
    for x in pg:
        if kind == I8:
            x[free[:, 0], :, free[:, 1]] = 127
        elif kind == E4M3:
            x.view(I8)[free[:, 0], :, free[:, 1]] = 127            # NaN
        else:
            x[free[:, 0], :, free[:, 1]] = bad
    for x in sc:
        x[free[:, 0], :, free[:, 1]] = bad
    for b, n in enumerate(lens):                       # two nodes hold what is no number
        for j, value in ((1, float("inf")), (3, bad)):
            p, at = int(table[b, (n + j) // places]), (n + j) % places
            if kind == I8:
                sc[0][p, :, at] = sc[1][p, :, at] = bad
            elif kind == E4M3:
                pg[0].view(I8)[p, :, at, 2] = 127
                pg[1].view(I8)[p, 0, at, 5] = 127
            else:
                pg[0][p, :, at, 2] = 1.0
                pg[1][p, 0, at, 5] = value
                pg[1][p, 0, at, 6] = -value
    scale = 0.2
    out, lse = attend(case, pg, sc, table, q, mask, scale)
    if kind in (F16, BF16):
        check_attend(case, pg, sc, table, q, mask, scale, out, lse)
        return
    # rows that see one of them are NaN, the others as if those nodes were not there
    clean = [x.clone() for x in sc]
    cp = [x.clone() for x in pg]
    for b, n in enumerate(lens):
        for j in (1, 3):
            p, at = int(table[b, (n + j) // places]), (n + j) % places
            for x in clean:
                x[p, :, at] = 1.0
            for x in cp:
                x.view(I8)[p, :, at] = 0
    sees = ((mask >> 1 | mask >> 3) & 1).bool()
    for b in range(len(lens)):
        for i in range(counts[b]):
            if sees[b, i]:
                assert lse[b, i].isnan().all() and out[b, i].isnan().all()
    out, lse = out.cpu(), lse.cpu()
    ref_out, ref_lse = (x.cpu() for x in attend(case, cp, clean, table, q, mask, scale))
    blind = ~sees & (torch.arange(nodes) < torch.tensor(counts)[:, None])
    assert torch.equal(out[blind], ref_out[blind]) and torch.equal(lse[blind], ref_lse[blind])


def test_tree_attention_bad_pages_and_lengths():
    """Pages outside the cache read as zeros; lengths beyond max_len or the
    table are cut; q and out with strides of their own."""
    case = ([200, 50], 4, 4, 2, 64, 16, False, None, F16, F16, "own")
    pg, sc, table, q, mask = attend_inputs(case, 14)
    table[0, 3], table[0, 7], table[1, 1] = -5, 1 << 30, pg[0].shape[0]
    out, lse = attend(case, pg, sc, table, q, mask, 0.125)
    check_attend(case, pg, sc, table, q, mask, 0.125, out, lse)
    cut = ([100, 50], *case[1:])
    a = attend(([100, 50], *case[1:7], [0, 4], *case[8:]), pg, sc, table, q, mask, 0.125)
    wide = torch.zeros(2, 4, 9, 64, dtype=F16, device=DEV)[:, :, 3:7]
    wide.copy_(q)
    to = torch.full((2, 4, 6, 64), 7.0, dtype=F16, device=DEV)
    b = attend(cut, pg, sc, table, wide, mask, 0.125, out=to[:, :, 1:5])
    assert torch.equal(a[0][1], b[0][1]) and torch.equal(a[1][1], b[1][1]) and (to[:, :, 0] == 7).all() and (to[:, :, 5] == 7).all()
    # 100 tokens of the 200 (and none of the nodes) where max_len is 100
    full = ([100], 4, 4, 2, 64, 16, True, [4], F16, F16, "own")
    none = torch.zeros(1, 4, dtype=torch.int64)
    c = attend(([200], 4, 4, 2, 64, 16, False, None, F16, F16, "own"), pg, sc, table[:1], q[:1], None, 0.125, max_len=100)
    d = attend(full, pg, sc, table[:1], q[:1], none, 0.125)
    assert torch.equal(c[0], d[0]) and torch.equal(c[1], d[1])
    e = attend(([200], 4, 4, 2, 64, 16, False, None, F16, F16, "own"), pg, sc, table[:1, :0], q[:1], None, 0.125)
    assert not e[0].any() and (e[1] == -math.inf).all()


# ---------------------------------------------------------------------------
# Verification of drafted tokens
# ---------------------------------------------------------------------------
VERIFY = [  # batch, drafts, vocab, dtype, given, sharpness, layout
    (1, 4, 32000, F32, True, 2.5, "own"), (5, 6, 1001, F32, True, 2.5, "own"), (3, 10, 4099, BF16, True, 2.0, "own"),
    (7, 3, 2048, F16, False, 4.0, "own"), (2, 70, 300, F32, True, 1.0, "own"), (9, 1, 1, F32, True, 1.0, "own"),
    (4, 0, 777, F32, False, 1.0, "own"), (33, 5, 131071, F32, True, 2.5, "own"), (6, 4, 5003, BF16, False, 6.0, "odd"),
    (6, 4, 1023, F32, True, 2.5, "odd"), (300, 2, 50, F16, True, 2.0, "own"), (0, 2, 50, F16, True, 2.0, "own"),
]


def verify_inputs(case, seed=21):
    b, k, v, dt, given, sharp, layout = case
    g = gen(seed)
    x = sharp * torch.randn(b, k + 1, v, generator=g)
    p = torch.softmax(x, -1).to(dt)
    y = x[:, :k] + 0.7 * torch.randn(b, k, v, generator=g)
    q = torch.softmax(y, -1).to(dt) if given else None
    drafted = (y + torch.empty(b, k, v).exponential_(generator=g).log_().neg_()).argmax(-1) if k else torch.zeros(b, 0, dtype=torch.int64)
    if not given and k:
        drafted = p[:, :k].float().argmax(-1)          # certain drafts: the likeliest
    u, r = torch.rand(b, k, generator=g), torch.rand(b, generator=g)
    count = torch.randint(0, k + 1, (b,), generator=g).to(torch.int32)
    return p, q, drafted, u, r, count


def check_verify(p, q, drafted, u, r, count, got, layout="own"):
    n, tokens = (x.cpu() for x in got)
    for b in range(p.shape[0]):
        want = R.verify(p[b], q[b] if q is not None else None, drafted[b], u[b], r[b], int(count[b]) if count is not None else p.shape[1] - 1)
        assert (int(n[b]), tokens[b].tolist()) == want, b


@pytest.mark.parametrize("case", VERIFY, ids=str)
def test_verify_drafts(case):
    say(case)
    p, q, drafted, u, r, count = verify_inputs(case)
    pd, qd = (place(x, case[6]) if x is not None else None for x in (p, q))
    d = [x.to(DEV) for x in (drafted, u, r, count)]
    check_verify(p, q, drafted, u, r, count, rl.red_verify_drafts(pd, qd, *d[:3], draft_count=d[3]))
    check_verify(p, q, drafted, u, r, None, rl.red_verify_drafts(pd, qd, *d[:3]))
    low, high = torch.zeros_like(d[2]), torch.full_like(d[2], 1 - 2.0 ** -24)
    for e in (low, high):
        check_verify(p, q, drafted, u, e.cpu(), count, rl.red_verify_drafts(pd, qd, *d[:2], e, draft_count=d[3]))


def test_verify_drafts_corners():
    b, k, v = 8, 3, 3001
    p, q, drafted, u, r, _ = verify_inputs((b, k, v, F32, True, 2.0, "own"), 22)
    q[0], u[0] = p[0, :k], 1.0                          # refused, and p - q is 0 everywhere
    drafted[1] = torch.tensor([-1, 5, 6])               # outside the vocabulary
    drafted[2, 1] = v
    u[2, 0] = 0.0
    p[3] = 0.0                                          # no weight at all
    p[4, 0, 7] = float("nan")
    drafted[4, 0], u[4, 0] = 7, 0.5
    p[5, :, : v // 2] = 0.0                             # weight in the second half only
    r[5], r[6] = 0.0, 1.0                               # r of 1: the last of positive weight
    u[6], p[6, 0, -5:] = 1.0, 0.0
    u[7] = 0.0                                          # everything accepted
    p[7] = p[7] + 1e-30
    args = [x.to(DEV) for x in (p, q, drafted, u, r)]
    got = rl.red_verify_drafts(*args)
    check_verify(p, q, drafted, u, r, None, got)
    assert int(got[0][0]) == 0 and int(got[0][7]) == k and got[1][3].tolist() == [-1] * 4 and int(got[1][4, 0]) == -1
    # counts out of range are cut
    count = torch.tensor([-4, 0, 99, 2, 2, 1, 3, 1 << 30], dtype=torch.int32)
    got = rl.red_verify_drafts(*args, draft_count=count.to(DEV))
    check_verify(p, q, drafted, u, r, count.clamp(0, k), got)


@pytest.mark.parametrize("case", [(130, 2, 20011, F16, True, 2.0, "own"), (256, 1, 60001, BF16, False, 6.0, "odd"),
                                  (520, 3, 999, F32, True, 2.0, "own"), (1, 2, 16384, F32, True, 2.0, "own")], ids=str)
def test_verify_drafts_many(case):
    """Rows and numbers of sequences at the borders between one launch and two."""
    test_verify_drafts(case)


@pytest.mark.parametrize("dt", [F32, F16, BF16])
def test_verify_drafts_wide(dt):
    """A vocabulary that is widened by tokens of no weight (and takes two
    launches for it) has the same tokens drawn, in the corners too."""
    b, k, v, wide = 7, 3, 3001, 40003
    p, q, drafted, u, r, _ = verify_inputs((b, k, v, dt, True, 2.0, "own"), 23)
    q[0], u[0] = p[0, :k], 1.0                          # refused, and p - q is 0 everywhere
    p[1] = 0.0                                          # no weight at all
    p[2, 0, 7] = float("nan")
    drafted[2, 0], u[2, 0] = 7, 0.5
    r[3], r[4] = 0.0, 1.0
    u[5] = 0.0                                          # everything accepted
    p[5] = p[5] + 1e-4
    args = [x.to(DEV) for x in (p, q, drafted, u, r)]
    wider = [torch.nn.functional.pad(x, (0, wide - v)) for x in args[:2]] + args[2:]
    got, want = rl.red_verify_drafts(*args), rl.red_verify_drafts(*wider)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check_verify(p, q, drafted, u, r, None, got)


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
    probs, d = torch.zeros(2, 4, 9, device=DEV), torch.zeros(2, 3, dtype=torch.int64, device=DEV)
    u, r = torch.zeros(2, 3, device=DEV), torch.zeros(2, device=DEV)
    f = rl.red_verify_drafts
    for args, kw, error in (((probs.double(), None, d, u, r), {}, TypeError), ((probs[0], None, d, u, r), {}, ValueError),
                            ((probs, probs, d, u, r), {}, ValueError), ((probs, None, d.int(), u, r), {}, TypeError),
                            ((probs, None, d, u[:, :2], r), {}, ValueError), ((probs, None, d, u, u), {}, ValueError),
                            ((probs, None, d, u, r), dict(draft_count=d[:, 0]), TypeError),
                            ((probs, probs[:, :3].half(), d, u, r), {}, TypeError)):
        with pytest.raises(error):
            f(*args, **kw)
    q4, pg = torch.zeros(2, 3, 4, 64, dtype=F16, device=DEV), torch.zeros(5, 2, 8, 64, dtype=F16, device=DEV)
    table, lens = torch.zeros(2, 2, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    f = rl.red_tree_attention
    for args, kw, error in (((q4.float(), pg, pg, table, lens, 1.0), {}, TypeError), ((q4.bfloat16(), pg, pg, table, lens, 1.0), {}, rl.RedError),
                            ((q4[..., :32], pg, pg, table, lens, 1.0), {}, ValueError), ((q4, pg, pg, table.long(), lens, 1.0), {}, TypeError),
                            ((q4, pg, pg, table[:1], lens, 1.0), {}, ValueError), ((q4, pg, pg, table, lens[:1], 1.0), {}, ValueError),
                            ((q4, pg, pg[:, :1], table, lens, 1.0), {}, ValueError), ((q4, pg, pg, table, lens, float("nan")), {}, rl.RedError),
                            ((q4[:, :, :3], pg, pg, table, lens, 1.0), {}, rl.RedError),
                            ((q4, pg, pg, table, lens, 1.0), dict(tree_mask=torch.zeros(2, 4, dtype=torch.int64, device=DEV)), ValueError),
                            ((q4, pg, pg, table, lens, 1.0), dict(node_count=lens.long()), TypeError),
                            ((q4, pg, pg, table, lens, 1.0), dict(out=q4), rl.RedError),
                            ((torch.zeros(2, 65, 4, 64, dtype=F16, device=DEV), pg, pg, table, lens, 1.0), {}, rl.RedError)):
        with pytest.raises(error):
            f(*args, **kw)
