"""The serving step's operators on the GPU, against their definitions on the CPU.

Whole numbers are equal: slots, pages, tokens. Where a token or a kept set hangs
on a sum of weights, the reference says how close a border came to its target,
relative to the largest weight; the library's sums are whole multiples of
2^(ceil(log2 vocab) - 62) of that, each weight off by half of one and by the
2^-50 of a float64 exponential. In rows that are cut into chunks of 8192, sums
are those of bins: a weight counts in them as a whole number of 2^-36 of its
bin's upper edge, which is at most 2^(1/8) of it, so it is off by 1.1 * 2^-37,
by 2^-41 of the polynomial, and by as much again by the largest weight's own
number, which all are divided by: less than 2^-35 of itself in all. The sum of a
bin of a chunk is cut off to a whole unit: 512 bins of vocab / 8192 chunks and of
at most 2 vocab 2^-62 each are off by vocab^2 2^-65, which is at most vocab *
2^-45. So a border further away than sum * 2^-35 + vocab * 2^-45 + 2^-40 is
certain. Cases that come closer by chance are not (none is known to); those that
meet a border exactly do so with whole weights, which are exact."""
import math
import random
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected only with a GPU
    pytest.skip("no GPU visible", allow_module_level=True)

import decode_reference as R  # noqa: E402
import serve_reference as S  # noqa: E402
import reduction_libred_amd as rl  # noqa: E402

DEV = torch.device("cuda:0")
F32, F16, BF16, I8, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.int8, torch.float8_e4m3fn
I32 = torch.int32


def say(*a):
    print("[serve-gpu]", *a, flush=True)
    sys.stdout.flush()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def ints(x):
    return torch.tensor(x, dtype=I32, device=DEV)


# ---------------------------------------------------------------------------
# Slots
# ---------------------------------------------------------------------------
def plan_case(seed, batch, cols, places, longest, high, done=0.3, free=1.0, room=7, odd=False):
    rng = random.Random(seed)
    lens = [rng.randint(0, longest) for _ in range(batch)]
    held = [min(cols, -(-n // places) + (rng.randint(0, 2) if rng.random() < 0.3 else 0)) for n in lens]
    gone = [int(rng.random() < done) * rng.choice([1, -5, 7]) for _ in range(batch)]
    lens = [0 if g and rng.random() < 0.8 else n for n, g in zip(lens, gone)]
    counts = [rng.randint(0, high) for _ in range(batch)]
    if odd:      # numbers out of range, which the call bounds
        lens = [n if rng.random() < 0.8 else -rng.randint(1, 1 << 31) for n in lens]
        counts = [n if rng.random() < 0.8 else -rng.randint(1, 1 << 31) for n in counts]
    pages = sum(held) + rng.randint(0, 3) + int(free * sum(-(-(max(a, 0) + max(b, 0)) // places) for a, b in zip(lens, counts)))
    order = rng.sample(range(pages), pages)
    table, at = [], 0
    for h in held:
        table.append(order[at:at + h] + [-7] * (cols - h))
        at += h
    height = pages - at if free >= 1 else int(free * (pages - at))
    stack = order[at:at + height] + [-1] * (pages - height)
    if odd:
        held = [h if rng.random() < 0.8 or h not in (0, cols) else (-3 if h == 0 else cols + 5) for h in held]
    total = sum(max(c, 0) for c in counts)
    return dict(lens=lens, counts=counts, done=gone, table=table, held=held, stack=stack, height=height, places=places,
                tokens=max(0, total + room))


def run_plan(c, view=False, **kw):
    batch, cols = len(c["lens"]), len(c["table"][0]) if c["table"] else 3
    table = ints(c["table"]).view(batch, cols)
    if view:      # rows of a wider table
        wide = torch.full((batch, cols + 5), -99, dtype=I32, device=DEV)
        wide[:, 2:2 + cols] = table
        table = wide[:, 2:2 + cols]
    held, stack, height = ints(c["held"]), ints(c["stack"]), ints([c["height"]])
    done = None if c["done"] is None else ints(c["done"])
    slots, pos, starts, granted = rl.red_plan_slots(ints(c["lens"]), ints(c["counts"]), table, held, stack, height, c["places"], c["tokens"],
                                                    done=done, **kw)
    torch.cuda.synchronize()
    if view:
        assert (wide[:, :2] == -99).all() and (wide[:, 2 + cols:] == -99).all()
    return dict(slots=slots, pos=pos, starts=starts, granted=granted, table=table, held=held, stack=stack, height=height)


def check_plan(c, got):
    want = S.plan_slots(**c)
    for k, w in want.items():
        assert got[k].tolist() == w, k


PLANS = [  # batch, columns, places, longest, high, done, free, room, odd
    (1, 4, 16, 0, 1, 0.0, 1.0, 0, False), (1, 9, 1, 5, 3, 0.0, 1.0, 2, False), (3, 70, 16, 1000, 9, 0.3, 1.0, 7, False),
    (32, 70, 16, 1000, 9, 0.2, 1.0, 7, False), (64, 70, 7, 400, 40, 0.5, 0.6, 0, False), (65, 40, 24, 700, 300, 0.4, 0.4, 3, True),
    (200, 12, 64, 500, 300, 1.0, 1.0, 7, False), (255, 30, 8, 200, 60, 0.5, 0.0, 9, True), (1024, 6, 16, 60, 20, 0.3, 0.7, 1, True),
    (1025, 6, 16, 60, 20, 0.3, 1.0, 1, False), (3000, 5, 3, 9, 6, 0.5, 0.8, 30, True), (50, 30, 16, 300, 200, 0.3, 1.0, -900, False),
    (256, 40, 64, 1000, 1000, 0.5, 1.0, 100, False), (300, 100, 16, 900, 500, 0.6, 0.7, -5000, True), (7, 300, 1, 40, 250, 0.4, 1.0, 0, False),
    (5000, 8, 16, 40, 60, 0.5, 0.9, 11, True), (4, 3, 1 << 20, 2000000, 5, 0.3, 1.0, 5, False),
]


@pytest.mark.parametrize("view", [False, True])
@pytest.mark.parametrize("case", PLANS, ids=str)
def test_plan_slots(case, view):
    say("plan", case, view)
    c = plan_case(hash(case) % 1000, *case)
    check_plan(c, run_plan(c, view))
    c["done"] = None
    check_plan(c, run_plan(c, view))


def test_plan_slots_of_nothing():
    c = dict(lens=[], counts=[], done=[], table=[], held=[], stack=[4, -1], height=1, places=16, tokens=5)
    got = run_plan(c)
    assert got["slots"].tolist() == [-1] * 5 and got["pos"].tolist() == [0] * 5 and got["starts"].tolist() == [0]
    assert got["stack"].tolist() == [4, -1] and got["height"].tolist() == [1]
    c = dict(lens=[5, 0], counts=[0, 0], done=[0, 1], table=[[3, -1], [2, 1]], held=[1, 2], stack=[0, -1, -1], height=1, places=16, tokens=0)
    check_plan(c, run_plan(c))


def test_plan_slots_far_positions():
    """Positions beyond 2^31 and slots beyond 2^32."""
    c = dict(lens=[(1 << 31) - 3, 5], counts=[9, 2], done=[0, 0], table=[[1] * 4096, [(1 << 31) - 9] * 4096], held=[4096, 1], stack=[-1] * 4,
             height=0, places=1 << 20, tokens=11)
    check_plan(c, run_plan(c))


def test_plan_slots_step_after_step():
    """Sequences that grow, end and are followed by others: no page is ever in two places, and all come back."""
    rng = random.Random(3)
    batch, cols, places, pages = 40, 20, 4, 300
    table, held = torch.full((batch, cols), -1, dtype=I32, device=DEV), torch.zeros(batch, dtype=I32, device=DEV)
    stack, height = torch.randperm(pages, generator=gen(1)).to(I32).to(DEV), ints([pages])
    lens = [0] * batch
    for step in range(25):
        done = [int(rng.random() < 0.15 and step > 0) for _ in range(batch)]
        lens = [0 if d else n for n, d in zip(lens, done)]
        counts = [rng.randint(0, 9) for _ in range(batch)]
        *_, granted = rl.red_plan_slots(ints(lens), ints(counts), table, held, stack, height, places, 400, done=ints(done))
        lens = [n + g for n, g in zip(lens, granted.tolist())]
        used = [p for row, h in zip(table.tolist(), held.tolist()) for p in row[:h]]
        free = stack.tolist()[:int(height)]
        assert sorted(used + free) == list(range(pages))
        assert stack.tolist()[int(height):] == [-1] * (pages - int(height))
        assert all(h >= -(-n // places) for h, n in zip(held.tolist(), lens))
    rl.red_plan_slots(ints([0] * batch), ints([0] * batch), table, held, stack, height, places, 0, done=ints([1] * batch))
    assert sorted(stack.tolist()) == list(range(pages)) and int(height) == pages and held.sum() == 0


# ---------------------------------------------------------------------------
# Bounds and selection
# ---------------------------------------------------------------------------
def make_cache(g, kind, pages, heads, places, dim, layout):
    """Keys and their scales, on the CPU and on the GPU: 'own', pages of (places, heads) rows ('tokens'), or rows at odd addresses ('odd')."""
    x = torch.randn(pages, heads, places, dim, generator=g) * torch.exp(torch.randn(1, heads, 1, dim, generator=g))
    scales = None
    if kind is I8:
        x, scales = (x * 30).clamp(-127, 127).round().to(I8), torch.rand(pages, heads, places, generator=g) / 30
    elif kind is E4M3:
        x, scales = (x * 60).clamp(-448, 448).to(E4M3), torch.rand(pages, heads, places, generator=g) / 60
    else:
        x = x.to(kind)
    if layout == "own":
        d = x.to(DEV)
    elif layout == "tokens":
        d = x.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
    else:
        buf = torch.zeros(pages * heads * places * (dim + 1) + 1, dtype=x.dtype, device=DEV)
        d = buf[1:].view(pages, heads, places, dim + 1)[..., :dim]
        d.copy_(x)
    return x, scales, d, None if scales is None else scales.to(DEV)


def bounds_like(x, dtype, layout, fill=5.0):
    shape = (x.shape[0], x.shape[1], x.shape[3])
    if layout == "odd":
        return torch.full((shape[0] * shape[1] * (shape[2] + 1) + 1,), fill, dtype=dtype, device=DEV)[1:].view(*shape[:2], -1)[..., :shape[2]]
    return torch.full((shape[0], shape[1] + 1, shape[2]), fill, dtype=dtype, device=DEV)[:, 1:]


BOUNDS = [  # batch, heads, places, dim, lens up to, columns, first, most, type of bounds, of cache, layout
    (1, 1, 1, 16, 1, 1, False, None, BF16, BF16, "own"), (3, 8, 16, 128, 200, 13, False, None, BF16, BF16, "own"),
    (3, 8, 16, 128, 200, 13, True, 2, F16, F16, "own"), (4, 2, 7, 64, 90, 13, True, None, BF16, I8, "own"),
    (4, 3, 24, 80, 300, 13, True, 3, F16, E4M3, "tokens"), (2, 2, 64, 256, 500, 8, False, 5, F16, I8, "own"),
    (2, 2, 32, 192, 300, 10, False, None, BF16, E4M3, "own"), (5, 3, 5, 7, 40, 8, True, None, F16, F16, "own"),
    (3, 2, 16, 100, 100, 7, False, None, BF16, I8, "own"), (2, 4, 16, 128, 90, 6, True, None, BF16, BF16, "odd"),
    (2, 2, 128, 96, 700, 6, False, None, BF16, BF16, "tokens"), (3, 2, 16, 255, 90, 6, False, None, F16, E4M3, "odd"),
    (2, 1, 130, 8, 500, 4, False, None, BF16, BF16, "own"), (200, 1, 4, 32, 20, 5, True, 1, BF16, BF16, "own"),
]


@pytest.mark.parametrize("case", BOUNDS, ids=str)
def test_page_bounds(case):
    say("bounds", case)
    batch, heads, places, dim, longest, cols, from_first, most, dtype, kind, layout = case
    g = gen(sum(case[:6]))
    pages = batch * cols + 3
    x, scales, d, ds = make_cache(g, kind, pages, heads, places, dim, layout)
    if kind in (F16, BF16, E4M3):      # a NaN among them, and a page of nothing else in one element
        x.view(torch.int8 if kind is E4M3 else torch.int16)[::3, 0, 0, ::2] = 0x7F if kind is E4M3 else 0x7FFF
        x.view(torch.int8 if kind is E4M3 else torch.int16)[1, :, :, 3] = 0x7F if kind is E4M3 else 0x7FFF
        d.view(torch.int8 if kind is E4M3 else torch.int16).copy_(x.view(torch.int8 if kind is E4M3 else torch.int16))
    table = torch.randperm(pages, generator=g)[:batch * cols].view(batch, cols).to(I32)
    table[0, -1] = -1
    if cols > 2:
        table[-1, 1] = pages
    lens = torch.randint(0, longest + 1, (batch,), generator=g, dtype=I32)
    lens[0] = longest
    first = torch.randint(-3, longest + 1, (batch,), generator=g, dtype=I32) if from_first else None
    lo, hi = (bounds_like(x, dtype, layout) for _ in range(2))
    base = lo.cpu()
    rl.red_page_bounds(d, table.to(DEV), lens.to(DEV), lo, hi, first=None if first is None else first.to(DEV), most=most, k_scales=ds)
    want = S.page_bounds(x, scales, table, lens.tolist(), base, base, None if first is None else first.tolist(), cols if most is None else most)
    for got, w in zip((lo, hi), want):
        assert torch.equal(got.cpu(), w)


def test_page_bounds_of_a_sequence_without_tokens_or_pages():
    x = torch.zeros(2, 1, 4, 16, dtype=BF16, device=DEV)
    lo, hi = torch.ones(2, 1, 16, dtype=BF16, device=DEV), torch.ones(2, 1, 16, dtype=BF16, device=DEV)
    table = ints([[0, 1]])
    for lens, first, most in ((0, None, None), (-5, None, None), (8, 8, None), (8, None, 0)):
        rl.red_page_bounds(x, table, ints([lens]), lo, hi, first=None if first is None else ints([first]), most=most)
        assert (lo == 1).all() and (hi == 1).all()
    rl.red_page_bounds(x, table, ints([1000]), lo, hi)
    assert (lo == 0).all() and (hi == 0).all()
    rl.red_page_bounds(x[:0], table, ints([8]), lo[:0], hi[:0])
    rl.red_page_bounds(x, table[:0], ints([])[:0], lo, hi)


SELECTS = [  # batch, nodes, q heads, kv heads, dim, places, columns, budget, first, last, dtype, whole numbers, layout
    (1, 1, 1, 1, 16, 1, 9, 4, 0, 0, BF16, False, "own"), (3, 1, 8, 2, 128, 16, 100, 20, 1, 1, BF16, False, "own"),
    (3, 1, 8, 8, 64, 16, 100, 20, 1, 2, F16, False, "own"), (2, 8, 32, 8, 128, 32, 200, 64, 1, 2, BF16, False, "own"),
    (4, 1, 4, 2, 80, 24, 300, 17, 2, 3, F16, False, "own"), (2, 64, 16, 2, 64, 8, 130, 30, 3, 4, BF16, False, "own"),
    (2, 3, 6, 3, 100, 5, 90, 16, 0, 4, F16, False, "own"), (2, 1, 4, 4, 256, 16, 70, 9, 0, 0, BF16, False, "odd"),
    (2, 2, 4, 2, 7, 16, 70, 9, 1, 1, F16, False, "own"), (2, 1, 8, 2, 192, 64, 1500, 1100, 1, 1, BF16, False, "own"),
    (1, 1, 8, 2, 128, 16, 3000, 100, 1, 1, F16, False, "own"), (3, 1, 4, 2, 16, 16, 300, 40, 1, 1, BF16, True, "own"),
    (2, 4, 4, 1, 32, 4, 2100, 1030, 2, 2, F16, True, "own"), (5, 1, 2, 2, 64, 16, 40, 40, 1, 1, BF16, False, "own"),
]


@pytest.mark.parametrize("case", SELECTS, ids=str)
def test_select_pages(case):
    """Scores are float64 sums of exact products; those of whole numbers are
    exact, so pages of equal scores are many and the lower ones win."""
    say("select", case)
    batch, nodes, q_heads, heads, dim, places, cols, budget, first, last, dtype, whole, layout = case
    g = gen(sum(case[:10]))
    pages = batch * cols + 5
    a, b = (torch.randint(-1, 2, (pages, heads, dim), generator=g).float() if whole else torch.randn(pages, heads, dim, generator=g) for _ in range(2))
    lo, hi = torch.minimum(a, b).to(dtype), torch.maximum(a, b).to(dtype)
    q = (torch.randint(-2, 3, (batch, nodes, q_heads, dim), generator=g).float() if whole else torch.randn(batch, nodes, q_heads, dim, generator=g)).to(dtype)
    table = torch.randperm(pages, generator=g)[:batch * cols].view(batch, cols).to(I32)
    if cols > 50:
        table[0, 20], table[0, 30] = -1, pages         # not in the cache: below all others
        hi[int(table[-1, 25]), 0, 0] = math.nan          # no number: as those
    lens = torch.randint(0, cols * places - nodes + 1, (batch,), generator=g, dtype=I32)
    lens[0] = cols * places - nodes
    if batch > 2:
        lens[1], lens[2] = 0, (budget + 1) * places + 1 if (budget + 1) * places + 1 + nodes <= cols * places else 3
    counts = torch.randint(0, nodes + 1, (batch,), generator=g, dtype=I32)
    counts[0] = nodes
    for count, max_len in ((None, None), (counts, None), (counts, cols * places - 2 * places - 1)):
        dl, dh = (bounds_like(torch.empty(pages, heads, 1, dim), dtype, layout) for _ in range(2))
        dl.copy_(lo), dh.copy_(hi)
        n = counts.tolist() if count is not None else [nodes] * batch
        sel, left = rl.red_select_pages(q.to(DEV), dl, dh, table.to(DEV), lens.to(DEV), places, budget, first=first, last=last, max_len=max_len,
                                        node_count=None if count is None else count.to(DEV))
        sel, left = sel.cpu(), left.tolist()
        for i in range(batch):
            chosen, rest = S.select_pages(q[i], lo, hi, table[i], int(lens[i]), n[i], places, budget, first, last,
                                          cols * places if max_len is None else max_len)
            assert left[i] == rest
            for h in range(heads):
                assert sel[i, h].tolist() == [int(table[i, p]) for p in chosen[h]] + [-1] * (budget - len(chosen[h])), (i, h)


@pytest.mark.parametrize("value", [0.0, 1.0, -2.5, math.nan, math.inf])
def test_select_pages_of_equal_scores(value):
    """Nothing tells the pages apart: the lower ones are selected."""
    q = torch.full((2, 1, 4, 32), value, dtype=BF16, device=DEV)
    lo = torch.ones(90, 2, 32, dtype=BF16, device=DEV)
    table = torch.arange(90, dtype=I32, device=DEV).flip(0).view(2, 45)
    sel, left = rl.red_select_pages(q, lo, lo.clone(), table, ints([700, 719]), 16, 10, first=0, last=1)
    for b, tail in enumerate(([42, 43], [43, 44])):
        assert sel[b].tolist() == [[int(table[b, p]) for p in [*range(8), *tail]]] * 2
    assert left.tolist() == [700 - 16 * 34, 719 - 16 * 35]


def test_select_pages_queries_with_strides():
    g = gen(4)
    q = torch.randn(2, 3, 12, 64, generator=g).to(BF16)
    lo = torch.randn(50, 2, 64, generator=g).to(BF16)
    hi = lo + 1
    table = torch.randperm(50, generator=g)[:40].view(2, 20).to(I32)
    args = (lo.to(DEV), hi.to(DEV), table.to(DEV), ints([300, 200]), 16, 9)
    want = rl.red_select_pages(q[:, :, 2:10].contiguous().to(DEV), *args)
    got = rl.red_select_pages(q.to(DEV)[:, :, 2:10], *args)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    one = rl.red_select_pages(q[:, :1, 2:10].to(DEV).expand(-1, 3, -1, -1), *args)      # every node the same query: strides of 0
    same = rl.red_select_pages(q[:, :1, 2:10].contiguous().to(DEV).repeat(1, 3, 1, 1), *args)
    assert torch.equal(one[0], same[0])


# ---------------------------------------------------------------------------
# Attention over selected pages
# ---------------------------------------------------------------------------
SPARSE = [  # batch, nodes, group, kv heads, dim, places, columns, budget, type, cache
    (2, 1, 4, 2, 128, 16, 60, 12, BF16, BF16), (2, 1, 1, 3, 64, 16, 60, 40, F16, F16), (2, 5, 4, 2, 80, 24, 30, 9, BF16, I8),
    (1, 33, 2, 2, 64, 8, 40, 12, F16, E4M3), (3, 1, 8, 1, 256, 32, 20, 6, BF16, BF16), (2, 64, 8, 2, 128, 32, 30, 9, BF16, I8),
]


@pytest.mark.parametrize("case", SPARSE, ids=str)
def test_sparse_attention(case):
    """Pages of its own for every kv head: against a cache in which each kv head
    has its selected pages one after the other. The tolerances are those of
    red_tree_attention: a rounding of the exponentials and of the output, each of
    the output's type, against the largest value a row sees."""
    say("sparse", case)
    batch, nodes, group, heads, dim, places, cols, budget, dtype, kind = case
    g = gen(sum(case[:8]))
    pages = batch * cols
    k, ks, dk, dks = make_cache(g, kind, pages, heads, places, dim, "own")
    v, vs, dv, dvs = make_cache(g, kind, pages, heads, places, dim, "own")
    q = torch.randn(batch, nodes, group * heads, dim, generator=g).to(dtype)
    lens = torch.randint(0, budget * places - nodes + 1, (batch,), generator=g, dtype=I32)
    lens[0] = budget * places - nodes
    table = torch.stack([torch.stack([torch.randperm(pages, generator=g)[:budget] for _ in range(heads)]) for _ in range(batch)]).to(I32)
    scale = dim ** -0.5
    out, lse = rl.red_sparse_attention(q.to(DEV), dk, dv, table.to(DEV), lens.to(DEV), scale, k_scales=dks, v_scales=dvs)
    out, lse = out.cpu().double(), lse.cpu().double()
    value = [x.double() if s is None else x.double() * s[..., None].double() for x, s in ((k, ks), (v, vs))]
    for b in range(batch):
        seen = R.visible(int(lens[b]), nodes, None, nodes, budget * places).repeat_interleave(group, 0)
        for h in range(heads):
            kk, vv = (x[table[b, h].long(), h].reshape(-1, dim) for x in value)
            want, want_lse, _, size = R.tree_attention(q[b, :, h * group:(h + 1) * group].reshape(-1, dim), kk, vv, seen, scale)
            got = out[b, :, h * group:(h + 1) * group].reshape(-1, dim)
            top = torch.stack([vv[s].abs().amax(0) for s in seen])
            # scores: dim products and sums in float32 at most; exponentials and outputs: one rounding each
            of_scores = (dim + 8) * 2.0 ** -24 * size[:, None] + 2.0 ** -20
            step = R.step(F16 if kind in (I8, E4M3) else dtype)
            assert ((got - want).abs() <= R.step(dtype) * want.abs() + (2 * of_scores + step) * top + R.tiny(dtype)).all()
            assert ((lse[b, :, h * group:(h + 1) * group].reshape(-1) - want_lse).abs() <= of_scores[:, 0] + 2.0 ** -22 * want_lse.abs()).all()


@pytest.mark.parametrize("kind", [BF16, I8])
@pytest.mark.parametrize("lens", [[5, 900], [0, 31], [3000, 2000]])
def test_sparse_attention_with_one_table_for_all_heads(kind, lens):
    """The same bits as red_tree_attention; heads a stride of 0 apart, or copied."""
    g = gen(7)
    _, _, k, ks = make_cache(g, kind, 400, 4, 16, 128, "own")
    _, _, v, vs = make_cache(g, kind, 400, 4, 16, 128, "own")
    q = torch.randn(2, 3, 16, 128, generator=g).to(BF16).to(DEV)
    table = torch.randperm(400, generator=g).view(2, 200).to(I32).to(DEV)
    want = rl.red_tree_attention(q, k, v, table, ints(lens), 0.1, k_scales=ks, v_scales=vs)
    for t in (table[:, None].expand(-1, 4, -1), table[:, None].repeat(1, 4, 1)):
        got = rl.red_sparse_attention(q, k, v, t, ints(lens), 0.1, k_scales=ks, v_scales=vs)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_sparse_attention_pages_outside_and_masked_nan():
    """Pages of -1 read as zeros, for the head that has them; a NaN of a node that a row does not see stays out, for the head whose page holds it."""
    g = gen(8)
    _, _, k, _ = make_cache(g, BF16, 8, 2, 16, 64, "own")
    _, _, v, _ = make_cache(g, BF16, 8, 2, 16, 64, "own")
    v[5, 1, 3] = math.nan         # token 19 of head 1, node 1
    q = torch.randn(1, 2, 2, 64, generator=g).to(BF16).to(DEV)
    table = ints([[[0, 1], [4, 5]]])
    out, _ = rl.red_sparse_attention(q, k, v, table, ints([18]), 0.125)
    assert not out[0, 0].isnan().any() and not out[0, 1, 0].isnan().any() and out[0, 1, 1].isnan().all()
    table = ints([[[-1, -1], [2, 3]]])
    out, lse = rl.red_sparse_attention(q, k, v, table, ints([30]), 0.125)
    assert (out[0, :, 0] == 0).all() and torch.allclose(lse[0, :, 0].cpu(), torch.log(torch.tensor([31.0, 32.0])))
    assert (out[0, :, 1] != 0).any()


# ---------------------------------------------------------------------------
# Sampling
# ---------------------------------------------------------------------------
def certain(weights):
    """weights: those of the whole row, the largest 1."""
    return float(np.sum(weights)) * 2.0 ** -35 + len(weights) * 2.0 ** -45 + 2.0 ** -40


def check_sample(x, r, t=None, k=None, p=None, m=None, probs=F32, exact=False):
    """x (batch, steps, vocab) on the CPU, settings lists of `batch`."""
    batch, steps, vocab = x.shape
    settings = dict(temperature=t, top_p=p, min_p=m)
    settings = {n: None if y is None else torch.tensor(y, dtype=F32, device=DEV) for n, y in settings.items()}
    settings["top_k"] = None if k is None else ints(k)
    tokens, given = rl.red_sample(x.to(DEV), r.to(DEV), probs=probs, **settings)
    again, none = rl.red_sample(x.to(DEV), r.to(DEV), **settings)
    assert none is None and torch.equal(tokens, again)
    tokens, got = tokens.tolist(), given.cpu().double().numpy()
    wide = x.double().numpy()
    for b in range(batch):
        of = {n: None if y is None else float(y[b]) for n, y in settings.items()}
        for s in range(steps):
            kept, near = S.sample(wide[b, s], of["temperature"], None if k is None else k[b], of["top_p"], of["min_p"])
            every, _ = S.sample(wide[b, s], of["temperature"])
            sure = exact or near > certain(every)
            assert sure, "a border closer to its target than sums of 64 bits tell"
            # weights below half a unit count as 0 where they are summed
            unit = 2.0 ** -min(51, 62 - math.ceil(math.log2(vocab)))
            token, close = S.token_of(np.where(kept < unit / 2, 0, kept), float(r[b, s]))
            assert exact or close > certain(every)
            assert tokens[b][s] == token, (b, s, tokens[b][s], token)
            want = (kept / kept.sum() if kept.sum() > 0 else kept).astype(np.float64)
            # one rounding to the type, one to float32, and the weights' own
            allowed = want * (R.step(probs) + 2.0 ** -24 + 2.0 ** -30) + R.tiny(probs) + R.tiny(F32)
            assert (np.abs(got[b, s] - want) <= allowed).all(), (b, s, np.abs(got[b, s] - want).max())
            assert ((got[b, s] > 0) <= (want > 0)).all()


SAMPLES = [  # batch, steps, vocab, dtype, spread, k, p, m, masked, probs
    (1, 1, 1, F32, 1.0, None, True, True, 0.0, F32), (3, 1, 2, BF16, 1.0, 1, True, False, 0.0, F32), (2, 2, 7, F16, 2.0, 3, False, True, 0.0, BF16),
    (5, 1, 1000, F32, 2.0, 50, True, False, 0.0, F32), (4, 3, 1023, BF16, 2.0, None, True, True, 0.3, F16),
    (2, 1, 4096, F32, 3.0, 4000, True, True, 0.3, F32), (2, 1, 4097, F16, 3.0, None, True, False, 0.5, F32),
    (6, 1, 32000, F32, 2.5, 50, True, False, 0.0, F32), (3, 1, 32003, BF16, 2.5, 9000, True, False, 0.4, F32),
    (2, 2, 131071, F32, 1.0, None, True, False, 0.0, F32), (2, 1, 131071, BF16, 4.0, None, False, True, 0.4, BF16),
    (2, 1, 131072, F16, 0.1, 70000, True, True, 0.0, F32), (1, 1, 1 << 20, F32, 2.5, None, True, False, 0.2, F32),
    (1, 1, (1 << 20) - 5, BF16, 2.5, 1000, True, False, 0.0, F32), (300, 1, 513, F32, 2.0, 20, True, True, 0.1, F32),
    (3, 1, 20000, F32, 2.0, None, False, False, 0.1, F32), (3, 1, 8191, BF16, 1.0, 3000, True, True, 0.2, BF16),
    (3, 1, 8192, F32, 0.2, 5000, True, False, 0.0, F16), (3, 2, 8193, F16, 2.0, 4000, True, True, 0.1, F32), (9, 1, 6001, F32, 2.5, 70, True, False, 0.5, F32),
    (70, 1, 33000, F32, 2.0, None, True, False, 0.1, F32), (30, 2, 50001, BF16, 2.5, 400, True, True, 0.3, F16),
]


@pytest.mark.parametrize("case", SAMPLES, ids=str)
def test_sample(case):
    say("sample", case)
    batch, steps, vocab, dtype, spread, k, p, m, masked, probs = case
    g, rng = gen(vocab + batch), random.Random(vocab + batch)
    x = torch.randn(batch, steps, vocab, generator=g) * spread
    if masked:
        hidden = torch.rand(batch, steps, vocab, generator=g) < masked
        hidden[..., 0] = False
        x[hidden] = -math.inf
        if batch > 1:
            x[0][hidden[0]] = torch.finfo(dtype).min       # the other way of masking
    r = torch.rand(batch, steps, generator=g)
    check_sample(x.to(dtype), r, t=[rng.choice([0.0, 0.3, 0.7, 1.0, 1.9]) for _ in range(batch)],
                 k=None if k is None else [rng.choice([k, 0, 1, vocab, k // 2 + 1, -4, vocab + 9]) for _ in range(batch)],
                 p=[rng.uniform(0.3, 0.999) for _ in range(batch)] if p else None, m=[rng.uniform(0.0, 0.2) for _ in range(batch)] if m else None,
                 probs=probs)


@pytest.mark.parametrize("vocab", [5, 2049, 9001, 16001, 40000, 131071])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_of_equal_logits(vocab, dtype):
    """Whole rows of ties: weights are whole, sums exact, and the lower numbers are kept."""
    say("ties", vocab, dtype)
    x = torch.full((6, 1, vocab), -3.25).to(dtype)
    x[5, 0, ::2] = 2.0       # two values, the larger at the even numbers
    r = torch.tensor([0.0, 0.5, 0.999, 0.25, 1.0, 0.75])[:, None]
    check_sample(x, r, t=[1.0, 1.0, 2.0, 0.0, 1.0, 1e9], k=[0, vocab // 2 + 1, 1, 9, vocab, (vocab + 1) // 2 - 1], p=None, exact=True)
    # halves and quarters of the sum are met exactly
    check_sample(x[:5], r[:5], p=[0.5, 0.25, 0.0, 0.75, 1.0], exact=True)
    check_sample(x[:5], r[:5], k=[4, 4, 0, vocab, 2], p=[0.5, 0.25, 0.5, 0.75, 0.5], m=[1.0, 5.0, 0.5, 0.0, -1.0], exact=True)


@pytest.mark.parametrize("vocab", [100, 9000, 131071])
def test_sample_of_a_few_equal_logits_among_masked_ones(vocab):
    """What a grammar leaves: borders and draws at whole multiples of one weight."""
    x = torch.full((8, 1, vocab), -math.inf)
    x[:, 0, [3, 50, vocab // 2, vocab - 1]] = 7.3
    r = torch.tensor([0.0, 0.25, 0.5, 0.75, 0.2499, 0.99, 1.0, 0.5])[:, None]
    check_sample(x, r, exact=True)
    check_sample(x, r, p=[0.25, 0.5, 0.75, 0.5, 0.5001, 0.9, 0.0, 0.24], exact=True)
    check_sample(x, r, k=[1, 2, 3, 4, 5, 2, 3, 0], p=[0.5] * 8, m=[1.0] * 8, exact=True)
    x[:, 0, [5, 60]] = 7.3 - 60 * math.log(2)        # 2^-60 of the others: more than nothing, less than a unit
    check_sample(x, r[:6].repeat(2, 1)[:8], k=[5] * 8, exact=True)


@pytest.mark.parametrize("case", [(0.7, 900, 0.93, None), (1.3, 40, 0.2, 0.3), (1.0, 3000, 0.999, 0.001), (0.4, 20000, 0.95, None), (1.0, 5, 0.9999, 0.9),
                                  (2.0, 30000, None, None), (2.0, None, 0.5, 0.0001), (1.0, None, None, 0.02), (8.0, 15000, 0.5, 0.7),
                                  (30.0, 25000, 0.97, None), (0.01, None, 0.999999, 1e-30), (1e-4, 20, 0.9, None)], ids=str)
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_sample_filters_together(case, dtype):
    """Borders of one filter above, within and below those of the others, in bins of few and of most tokens."""
    t, k, p, m = case
    g = gen(77)
    x = torch.randn(3, 1, 32768, generator=g) * torch.tensor([1.0, 2.0, 4.0])[:, None, None] + torch.tensor([0.0, 30.0, -100.0])[:, None, None]
    x = x.to(dtype)
    check_sample(x, torch.rand(3, 1, generator=g), t=[t] * 3, k=None if k is None else [k] * 3, p=None if p is None else [p] * 3,
                 m=None if m is None else [m] * 3)


def test_sample_of_few_values_over_many_tokens():
    """More tokens in the border's bin, and of its value, than are gathered."""
    g = gen(5)
    x = torch.randint(0, 3, (4, 1, 100001), generator=g).float()
    r = torch.rand(4, 1, generator=g)
    check_sample(x, r, k=[20000, 50000, 90000, 100000])
    check_sample(x, r, p=[0.1, 0.61803, 0.8123, 0.97777])
    check_sample(x, r, t=[100.0, 3.0, 0.05, 0.001], k=[20000, 50000, 90000, 100000], p=[0.1, 0.61803, 0.8123, 0.97777])


def test_sample_corners():
    inf, nan = math.inf, math.nan
    rows = [[-inf, -inf, -inf, -inf], [nan, nan, nan, -inf], [nan, 1.0, 2.0, nan], [inf, 1.0, inf, 3.0], [inf, nan, -inf, inf],
            [-0.0, 0.0, -0.0, 0.0], [3e38, -3e38, 3e38, 0.0], [1.0, -inf, 1.0, -inf], [5.0, 5.0, 5.0, 5.0]]
    x = torch.tensor(rows)[:, None]
    n = len(rows)
    for r in (0.0, 0.3, 0.5, 0.75, 1.0, 7.0, nan, -1.0, inf):
        given = torch.full((n, 1), r)
        check_sample(x, given, exact=True)
        check_sample(x, given, t=[0.0] * n, exact=True)
        check_sample(x, given, k=[1, 2, 3, 3, 1, 3, 2, 3, 2], exact=True)
        check_sample(x, given, t=[inf] * n, exact=True)
        check_sample(x, given, t=[nan] * n, p=[nan] * n, m=[nan] * n, exact=True)
        check_sample(x, given, t=[-1.0] * n, exact=True)
        check_sample(x, given, t=[1e-45] * n, p=[0.5] * n, exact=True)
        check_sample(x, given, p=[0.0] * n, m=[1.0] * n, exact=True)
        check_sample(x, given, p=[-3.0] * n, m=[9.0] * n, exact=True)
    for dtype in (F16, BF16):
        check_sample(x.to(dtype), torch.full((n, 1), 0.6), m=[0.01] * n, probs=dtype, exact=True)


def test_sample_far_tails():
    """Weights down to 2^-1000 of the largest: kept by top-k, in the probabilities as far as their type goes."""
    x = (-torch.arange(3000.0) / 4)[None, None].repeat(3, 1, 1)
    check_sample(x, torch.tensor([[0.5], [0.999999], [1.0]]), k=[2999, 500, 100], exact=True)
    check_sample(x.flip(-1).contiguous(), torch.tensor([[0.5], [0.999999], [0.1]]), p=[0.9, 0.99, 0.5])


@pytest.mark.parametrize("power", [26, 27])
@pytest.mark.parametrize("sign", [1, -1])
def test_sample_of_large_logits(power, sign):
    """Eighths of powers of two of the weights whose numbers pass 2^26 and 2^27
    within the row, in other chunks than the largest logit's."""
    border = sign * round(2.0 ** power / (8 * math.log2(math.e)))
    x = torch.full((4, 1, 40000), float(border - 30))
    x[:, 0, ::9] = border - 4
    x[:, 0, 9000:9100] = border + 4
    x[:, 0, 20000:20007] = border - 1
    x[1, 0, :16384], x[2, 0, :24576] = border - 9, -torch.finfo(F32).max
    x[3, 0, 9000:9100], x[3, 0, 30000] = border - 6, border + 2
    r = torch.tensor([0.3, 0.999, 0.7, 0.05])[:, None]
    check_sample(x, r)
    check_sample(x, r, p=[0.99, 0.9995, 0.7, 0.6], k=[2000, 39000, 40000, 300])
    check_sample(x, r, t=[3.0] * 4, p=[0.99, 0.9995, 0.7, 0.6], m=[0.0, 0.001, 0.02, 0.3])


def test_sample_layouts():
    """Logits with strides, also 0; two and three dimensions; what is not asked for is not given."""
    g = gen(9)
    wide = torch.randn(4, 3, 1100, generator=g).to(BF16).to(DEV)
    r = torch.rand(4, 3, generator=g).to(DEV)
    t = torch.tensor([0.5, 1.0, 2.0, 0.0], device=DEV)
    want = rl.red_sample(wide[..., 5:1050].contiguous(), r, temperature=t, probs=F32)
    got = rl.red_sample(wide[..., 5:1050], r, temperature=t, probs=F32)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    one = rl.red_sample(wide[:, 1, 5:1050], r[:, 1].contiguous(), temperature=t, probs=F32)
    assert torch.equal(one[0], want[0][:, 1]) and torch.equal(one[1], want[1][:, 1])
    spread = rl.red_sample(wide[:1, :1, 5:1050].expand(4, 3, -1), r)
    assert torch.equal(spread[0], rl.red_sample(wide[:1, :1, 5:1050].repeat(4, 3, 1), r)[0])
    only = rl.red_sample(wide, probs=F16)
    assert only[0] is None and only[1].dtype is F16
    assert rl.red_sample(wide[:0], r[:0])[0].shape == (0, 3)
    none = rl.red_sample(wide[:, :0], r[:, :0], probs=F32)
    assert none[0].shape == (4, 0) and none[1].shape == (4, 0, 1100)


def test_sample_then_verification():
    """Filtered probabilities are those that red_verify_drafts takes: with target
    and draft alike every draft with weight is accepted for u below 1."""
    g = gen(10)
    x = (2 * torch.randn(5, 4, 3001, generator=g)).to(DEV)
    r = torch.rand(5, 4, generator=g).to(DEV)
    top = ints([20, 30, 0, 5, 1])
    tokens, p = rl.red_sample(x, r, top_k=top, probs=F32)
    q = p[:, :3].contiguous()
    n, got = rl.red_verify_drafts(p, q, tokens[:, :3].contiguous(), torch.full((5, 3), 0.99, device=DEV), r[:, 3].contiguous())
    assert (n == 3).all() and torch.equal(got[:, :3], tokens[:, :3])
    assert (p.gather(2, got[..., None]) > 0).all()


# ---------------------------------------------------------------------------
# Refusals of the binding
# ---------------------------------------------------------------------------
def test_binding_refuses():
    x = torch.zeros(2, 5, device=DEV)
    r = torch.zeros(2, device=DEV)
    with pytest.raises(TypeError):
        rl.red_sample(x.double(), r)
    with pytest.raises(TypeError):
        rl.red_sample(x.cpu(), r)
    with pytest.raises(ValueError):
        rl.red_sample(x.t(), torch.zeros(5, device=DEV))
    with pytest.raises(ValueError):
        rl.red_sample(x[0], r)
    with pytest.raises(ValueError):
        rl.red_sample(x, torch.zeros(3, device=DEV))
    with pytest.raises(TypeError):
        rl.red_sample(x, r, top_k=r)
    with pytest.raises(TypeError):
        rl.red_sample(x, r, probs=torch.int32)
    with pytest.raises(ValueError):
        rl.red_sample(x, r, temperature=torch.zeros(1, device=DEV))
    one = ints([1])
    with pytest.raises(ValueError):
        rl.red_plan_slots(one, ints([1, 2]), ints([[1]]), one, one, one, 16, 4)
    with pytest.raises(TypeError):
        rl.red_plan_slots(one, one.long(), ints([[1]]), one, one, one, 16, 4)
    with pytest.raises(ValueError):
        rl.red_plan_slots(one, one, ints([1]), one, one, one, 16, 4)
    with pytest.raises(ValueError):
        rl.red_plan_slots(one, one, ints([[1]]), one, one, one, 0, 4)
    with pytest.raises(ValueError):
        rl.red_plan_slots(one, one, ints([[1]]), one, one, one, 16, -4)
    with pytest.raises(rl.RedError):       # held is also an input
        rl.red_plan_slots(one, ints([2]), ints([[1]]), one, ints([3]), ints([1]), 16, 4)
    k = torch.zeros(4, 2, 16, 64, dtype=BF16, device=DEV)
    lo = torch.zeros(4, 2, 64, dtype=BF16, device=DEV)
    with pytest.raises(TypeError):
        rl.red_page_bounds(k, ints([[1]]), one, lo.half(), lo.half())
    with pytest.raises(ValueError):
        rl.red_page_bounds(k, ints([[1]]), one, lo[:3], lo[:3].clone())
    with pytest.raises(ValueError):
        rl.red_page_bounds(k, ints([[1]]), one, lo, lo.clone(), k_scales=torch.zeros(4, 2, 16, device=DEV))
    with pytest.raises(ValueError):
        rl.red_page_bounds(k.to(I8), ints([[1]]), one, lo, lo.clone())
    with pytest.raises(rl.RedError):
        rl.red_page_bounds(k, ints([[1]]), one, lo, lo)
    q = torch.zeros(1, 1, 4, 64, dtype=BF16, device=DEV)
    with pytest.raises(rl.RedError):       # no room for the pages that are always selected
        rl.red_select_pages(q, lo, lo, ints([[1, 2]]), one, 16, 3, first=1, last=1)
    with pytest.raises(ValueError):
        rl.red_select_pages(q, lo, lo, ints([[1, 2]]), one, 16, 9, first=-1)
    with pytest.raises(TypeError):
        rl.red_select_pages(q.half(), lo, lo, ints([[1, 2]]), one, 16, 9)
    with pytest.raises(ValueError):
        rl.red_sparse_attention(q, k, k, ints([[1, 2]]), one, 0.1)
    with pytest.raises(ValueError):
        rl.red_sparse_attention(q, k, k, ints([[[1, 2]]]), one, 0.1)
    with pytest.raises(ValueError):
        rl.red_tree_attention(q, k, k, ints([[[1, 2], [1, 2]]]), one, 0.1)
