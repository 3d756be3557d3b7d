"""Corners of the serving step's operators on the GPU: nothing to read, offsets
beyond 32 bits, more rows than one pass takes, shared pages, extreme temperatures."""
import math
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected only with a GPU
    pytest.skip("no GPU visible", allow_module_level=True)

import serve_reference as S  # noqa: E402
import reduction_libred_amd as rl  # noqa: E402
from test_serve_gpu import DEV, F16, F32, BF16, I8, I32, check_plan, check_sample, gen, ints, run_plan  # noqa: E402

FAR = (1 << 31) + 64


def say(*a):
    print("[serve-corners]", *a, flush=True)
    sys.stdout.flush()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("dim", [64, 7])
def test_selection_from_an_empty_cache(dtype, dim):
    """No page is in the cache, so all scores are NaN and the lower pages are selected; no bound is read."""
    say("empty cache", dtype, dim)
    none = torch.empty(0, 2, dim, dtype=dtype, device=DEV)
    q = torch.ones(2, 3, 4, dim, dtype=dtype, device=DEV)
    table = torch.arange(80, dtype=I32, device=DEV).view(2, 40)
    sel, left = rl.red_select_pages(q, none, none.clone(), table, ints([600, 30]), 16, 6)
    assert sel[0].tolist() == [[0, 1, 2, 3, 36, 37]] * 2 and sel[1].tolist() == [[40, 41, 42, -1, -1, -1]] * 2
    assert left.tolist() == [600 - 16 * 32, 30]


def test_selection_without_nodes_or_tokens():
    q = torch.ones(2, 0, 4, 64, dtype=BF16, device=DEV)
    lo = torch.zeros(5, 2, 64, dtype=BF16, device=DEV)
    table = torch.arange(40, dtype=I32, device=DEV).view(2, 20)
    sel, left = rl.red_select_pages(q, lo, lo.clone(), table, ints([300, 0]), 16, 6)
    assert (sel == -1).all() and left.tolist() == [0, 0]
    q = torch.ones(2, 2, 4, 64, dtype=BF16, device=DEV)
    sel, left = rl.red_select_pages(q, lo, lo.clone(), table, ints([-7, 0]), 16, 6)
    assert sel[0].tolist() == [[0, -1, -1, -1, -1, -1]] * 2 and left.tolist() == [0, 0]
    sel, left = rl.red_select_pages(q, lo, lo.clone(), table[:, :0], ints([300, 3]), 16, 6)
    assert (sel == -1).all()


@pytest.mark.parametrize("shift, pad", [(1, 0), (4, 0), (0, 1), (0, 4)])
def test_selection_by_queries_at_any_address(shift, pad):
    """Queries that begin or follow each other off the boundaries that wide loads need."""
    g = gen(9)
    lo = torch.randn(60, 2, 128, generator=g).to(BF16)
    hi = lo + 1
    q = torch.randn(2, 5, 6, 128, generator=g).to(BF16)
    table = torch.randperm(60, generator=g).view(2, 30).to(I32)
    buf = torch.zeros(2 * 5 * 6 * (128 + pad) + shift, dtype=BF16, device=DEV)
    d = buf[shift:].view(2, 5, 6, 128 + pad)[..., :128]
    d.copy_(q)
    sel, _ = rl.red_select_pages(d, lo.to(DEV), hi.to(DEV), table.to(DEV), ints([440, 333]), 16, 9)
    for b, n in enumerate((440, 333)):
        chosen, _ = S.select_pages(q[b], lo, hi, table[b], n, 5, 16, 9, 1, 1, 480)
        for h in range(2):
            assert sel[b, h].tolist() == [int(table[b, p]) for p in chosen[h]]


def test_slots_without_pages_or_sequences():
    say("no pages")
    c = dict(lens=[3, 0], counts=[1, 2], done=[0, 1], table=[[], []], held=[0, 4], stack=[], height=0, places=16, tokens=6)
    batch, none = 2, torch.empty(2, 0, dtype=I32, device=DEV)
    held, stack, height = ints(c["held"]), ints([])[:0], ints([5])
    slots, pos, starts, granted = rl.red_plan_slots(ints(c["lens"]), ints(c["counts"]), none, held, stack, height, 16, 6, done=ints(c["done"]))
    assert slots.tolist() == [-1] * 6 and pos.tolist() == [3, 0, 1, 0, 0, 0] and starts.tolist() == [0, 1, 3] and granted.tolist() == [0] * batch
    assert held.tolist() == [0, 0] and height.tolist() == [0]
    c = dict(lens=[], counts=[], done=None, table=[], held=[], stack=[4, -1], height=1, places=16, tokens=5000)
    got = run_plan(c)
    assert got["slots"].tolist() == [-1] * 5000 and got["starts"].tolist() == [0] and got["stack"].tolist() == [4, -1]


@pytest.mark.parametrize("height", [-5, 0, 3, 1000])
@pytest.mark.parametrize("room", [5, 3000, 9000])
def test_slots_with_a_height_out_of_range(height, room):
    """The height counts as 0 below, as the stack's size above; pages that the stack has no room for are dropped."""
    stack = list(range(100, 103)) + list(range(7))
    check_plan(dict(lens=[40, 3, 0], counts=[9, 2, 4], done=[1, 0, 0], table=[[11, 12, 13, 14]] + [[20, 21, 22, 23]] + [[30, 31, 32, 33]],
                    held=[4, 1, 0], stack=stack, height=height, places=16, tokens=room),
               run_plan(dict(lens=[40, 3, 0], counts=[9, 2, 4], done=[1, 0, 0], table=[[11, 12, 13, 14]] + [[20, 21, 22, 23]] + [[30, 31, 32, 33]],
                             held=[4, 1, 0], stack=stack, height=height, places=16, tokens=room)))


@pytest.mark.parametrize("total", [2047, 2048, 2049, 4097])
@pytest.mark.parametrize("places", [1, 16])
def test_slots_at_the_borders_between_launches(total, places):
    cols = -(-total // places)
    order = torch.randperm(3 * cols + 5, generator=gen(total)).tolist()
    c = dict(lens=[0, 5, 0], counts=[total - 40, 7, 33], done=[1, 0, 0], table=[order[:cols], order[cols:2 * cols], order[2 * cols:3 * cols]],
             held=[cols, min(cols, -(-5 // places)), 0], stack=order[3 * cols:] + [-1] * (3 * cols), height=5, places=places, tokens=total)
    check_plan(c, run_plan(c))


def test_bounds_of_shared_pages():
    """Pages that are whole in two sequences, and twice in one."""
    g = gen(6)
    k = torch.randn(9, 3, 16, 128, generator=g).to(BF16)
    table = torch.tensor([[1, 2, 3, 4], [1, 2, 5, 6], [7, 7, 7, 8]], dtype=I32)
    lens = torch.tensor([60, 55, 64], dtype=I32)
    lo, hi = (torch.full((9, 3, 128), 9.0, dtype=BF16, device=DEV) for _ in range(2))
    rl.red_page_bounds(k.to(DEV), table.to(DEV), lens.to(DEV), lo, hi)
    want = S.page_bounds(k, None, table, lens.tolist(), torch.full((9, 3, 128), 9.0, dtype=BF16), torch.full((9, 3, 128), 9.0, dtype=BF16), None, 4)
    assert torch.equal(lo.cpu(), want[0]) and torch.equal(hi.cpu(), want[1])


def test_pages_beyond_32_bit_offsets():
    """Elements of the cache, of the bounds and of the queries further than 2^31 from the first."""
    say("far pages")
    g = gen(7)
    x = torch.randint(-127, 128, (2, 2, 16, 64), generator=g, dtype=I32).to(I8)
    scales = torch.rand(2, 2, 16, generator=g)
    buf = torch.empty(FAR + 2 * 16 * 64, dtype=I8, device=DEV)
    k = buf.as_strided((2, 2, 16, 64), (FAR, 16 * 64, 64, 1))
    k.copy_(x)
    wide = [torch.empty(FAR + 2 * 64, dtype=BF16, device=DEV) for _ in range(2)]
    lo, hi = (w.as_strided((2, 2, 64), (FAR, 64, 1)) for w in wide)
    lo.zero_(), hi.zero_()
    table = torch.tensor([[1, 0]], dtype=I32)
    rl.red_page_bounds(k, table.to(DEV), ints([32]), lo, hi, k_scales=scales.to(DEV))
    want = S.page_bounds(x, scales, table, [32], torch.zeros(2, 2, 64, dtype=BF16), torch.zeros(2, 2, 64, dtype=BF16), None, 2)
    assert torch.equal(lo.cpu(), want[0]) and torch.equal(hi.cpu(), want[1])
    del buf, k
    q = torch.randn(2, 1, 4, 64, generator=g).to(BF16)
    far = torch.empty(FAR + 4 * 64, dtype=BF16, device=DEV).as_strided((2, 1, 4, 64), (FAR, 4 * 64, 64, 1))
    far.copy_(q)
    table = torch.tensor([[0, 1] * 10, [1, 0] * 10], dtype=I32)
    lens = torch.tensor([300, 319], dtype=I32)
    sel, left = rl.red_select_pages(far, lo, hi, table.to(DEV), lens.to(DEV), 16, 9)
    for b in range(2):
        chosen, rest = S.select_pages(q[b], want[0], want[1], table[b], int(lens[b]), 1, 16, 9, 1, 1, 320)
        assert int(left[b]) == rest
        for h in range(2):
            assert sel[b, h].tolist() == [int(table[b, p]) for p in chosen[h]]


@pytest.mark.parametrize("vocab", [1000, 5000, 9000])
def test_rows_beyond_32_bit_offsets(vocab):
    say("far rows", vocab)
    g = gen(8)
    x = (2 * torch.randn(2, 2, vocab, generator=g)).to(BF16)
    far = torch.empty(2 * FAR + vocab, dtype=BF16, device=DEV).as_strided((2, 2, vocab), (FAR, FAR // 2, 1))
    r = torch.rand(2, 2, generator=g)
    far.copy_(x)
    p = torch.tensor([0.9, 0.6], device=DEV)
    got = rl.red_sample(far, r.to(DEV), top_p=p, probs=F32)
    want = rl.red_sample(x.to(DEV), r.to(DEV), top_p=p, probs=F32)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("vocab", [4097, 8193, 9000])
def test_more_rows_than_a_pass(vocab):
    """Rows go through the scratch some two thousand at a time: the same results as a few at a time."""
    say("many rows", vocab)
    g = gen(vocab)
    x = (2.5 * torch.randn(1100, 2, vocab, generator=g)).to(BF16).to(DEV)
    r = torch.rand(1100, 2, generator=g).to(DEV)
    t, p, k = torch.rand(1100, device=DEV) + 0.5, torch.rand(1100, device=DEV), torch.randint(0, 300, (1100,), dtype=I32, device=DEV)
    tokens, probs = rl.red_sample(x, r, temperature=t, top_p=p, top_k=k, probs=BF16)
    for a in range(0, 1100, 100):
        b = a + 100
        some = rl.red_sample(x[a:b], r[a:b], temperature=t[a:b].contiguous(), top_p=p[a:b].contiguous(), top_k=k[a:b].contiguous(), probs=BF16)
        assert torch.equal(tokens[a:b], some[0]) and torch.equal(probs[a:b], some[1])


@pytest.mark.parametrize("vocab", [7, 4097, 30000])
@pytest.mark.parametrize("t", [1e-45, 1e-38, 1e-7, 3e38, math.inf, -1.0, math.nan])
def test_sample_extreme_temperatures(vocab, t):
    """Whole logits: neighbours are far apart or alike, and no target is a whole number of weights."""
    g = gen(vocab)
    x = torch.randint(-4, 1, (3, 1, vocab), generator=g).float()
    x[1] += 9
    x[2, 0, ::2] = -math.inf
    r = torch.tensor([[0.1], [0.3], [0.87]])
    check_sample(x, r, t=[t] * 3, k=[vocab // 2 + 1, 3, 0], p=[0.43, 0.71, 1.0])
    check_sample(x, r, t=[t] * 3, m=[0.5, 1.0, 0.0])


@pytest.mark.parametrize("vocab", [6, 4099, 20000])
def test_sample_of_infinite_and_missing_logits(vocab):
    inf, nan = math.inf, math.nan
    x = torch.full((6, 1, vocab), -inf)
    x[1] = nan
    x[2, 0, 1::2] = inf
    x[3, 0, vocab - 1] = -3e38
    x[4, 0, ::3], x[4, 0, 2] = nan, 5.0
    x[5, 0, -2:] = torch.tensor([inf, nan])
    for r in (0.0, 0.5, 1.0):
        check_sample(x, torch.full((6, 1), r), exact=True)
        check_sample(x, torch.full((6, 1), r), t=[0.7] * 6, k=[2] * 6, p=[0.5] * 6, m=[0.25] * 6, exact=True)
