"""The serving step's operators in forms that tests/test_serve_gpu.py leaves out: trees
over selected pages, tables that are views of wider ones, steps that give many pages
back, flat rows of distinct logits."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected only with a GPU
    pytest.skip("no GPU visible", allow_module_level=True)

import decode_reference as R  # noqa: E402
import serve_reference as S  # noqa: E402
import reduction_libred_amd as rl  # noqa: E402
from test_serve_gpu import BF16, DEV, E4M3, F16, F32, I8, I32, check_plan, check_sample, gen, ints, make_cache, run_plan  # noqa: E402


def say(*a):
    print("[serve-more]", *a, flush=True)


def tree_masks(g, batch, nodes):
    """Trees whose nodes see their forebears, and rows that see themselves alone, or nothing."""
    mask = torch.zeros(batch, nodes, dtype=torch.int64)
    for b in range(batch):
        for i in range(nodes):
            parent = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
            word = (int(mask[b, parent]) & (1 << 64) - 1 if parent >= 0 else 0) | 1 << i
            mask[b, i] = word - (1 << 64) if word >> 63 else word
        mask[b, nodes // 2] = 0
    return mask


TREES = [  # batch, nodes, group, kv heads, dim, places, budget, type, cache
    (2, 5, 4, 2, 128, 16, 12, BF16, BF16), (2, 8, 4, 2, 128, 16, 9, BF16, BF16), (2, 3, 8, 2, 64, 24, 9, F16, F16), (3, 6, 4, 2, 80, 8, 11, BF16, I8),
    (1, 33, 2, 2, 64, 8, 40, F16, E4M3), (2, 64, 1, 3, 128, 32, 6, BF16, E4M3), (2, 7, 3, 1, 256, 16, 20, F16, I8), (1, 64, 8, 1, 128, 64, 5, BF16, BF16),
]


@pytest.mark.parametrize("case", TREES, ids=str)
def test_sparse_attention_of_trees(case):
    """Masks of the nodes with a table for each kv head: against the selected pages one
    after the other. Tolerances as in test_sparse_attention. The same call again has
    the same bits."""
    say("trees", case)
    batch, nodes, group, heads, dim, places, budget, dtype, kind = case
    g = gen(sum(case[:7]))
    pages = batch * budget * 2 + 3
    k, ks, dk, dks = make_cache(g, kind, pages, heads, places, dim, "own")
    v, vs, dv, dvs = make_cache(g, kind, pages, heads, places, dim, "own")
    q = torch.randn(batch, nodes, group * heads, dim, generator=g).to(dtype)
    lens = torch.randint(0, budget * places - nodes + 1, (batch,), generator=g, dtype=I32)
    lens[-1] = 0
    lens[0] = budget * places - nodes
    counts = torch.randint(0, nodes + 1, (batch,), generator=g, dtype=I32)
    counts[0] = nodes
    mask = tree_masks(g, batch, nodes)
    table = torch.stack([torch.stack([torch.randperm(pages, generator=g)[:budget] for _ in range(heads)]) for _ in range(batch)]).to(I32)
    scale = dim ** -0.5
    value = [x.double() if s is None else x.double() * s[..., None].double() for x, s in ((k, ks), (v, vs))]
    for count in (None, counts):
        def call():
            return rl.red_sparse_attention(q.to(DEV), dk, dv, table.to(DEV), lens.to(DEV), scale, tree_mask=mask.to(DEV),
                                           node_count=None if count is None else count.to(DEV), k_scales=dks, v_scales=dvs)

        first = call()
        assert all(torch.equal(a, b) for _ in range(5) for a, b in zip(first, call()))
        out, lse = (x.cpu().double() for x in first)
        for b in range(batch):
            n = nodes if count is None else int(count[b])
            seen = R.visible(int(lens[b]), nodes, mask[b], n, budget * places)
            seen[n:] = False
            seen = seen.repeat_interleave(group, 0)
            for h in range(heads):
                kk, vv = (x[table[b, h].long(), h].reshape(-1, dim) for x in value)
                want, want_lse, _, size = R.tree_attention(q[b, :, h * group:(h + 1) * group].reshape(-1, dim), kk, vv, seen, scale)
                got, got_lse = out[b, :, h * group:(h + 1) * group].reshape(-1, dim), lse[b, :, h * group:(h + 1) * group].reshape(-1)
                top = torch.stack([vv[s].abs().amax(0) if s.any() else torch.zeros(dim, dtype=torch.float64) for s in seen])
                of_scores = (dim + 8) * 2.0 ** -24 * size[:, None] + 2.0 ** -20
                step = R.step(F16 if kind in (I8, E4M3) else dtype)
                assert ((got - want).abs() <= R.step(dtype) * want.abs() + (2 * of_scores + step) * top + R.tiny(dtype)).all()
                none = ~seen.any(1)
                assert (got[none] == 0).all() and (got_lse[none] == -math.inf).all()
                assert ((got_lse - want_lse)[~none].abs() <= of_scores[~none, 0] + 2.0 ** -22 * want_lse[~none].abs()).all()


def wider(x, fill):
    """The same numbers as columns of a wider tensor."""
    w = torch.full((*x.shape[:-1], x.shape[-1] + 7), fill, dtype=x.dtype, device=DEV)
    w[..., 3:-4] = x.to(DEV)
    return w[..., 3:-4]


def test_tables_within_wider_ones():
    """Rows of the table further apart than they are long; what lies between is not followed."""
    g = gen(3)
    k = torch.randn(50, 2, 16, 64, generator=g).to(BF16)
    table = torch.randperm(50, generator=g)[:48].view(2, 24).to(I32)
    lens = torch.tensor([370, 290], dtype=I32)
    got = []
    for t in (table.to(DEV), wider(table, 49)):
        lo, hi = (torch.full((50, 2, 64), 9.0, dtype=BF16, device=DEV) for _ in range(2))
        rl.red_page_bounds(k.to(DEV), t, lens.to(DEV), lo, hi)
        q = torch.randn(2, 3, 8, 64, generator=gen(4)).to(BF16).to(DEV)
        sel, left = rl.red_select_pages(q, lo, hi, t, lens.to(DEV), 16, 9)
        out, lse = rl.red_sparse_attention(q, k.to(DEV), k.to(DEV), wider(sel, 49) if t.stride(0) > 24 else sel, left, 0.125)
        got.append((lo, hi, sel, left, out, lse))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    want = S.page_bounds(k, None, table, lens.tolist(), *(torch.full((50, 2, 64), 9.0, dtype=BF16) for _ in range(2)), None, 24)
    assert torch.equal(got[1][0].cpu(), want[0]) and torch.equal(got[1][1].cpu(), want[1])


@pytest.mark.parametrize("places, tokens", [(16, 80), (1, 80), (16, 2100), (1, 9000), (128, 9000)])
@pytest.mark.parametrize("room", [1.0, 0.9])
def test_plan_slots_gives_many_pages_back(places, tokens, room):
    """Tens of thousands of pages come back in a step of few tokens, and in longer ones;
    the stack has room for all of them, or drops some."""
    say("many pages", places, tokens, room)
    g, batch, cols = gen(places + tokens), 70, 700
    order = torch.randperm(batch * cols + 40, generator=g).tolist()
    held = [int(torch.randint(0, cols + 1, (1,), generator=g)) if b % 9 else cols for b in range(batch)]
    done = [int(b % 10 != 3) * (b + 1) for b in range(batch)]
    counts = [tokens // batch + b % 2 for b in range(batch)]
    lens = [0 if d else min(h * places, cols * places - c) for d, h, c in zip(done, held, counts)]
    pages = int(room * (sum(held) + 40))
    c = dict(lens=lens, counts=counts, done=done, table=[order[b * cols:(b + 1) * cols] for b in range(batch)], held=held,
             stack=order[batch * cols:] + [-1] * (pages - 40), height=40, places=places, tokens=tokens)
    check_plan(c, run_plan(c))


@pytest.mark.parametrize("vocab, spread, t, p", [(262144, 1.0, 2.0, 0.8), (262144, 1.0, 3.0, 0.9), (262144, 0.5, 1.0, 0.31), ((1 << 20) - 3, 1.0, 0.7, 0.9),
                                                 (1 << 20, 1.0, 1.0, 0.95), (131071, 0.01, 1.0, 0.5)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_of_flat_rows(vocab, spread, t, p, dtype):
    """More distinct logits near the border than are gathered: the whole row again, for each border."""
    say("flat", vocab, spread, t, p, dtype)
    g = gen(vocab % 1000 + int(10 * t))
    x = (spread * torch.randn(2, 1, vocab, generator=g)).to(dtype)
    r = torch.rand(2, 1, generator=g)
    check_sample(x, r, t=[t] * 2, p=[p] * 2)
    check_sample(x, r, t=[t] * 2, k=[vocab // 3, vocab - 9], p=[p, 0.4], m=[0.0, 0.01])
