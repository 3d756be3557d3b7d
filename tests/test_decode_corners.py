"""The decoding step's operators where they could go wrong without a usual case
noticing, on the GPU against float64 on the CPU."""
import math

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


def gen(seed):
    return torch.Generator().manual_seed(seed)


def integers(n):
    return torch.zeros(n, dtype=torch.int64, device=DEV)


@pytest.mark.parametrize("batch, vocab", [(200, 2999), (130, 60001), (700, 2999), (40, 60001)])
def test_verify_token_of_every_wave(batch, vocab):
    """Tokens spread over all waves of a block, by one launch (the first two)
    and by two: weights of 1, so that r draws token floor(r * vocab)."""
    r = torch.rand(batch, generator=gen(1))
    want = torch.floor(r.double() * vocab).long()
    p = torch.ones(batch, 1, vocab, device=DEV)
    for _ in range(3):
        n, tokens = rl.red_verify_drafts(p, None, torch.zeros(batch, 0, dtype=torch.int64, device=DEV),
                                         torch.zeros(batch, 0, device=DEV), r.to(DEV))
        assert not n.any() and torch.equal(tokens[:, 0].cpu(), want)


@pytest.mark.parametrize("kind", [I8, E4M3, F16])
@pytest.mark.parametrize("tokens, heads, places, dim", [(1, 8, 128, 128), (3, 40, 64, 100)])
def test_read_of_no_pages(kind, tokens, heads, places, dim):
    pg = torch.empty(0, heads, places, dim, dtype=kind, device=DEV)
    sc = {n: torch.empty(0, heads, places, device=DEV) for n in ("k_scales", "v_scales")} if kind in R.TOP else {}
    out = [torch.full((tokens, heads, dim), math.nan, dtype=F16, device=DEV) for _ in range(2)]
    rl.red_cache_read(pg, pg, integers(tokens), F16, k_out=out[0], v_out=out[1], **sc)
    assert not out[0].any() and not out[1].any()


def on_a_new_stream(first, then):
    """then() captured on a stream on which only first() has run, replayed."""
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        first()
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            got = then()
    for _ in range(3):
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, then()):
            assert torch.equal(x, y)
        torch.cuda.synchronize()


def test_attention_captured_after_more_nodes():
    """64 nodes of 2 heads (one tile of 64 tokens) before 32 (two of 32)."""
    g = gen(2)
    pages = [torch.randn(4, 1, 16, 128, generator=g).to(F16).to(DEV) for _ in range(2)]
    q = torch.randn(1, 64, 2, 128, generator=g).to(F16).to(DEV)
    table, lens = torch.arange(4, dtype=torch.int32, device=DEV)[None], torch.tensor([30], dtype=torch.int32, device=DEV)

    def call(nodes):
        return rl.red_tree_attention(q[:, :nodes], *pages, table, lens, 0.1)

    on_a_new_stream(lambda: call(64), lambda: call(32))


def eight_bit_cache(kind, pages, heads, places, dim, seed, scale=1.0):
    """A cache of random rows with scales around `scale` / 64."""
    g = gen(seed)
    codes = [torch.randn(pages, heads, places, dim, generator=g) for _ in range(2)]
    codes = [(x * 36).clamp(-127, 127).round().to(I8) if kind == I8 else (x * 120).clamp(-448, 448).to(E4M3) for x in codes]
    scales = [(0.5 + torch.rand(pages, heads, places, generator=g)) / 64 * s for s in (1.0, scale)]
    return codes, scales


def on_device(x):
    return x.view(I8).to(DEV).view(E4M3) if x.dtype == E4M3 else x.to(DEV)


def attention_reference(q, codes, scales, table, lens, mask, scale):
    """-> out (batch, nodes, heads, dim), lse, and what errors of them are
    relative to: the sum of the magnitudes of a score's terms, the largest
    value; in float64. A value row whose scale is no number is NaN."""
    batch, nodes, hq, dim = q.shape
    hk, places = codes[0].shape[1], codes[0].shape[2]
    out, (lse, size, top) = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(3, batch, nodes, hq, dtype=torch.float64)
    for b, n in enumerate(lens):
        t = torch.arange(n + nodes)
        page, at = table[b, t // places].long(), t % places
        seen = R.visible(n, nodes, mask[b], nodes, n + nodes)
        for h in range(hk):
            k, v = (c[page, h, at].double() * s[page, h, at].double()[:, None] for c, s in zip(codes, scales))
            bad = ~scales[1][page, h, at].isfinite()
            v = torch.where(bad[:, None], torch.zeros((), dtype=torch.float64), v)
            group = hq // hk
            for j in range(group):
                x, l, _, z = R.tree_attention(q[b, :, h * group + j], k, v, seen, scale)
                x[(seen & bad).any(1)] = math.nan
                out[b, :, h * group + j], lse[b, :, h * group + j], size[b, :, h * group + j] = x, l, z
                top[b, :, h * group + j] = (seen * v.abs().amax(1)).amax(1)
    return out, lse, size, top


def check_attention(got, want, total, dim, log_scales=8):
    """Scores: dim products and sums in float32, the logarithm of a value's
    scale (`log_scales` at most) joins them. Sums: `total` terms. The
    exponentials are rounded to float16 for the product (2^-11, or 2^-25 below
    its range), the result to bfloat16."""
    (out, lse), (wout, wlse, size, top) = got, want
    es = (dim + 8) * U * size + 16 * U * (1 + log_scales)
    off = (lse - wlse).abs()
    assert (off <= es + (total + 32) * U + 4 * U * wlse.abs()).all(), off.max()
    allowed = 2.0 ** -8 * wout.abs() + (top * (2.0 ** -11 + total * 2.0 ** -25 + (total + 32) * U + 2 * es))[..., None]
    assert torch.equal(out.isnan(), wout.isnan())
    fine = ~wout.isnan()
    assert ((out - wout).abs()[fine] <= allowed[fine]).all(), (out - wout).abs()[fine].max()


def chains_and_branches(batch, nodes):
    """Even sequences: a chain; odd ones: every node by itself."""
    words = [[(1 << (i + 1)) - 1 if b % 2 == 0 else 1 << i for i in range(nodes)] for b in range(batch)]
    return torch.tensor([[w - 2 ** 64 if w >= 2 ** 63 else w for w in row] for row in words])


SHAPES = [  # lens, nodes, q heads, kv heads, dim, places
    ([70, 33, 0], 4, 4, 2, 64, 16), ([3000, 1700], 3, 4, 1, 128, 32), ([60, 20], 20, 2, 1, 96, 16), ([2500], 24, 4, 1, 128, 16),
    ([90, 41], 40, 4, 2, 64, 8), ([1800, 2000], 64, 2, 1, 192, 64),
]


def call_attention(q, codes, scales, table, lens, mask, scale):
    out, lse = rl.red_tree_attention(q.to(DEV), on_device(codes[0]), on_device(codes[1]), table.to(DEV),
                                     torch.tensor(lens, dtype=torch.int32, device=DEV), scale, tree_mask=mask.to(DEV),
                                     k_scales=scales[0].to(DEV), v_scales=scales[1].to(DEV))
    return out.cpu().double(), lse.cpu().double()


@pytest.mark.parametrize("where", ["tokens", "nodes"])
@pytest.mark.parametrize("kind", [I8, E4M3], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_value_rows_that_are_no_numbers(shape, kind, where):
    """A value row stored with an infinity or a NaN reads back as NaN: the rows
    that see it are NaN, their lse is the scores' alone, and the others are what
    they are without it."""
    lens, nodes, hq, hk, dim, places = shape
    print(shape, kind, where, flush=True)
    batch, per = len(lens), -(-(max(lens) + nodes) // places)
    codes, scales = eight_bit_cache(kind, batch * per, hk, places, dim, 3)
    table = torch.randperm(batch * per, generator=gen(4)).to(torch.int32).view(batch, per)
    q = torch.randn(batch, nodes, hq, dim, generator=gen(5)).to(BF16)
    mask = chains_and_branches(batch, nodes)
    hit = [n + nodes // 2 if where == "nodes" else n // 3 for n in lens]
    for b, t in enumerate(hit):
        if where == "nodes" or lens[b] > 0:
            codes[1].view(I8)[table[b, t // places].long(), :, t % places] = 0
            scales[1][table[b, t // places].long(), :, t % places] = math.inf if b % 2 else math.nan
    want = attention_reference(q, codes, scales, table, lens, mask, dim ** -0.5)
    got = call_attention(q, codes, scales, table, lens, mask, dim ** -0.5)
    assert want[0].isnan().any() and not (where == "nodes" and want[0].isnan().all())
    check_attention(got, want, max(lens) + nodes, dim)


@pytest.mark.parametrize("spread", ["mixed", "zeros first", "zeros last", "far apart"])
@pytest.mark.parametrize("kind", [I8, E4M3], ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_value_scales_far_apart(shape, kind, spread):
    """Rows of zeros among values of 2^50 and more, and scales 2^130 apart: every
    token has its full weight."""
    lens, nodes, hq, hk, dim, places = shape
    print(shape, kind, spread, flush=True)
    batch, per = len(lens), -(-(max(lens) + nodes) // places)
    codes, scales = eight_bit_cache(kind, batch * per, hk, places, dim, 6)
    table = torch.randperm(batch * per, generator=gen(7)).to(torch.int32).view(batch, per)
    q = (0.5 * torch.randn(batch, nodes, hq, dim, generator=gen(8))).to(BF16)
    for b, n in enumerate(lens):
        t = torch.arange(n + nodes)
        page, at = table[b, t // places].long(), t % places
        low = {"mixed": t % 2 == 0, "zeros first": t < n * 2 // 3, "zeros last": t >= n // 3, "far apart": t % 3 == 0}[spread]
        if spread == "far apart":
            scales[1][page[low], :, at[low]] *= 2.0 ** -60
            scales[1][page[~low], :, at[~low]] *= 2.0 ** 70
        else:
            scales[1][page[low], :, at[low]] = 0.0
            codes[1].view(I8)[page[low], :, at[low]] = 0
            scales[1][page[~low], :, at[~low]] *= 2.0 ** (50 + 20 * b)
    mask = chains_and_branches(batch, nodes)
    want = attention_reference(q, codes, scales, table, lens, mask, dim ** -0.5)
    got = call_attention(q, codes, scales, table, lens, mask, dim ** -0.5)
    check_attention(got, want, max(lens) + nodes, dim, 130)


@pytest.mark.parametrize("dt", [F32, F16, BF16], ids=str)
@pytest.mark.parametrize("vocab", [3001, 40003])
def test_verify_nan_in_either_row(dt, vocab):
    """A NaN among the weights of the row that a token is drawn from draws none
    (-1), whether it is the target's or the draft's; elsewhere it is not looked at."""
    b, k = 6, 2
    p = torch.softmax(torch.randn(b, k + 1, vocab, generator=gen(9)), -1).to(dt)
    q = torch.softmax(torch.randn(b, k, vocab, generator=gen(10)), -1).to(dt)
    drafted = torch.full((b, k), 5)
    u, r = torch.full((b, k), 1.0), torch.rand(b, generator=gen(11))
    q[:, :, 5], p[:, :, 5] = 0.5, 0.25                 # refused by u of 1
    u[3:, 0] = 0.0                                     # the first is accepted
    q[0, 0, 9] = q[1, 0, vocab - 1] = p[2, 0, 7] = math.nan
    q[3, 1, 9], q[4, 0, 9], p[5, 2, 9] = math.nan, math.nan, math.nan
    n, tokens = rl.red_verify_drafts(*(x.to(DEV) for x in (p, q, drafted, u, r)))
    assert n.tolist() == [0, 0, 0, 1, 1, 1]
    assert tokens[:4].tolist() == [[-1, -1, -1]] * 3 + [[5, -1, -1]]
    for i in (4, 5):
        w = (p[i, 1].double() - q[i, 1].double()).clamp(min=0)
        run = torch.cumsum(w, 0)
        want = int((run > float(r[i]) * run[-1]).nonzero()[0])
        assert tokens[i].tolist() == [5, want, -1]


MANY = (1 << 26) + 5   # a wave or a row each: more than a launch has threads for


def test_norms_of_many_tokens():
    x = torch.randn(MANY, 1, 2, dtype=F16, device=DEV)
    pos, freq = torch.arange(MANY, device=DEV), torch.tensor([1e-4], device=DEV)
    got, _ = rl.red_qk_norm_rope(x, x[:, :0], pos, freq)
    half = MANY // 2
    for part in (slice(0, half), slice(half, MANY)):
        want, _ = rl.red_qk_norm_rope(x[part], x[part, :0], pos[part], freq)
        assert torch.equal(got[part], want)


@pytest.mark.parametrize("kind", [F16, I8], ids=str)
def test_cache_of_many_tokens(kind):
    x = [torch.randn(MANY, 1, 1, dtype=F16, device=DEV) for _ in range(2)]
    pages = -(-MANY // 64)
    pg = [torch.zeros(pages, 1, 64, 1, dtype=kind, device=DEV) for _ in range(2)]
    sc = dict(k_scales=torch.zeros(pages, 1, 64, device=DEV), v_scales=torch.zeros(pages, 1, 64, device=DEV)) if kind == I8 else {}
    slots = torch.arange(MANY - 1, -1, -1, device=DEV)
    rl.red_cache_write(*x, slots, *pg, **sc)
    for i, s in enumerate(("k_scales", "v_scales")):
        cached = pg[i].view(-1)[:MANY].flip(0)
        if kind == I8:      # a row of one element is its own largest: 127 and its sign, or 0
            assert torch.equal(cached.half() * 1.0, torch.sign(x[i].view(-1)) * 127)
            top = x[i].view(-1).abs().float()      # by a tensor: torch divides by a number as a product with 1 / 127
            assert torch.equal(sc[s].view(-1)[:MANY].flip(0), top / torch.full_like(top, 127))
        else:
            assert torch.equal(cached, x[i].view(-1))
    back = rl.red_cache_read(*pg, slots, F16, **sc)
    for a, b in zip(back, x):
        assert torch.equal(a, b) if kind == F16 else (a - b).abs().max() <= 2.0 ** -9 * b.abs().max()


def test_attention_of_many_segments():
    """65535 sequences of 257 kv heads, a block each."""
    batch, heads, dim = 65535, 257, 16
    pages = [torch.randn(3, heads, 16, dim, generator=gen(12)).to(F16).to(DEV) for _ in range(2)]
    table = (torch.arange(batch, dtype=torch.int32, device=DEV) % 3)[:, None]
    lens = torch.arange(batch, dtype=torch.int32, device=DEV) % 16
    q = torch.randn(batch, 1, heads, dim, dtype=F16, device=DEV)
    out, lse = rl.red_tree_attention(q, *pages, table, lens, 0.25)
    half = batch // 2
    for part in (slice(0, half), slice(half, batch)):
        want = rl.red_tree_attention(q[part], *pages, table[part], lens[part], 0.25)
        assert torch.equal(out[part], want[0]) and torch.equal(lse[part], want[1])


def norm_tensors(dt, seed):
    g = gen(seed)
    x = [torch.randn(37, h, 64, generator=g).to(dt).to(DEV) for h in (6, 2)]
    w = [(1 + 0.2 * torch.randn(64, generator=g)).to(dt).to(DEV) for _ in range(2)]
    dy = [torch.randn(37, h, 64, generator=g).to(dt).to(DEV) for h in (6, 2)]
    return x, w, dy, torch.randint(0, 5000, (37,), generator=g).to(DEV), R.frequencies(48).to(DEV)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dt", [F32, F16, BF16], ids=str)
def test_norms_have_gradients(dt, interleaved):
    """The gradients that autograd finds are those of the backward call."""
    x, w, dy, pos, freq = norm_tensors(dt, 13)
    leaves = [y.detach().clone().requires_grad_() for y in x + w]
    out = rl.red_qk_norm_rope(leaves[0], leaves[1], pos, freq, leaves[2], leaves[3], eps=1e-5, interleaved=interleaved)
    plain = rl.red_qk_norm_rope(x[0], x[1], pos, freq, w[0], w[1], eps=1e-5, interleaved=interleaved)
    assert torch.equal(out[0], plain[0]) and torch.equal(out[1], plain[1]) and plain[0].grad_fn is None
    torch.autograd.backward(out, dy)
    want = rl.red_qk_norm_rope_backward(dy[0], dy[1], x[0], x[1], pos, freq, w[0], w[1], eps=1e-5, interleaved=interleaved)
    for y, z in zip(leaves, want):
        assert y.grad.dtype == dt and torch.equal(y.grad, z.to(dt))


def test_norms_gradients_of_some_inputs():
    x, w, dy, pos, freq = norm_tensors(F32, 14)
    zero = torch.zeros_like(dy[0])
    want = rl.red_qk_norm_rope_backward(zero, dy[1], x[0], x[1], pos, freq, None, w[1])
    # only k's output is used, only the weight of k wants a gradient
    kw = w[1].clone().requires_grad_()
    _, k = rl.red_qk_norm_rope(x[0], x[1], pos, freq, None, kw)
    k.backward(dy[1])
    assert torch.equal(kw.grad, want[3])
    # q within a larger tensor, no weights; a sum's gradient is broadcast
    fused = torch.cat(x, 1).requires_grad_()
    q, k = rl.red_qk_norm_rope(fused[:, :6], fused[:, 6:], pos, freq)
    (q.sum() + 2 * k.sum()).backward()
    want = rl.red_qk_norm_rope_backward(torch.ones_like(dy[0]), torch.full_like(dy[1], 2), x[0], x[1], pos, freq)
    assert torch.equal(fused.grad, torch.cat(want[:2], 1))
    # on a stream of its own, where the backward pass follows it
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    leaf = x[0].clone().requires_grad_()
    torch.cuda.synchronize()
    q, _ = rl.red_qk_norm_rope(leaf, x[1], pos, freq, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    q.sum().backward()
    torch.cuda.synchronize()
    assert torch.equal(leaf.grad, rl.red_qk_norm_rope_backward(torch.ones_like(dy[0]), torch.zeros_like(dy[1]), x[0], x[1], pos, freq)[0])


def test_norms_without_gradients():
    x, w, dy, pos, freq = norm_tensors(F16, 15)
    leaf = x[0].clone().requires_grad_()
    with torch.no_grad():
        assert not rl.red_qk_norm_rope(leaf, x[1], pos, freq)[0].requires_grad
    assert not rl.red_qk_norm_rope(leaf.detach(), x[1], pos, freq)[0].requires_grad
    to = torch.empty_like(x[0])
    with pytest.warns(UserWarning, match="no history"):
        got, _ = rl.red_qk_norm_rope(leaf, x[1], pos, freq, q_out=to)
    assert got is to and not got.requires_grad
    with pytest.raises(TypeError):
        rl.red_qk_norm_rope(leaf, x[1], pos.int(), freq)
    # an input that is changed before the backward pass is found out
    y = leaf * 1.0
    q, _ = rl.red_qk_norm_rope(y, x[1], pos, freq)
    y.zero_()
    with pytest.raises(RuntimeError):
        q.sum().backward()


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("dt", [F32, F16, BF16], ids=str)
@pytest.mark.parametrize("dim, rot, interleaved", [(128, 64, False), (128, 64, True), (128, 128, False), (100, 50, False), (66, 30, True),
                                                   (96, 0, False), (255, 128, False)])
def test_norms_weight_that_is_no_number(dim, rot, interleaved, dt, bad):
    """It reaches its own column and the one that turns with it, no other."""
    x = [torch.randn(5, h, dim, generator=gen(16)).to(dt).to(DEV) for h in (3, 1)]
    pos, freq = torch.arange(1, 6, device=DEV), R.frequencies(rot).to(DEV)
    w = torch.ones(dim, dtype=dt, device=DEV)
    clean = rl.red_qk_norm_rope(*x, pos, freq, w, w, interleaved=interleaved)
    for at in {0, dim - 1, rot // 2, max(rot - 1, 0), min(rot, dim - 1)}:
        v = w.clone()
        v[at] = bad
        a, b = R.pairs(rot, interleaved)
        hit = {at} | {int(q) for p, q in zip(a, b) if p == at} | {int(p) for p, q in zip(a, b) if q == at}
        rest = [c for c in range(dim) if c not in hit]
        for got, want in zip(rl.red_qk_norm_rope(*x, pos, freq, v, v, interleaved=interleaved), clean):
            assert torch.equal(got[..., rest], want[..., rest]), at
            assert not got[..., sorted(hit)].isfinite().any(), at
            if at >= rot and bad == math.inf:       # times a number, and nothing else
                assert got[..., at].isinf().all(), at


@pytest.mark.parametrize("strides", [(1, 70, 1), (8, 1, 1), (0, 8, 1), (8, 0, 1), (3, 1, 1)])
def test_norms_of_rows_that_overlap(strides):
    """Heads that are windows of one another, or broadcast."""
    x = torch.randn(500, generator=gen(17)).to(DEV)
    q, k = (x.as_strided((6, h, 8), strides) for h in (3, 2))
    pos, freq = torch.arange(6, device=DEV), R.frequencies(8).to(DEV)
    # The roundings of the norms' other tests: 20 of float32 forward, 48 back, and
    # 200 more in the weights' sums.
    for got, y in zip(rl.red_qk_norm_rope(q, k, pos, freq), (q, k)):
        want, size = R.qk_norm_rope(y.cpu(), None, pos.cpu(), freq.cpu(), 1e-6, False)
        assert ((got.cpu() - want).abs() <= U * (want.abs() + 21 * size)).all()
    dq, dk = torch.randn(6, 3, 8, generator=gen(18)), torch.randn(6, 2, 8, generator=gen(19))
    got = rl.red_qk_norm_rope_backward(dq.to(DEV), dk.to(DEV), q, k, pos, freq)
    for i, (dy, y) in enumerate(((dq, q), (dk, k))):
        dx, size, dw, dsize = R.qk_norm_rope_backward(dy, y.cpu(), None, pos.cpu(), freq.cpu(), 1e-6, False)
        assert ((got[i].cpu() - dx).abs() <= U * (dx.abs() + 49 * size)).all()
        assert ((got[2 + i].cpu() - dw).abs() <= U * (dw.abs() + 249 * dsize)).all()


def test_attention_refuses_a_negative_length():
    pages = torch.zeros(2, 1, 16, 64, dtype=F16, device=DEV)
    q, table, lens = torch.zeros(1, 1, 1, 64, dtype=F16, device=DEV), torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        rl.red_tree_attention(q, pages, pages, table, lens, 1.0, max_len=-1)
    out, lse = rl.red_tree_attention(q, pages, pages, table, lens, 1.0, max_len=0)
    assert not out.any() and (lse == -math.inf).all()


@pytest.mark.parametrize("kind", [I8, E4M3], ids=str)
@pytest.mark.parametrize("dt", [F16, BF16], ids=str)
@pytest.mark.parametrize("dim", [61, 64, 100])
def test_cache_reads_the_same_whatever_the_alignment(dim, dt, kind):
    """A product in float32 and its rounding, for subnormal results too, where
    one rounding of the two would differ."""
    x = (torch.randn(8000, 2, dim, generator=gen(20)) * torch.exp(2 * torch.randn(8000, 2, 1, generator=gen(21)) - 4)).to(dt).to(DEV)
    raw = [torch.zeros(500 * 2 * 16 * dim + 1, dtype=I8, device=DEV).view(kind) for _ in range(2)]
    sc = [torch.zeros(500, 2, 16, device=DEV) for _ in range(2)]
    slots = torch.arange(8000, device=DEV)
    for first in (0, 1):        # rows on their boundaries, and one byte behind
        pg = [y[first:first + 500 * 2 * 16 * dim].view(500, 2, 16, dim) for y in raw]
        rl.red_cache_write(x, -x, slots, *pg, *sc)
        for got, p, s in zip(rl.red_cache_read(*pg, slots, dt, *sc), pg, sc):
            want = (p.float() * s[..., None]).to(dt).transpose(1, 2).reshape(8000, 2, dim)
            assert torch.equal(got, want)
