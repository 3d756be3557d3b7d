"""The serving step's calls as they are used: one after the other against their
definitions, the example, their graphs, and streams other than the tensors'."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected only with a GPU
    pytest.skip("no GPU visible", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode_reference as R  # noqa: E402
import serve_reference as S  # noqa: E402
import serve_step as E  # noqa: E402
import reduction_libred_amd as rl  # noqa: E402

DEV = torch.device("cuda:0")
BF16, I32 = torch.bfloat16, torch.int32
B, HQ, HK, D, PLACES, COLS, PAGES, CAP, BUDGET, NODES, VOCAB = 4, 8, 2, 64, 16, 40, 120, 24, 9, 6, 9000
STATE = ("table", "held", "stack", "height", "kp", "vp", "ks", "vs", "lo", "hi")


def inputs(seed):
    """Sequences of up to 30 pages, of which one ends and gives its pages back, and their caches."""
    g = torch.Generator().manual_seed(seed)
    lens = torch.tensor([int(torch.randint(1, 450, (1,), generator=g)), 0, 16, 333], dtype=I32)
    counts = torch.randint(1, NODES + 1, (B,), generator=g, dtype=I32)
    done = torch.tensor([0, 1, 0, 0], dtype=I32)
    held = -(-lens // PLACES)
    held[1] = 7
    order, at = torch.randperm(PAGES, generator=g).to(I32), 0
    table = torch.full((B, COLS), -1, dtype=I32)
    for b in range(B):
        table[b, :held[b]] = order[at:at + int(held[b])]
        at += int(held[b])
    stack = torch.cat((order[at:], torch.full((at,), -1, dtype=I32)))
    q, k, v = (torch.randn(CAP, h, D, generator=g).to(BF16) for h in (HQ, HK, HK))
    cache = [torch.randint(-127, 128, (PAGES, HK, PLACES, D), generator=g, dtype=I32).to(torch.int8) for _ in range(2)]
    scales = [torch.rand(PAGES, HK, PLACES, generator=g) / 64 for _ in range(2)]
    lo, hi = S.page_bounds(cache[0], scales[0], table, lens.tolist(), torch.zeros(PAGES, HK, D, dtype=BF16), torch.zeros(PAGES, HK, D, dtype=BF16),
                           None, COLS)
    s = dict(lens=lens, counts=counts, done=done, table=table, held=held.to(I32), stack=stack, height=torch.tensor([PAGES - at], dtype=I32), q=q, k=k, v=v,
             kp=cache[0], vp=cache[1], ks=scales[0], vs=scales[1], lo=lo, hi=hi, x=(2 * torch.randn(B, VOCAB, generator=g)).to(BF16),
             r=torch.rand(B, generator=g), t=torch.tensor([0.7, 0.0, 1.0, 1.3]), top_k=torch.tensor([50, 0, 9, 700], dtype=I32),
             top_p=torch.tensor([0.9, 1.0, 0.95, 0.8]), min_p=torch.tensor([0.0, 0.0, 0.01, 0.002]), rows=torch.arange(NODES))
    return {n: x.to(DEV) for n, x in s.items()}


def step(s, stream=None, only=None):
    """Every call of a step; all results. The state is updated."""
    slots, pos, starts, granted = rl.red_plan_slots(s["lens"], s["counts"], s["table"], s["held"], s["stack"], s["height"], PLACES, CAP, done=s["done"],
                                                    stream=stream)
    rl.red_cache_write(s["k"], s["v"], slots, s["kp"], s["vp"], s["ks"], s["vs"], stream=stream)
    with torch.cuda.stream(stream):
        after = s["lens"] + granted
        q = s["q"][(starts[:-1, None] + s["rows"]).clamp(max=CAP - 1)]
    rl.red_page_bounds(s["kp"], s["table"], after, s["lo"], s["hi"], first=s["lens"], most=3, k_scales=s["ks"], stream=stream)
    table, left = rl.red_select_pages(q, s["lo"], s["hi"], s["table"], s["lens"], PLACES, BUDGET, node_count=granted, stream=stream)
    out, lse = rl.red_sparse_attention(q, s["kp"], s["vp"], table, left, 0.125, node_count=granted, k_scales=s["ks"], v_scales=s["vs"], stream=stream)
    tokens, probs = rl.red_sample(s["x"], s["r"], s["t"], s["top_k"], s["top_p"], s["min_p"], probs=torch.float32, stream=stream)
    return [slots, pos, starts, granted, table, left, out, lse, tokens, probs, q]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b)) and len(a) == len(b)


@pytest.mark.parametrize("seed", [1, 2])
def test_calls_of_a_step_against_their_definitions(seed):
    s = inputs(seed)
    was = {n: x.cpu() for n, x in s.items()}
    slots, pos, starts, granted, table, left, out, lse, tokens, probs, q = (x.cpu() for x in step(s))
    now = {n: x.cpu() for n, x in s.items()}
    # whole numbers: the slots and pages
    want = S.plan_slots(lens=was["lens"].tolist(), counts=was["counts"].tolist(), done=was["done"].tolist(), table=was["table"].tolist(),
                        held=was["held"].tolist(), stack=was["stack"].tolist(), height=int(was["height"]), places=PLACES, tokens=CAP)
    for name, got in dict(slots=slots, pos=pos, starts=starts, granted=granted, table=now["table"], held=now["held"], stack=now["stack"],
                          height=now["height"]).items():
        assert got.tolist() == want[name], name
    assert granted.tolist() == was["counts"].tolist()
    # bounds: of what the cache holds now
    lo, hi = S.page_bounds(now["kp"], now["ks"], now["table"], (was["lens"] + granted).tolist(), was["lo"], was["hi"], was["lens"].tolist(), 3)
    assert torch.equal(now["lo"], lo) and torch.equal(now["hi"], hi)
    values = [(c.double() * sc.double()[..., None]) for c, sc in ((now["kp"], now["ks"]), (now["vp"], now["vs"]))]
    for b in range(B):
        n = int(granted[b])
        chosen, rest = S.select_pages(q[b], lo, hi, now["table"][b], int(was["lens"][b]), n, PLACES, BUDGET, 1, 1, COLS * PLACES)
        assert int(left[b]) == rest
        for h in range(HK):
            pages = [int(now["table"][b, p]) for p in chosen[h]]
            assert table[b, h].tolist() == pages + [-1] * (BUDGET - len(pages))
            kk, vv = (x[pages, h].reshape(-1, D) for x in values)
            group = HQ // HK
            rows = q[b, :n, h * group:(h + 1) * group].reshape(-1, D)
            seen = R.visible(rest, n, None, n, len(pages) * PLACES).repeat_interleave(group, 0)
            o, l, _, size = R.tree_attention(rows, kk, vv, seen, 0.125)
            top = torch.stack([vv[x].abs().amax(0) for x in seen])
            # as in the tests of the attention: products and sums in float32, exponentials and outputs rounded once
            of_scores = (D + 8) * 2.0 ** -24 * size[:, None] + 2.0 ** -20
            got = out[b, :n, h * group:(h + 1) * group].reshape(-1, D).double()
            assert ((got - o).abs() <= R.step(BF16) * o.abs() + (2 * of_scores + R.step(torch.float16)) * top + R.tiny(BF16)).all()
            assert ((lse[b, :n, h * group:(h + 1) * group].reshape(-1).double() - l).abs() <= of_scores[:, 0] + 2.0 ** -22 * l.abs()).all()
        kept, _ = S.sample(was["x"][b].double().numpy(), float(was["t"][b]), int(was["top_k"][b]), float(was["top_p"][b]), float(was["min_p"][b]))
        token, _ = S.token_of(kept, float(was["r"][b]))
        assert int(tokens[b]) == token
        p = torch.from_numpy((kept / kept.sum()).astype("float64"))
        assert ((probs[b].double() - p).abs() <= p * 2.0 ** -23 + R.tiny(torch.float32)).all() and ((probs[b] > 0) == (p > 0)).all()


def test_graph_of_a_step():
    s = inputs(5)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        # no scratch yet: refused, and the capture stays usable
        q = s["q"][:4, None].contiguous()
        with torch.cuda.graph(graph, stream=stream):
            for refused in (lambda: rl.red_plan_slots(s["lens"], s["counts"], s["table"], s["held"], s["stack"], s["height"], PLACES, CAP),
                            lambda: rl.red_select_pages(q, s["lo"], s["hi"], s["table"], s["lens"], PLACES, BUDGET),
                            lambda: rl.red_sample(s["x"], s["r"])):
                with pytest.raises(rl.RedError) as e:
                    refused()
                assert e.value.status == rl.RED_ERR_CAPTURE
            s["q"] + 0
        step(s)                                     # scratch
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            captured = step(s)
        # another graph of the stream, replayed in between
        other, given = torch.cuda.CUDAGraph(), inputs(21)
        torch.cuda.synchronize()
        with torch.cuda.graph(other, stream=stream):
            others = step(given)
    torch.cuda.synchronize()
    for seed in (6, 7, 8, 9):
        fresh = inputs(seed)
        for name, x in s.items():
            x.copy_(fresh[name])
        again = inputs(21)
        for name, x in given.items():
            x.copy_(again[name])
        graph.replay()
        torch.cuda.synchronize()
        got, state = [x.clone() for x in captured], [s[n].clone() for n in STATE]
        other.replay()
        torch.cuda.synchronize()
        assert same(captured, got)
        want = step(fresh)                          # eager work between the replays
        torch.cuda.synchronize()
        assert same(got, want) and same(state, [fresh[n] for n in STATE])
        want = step(again)
        torch.cuda.synchronize()
        assert same(others, want) and same([given[n] for n in STATE], [again[n] for n in STATE])


def test_capture_after_a_larger_call():
    """What a call of no less of anything leaves is enough; also one whose budget takes all pages."""
    stream = torch.cuda.Stream()
    s = inputs(3)
    stream.wait_stream(torch.cuda.current_stream())
    q = s["q"][:4, None].contiguous()
    table = torch.arange(120, dtype=I32, device=DEV).repeat(4, 400)      # keys of 3 MB: more than the least scratch
    args = (q, s["lo"], s["hi"], table, s["lens"] * 1500, PLACES)
    want = rl.red_select_pages(*args, 70)
    wide = s["x"].repeat(700, 1)
    tokens = rl.red_sample(wide[:650], torch.full((650,), 0.5, device=DEV))[0]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        rl.red_select_pages(*args, 48000)
        rl.red_sample(wide, torch.full((wide.shape[0],), 0.5, device=DEV))
        half = torch.full((650,), 0.5, device=DEV)
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            got = rl.red_select_pages(*args, 70)
            drawn = rl.red_sample(wide[:650], half)[0]
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want) and torch.equal(drawn, tokens)
        drawn.zero_(), got[0].zero_()
        torch.cuda.synchronize()


def test_other_streams():
    """Given streams, by argument and as the current one, at the same time."""
    want = []
    for seed in (9, 10):
        s = inputs(seed)
        want.append([x.cpu() for x in step(s)] + [s[n].cpu() for n in STATE])
    torch.cuda.synchronize()
    s = [inputs(seed) for seed in (9, 10)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    with torch.cuda.stream(streams[0]):
        a = step(s[0])
    b = step(s[1], stream=streams[1])
    torch.cuda.synchronize()
    assert same([x.cpu() for x in a + [s[0][n] for n in STATE]], want[0])
    assert same([x.cpu() for x in b + [s[1][n] for n in STATE]], want[1])


def test_poisoned_scratch():
    """Every intermediate that a call reads is one that it wrote."""
    stream = torch.cuda.Stream()
    keep = inputs(11)
    s = {n: x.clone() for n, x in keep.items()}
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        def poisoned(word, f):
            if word is not None:
                rl.red_probe_fill_workspace(word)
            return [x.clone() for x in f()]

        def run(word):
            for n, x in keep.items():
                s[n].copy_(x)
            plan = poisoned(word, lambda: rl.red_plan_slots(s["lens"], s["counts"], s["table"], s["held"], s["stack"], s["height"], PLACES, CAP,
                                                            done=s["done"]))
            wide = poisoned(word, lambda: rl.red_plan_slots(s["lens"], s["counts"] * 20, s["table"], s["held"], s["stack"], s["height"], PLACES, 9000))
            q = s["q"][:4, None].contiguous()
            chosen = poisoned(word, lambda: rl.red_select_pages(q, s["lo"], s["hi"], s["table"], s["lens"], PLACES, BUDGET))
            out = poisoned(word, lambda: rl.red_sparse_attention(q, s["kp"], s["vp"], *chosen, 0.125, k_scales=s["ks"], v_scales=s["vs"]))
            drawn = poisoned(word, lambda: rl.red_sample(s["x"], s["r"], s["t"], s["top_k"], s["top_p"], s["min_p"], probs=torch.float32))
            # chunks without a logit, and far below the largest
            x = s["x"].repeat(1, 4)
            x[:, 9000:18000] = -torch.inf
            x[:, 18000:27000] = -3e38
            few = poisoned(word, lambda: rl.red_sample(x, s["r"], s["t"], s["top_k"], s["top_p"], s["min_p"], probs=torch.float32))
            return plan + wide + chosen + out + drawn + few + [s[n].clone() for n in STATE]

        want = run(None)
        for word in (0x7FC00000, 0x00000001, 0xFFFFFFFF, 0x3F800000):
            assert same(run(word), want), hex(word)
    torch.cuda.synchronize()


def test_outputs_belong_to_the_stream():
    """What a call on a given stream allocates is not handed to another stream's
    tensors while the call may still write it."""
    s = inputs(12)
    want = rl.red_sample(s["x"], s["r"], probs=torch.float32)[1]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _, probs = rl.red_sample(s["x"], s["r"], probs=torch.float32, stream=side)
    at = probs.data_ptr()
    del probs
    others = [torch.empty_like(want) for _ in range(8)]
    assert all(x.data_ptr() != at for x in others)
    _, again = rl.red_sample(s["x"], s["r"], probs=torch.float32, stream=side)
    side.synchronize()
    assert torch.equal(again, want)


@pytest.mark.parametrize("pages", [64, 21])
def test_example_serves(pages):
    """All requests are answered, also where some wait for pages, and all pages come back."""
    g = torch.Generator().manual_seed(4)
    requests = [torch.randint(0, E.VOCAB, (int(torch.randint(1, 200, (1,), generator=g)),), generator=g).tolist() for _ in range(7)]
    model = E.Toy(3, 256, pages, 6, DEV)
    answers, steps = E.serve(model, requests, 5)
    assert all(len(a) == 5 and all(0 <= t < E.VOCAB for t in a) for a in answers)
    again, _ = E.serve(E.Toy(3, 256, pages, 6, DEV), requests, 5)
    assert again == answers
    rl.red_plan_slots(model.lens * 0, model.lens * 0, model.table, model.held, model.free_pages, model.free_count, E.PLACES, 0,
                      done=torch.ones_like(model.lens))
    assert sorted(model.free_pages.tolist()) == list(range(pages)) and int(model.free_count) == pages


def test_example_without_selection():
    """A step whose budget takes all pages: red_tree_attention over the table, the same bits."""
    model = E.Toy(3, 128, 24, 8, DEV)
    g = torch.Generator().manual_seed(5)
    seen = []
    attend = rl.red_sparse_attention

    def watched(q, k, v, table, left, scale, node_count):
        lens = model.lens - node_count
        assert torch.equal(left, lens * (node_count > 0))
        got = attend(q, k, v, table, left, scale, node_count=node_count)
        want = rl.red_tree_attention(q, k, v, model.table, lens, scale, node_count=node_count)
        seen.append(all(torch.equal(a, b) for a, b in zip(got, want)))
        return got

    rl.red_sparse_attention = watched
    try:
        E.serve(model, [torch.randint(0, E.VOCAB, (n,), generator=g).tolist() for n in (70, 5, 33, 90)], 4)
    finally:
        rl.red_sparse_attention = attend
    assert seen and all(seen)
