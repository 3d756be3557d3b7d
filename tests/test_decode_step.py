"""The decoding step's calls together: the example against a plain forward pass
in float32 without a cache, their graphs, and streams other than the tensors'."""
import math
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected only with a GPU
    pytest.skip("no GPU visible", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode_step as E  # noqa: E402
import decode_reference as R  # noqa: E402
import reduction_libred_amd as rl  # noqa: E402

DEV = torch.device("cuda:0")


def plain_probabilities(model, tokens):
    """Probabilities after every token of one sequence, in float32 on the CPU,
    from the same weights, nothing quantised."""
    w = {k: getattr(model, k).float().cpu() for k in ("embed", "qkv", "out", "head", "freq")}
    x = w["embed"][tokens]
    n = len(tokens)
    qkv = (x @ w["qkv"]).view(n, -1, E.DIM)
    q, k, v = torch.split(qkv, [E.HEADS, E.KV_HEADS, E.KV_HEADS], dim=1)
    pos = torch.arange(n)
    q, k = (R.qk_norm_rope(y, None, pos, w["freq"], 1e-6, False)[0].float() for y in (q, k))
    group = E.HEADS // E.KV_HEADS
    out = torch.empty(n, E.HEADS, E.DIM)
    for h in range(E.HEADS):
        s = q[:, h] @ k[:, h // group].t().contiguous() * E.DIM ** -0.5
        s = s.masked_fill(torch.triu(torch.ones(n, n, dtype=torch.bool), 1), -math.inf)
        out[:, h] = torch.softmax(s, -1) @ v[:, h // group]
    return torch.softmax((x + out.reshape(n, -1) @ w["out"]) @ w["head"], -1)


def test_example_against_a_plain_forward_pass():
    """A prompt, then chains of tokens step by step through the cache: the same
    probabilities as all tokens at once without one. The int8 cache is off by at
    most half a step of 1/127 of a row's largest element, bfloat16 by 2^-8 a
    rounding; the probabilities have to agree to a few of those (total
    variation, 0.05)."""
    model = E.Toy(2, 96, DEV)
    tokens = torch.randint(0, E.VOCAB, (2, 70), generator=torch.Generator().manual_seed(3))
    got, at = [], 0
    for n in (33, 5, 1, 12, 19):
        got.append(model.forward(tokens[:, at:at + n].to(DEV)).cpu())
        model.lens += n
        at += n
    got = torch.cat(got, 1)
    for b in range(2):
        want = plain_probabilities(model, tokens[b])
        assert ((got[b] - want).abs().sum(-1) / 2).max() < 0.05


def test_example_decodes():
    model = E.Toy(3, 128, DEV)
    prompt = torch.randint(0, E.VOCAB, (3, 20), generator=torch.Generator().manual_seed(4)).to(DEV)
    tokens, accepted = E.decode(model, prompt, 10)
    assert accepted > 0 and all(len(t) >= 10 and all(0 <= x < E.VOCAB for x in t) for t in tokens)
    assert sum(len(t) for t in tokens) == accepted + 30
    assert model.lens.tolist() == [19 + len(t) for t in tokens]
    again, _ = E.decode(E.Toy(3, 128, DEV), prompt, 10)
    assert again == tokens


def step_inputs(seed):
    g = torch.Generator().manual_seed(seed)
    t, hq, hk, d, b, pages, places = 12, 8, 2, 64, 3, 40, 16
    q, k, v = (torch.randn(t, h, d, generator=g).to(torch.bfloat16).to(DEV) for h in (hq, hk, hk))
    pos = torch.randint(0, 1000, (t,), generator=g).to(DEV)
    cache = [torch.randint(-127, 128, (pages, hk, places, d), generator=g, dtype=torch.int32).to(torch.int8).to(DEV) for _ in range(2)]
    scales = [(torch.rand(pages, hk, places, generator=g) / 64).to(DEV) for _ in range(2)]
    slots = torch.randperm(pages * places, generator=g)[:t].to(DEV)
    table = torch.randperm(pages, generator=g)[:b * 13].to(torch.int32).view(b, 13).to(DEV)
    lens = torch.tensor([150, 0, 77], dtype=torch.int32, device=DEV)
    p = torch.softmax(torch.randn(b, 5, 5000, generator=g) * 2, -1).to(DEV)
    draft = torch.softmax(torch.randn(b, 4, 5000, generator=g) * 2, -1).to(DEV)
    drafted = torch.randint(0, 5000, (b, 4), generator=g).to(DEV)
    u, r = torch.rand(b, 4, generator=g).to(DEV), torch.rand(b, generator=g).to(DEV)
    return dict(q=q, k=k, v=v, pos=pos, kp=cache[0], vp=cache[1], ks=scales[0], vs=scales[1], slots=slots, table=table,
                lens=lens, p=p, draft=draft, drafted=drafted, u=u, r=r, freq=R.frequencies(64).to(DEV))


def step(s, stream=None):
    """Every call of a step (and the norms' backward pass); all results."""
    q, k = rl.red_qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], stream=stream)
    back = rl.red_qk_norm_rope_backward(q, k, s["q"], s["k"], s["pos"], s["freq"], stream=stream)
    rl.red_cache_write(k, s["v"], s["slots"], s["kp"], s["vp"], s["ks"], s["vs"], stream=stream)
    read = rl.red_cache_read(s["kp"], s["vp"], s["slots"], torch.bfloat16, s["ks"], s["vs"], stream=stream)
    out = rl.red_tree_attention(q.view(3, 4, 8, 64), s["kp"], s["vp"], s["table"], s["lens"], 0.125, k_scales=s["ks"],
                                v_scales=s["vs"], stream=stream)
    return [q, k, *back, *read, *out, *rl.red_verify_drafts(s["p"], s["draft"], s["drafted"], s["u"], s["r"], stream=stream)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b)) and len(a) == len(b)


def test_graph_of_a_step():
    s = step_inputs(5)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        # no scratch yet: refused, and the capture stays usable
        with torch.cuda.graph(graph, stream=stream):
            with pytest.raises(rl.RedError) as e:
                rl.red_tree_attention(s["q"].view(3, 4, 8, 64), s["kp"], s["vp"], s["table"], s["lens"], 0.125,
                                      k_scales=s["ks"], v_scales=s["vs"])
            assert e.value.status == rl.RED_ERR_CAPTURE
            with pytest.raises(rl.RedError):
                rl.red_verify_drafts(s["p"], s["draft"], s["drafted"], s["u"], s["r"])
            with pytest.raises(rl.RedError):
                rl.red_qk_norm_rope_backward(s["q"], s["k"], s["q"], s["k"], s["pos"], s["freq"])
            s["q"] + 0
        step(s)                                     # scratch
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            captured = step(s)
    torch.cuda.synchronize()
    for seed in (6, 7, 8):
        fresh = step_inputs(seed)
        for name, x in s.items():
            x.copy_(fresh[name])
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in captured]
        cache = [s[n].clone() for n in ("kp", "vp", "ks", "vs")]
        want = step(fresh)                          # eager work between the replays
        torch.cuda.synchronize()
        assert same(got, want) and same(cache, [fresh[n] for n in ("kp", "vp", "ks", "vs")])


def test_other_streams():
    """Given streams, by argument and as the current one, at the same time."""
    want = []
    for seed in (9, 10):
        want.append([x.cpu() for x in step(step_inputs(seed))])
    torch.cuda.synchronize()
    s = [step_inputs(seed) for seed in (9, 10)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    with torch.cuda.stream(streams[0]):
        a = step(s[0])
    b = step(s[1], stream=streams[1])
    torch.cuda.synchronize()
    assert same([x.cpu() for x in a], want[0]) and same([x.cpu() for x in b], want[1])


def test_poisoned_scratch():
    """Every partial that a call reads is one that it wrote."""
    s = step_inputs(11)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    keep = {n: s[n].clone() for n in ("kp", "vp", "ks", "vs")}
    with torch.cuda.stream(stream):
        want = [x.clone() for x in step(s)]
        for word in (0x7FC00000, 0x7F800000, 0xFF800000, 0xFFFFFFFF):
            for n, x in keep.items():
                s[n].copy_(x)
            for call in range(4):
                rl.red_probe_fill_workspace(word)
                if call == 0:
                    got = rl.red_qk_norm_rope_backward(want[0], want[1], s["q"], s["k"], s["pos"], s["freq"])
                    assert same(got, want[2:6])
                elif call == 1:
                    rl.red_cache_write(want[1], s["v"], s["slots"], s["kp"], s["vp"], s["ks"], s["vs"])
                elif call == 2:
                    got = rl.red_tree_attention(want[0].view(3, 4, 8, 64), s["kp"], s["vp"], s["table"], s["lens"], 0.125,
                                                k_scales=s["ks"], v_scales=s["vs"])
                    assert same(got, want[8:10])
                else:
                    assert same(rl.red_verify_drafts(s["p"], s["draft"], s["drafted"], s["u"], s["r"]), want[10:12])
    torch.cuda.synchronize()


@pytest.mark.parametrize("as_handle", [False, True])
def test_outputs_belong_to_the_stream(as_handle):
    """What a call on a given stream allocates and frees is not handed to
    another stream's tensors while the call may still write it."""
    s = step_inputs(11)
    q = s["q"]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    given = side.cuda_stream if as_handle else side
    a, b = rl.red_qk_norm_rope(q, s["k"], s["pos"], s["freq"], stream=given)
    at = a.data_ptr()
    del a, b
    others = [torch.empty_like(q) for _ in range(8)]
    assert all(x.data_ptr() != at for x in others)
    again, _ = rl.red_qk_norm_rope(q, s["k"], s["pos"], s["freq"], stream=given)
    side.synchronize()
    want, _ = rl.red_qk_norm_rope(q, s["k"], s["pos"], s["freq"])
    torch.cuda.synchronize()
    assert torch.equal(again, want)
