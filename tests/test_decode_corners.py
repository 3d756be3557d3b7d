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
