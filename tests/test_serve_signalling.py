"""Signalling NaNs (the bit patterns that no arithmetic leaves, but memory may hold)
count as NaNs in the serving step's operators."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected only with a GPU
    pytest.skip("no GPU visible", allow_module_level=True)

import serve_reference as S  # noqa: E402
import reduction_libred_amd as rl  # noqa: E402

DEV = torch.device("cuda:0")
F32, F16, BF16, I32 = torch.float32, torch.float16, torch.bfloat16, torch.int32
# the least and the largest of either sign
BITS = {BF16: (0x7F81, 0x7FBF, -0x7F, -0x41), F16: (0x7C01, 0x7DFF, -0x3FF, -0x201), F32: (0x7F800001, 0x7FBFFFFF, -0x7FFFFF, -0x400001)}
INTS = {BF16: torch.int16, F16: torch.int16, F32: I32}


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("dim", [64, 128, 256, 7])
def test_page_bounds_pass_over_signalling_nans(dtype, dim):
    print("[signalling] bounds", dtype, dim, flush=True)
    places = 40
    k = torch.randn(places, 1, places, dim, generator=torch.Generator().manual_seed(dim)).to(dtype)
    for p in range(places):      # page p: token p, of which every element is one of them
        for i, bits in enumerate(BITS[dtype]):
            k.view(torch.int16)[p, 0, p, i::4] = bits
    k.view(torch.int16)[3, :, :, 1] = BITS[dtype][0]       # an element of which all are
    assert k.isnan().sum() == (places * dim + places - 1)
    table, lens = torch.arange(places, dtype=I32)[None], torch.tensor([places * places], dtype=I32)
    lo, hi = (torch.full((places, 1, dim), 9.0, dtype=dtype, device=DEV) for _ in range(2))
    rl.red_page_bounds(k.to(DEV), table.to(DEV), lens.to(DEV), lo, hi)
    want = S.page_bounds(k, None, table, lens.tolist(), lo.cpu(), hi.cpu(), None, places)
    assert torch.equal(lo.cpu(), want[0]) and torch.equal(hi.cpu(), want[1])


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("vocab", [5, 1000, 6000, 9001, 40000])
def test_sample_counts_signalling_nans_as_minus_infinity(dtype, vocab):
    print("[signalling] sample", dtype, vocab, flush=True)
    g = torch.Generator().manual_seed(vocab)
    x = (3 * torch.randn(6, vocab, generator=g)).to(dtype)
    hidden = torch.rand(6, vocab, generator=g) < torch.tensor([0.01, 0.3, 0.9, 0.5, 0.5, 0.0])[:, None]
    hidden[3, :-1] = True                               # one is left, or none
    hidden[4] = True                                     # none is
    hidden[5, torch.arange(vocab) != int(x[5].argmax())] = torch.rand(vocab - 1, generator=g) < 0.5
    bits = torch.tensor(BITS[dtype], dtype=INTS[dtype])[torch.randint(0, 4, (6, vocab), generator=g)]
    masked = x.masked_fill(hidden, -torch.inf)
    x.view(INTS[dtype])[hidden] = bits[hidden]
    assert (x.isnan() == hidden).all()
    r = torch.rand(6, generator=g).to(DEV)
    t, p = torch.tensor([1.0, 0.7, 2.0, 1.0, 1.0, 0.9], device=DEV), torch.full((6,), 0.9, device=DEV)
    k, m = torch.full((6,), vocab // 3 + 1, dtype=I32, device=DEV), torch.full((6,), 0.02, device=DEV)
    for settings in ({}, dict(temperature=t), dict(top_p=p), dict(top_k=k, temperature=t), dict(temperature=t, top_k=k, top_p=p, min_p=m)):
        got, want = (rl.red_sample(y.to(DEV), r, probs=F32, **settings) for y in (x, masked))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert int(got[0][4]) == -1 and int(got[0][3]) == (-1 if hidden[3, -1] else vocab - 1)
