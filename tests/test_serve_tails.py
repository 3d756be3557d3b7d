"""Sampling from rows that are a few large logits and a long tail of weights about as
large as the unit in which sums are held: a weight below half a unit counts as 0 and
is not drawn, however many there are, and r of 1 draws the last that counts."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected only with a GPU
    pytest.skip("no GPU visible", allow_module_level=True)

import serve_reference as S  # noqa: E402
import reduction_libred_amd as rl  # noqa: E402

DEV = torch.device("cuda:0")
F32, I32 = torch.float32, torch.int32
RS = (0.0, 0.3, 0.6, 0.9, 1.0, 7.0, math.nan, -1.0)


def unit(vocab):
    return 2.0 ** -min(51, 62 - math.ceil(math.log2(vocab)))


def check(rows, **settings):
    """rows (n, vocab): every row with every r against the definition, weights below half a unit being 0."""
    n, vocab = rows.shape
    x = rows.repeat_interleave(len(RS), 0).to(DEV)
    given = {k: torch.full((n * len(RS),), v, dtype=I32 if k == "top_k" else F32, device=DEV) for k, v in settings.items()}
    tokens = rl.red_sample(x, torch.tensor(RS * n, device=DEV), **given)[0].view(n, -1).tolist()
    for i in range(n):
        kept, _ = S.sample(rows[i].double().numpy(), k=settings.get("top_k"), p=settings.get("top_p"), m=settings.get("min_p"))
        want = [S.token_of(np.where(kept < unit(vocab) / 2, 0, kept), r)[0] for r in RS]
        assert tokens[i] == want, (i, settings)


@pytest.mark.parametrize("units", [0.01, 0.4, 0.6, 1.4, 30.0, 3000.0])
@pytest.mark.parametrize("vocab", [700, 8192, 9001, 40000, 131071, 1 << 20])
def test_long_tails(vocab, units):
    """Weights 1 and 1/2 and all others the same; at the row's begin, at its end, and within."""
    print("[tails]", vocab, units, flush=True)
    tail = math.log(units * unit(vocab))
    rows = torch.full((4, vocab), tail)
    for i, (one, half) in enumerate(((5, 100), (vocab - 6, vocab - 101), (vocab // 2, vocab // 2 + 9), (vocab - 1, 0))):
        rows[i, one], rows[i, half] = 0.0, math.log(0.5)
    check(rows)
    check(rows, top_k=2)
    check(rows, top_k=vocab)
    check(rows, min_p=units * unit(vocab) / 2)
    check(rows, top_p=0.9)


@pytest.mark.parametrize("vocab", [9001, 40000, 131071])
def test_the_last_of_positive_weight(vocab):
    """For r of 1, also where it is alone in its chunk, or less than a sum of bins can tell."""
    rows = torch.full((4, vocab), -math.inf)
    rows[:, 5], rows[:, 100] = 0.0, math.log(0.5)
    for i, units in enumerate((0.6, 0.4, 1.2, 700.0)):
        rows[i, vocab - 3] = math.log(units * unit(vocab))
    got = rl.red_sample(rows.to(DEV), torch.ones(4, device=DEV))[0].tolist()
    assert got == [vocab - 3, 100, vocab - 3, vocab - 3]
    # weights that fall by powers of two until they are less than a unit, among large ones
    fall = torch.arange(vocab, dtype=torch.float64).mul(-80 / vocab).float()[None]
    got = rl.red_sample(fall.to(DEV), torch.ones(1, device=DEV))[0].tolist()
    assert got == [int(torch.nonzero(fall[0].double().exp() >= unit(vocab) / 2)[-1])]
