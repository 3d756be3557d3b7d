"""Signalling NaNs in float32 arrays: the maxima, minima and their indices pass over
them, as over quiet ones."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected only with a GPU
    pytest.skip("no GPU visible", allow_module_level=True)

import reduction_libred_amd as rl  # noqa: E402


def array(n, seed, among):
    """n numbers, signalling NaNs among them, side by side around the extremes where `among` is 0; and the numbers alone."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, generator=g)
    hidden = torch.rand(n, generator=g) < among
    ends = [int(x.argmax()), int(x.argmin())]
    if among == 0:
        for i in ends:
            hidden[max(i - 4, 0):i + 5] = True
    hidden[ends] = False
    numbers = x.numpy().copy()
    numbers[hidden.numpy()] = np.nan
    bits = torch.tensor([0x7F800001, 0x7FBFFFFF, -0x7FFFFF, -0x400001], dtype=torch.int32)
    x.view(torch.int32)[hidden] = bits[torch.randint(0, 4, (int(hidden.sum()),), generator=g)]
    return x, numbers


@pytest.mark.parametrize("among", [0.0, 0.01, 0.3, 0.9])
@pytest.mark.parametrize("n", [1, 5, 64, 1000, 5003, 40000, 1 << 20, (1 << 24) + 3, 1 << 25])
def test_extremes_pass_over_signalling_nans(n, among):
    print("[signalling]", n, among, flush=True)
    for seed in range(3 if n < 1 << 22 else 1):
        x, numbers = array(n, n + seed, among)
        for skip in (0, 1):
            if skip >= n or np.isnan(numbers[skip:]).all():
                continue
            d, w = x[skip:].cuda(), numbers[skip:]
            assert int(rl.red_argmax_f32(d)) == np.nanargmax(w) and int(rl.red_argmin_f32(d)) == np.nanargmin(w)
            assert float(rl.red_max_f32(d)) == np.nanmax(w) and float(rl.red_min_f32(d)) == np.nanmin(w)


@pytest.mark.parametrize("rows, cols", [(300, 7), (100, 33), (64, 1000), (9, 20000), (3, 400000)])
def test_rows_and_columns_pass_over_signalling_nans(rows, cols):
    x, numbers = array(rows * cols, cols, 0.3)
    d, w = x.view(rows, cols).cuda(), numbers.reshape(rows, cols)
    w = np.where(np.isnan(w), -np.inf, w)
    assert np.array_equal(rl.red_rows_max_f32(d).cpu().numpy(), w.max(1)) and np.array_equal(rl.red_cols_max_f32(d).cpu().numpy(), w.max(0))
