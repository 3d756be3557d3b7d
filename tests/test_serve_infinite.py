"""Selection by bounds of pages that are infinite: a bound that no query takes does
not count, the others make a score infinite. A bound that is NaN always counts."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected only with a GPU
    pytest.skip("no GPU visible", allow_module_level=True)

import reduction_libred_amd as rl  # noqa: E402

DEV = torch.device("cuda:0")
F16, BF16, F64, I32 = torch.float16, torch.bfloat16, torch.float64, torch.int32
INF = math.inf


def scores(q, lo, hi):
    """The largest q . k of a key between the bounds, summed over the rows of q (rows, dim): of (pages, dim)."""
    x, l, h = (v.to(F64) for v in (q, lo, hi))
    each = torch.where(x[:, None] > 0, x[:, None] * h, torch.where(x[:, None] < 0, x[:, None] * l, 0.0))
    each = torch.where(x[:, None].isnan(), x[:, None], each)
    return each.sum((0, 2)) + torch.where(l.isnan() | h.isnan(), math.nan, 0.0).sum(1)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("nodes, group, dim", [(1, 1, 128), (1, 4, 64), (3, 2, 256), (1, 1, 7), (2, 3, 100), (64, 8, 128)])
@pytest.mark.parametrize("cols", [40, 700])
def test_infinite_bounds(dtype, nodes, group, dim, cols):
    print("[infinite]", dtype, nodes, group, dim, cols, flush=True)
    g = torch.Generator().manual_seed(dim + cols)
    heads, places, budget = 2, 16, 12
    a, b = (torch.randint(-3, 4, (cols, heads, dim), generator=g).float() for _ in range(2))
    lo, hi = torch.minimum(a, b), torch.maximum(a, b)
    q = torch.randint(-2, 3, (1, nodes, heads * group, dim), generator=g).float()
    # element 0: every query above 0; 1: every one below; 2: all 0; 3: of either sign where there are several
    q[..., 0], q[..., 1], q[..., 2] = q[..., 0].abs() + 1, -q[..., 1].abs() - 1, 0.0
    lo[5, :, 0], hi[6, :, 1] = -INF, INF              # no query takes these
    lo[7, :, 2], hi[7, :, 2] = -INF, INF
    hi[9, :, 0] = INF                                  # the score is infinite
    hi[11, :, 0], lo[11, :, 0] = -INF, -INF           # and minus that
    hi[13, :, 0], hi[13, 0, 1], lo[13, 0, 1] = INF, INF, INF      # inf - inf: no number in head 0
    lo[15], hi[15] = INF, -INF                        # a page of NaN alone
    hi[17, 1, 2] = math.nan                            # no number, taken or not
    hi[19, 0, 0] = math.nan
    lo, hi, q = lo.to(dtype), hi.to(dtype), q.to(dtype)
    table = torch.randperm(cols, generator=g).to(I32)[None]
    lens = torch.tensor([cols * places - nodes], dtype=I32)
    sel, left = rl.red_select_pages(q.to(DEV), lo.to(DEV), hi.to(DEV), table.to(DEV), lens.to(DEV), places, budget, first=1, last=0)
    tail = int(lens) // places
    forced = {0, *range(tail, cols)}
    for h in range(heads):
        of = scores(q[0, :, h * group:(h + 1) * group].reshape(-1, dim), lo[table[0].long(), h], hi[table[0].long(), h])
        order = sorted((p for p in range(cols) if p not in forced), key=lambda p: (bool(of[p].isnan()), -float(of[p].nan_to_num(0.0)), p)
                       if not of[p].isinf() else (False, -float(of[p]), p))
        want = sorted([*forced, *order[:budget - len(forced)]])
        assert sel[0, h].tolist() == [int(table[0, p]) for p in want], h
    assert int(left) == int(lens) - places * (cols - budget)


def test_infinite_bounds_leave_other_scores_as_they_are():
    """The same pages as with a finite bound in its place, where no query takes it."""
    g = torch.Generator().manual_seed(1)
    lo = torch.randn(300, 2, 128, generator=g).to(BF16)
    hi = lo + 1
    q = torch.randn(1, 2, 8, 128, generator=g).abs().to(BF16).to(DEV)
    table = torch.randperm(300, generator=g).to(I32)[None].to(DEV)
    lens = torch.tensor([4700], dtype=I32, device=DEV)
    got = []
    for value in (-300.0, -INF):
        lo[int(table[0, 9])] = value
        got.append(rl.red_select_pages(q, lo.to(DEV), hi.to(DEV), table, lens, 16, 60)[0])
    assert torch.equal(*got)
