"""Several host threads that call on the same stream, on the GPU: calls of more
than one launch, each with results of its own, come out as they do alone."""
import sys
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - collected only with a GPU
    pytest.skip("no GPU visible", allow_module_level=True)

import reduction_libred_amd as rl  # noqa: E402

DEV = torch.device("cuda:0")
F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32
THREADS, TIMES = 4, 25


def gen(seed):
    return torch.Generator().manual_seed(seed)


def slots(seed):
    """5000 tokens of 60 rows, of which a third gives its pages back: two or three launches."""
    g, batch, cols = gen(seed), 60, 40 + seed
    table = torch.randperm(2 * batch * cols, generator=g).to(I32)
    held = torch.randint(0, 9, (batch,), generator=g, dtype=I32)
    state = [x.to(DEV) for x in (table[:batch * cols].view(batch, cols), held, table[batch * cols:].contiguous(),
                                 torch.tensor([batch * cols], dtype=I32))]
    lens, counts = held * 16, torch.randint(0, 150, (batch,), generator=g, dtype=I32)
    done = (torch.rand(batch, generator=g) < 0.3).to(I32)
    lens, counts, done = (x.to(DEV) for x in (torch.where(done == 1, 0, lens), counts, done))

    def call():
        now = [x.clone() for x in state]
        return [*rl.red_plan_slots(lens, counts, *now, 16, 5000, done=done), *now]
    return call


def selection(seed):
    g, pages = gen(seed), 700
    lo = torch.randn(pages, 2, 128, generator=g).to(BF16).to(DEV)
    args = (torch.randn(2, 3, 8, 128, generator=g).to(BF16).to(DEV), lo, lo + 1, torch.randperm(pages, generator=g).view(2, 350).to(I32).to(DEV),
            torch.tensor([5000, 4000 + seed], dtype=I32, device=DEV), 16, 20)
    return lambda: rl.red_select_pages(*args)


def sampling(seed):
    g, rows = gen(seed), 3 + seed
    x, r = (2 * torch.randn(rows, 40000, generator=g)).to(DEV), torch.rand(rows, generator=g).to(DEV)
    p, k = torch.full((rows,), 0.9, device=DEV), torch.full((rows,), 700, dtype=I32, device=DEV)
    return lambda: rl.red_sample(x, r, top_k=k, top_p=p, probs=F32)


def attention(seed):
    g = gen(seed)
    k, v = (torch.randn(300, 2, 16, 128, generator=g).to(BF16).to(DEV) for _ in range(2))
    args = (torch.randn(2, 5, 8, 128, generator=g).to(BF16).to(DEV), k, v, torch.randperm(300, generator=g).view(2, 150).to(I32).to(DEV),
            torch.tensor([2000, 1500 + seed], dtype=I32, device=DEV), 0.1)
    return lambda: rl.red_tree_attention(*args)


def verification(seed):
    g = gen(seed)
    p, q = (torch.rand(3, n, 70000, generator=g).to(DEV) for n in (3, 2))
    args = (p, q, torch.randint(0, 70000, (3, 2), generator=g).to(DEV), torch.rand(3, 2, generator=g).to(DEV), torch.rand(3, generator=g).to(DEV))
    return lambda: rl.red_verify_drafts(*args)


def norms(seed):
    g = gen(seed)
    q, k, dq, dk = (torch.randn(400, h, 64, generator=g).to(DEV) for h in (4, 2, 4, 2))
    pos, freq = torch.arange(400, device=DEV), torch.rand(16, generator=g).to(DEV)
    return lambda: rl.red_qk_norm_rope_backward(dq, dk, q, k, pos, freq)


def reductions(seed):
    g = gen(seed)
    x, rows, cols = (torch.randn(*s, generator=g).to(DEV) for s in ((3000000 + seed,), (3, 400000), (3000, 300 + seed)))
    return lambda: (rl.red_sum_f32(x), rl.red_argmax_f32(x), rl.red_rows_sum_f32(rows), rl.red_cols_sum_f32(cols))


CALLS = (slots, selection, sampling, attention, verification, norms, reductions)


@pytest.mark.parametrize("what", [*((c,) for c in CALLS), CALLS], ids=lambda w: w[0].__name__ if len(w) == 1 else "all")
def test_host_threads_on_one_stream(what):
    print("[stream-turns]", *(f.__name__ for f in what), flush=True)
    calls = [[f(7 * t + 1) for f in what] for t in range(THREADS)]
    want = [[f() for f in own] for own in calls]
    torch.cuda.synchronize()
    wrong, errors, begin = [], [], threading.Barrier(THREADS)

    def work(t):
        try:
            begin.wait(60)
            for i in range(TIMES):
                for f, w in zip(calls[t], want[t]):
                    got = f()
                    if not all(torch.equal(a, b) for a, b in zip(got, w)):
                        wrong.append((t, i))
        except Exception as e:      # reported below, in the test's thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(t,)) for t in range(THREADS)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    sys.stdout.flush()
    assert not errors and not wrong, (errors, wrong)
