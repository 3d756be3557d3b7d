"""What the entry points of libred_serve.h make of valid arguments on the host:
serve.cpp compiled for it, over launchers that only note what they are asked
for. No GPU is needed and no kernel runs."""
import ctypes
import os
import random
import subprocess

import pytest

import reduction_libred_amd as rl
from reduction_libred_amd import build, decode as D, serve as S

HERE = os.path.dirname(os.path.abspath(__file__))
P = [(i + 1) << 44 for i in range(20)]   # aligned fake addresses far apart, never dereferenced
I64 = ctypes.c_int64
CALLS = ("red_plan_slots", "red_page_bounds", "red_select_pages", "red_sample")


@pytest.fixture(scope="module")
def calls(tmp_path_factory):
    at = tmp_path_factory.mktemp("serve_calls")
    os.makedirs(at / "hip")
    for name in ("hip_runtime.h", "hip_runtime_api.h"):
        (at / "hip" / name).write_text('#include "hip_block.hpp"\n')
    lib = str(at / "serve_calls.so")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{at}", f"-I{os.path.join(HERE, 'emulated')}",
                        f"-I{build.CSRC}", f"-I{build.INCLUDE}", os.path.join(HERE, "emulated", "serve_calls.cpp"), "-o", lib],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    L = ctypes.CDLL(lib)
    for name in CALLS:
        getattr(L, name).restype, getattr(L, name).argtypes = S.SIGNATURES[name]
    L.scratch_asked.restype, L.scratch_at.restype = ctypes.c_size_t, I64
    return L


def call(calls, name, a):
    """-> the scratch asked for, the launches"""
    calls.forget()
    assert getattr(calls, name)(ctypes.byref(a), None) == rl.RED_OK
    n = calls.launched(None, 0)
    to = (I64 * (5 * n))()
    calls.launched(to, n)
    got = [tuple(to[5 * i:5 * i + 5]) for i in range(n)]
    for blocks, threads, *_ in got:
        assert 0 < blocks * threads < 1 << 32
    return calls.scratch_asked(), got


def plan(batch, tokens, pages, places=16, cols=64):
    return S.PlanSlotsArgs(batch=batch, tokens=tokens, places=places, pages=pages, lens=P[0], counts=P[1], done=P[2], table=P[3], table_cols=cols,
                           table_stride=cols, held=P[4], free_pages=P[5], free_count=P[6], slots=P[7], pos=P[8], starts=P[9], granted=P[10])


def bounds(batch, cols, heads=8, dim=128, most=None):
    c = D.PagedCache(k=P[0], v=None, k_scales=None, v_scales=None, type=2, pages=1 << 20, heads=heads, places=16, dim=dim,
                     page_stride=heads * 16 * dim, head_stride=16 * dim, place_stride=dim, scale_page_stride=0, scale_head_stride=0, scale_place_stride=0)
    return S.PageBoundsArgs(type=2, batch=batch, most=cols if most is None else most, cache=c, table=P[4], table_cols=cols, table_stride=cols, lens=P[5],
                            first=None, lo=P[6], hi=P[7], bound_page_stride=heads * dim, bound_head_stride=dim)


def select(batch, cols, budget, heads=8, group=4, dim=128, places=16, nodes=1, max_len=None):
    h = heads * group
    return S.SelectPagesArgs(type=2, batch=batch, nodes=nodes, q_heads=h, kv_heads=heads, dim=dim, pages=1 << 20, places=places, budget=budget, first=1,
                             last=1, max_len=cols * places if max_len is None else max_len, q=P[0], q_batch_stride=nodes * h * dim, q_node_stride=h * dim,
                             q_head_stride=dim, lo=P[1], hi=P[2], bound_page_stride=heads * dim, bound_head_stride=dim, table=P[3], table_cols=cols,
                             table_stride=cols, lens=P[4], node_count=None, selected=P[5], selected_lens=P[6])


def sample(batch, vocab, steps=1):
    return S.SampleArgs(type=0, probs_type=0, batch=batch, steps=steps, vocab=vocab, logits=P[0], batch_stride=steps * vocab, step_stride=vocab,
                        temperature=P[1], top_k=P[2], top_p=P[3], min_p=P[4], r=P[5], tokens=P[6], probs=None, probs_batch_stride=0,
                        probs_step_stride=0)


def test_a_larger_shape_provides_the_scratch(calls):
    """A call with no less of anything asks for no less scratch."""
    rng = random.Random(3)
    more = lambda x, *steps: x + rng.choice([0, 0, 1, *steps])  # noqa: E731
    for _ in range(300):
        a = [rng.choice([1, 7, 300]), rng.choice([0, 5, 4096, 4097, 70000]), rng.choice([0, 9, 5000])]
        b = [more(x, 9, 1000) for x in a]
        assert call(calls, "red_plan_slots", plan(*a))[0] <= call(calls, "red_plan_slots", plan(*b))[0]
        a = [rng.choice([1, 2, 60]), rng.choice([0, 1, 63, 64, 700, 5000]), rng.choice([4, 64, 700, 6000])]
        b = [more(x, 9, 5000) for x in a]
        assert call(calls, "red_select_pages", select(*a))[0] <= call(calls, "red_select_pages", select(*b))[0], (a, b)
        a = [rng.choice([1, 3, 200, 1500, 2100]), rng.choice([1, 4096, 4097, 8192, 8193, 32000, 131071, (1 << 20) - 50000])]
        b = [more(a[0], 9, 1000), more(a[1], 4096, 8192, 50000 - 1)]
        assert call(calls, "red_sample", sample(*a))[0] <= call(calls, "red_sample", sample(*b))[0], (a, b)


def test_where_no_scratch_is_needed(calls):
    assert call(calls, "red_sample", sample(2000, 8192))[0] == 0
    assert call(calls, "red_page_bounds", bounds(200, 3000))[0] == 0


@pytest.mark.parametrize("batch, cols, many", [(1, 1, False), (65535, 8, False), (65535, 200, True), (300, 1 << 20, True)])
def test_bounds_of_any_number_of_pages(calls, batch, cols, many):
    _, got = call(calls, "red_page_bounds", bounds(batch, cols))
    done = 0
    for _, _, n, lens, table in got:
        assert (lens, table) == (P[5] + 4 * done, P[4] + 4 * done * cols)
        done += n
    assert done == batch and (len(got) > 1) == many


@pytest.mark.parametrize("batch, cols, heads, budget, many", [(1, 4, 1, 9, False), (32, 1000, 8, 60, False), (65535, 10, 200, 12, True),
                                                              (40000, 4, 12000, 4, True), (3, 1 << 20, 64, 1 << 20, False)])
def test_selection_of_any_number_of_pages(calls, batch, cols, heads, budget, many):
    scratch, got = call(calls, "red_select_pages", select(batch, cols, budget, heads=heads, group=1, dim=16))
    assert scratch >= batch * heads * cols * 8 or not many
    done = 0
    for _, _, n, lens, out in got:
        assert (lens, out) == (P[4] + 4 * done, P[5] + 4 * done * heads * budget)
        done += n
    assert done == batch and (len(got) > 1) == many


@pytest.mark.parametrize("batch, steps, vocab, many", [(1, 1, 1, False), (65535, 63, 8192, False), (65535, 8, 8193, True), (192, 1, 131071, False),
                                                       (5000, 3, 1 << 20, True)])
def test_sampling_of_any_number_of_rows(calls, batch, steps, vocab, many):
    """Rows in their order, as many at a time as the scratch holds."""
    scratch, got = call(calls, "red_sample", sample(batch, vocab, steps))
    done = 0
    for _, _, n, first, end in got:
        assert first == done
        done += n
        assert vocab <= 8192 or end <= calls.scratch_at() + scratch
    assert done == batch * steps and (len(got) > 1) == many
