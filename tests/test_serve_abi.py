"""Refusals of the serving step's entry points (include/libred_serve.h), without
a GPU: argument errors come back as RED_ERR_INVALID_ARG before any HIP call,
which on a machine without a GPU would turn the status into RED_ERR_NO_DEVICE.
No call here reaches a kernel. And the header as C, with the binding's structs."""
import ctypes
import os
import subprocess

import pytest

import reduction_libred_amd as rl
from reduction_libred_amd import decode as D
from reduction_libred_amd import serve as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID = rl.RED_ERR_INVALID_ARG
P = [0x10000000 * i for i in range(1, 20)]   # aligned fake addresses, never dereferenced


def ref(x):
    return ctypes.byref(x)


def with_fields(a, kw):
    for key, value in kw.items():
        setattr(a, key, value)
    return a


def _plan(**kw):
    return with_fields(S.PlanSlotsArgs(batch=4, tokens=10, places=16, pages=64, lens=P[0], counts=P[1], done=P[2], table=P[3], table_cols=8,
                                       table_stride=8, held=P[4], free_pages=P[5], free_count=P[6], slots=P[7], pos=P[8], starts=P[9],
                                       granted=P[10]), kw)


PLAN_BAD = [
    dict(batch=65536), dict(tokens=1 << 31), dict(pages=1 << 31), dict(places=0), dict(places=(1 << 20) + 1), dict(table_cols=(1 << 30) + 1),
    dict(table_cols=1 << 30, table_stride=1 << 30), dict(table_stride=-1), dict(table_stride=7), dict(table_stride=(1 << 40) + 1),
    dict(lens=None), dict(counts=None), dict(table=None), dict(held=None), dict(free_pages=None), dict(free_count=None), dict(slots=None),
    dict(pos=None), dict(starts=None), dict(granted=None), dict(lens=P[0] + 2), dict(done=P[2] + 1), dict(table=P[3] + 2),
    dict(slots=P[7] + 4), dict(pos=P[8] + 4), dict(starts=P[9] + 2),
    dict(held=P[0]), dict(granted=P[1]), dict(pos=P[7] + 72), dict(starts=P[10] - 16), dict(free_count=P[5] + 252), dict(table=P[5] - 4 * 31),
    dict(table=P[4]), dict(slots=P[8]),
]


@pytest.mark.parametrize("bad", PLAN_BAD, ids=lambda b: "-".join(b))
def test_plan_slots_refuses(bad):
    assert rl.lib().red_plan_slots(ref(_plan(**bad)), None) == INVALID


def _cache(kind=2, pages=6, heads=2, places=4, dim=16, **kw):
    scaled = kind >= 3
    return with_fields(D.PagedCache(k=P[0], v=None, k_scales=P[1] if scaled else None, v_scales=None, type=kind, pages=pages, heads=heads,
                                    places=places, dim=dim, page_stride=heads * places * dim, head_stride=places * dim, place_stride=dim,
                                    scale_page_stride=heads * places, scale_head_stride=places, scale_place_stride=1), kw)


def _bounds(cache=None, **kw):
    c = cache or _cache()
    return with_fields(S.PageBoundsArgs(type=2, batch=3, most=5, cache=c, table=P[2], table_cols=5, table_stride=5, lens=P[3], first=P[4],
                                        lo=P[5], hi=P[6], bound_page_stride=c.heads * c.dim, bound_head_stride=c.dim), kw)


BOUNDS_BAD = [
    dict(type=0), dict(type=1), dict(type=3), dict(batch=65536), dict(table_cols=(1 << 30) + 1), dict(table_stride=-1),
    dict(table_stride=(1 << 40) + 1), dict(table=None), dict(lens=None), dict(lo=None), dict(hi=None), dict(lo=P[5] + 1), dict(hi=P[6] + 1),
    dict(table=P[2] + 2), dict(lens=P[3] + 1), dict(first=P[4] + 2), dict(bound_page_stride=-1), dict(bound_head_stride=-1),
    dict(bound_page_stride=16), dict(bound_head_stride=8), dict(bound_page_stride=1 << 60), dict(hi=P[5]), dict(hi=P[5] + 300),
    dict(lo=P[0] + 64), dict(hi=P[0]),
    dict(most=1 << 26, table_cols=1 << 30, table_stride=1 << 30),
    dict(cache=_cache(0)), dict(cache=_cache(5)), dict(cache=_cache(heads=0)), dict(cache=_cache(places=0)), dict(cache=_cache(dim=0)),
    dict(cache=_cache(dim=257)), dict(cache=_cache(k=None)), dict(cache=_cache(k=P[0] + 1)), dict(cache=_cache(k_scales=P[1])),
    dict(cache=_cache(3, k_scales=None)), dict(cache=_cache(3, k_scales=P[1] + 2)), dict(cache=_cache(page_stride=-1)),
    dict(cache=_cache(1)),
]


@pytest.mark.parametrize("bad", BOUNDS_BAD, ids=lambda b: "-".join(b))
def test_page_bounds_refuses(bad):
    assert rl.lib().red_page_bounds(ref(_bounds(**bad)), None) == INVALID


def _select(**kw):
    return with_fields(S.SelectPagesArgs(type=2, batch=3, nodes=2, q_heads=4, kv_heads=2, dim=16, pages=40, places=4, budget=6, first=1,
                                         last=1, max_len=80, q=P[0], q_batch_stride=128, q_node_stride=64, q_head_stride=16, lo=P[1], hi=P[2],
                                         bound_page_stride=32, bound_head_stride=16, table=P[3], table_cols=20, table_stride=20, lens=P[4],
                                         node_count=P[5], selected=P[6], selected_lens=P[7]), kw)


SELECT_BAD = [
    dict(type=0), dict(type=4), dict(batch=65536), dict(nodes=65), dict(q_heads=3), dict(q_heads=0), dict(q_heads=65536 * 2), dict(kv_heads=0),
    dict(kv_heads=65536, q_heads=65536), dict(dim=0), dict(dim=257), dict(places=0), dict(places=(1 << 20) + 1), dict(pages=1 << 31),
    dict(max_len=(1 << 30) + 1), dict(table_cols=(1 << 30) + 1), dict(table_stride=-1), dict(budget=0), dict(budget=3), dict(first=4),
    dict(last=4), dict(first=1 << 63), dict(last=(1 << 64) - 2), dict(budget=(1 << 30) + 1), dict(q_batch_stride=-1), dict(q_head_stride=-16),
    dict(q_node_stride=(1 << 40) + 1), dict(bound_page_stride=-1), dict(bound_head_stride=1 << 60), dict(q=None), dict(lo=None), dict(hi=None),
    dict(table=None), dict(lens=None), dict(selected=None), dict(selected_lens=None), dict(q=P[0] + 1), dict(lo=P[1] + 1),
    dict(selected=P[6] + 2), dict(lens=P[4] + 2), dict(node_count=P[5] + 1), dict(selected=P[3]), dict(selected_lens=P[4]),
    dict(selected_lens=P[6] + 8), dict(selected_lens=P[5]), dict(budget=1 << 29, batch=60000),
]


@pytest.mark.parametrize("bad", SELECT_BAD, ids=lambda b: "-".join(b))
def test_select_pages_refuses(bad):
    assert rl.lib().red_select_pages(ref(_select(**bad)), None) == INVALID


def _sample(**kw):
    return with_fields(S.SampleArgs(type=0, probs_type=0, batch=3, steps=2, vocab=100, logits=P[0], batch_stride=200, step_stride=100,
                                    temperature=P[1], top_k=P[2], top_p=P[3], min_p=P[4], r=P[5], tokens=P[6], probs=P[7],
                                    probs_batch_stride=200, probs_step_stride=100), kw)


SAMPLE_BAD = [
    dict(type=3), dict(type=-1), dict(probs_type=3), dict(batch=65536), dict(steps=65536), dict(batch=65535, steps=65), dict(vocab=0),
    dict(vocab=(1 << 20) + 1), dict(logits=None), dict(logits=P[0] + 2), dict(r=None), dict(r=P[5] + 2), dict(temperature=P[1] + 1),
    dict(top_k=P[2] + 2), dict(top_p=P[3] + 1), dict(min_p=P[4] + 3), dict(tokens=P[6] + 4), dict(probs=P[7] + 2), dict(batch_stride=-1),
    dict(step_stride=-100), dict(batch_stride=1 << 60), dict(probs_step_stride=99), dict(probs_batch_stride=100), dict(probs_step_stride=-1),
    dict(probs=P[0]), dict(probs=P[0] + 4 * 300), dict(tokens=P[0] + 8), dict(tokens=P[7] + 16),
]


@pytest.mark.parametrize("bad", SAMPLE_BAD, ids=lambda b: "-".join(b))
def test_sample_refuses(bad):
    assert rl.lib().red_sample(ref(_sample(**bad)), None) == INVALID


def _attend(**kw):
    c = _cache(v=P[8])
    return with_fields(D.TreeAttentionArgs(type=2, scale=0.25, batch=1, nodes=1, q_heads=2, max_len=8, q=P[9], out=P[10], lse=P[11],
                                           q_batch_stride=32, q_node_stride=32, q_head_stride=16, out_batch_stride=32, out_node_stride=32,
                                           out_head_stride=16, cache=c, table=P[2], table_cols=2, table_stride=4, lens=P[3]), kw)


@pytest.mark.parametrize("stride", [-1, (1 << 40) + 1])
def test_sparse_attention_refuses_strides(stride):
    assert rl.lib().red_sparse_attention(ref(_attend()), stride, None) == INVALID


@pytest.mark.parametrize("bad", [dict(nodes=65), dict(q_heads=3), dict(q=None), dict(table=None), dict(scale=float("nan")),
                                 dict(q=P[9] + 2), dict(table_stride=-1), dict(out=P[9])], ids=lambda b: "-".join(b))
def test_sparse_attention_refuses_what_tree_attention_does(bad):
    assert rl.lib().red_sparse_attention(ref(_attend(**bad)), 2, None) == INVALID


def test_nothing_to_do():
    L = rl.lib()
    assert L.red_page_bounds(ref(_bounds(batch=0)), None) == rl.RED_OK
    assert L.red_page_bounds(ref(_bounds(most=0, lens=None)), None) == rl.RED_OK
    assert L.red_page_bounds(ref(_bounds(_cache(pages=0, k=None))), None) == rl.RED_OK
    assert L.red_select_pages(ref(_select(batch=0)), None) == rl.RED_OK
    assert L.red_sample(ref(_sample(batch=0)), None) == rl.RED_OK
    assert L.red_sample(ref(_sample(steps=0, logits=None)), None) == rl.RED_OK
    assert L.red_sample(ref(_sample(tokens=None, probs=None, r=None)), None) == rl.RED_OK
    for f in ("red_plan_slots", "red_page_bounds", "red_select_pages", "red_sample"):
        assert getattr(L, f)(None, None) == INVALID
    assert L.red_sparse_attention(None, 0, None) == INVALID


@pytest.mark.skipif(__import__("torch").cuda.device_count() > 0, reason="only meaningful where no GPU is visible")
def test_valid_calls_ask_for_a_device():
    """The arguments that the refusals start from are refused for nothing else."""
    L = rl.lib()
    for f, a in (("red_plan_slots", _plan()), ("red_page_bounds", _bounds()), ("red_page_bounds", _bounds(_cache(3))),
                 ("red_select_pages", _select()), ("red_sample", _sample())):
        assert getattr(L, f)(ref(a), None) == rl.RED_ERR_NO_DEVICE, f
    assert L.red_sparse_attention(ref(_attend()), 2, None) == rl.RED_ERR_NO_DEVICE


C_SOURCE = r"""
#include <stdio.h>
#include <string.h>
#include "libred_serve.h"

int main(void) {
    red_plan_slots_args p;
    red_page_bounds_args b;
    red_select_pages_args s;
    red_sample_args m;
    memset(&p, 0, sizeof p), memset(&b, 0, sizeof b), memset(&s, 0, sizeof s), memset(&m, 0, sizeof m);
    int fails = 0;
    fails += red_plan_slots(&p, 0) != RED_ERR_INVALID_ARG;
    fails += red_page_bounds(&b, 0) != RED_ERR_INVALID_ARG;
    fails += red_select_pages(&s, 0) != RED_ERR_INVALID_ARG;
    fails += red_sparse_attention(NULL, 0, 0) != RED_ERR_INVALID_ARG;
    fails += red_sample(&m, 0) != RED_ERR_INVALID_ARG;
    printf("%d %zu %zu %zu %zu\n", fails, sizeof p, sizeof b, sizeof s, sizeof m);
    return fails;
}
"""


def test_header_compiles_as_c_and_its_structs_are_the_bindings(tmp_path):
    src = tmp_path / "caller.c"
    src.write_text(C_SOURCE)
    exe = tmp_path / "caller"
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    libdir = os.path.dirname(rl.LIB_PATH)
    cmd = ["gcc", "-std=c99", "-Wall", "-Werror", "-D__HIP_PLATFORM_AMD__", f"-I{os.path.join(ROOT, 'include')}",
           f"-I{os.path.join(rocm, 'include')}", str(src), "-o", str(exe), f"-L{libdir}", "-l:libred.so", f"-Wl,-rpath,{libdir}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0 and "hip_runtime_api.h" in r.stderr:
        pytest.skip("HIP headers not found")
    assert r.returncode == 0, r.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stdout + run.stderr
    sizes = [ctypes.sizeof(c) for c in (S.PlanSlotsArgs, S.PageBoundsArgs, S.SelectPagesArgs, S.SampleArgs)]
    assert run.stdout.split() == ["0"] + [str(s) for s in sizes]
