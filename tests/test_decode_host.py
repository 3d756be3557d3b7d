"""What the entry points of libred_decode.h make of valid arguments on the host:
decode.cpp compiled for it, over launchers that only note what they are asked
for. No GPU is needed and no kernel runs."""
import ctypes
import os
import subprocess

import pytest

import reduction_libred_amd as rl
from reduction_libred_amd import build, decode as D

HERE = os.path.dirname(os.path.abspath(__file__))
A, B, C, E, F, G = (0x1000000 * i for i in range(1, 7))   # aligned fake addresses, never dereferenced
I64 = ctypes.c_int64


@pytest.fixture(scope="module")
def calls(tmp_path_factory):
    at = tmp_path_factory.mktemp("decode_calls")
    os.makedirs(at / "hip")
    for name in ("hip_runtime.h", "hip_runtime_api.h"):
        (at / "hip" / name).write_text('#include "hip_block.hpp"\n')
    lib = str(at / "decode_calls.so")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{at}", f"-I{os.path.join(HERE, 'emulated')}",
                        f"-I{build.CSRC}", f"-I{build.INCLUDE}", os.path.join(HERE, "emulated", "decode_calls.cpp"), "-o", lib],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    L = ctypes.CDLL(lib)
    for name, (res, args) in D.SIGNATURES.items():
        getattr(L, name).restype, getattr(L, name).argtypes = res, args
    L.outside_reads.restype, L.outside_reads.argtypes = I64, [ctypes.c_void_p, ctypes.c_int]
    L.forget()
    return L


def ref(x):
    return ctypes.byref(x)


@pytest.mark.parametrize("kind", [1, 2, 3, 4])
@pytest.mark.parametrize("tokens, heads, places, dim", [(1, 8, 128, 128), (3, 2, 4, 64), (1, 1, 1 << 20, 16), (2, 300, 16, 7)])
def test_read_of_no_pages_stays_in_its_buffers(calls, kind, tokens, heads, places, dim):
    """A cache without pages has no memory: what is loaded instead lies in the
    outputs and in the slots, whatever the strides."""
    scaled = kind >= 3
    cache = D.PagedCache(k=None, v=None, k_scales=None, v_scales=None, type=kind, pages=0, heads=heads, places=places, dim=dim,
                         page_stride=heads * places * dim, head_stride=places * dim, place_stride=dim,
                         scale_page_stride=heads * places, scale_head_stride=places, scale_place_stride=1)
    k = D.Heads(A, heads, heads * dim, dim)
    st = calls.red_cache_read(ref(cache), 1 if kind != 2 else 2, ref(k), ref(D.Heads(A, heads, heads * dim, dim)), C, tokens, None)
    assert st == rl.RED_OK
    assert calls.outside_reads(A, 0) <= 2 * tokens * heads * dim
    if scaled:
        assert calls.outside_reads(C, 1) <= 8 * tokens
