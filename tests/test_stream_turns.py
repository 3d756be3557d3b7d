"""Host threads that call on the same stream. A call of several launches hands
results from one to the next through the buffers of its stream, so no other
call's launches may come between them: decode.cpp and serve.cpp compiled for the
host, over launchers that look whose buffers they find. No GPU is needed."""
import ctypes
import os
import subprocess

import pytest

from reduction_libred_amd import build, decode as D
import test_decode_host as H
import test_serve_host as S

HERE = os.path.dirname(os.path.abspath(__file__))
P = S.P


@pytest.fixture(scope="module")
def turns(tmp_path_factory):
    at = tmp_path_factory.mktemp("turn_calls")
    os.makedirs(at / "hip")
    for name in ("hip_runtime.h", "hip_runtime_api.h"):
        (at / "hip" / name).write_text('#include "hip_block.hpp"\n')
    lib = str(at / "turn_calls.so")
    sources = [os.path.join(HERE, "emulated", "turn_calls.cpp"), *(os.path.join(build.CSRC, f) for f in ("decode.cpp", "serve.cpp"))]
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-pthread", f"-I{at}", f"-I{os.path.join(HERE, 'emulated')}",
                        f"-I{build.CSRC}", f"-I{build.INCLUDE}", *sources, "-o", lib], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return ctypes.CDLL(lib)


def norms():
    def heads(at, n):
        return D.Heads(P[at], n, n * 64, 64)

    a = D.QkNormRopeArgs(type=1, interleaved=0, tokens=500, dim=64, rot=2, eps=1e-6, q=heads(0, 2), k=heads(1, 1), q_out=heads(2, 2),
                         k_out=heads(3, 1), q_weight=None, k_weight=None, pos=P[4], freq=P[5])
    return a, heads(6, 2), heads(7, 1)


CALLS = {"slots": (0, S.plan(30, 5000, 700)), "slots of a short step": (0, S.plan(3, 20, 70)), "selection": (1, S.select(2, 600, 30)),
         "sampling": (2, S.sample(3, 32000)), "attention": (3, H.attention(2, 2, 3, 4, 2, 128, 5000)),
         "verification": (4, H.verify(3, 131071, 2)), "norms' backward pass": (5, *norms())}


def arguments(name):
    what, *structs = CALLS[name]
    return what, *(ctypes.byref(s) for s in structs), *[None] * (3 - len(structs))


@pytest.mark.parametrize("name", CALLS)
def test_calls_on_one_stream_take_turns(turns, name):
    assert turns.on_one_stream(*arguments(name), 4, 15) == 0


@pytest.mark.parametrize("name", CALLS)
def test_calls_on_two_streams_do_not_wait_for_each_other(turns, name):
    assert turns.on_two_streams(*arguments(name)) == 2
