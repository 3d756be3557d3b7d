"""The verification's choice of a token, its kernels compiled for the host and
run with one host thread a lane: with any one wave held back at every barrier
the token is the same."""
import os
import re
import subprocess

import pytest

from reduction_libred_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    at = tmp_path_factory.mktemp("emulated")
    os.makedirs(at / "hip")
    for name in ("hip_runtime.h", "hip_runtime_api.h"):
        (at / "hip" / name).write_text('#include "hip_block.hpp"\n')
    with open(os.path.join(build.CSRC, "verify_drafts.hip")) as f:
        source = f.read()
    kernels, launches = source.split("template <class T>\nhipError_t verify(")
    kernels = re.sub(r"asm volatile\([^;]*;", "", kernels)     # says where arguments lie; nothing on the host
    (at / "kernels.hpp").write_text(kernels + "}  // namespace\n}  // namespace libred\n")
    clang = os.path.join(os.path.dirname(os.path.dirname(build.hipcc())), "llvm", "bin", "clang++")
    if not os.path.exists(clang):
        pytest.skip("no clang++ beside hipcc")
    exe = str(at / "verify_choice")
    r = subprocess.run([clang, "-std=c++17", "-O1", "-w", f"-I{at}", f"-I{os.path.join(HERE, 'emulated')}", f"-I{build.CSRC}",
                        f"-I{build.INCLUDE}", f'-DSOURCE="{at}/kernels.hpp"', os.path.join(HERE, "emulated", "verify_choice.cpp"),
                        "-o", exe, "-lpthread"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


@pytest.mark.parametrize("late", [-1, 0, 1, 2, 3])
@pytest.mark.parametrize("token", [3, 261, 700, 1023, 1024 + 515, 2999])
def test_token_whichever_wave_is_late(program, token, late):
    """Two launches, 4 waves a block: tokens 256 w .. 256 w + 255 of a segment
    are wave w's."""
    r = subprocess.run([program, "0", "3000", repr((token + 0.5) / 3000), str(late)], capture_output=True, text=True, timeout=120)
    assert r.stdout.split() == ["0", str(token)], r.stdout + r.stderr


@pytest.mark.parametrize("late", [-1, 0, 5])
@pytest.mark.parametrize("token", [70, 999])
def test_token_whichever_wave_is_late_in_one_launch(program, token, late):
    """16 waves a block, 64 tokens of a segment each."""
    r = subprocess.run([program, "1", "1500", repr((token + 0.5) / 1500), str(late)], capture_output=True, text=True, timeout=120)
    assert r.stdout.split() == ["0", str(token)], r.stdout + r.stderr
