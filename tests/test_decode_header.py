"""libred_decode.h is plain C: gcc compiles a caller, links libred.so, and the
argument checks answer from C (no call reaches a kernel)."""
import os
import subprocess

import pytest

import reduction_libred_amd as rl
from reduction_libred_amd import decode as D

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

C_SOURCE = r"""
#include <stdio.h>
#include <string.h>
#include "libred_decode.h"

int main(void) {
    red_qk_norm_rope_args n;
    red_paged_cache c;
    red_tree_attention_args t;
    red_verify_drafts_args v;
    red_heads h;
    memset(&n, 0, sizeof n), memset(&c, 0, sizeof c), memset(&t, 0, sizeof t), memset(&v, 0, sizeof v), memset(&h, 0, sizeof h);
    int fails = 0;
    fails += red_qk_norm_rope(&n, 0) != RED_ERR_INVALID_ARG;
    fails += red_qk_norm_rope_backward(&n, &h, &h, NULL, NULL, 0) != RED_ERR_INVALID_ARG;
    fails += red_cache_write(&c, RED_F16, &h, &h, NULL, 0, 0) != RED_ERR_INVALID_ARG;
    fails += red_cache_read(&c, RED_BF16, &h, &h, NULL, 0, 0) != RED_ERR_INVALID_ARG;
    fails += red_tree_attention(&t, 0) != RED_ERR_INVALID_ARG;
    fails += red_verify_drafts(&v, 0) != RED_ERR_INVALID_ARG;
    printf("%d %zu %zu %zu %zu %zu\n", fails, sizeof h, sizeof n, sizeof c, sizeof t, sizeof v);
    return fails;
}
"""


def test_header_compiles_as_c_and_its_structs_are_the_bindings(tmp_path):
    import ctypes

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
    sizes = [ctypes.sizeof(c) for c in (D.Heads, D.QkNormRopeArgs, D.PagedCache, D.TreeAttentionArgs, D.VerifyDraftsArgs)]
    assert run.stdout.split() == ["0"] + [str(s) for s in sizes]
