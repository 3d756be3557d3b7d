"""What the entry points of libred_decode.h make of valid arguments on the host:
decode.cpp compiled for it, over launchers that only note what they are asked
for. No GPU is needed and no kernel runs."""
import ctypes
import os
import random
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
    L.scratch_asked.restype = ctypes.c_size_t
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


def asked(calls, f, *args):
    """The scratch that a call makes sure of: a buffer has 1 MiB at least."""
    calls.forget()
    assert getattr(calls, f)(*args, None) == rl.RED_OK
    n = calls.scratch_asked()
    return max(n, 1 << 20) if n else 0


def needs(calls, f, *args):
    calls.forget()
    assert getattr(calls, f)(*args, None) == rl.RED_OK
    return calls.scratch_asked()


def attention(kind, batch, nodes, group, heads, dim, max_len):
    scaled = kind >= 3
    c = D.PagedCache(k=A, v=B, k_scales=C if scaled else None, v_scales=E if scaled else None, type=kind, pages=4, heads=heads,
                     places=16, dim=dim, page_stride=heads * 16 * dim, head_stride=16 * dim, place_stride=dim,
                     scale_page_stride=heads * 16, scale_head_stride=16, scale_place_stride=1)
    h = heads * group
    cols = -(-max_len // 16)
    return D.TreeAttentionArgs(type=kind if not scaled else 1, scale=0.25, batch=batch, nodes=nodes, q_heads=h, max_len=max_len,
                               q=1 << 42, out=1 << 43, lse=F, q_batch_stride=nodes * h * dim, q_node_stride=h * dim,
                               q_head_stride=dim, out_batch_stride=nodes * h * dim, out_node_stride=h * dim, out_head_stride=dim,
                               cache=c, table=G, table_cols=cols, table_stride=cols, lens=A)


@pytest.mark.parametrize("kind", [1, 3])
@pytest.mark.parametrize("dim", [64, 96, 128, 144, 256])
def test_attention_of_a_larger_shape_provides_the_scratch(calls, kind, dim):
    """Types, kv heads and dim being the same, a call of no fewer sequences,
    nodes, query heads and tokens asks for no less."""
    rng = random.Random(dim + kind)
    lengths = [32, 33, 40, 63, 64, 65, 100, 128, 129, 200, 257, 1000, 5000, 40000]
    small = [(1, 32, 2, 1, 64), (1, 8, 8, 1, 64), (1, 1, 16, 8, 129)]
    large = [(1, 64, 2, 1, 64), (1, 9, 8, 1, 64), (1, 2, 16, 8, 129)]
    for _ in range(400):
        heads = rng.choice([1, 2, 8])
        a = [rng.choice([1, 2, 3, 20, 200]), rng.randint(1, 64), rng.choice([1, 2, 4, 8]), heads, rng.choice(lengths)]
        b = [a[0] + rng.choice([0, 0, 1, 50]), min(64, a[1] + rng.choice([0, 0, 1, 20])), a[2] + rng.choice([0, 0, 1, 8]), heads,
             a[4] + rng.choice([0, 0, 1, 32, 1000])]
        small.append(a), large.append(b)
    for a, b in zip(small, large):
        x = needs(calls, "red_tree_attention", ref(attention(kind, *a[:4], dim, a[4])))
        y = asked(calls, "red_tree_attention", ref(attention(kind, *b[:4], dim, b[4])))
        assert x <= y, (a, b)


def verify(batch, vocab, drafts):
    return D.VerifyDraftsArgs(type=0, batch=batch, drafts=drafts, vocab=vocab, p=A, p_batch_stride=vocab * (drafts + 1),
                              p_step_stride=vocab, q=B, q_batch_stride=vocab * drafts, q_step_stride=vocab, drafted=C, u=E, r=F,
                              draft_count=None, accepted=G, tokens=0x10000000)


def test_verification_of_a_larger_shape_provides_the_scratch(calls):
    """No fewer sequences, drafts and tokens of the vocabulary ask for no less."""
    rng = random.Random(5)
    vocabs = [1, 1024, 1025, 32000, 131071, 262144, 262145, 524288, 524289, 1000000, 5000000]
    pairs = [((2000, 262144), (2000, 262145)), ((600, 524288), (600, 524289)), ((40000, 200000), (40000, 300000))]
    for _ in range(400):
        a = (rng.choice([1, 2, 100, 513, 2000, 60000]), rng.choice(vocabs))
        pairs.append((a, (a[0] + rng.choice([0, 0, 1, 1000]), a[1] + rng.choice([0, 1, 1, 1024, 100000]))))
    for a, b in pairs:
        x = needs(calls, "red_verify_drafts", ref(verify(*a, 2)))
        y = asked(calls, "red_verify_drafts", ref(verify(*b, 2)))
        assert x <= y, (a, b)


def launched(calls):
    n = calls.launched(None, 0)
    to = (I64 * (5 * n))()
    calls.launched(to, n)
    return [tuple(to[5 * i:5 * i + 5]) for i in range(n)]


def check_launches(calls, items, in_bytes, out_bytes, by_bytes):
    """Every launch has fewer than 2^32 threads, and together they take all
    items in their order, from the tensors' starts on."""
    got = launched(calls)
    done, (_, _, in0, out0, by0) = 0, got[0]
    for blocks, n, at_in, at_out, at_by in got:
        assert 0 < blocks * 256 < 1 << 32 and n > 0
        assert (at_in - in0, at_out - out0, at_by - by0) == (done * in_bytes, done * out_bytes, done * by_bytes)
        done += n
    assert done == items
    return len(got)


BIG = 1 << 44    # fake addresses of large tensors


@pytest.mark.parametrize("tokens, many", [(5, False), ((1 << 26) - 4, False), ((1 << 26) + 5, True), (1 << 30, True), (1 << 33, True)])
@pytest.mark.parametrize("dim", [3, 64])
def test_norms_of_any_number_of_tokens(calls, tokens, many, dim):
    def heads(at, n=2):
        return D.Heads(BIG * at, n, n * dim, dim)

    calls.forget()
    a = D.QkNormRopeArgs(type=1, interleaved=0, tokens=tokens, dim=dim, rot=2, eps=1e-6, q=heads(1), k=heads(2, 1), q_out=heads(3),
                         k_out=heads(4, 1), q_weight=None, k_weight=None, pos=BIG * 5, freq=G)
    assert calls.red_qk_norm_rope(ref(a), None) == rl.RED_OK
    assert (check_launches(calls, tokens, 4 * dim, 4 * dim, 8) > 1) == many
    calls.forget()
    dq, dk = heads(6), heads(7, 1)
    assert calls.red_qk_norm_rope_backward(ref(a), ref(dq), ref(dk), None, None, None) == rl.RED_OK
    assert check_launches(calls, tokens, 4 * dim, 4 * dim, 8) == 1


@pytest.mark.parametrize("tokens, dim, many", [(5, 64, False), (1 << 26, 64, False), ((1 << 26) - 4, 3, False), ((1 << 26) + 5, 3, True),
                                               (1 << 32, 64, True), (1 << 30, 7, True)])
@pytest.mark.parametrize("kind", [1, 3])
def test_cache_calls_of_any_number_of_tokens(calls, tokens, dim, many, kind):
    scaled = kind >= 3
    c = D.PagedCache(k=A, v=B, k_scales=C if scaled else None, v_scales=E if scaled else None, type=kind, pages=1 << 36, heads=1,
                     places=16, dim=dim, page_stride=0, head_stride=dim * 16, place_stride=dim, scale_page_stride=0,
                     scale_head_stride=16, scale_place_stride=1)
    k, v = D.Heads(BIG, 1, dim, dim), D.Heads(BIG * 2, 1, dim, dim)
    for f in (calls.red_cache_write, calls.red_cache_read):
        calls.forget()
        assert f(ref(c), 1, ref(k), ref(v), BIG * 3, tokens, None) == rl.RED_OK
        assert (check_launches(calls, tokens, 2 * dim, 2 * dim, 8) > 1) == many


@pytest.mark.parametrize("batch, heads, many", [(3, 8, False), (65535, 256, False), (65535, 257, True), (65535, 65535, True)])
def test_attention_of_any_number_of_segments(calls, batch, heads, many):
    calls.forget()
    a = attention(1, batch, 1, 1, heads, 16, 16)
    assert calls.red_tree_attention(ref(a), None) == (rl.RED_OK if batch * heads < 1 << 31 else rl.RED_ERR_INVALID_ARG)
    if batch * heads < 1 << 31:
        assert (check_launches(calls, batch, 2 * 16 * heads, 2 * 16 * heads, 4) > 1) == many


@pytest.mark.parametrize("blocks", [1, 7, 512])
@pytest.mark.parametrize("tiles", [0, 1, 511, 513, 100000, (1 << 31) - 600, (1 << 31) - 1])
def test_shares_of_tiles_are_a_partition(calls, tiles, blocks):
    per = calls.share_size(tiles, blocks)
    assert per == -(-tiles // blocks)
    ends = [calls.share_begin(tiles, per, s) for s in range(blocks + 1)]
    assert ends[0] == 0 and ends[-1] == tiles and all(0 <= b - a <= per for a, b in zip(ends, ends[1:]))
