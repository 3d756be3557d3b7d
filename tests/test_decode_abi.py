"""Refusals of the decoding step's entry points (include/libred_decode.h),
without a GPU: argument errors come back as RED_ERR_INVALID_ARG before any HIP
call, which on a machine without a GPU would turn the status into
RED_ERR_NO_DEVICE. No call here reaches a kernel."""
import ctypes

import pytest

import reduction_libred_amd as rl
from reduction_libred_amd import decode as D

INVALID = rl.RED_ERR_INVALID_ARG
A, B, C, E, F, G = (0x1000000 * i for i in range(1, 7))   # aligned fake addresses, never dereferenced


def _heads(data, heads, dim=8, tokens_apart=None):
    return D.Heads(data, heads, heads * dim if tokens_apart is None else tokens_apart, dim)


def _norm(**kw):
    a = D.QkNormRopeArgs(type=1, interleaved=0, tokens=3, dim=8, rot=8, eps=1e-6, q=_heads(A, 4), k=_heads(B, 2),
                         q_out=_heads(C, 4), k_out=_heads(E, 2), q_weight=None, k_weight=None, pos=F, freq=G)
    for key, value in kw.items():
        setattr(a, key, value)
    return a


NORM_BAD = [
    dict(type=3), dict(type=4), dict(type=-1), dict(dim=0), dict(dim=257), dict(rot=10), dict(rot=3),
    dict(tokens=rl.RED_MAX_N + 1), dict(eps=-1.0), dict(eps=float("nan")),
    dict(q=_heads(None, 4)), dict(k=_heads(None, 2)), dict(q=_heads(A + 1, 4)), dict(q=_heads(A, -1)),
    dict(q=D.Heads(A, 4, -8, 8)), dict(q=D.Heads(A, 4, 1 << 60, 8)), dict(q=_heads(A, 3)),
    dict(q_out=_heads(None, 4)), dict(q_out=_heads(C + 1, 4)),
    dict(q_out=D.Heads(C, 4, 8, 8)), dict(q_out=D.Heads(C, 4, 32, 4)), dict(q_out=D.Heads(C, 4, 0, 8)),
    dict(q_out=_heads(A + 16, 4)), dict(q_out=D.Heads(A, 4, 40, 8)), dict(k_out=_heads(B + 16, 2)),
    dict(q_weight=A + 1), dict(pos=None), dict(freq=None), dict(pos=F + 4), dict(freq=G + 2),
]


@pytest.mark.parametrize("bad", NORM_BAD, ids=lambda b: "-".join(b))
def test_qk_norm_rope_refuses(bad):
    a = _norm(**bad)
    assert rl.lib().red_qk_norm_rope(ctypes.byref(a), None) == INVALID
    dq, dk = _heads(0x10000000, 4), _heads(0x11000000, 2)
    assert rl.lib().red_qk_norm_rope_backward(ctypes.byref(a), ctypes.byref(dq), ctypes.byref(dk), None, None,
                                              None) == INVALID


def test_qk_norm_rope_backward_refuses():
    f = rl.lib().red_qk_norm_rope_backward
    dq, dk = _heads(0x10000000, 4), _heads(0x11000000, 2)
    a = _norm()
    ref = ctypes.byref
    assert f(None, ref(dq), ref(dk), None, None, None) == INVALID
    assert f(ref(a), None, ref(dk), None, None, None) == INVALID
    assert f(ref(a), ref(dq), ref(_heads(0x11000000, 3)), None, None, None) == INVALID
    assert f(ref(a), ref(_heads(C + 16, 4)), ref(dk), None, None, None) == INVALID     # out over dq, shifted
    assert f(ref(a), ref(dq), ref(dk), ctypes.c_void_p(A + 2), None, None) == INVALID
    assert rl.lib().red_qk_norm_rope(None, None) == INVALID


def test_qk_norm_rope_nothing_to_do():
    L = rl.lib()
    a = _norm(tokens=0)
    assert L.red_qk_norm_rope(ctypes.byref(a), None) == rl.RED_OK
    a = _norm(q=_heads(None, 0), k=_heads(None, 0), q_out=_heads(None, 0), k_out=_heads(None, 0))
    assert L.red_qk_norm_rope(ctypes.byref(a), None) == rl.RED_OK
    dq, dk = _heads(None, 0), _heads(None, 0)
    assert L.red_qk_norm_rope_backward(ctypes.byref(a), ctypes.byref(dq), ctypes.byref(dk), None, None,
                                       None) == rl.RED_OK


def _cache(**kw):
    c = D.PagedCache(k=A, v=B, k_scales=C, v_scales=E, type=3, pages=4, heads=2, places=8, dim=16, page_stride=256,
                     head_stride=128, place_stride=16, scale_page_stride=16, scale_head_stride=8, scale_place_stride=1)
    for key, value in kw.items():
        setattr(c, key, value)
    return c


CACHE_BAD = [
    dict(type=0), dict(type=5), dict(k=None), dict(v=None), dict(k_scales=None), dict(v_scales=None), dict(heads=0),
    dict(places=0), dict(dim=0), dict(dim=257), dict(page_stride=-1), dict(page_stride=1 << 60), dict(scale_place_stride=-1),
    dict(k_scales=C + 2), dict(type=1), dict(pages=(1 << 40) + 1),
]


@pytest.mark.parametrize("bad", CACHE_BAD, ids=lambda b: "-".join(b))
def test_cache_refuses(bad):
    c, k, v = _cache(**bad), _heads(0x10000000, 2, 16), _heads(0x11000000, 2, 16)
    for f in (rl.lib().red_cache_write, rl.lib().red_cache_read):
        assert f(ctypes.byref(c), 1, ctypes.byref(k), ctypes.byref(v), F, 3, None) == INVALID


def test_cache_tokens_refuse():
    c, k, v = _cache(), _heads(0x10000000, 2, 16), _heads(0x11000000, 2, 16)
    ref = ctypes.byref
    for f in (rl.lib().red_cache_write, rl.lib().red_cache_read):
        assert f(None, 1, ref(k), ref(v), F, 3, None) == INVALID
        assert f(ref(c), 1, None, ref(v), F, 3, None) == INVALID
        for t in (0, 3, 4):
            assert f(ref(c), t, ref(k), ref(v), F, 3, None) == INVALID
        assert f(ref(c), 1, ref(_heads(0x10000000, 3, 16)), ref(v), F, 3, None) == INVALID
        assert f(ref(c), 1, ref(_heads(0x10000001, 2, 16)), ref(v), F, 3, None) == INVALID
        assert f(ref(c), 1, ref(k), ref(v), None, 3, None) == INVALID
        assert f(ref(c), 1, ref(k), ref(v), F + 4, 3, None) == INVALID
        assert f(ref(c), 1, ref(k), ref(v), F, rl.RED_MAX_N + 1, None) == INVALID
        assert f(ref(c), 1, ref(k), ref(v), F, 0, None) == rl.RED_OK
    half = _cache(type=1, k_scales=None, v_scales=None)
    assert rl.lib().red_cache_write(ref(half), 2, ref(k), ref(v), F, 3, None) == INVALID       # a cache of another type
    assert rl.lib().red_cache_read(ref(c), 1, ref(_heads(0x10000000, 2, 16, 8)), ref(v), F, 3, None) == INVALID
    none = _cache(pages=0, k=None, v=None, k_scales=None, v_scales=None)
    assert rl.lib().red_cache_write(ref(none), 1, ref(k), ref(v), F, 3, None) == rl.RED_OK


def _attend(**kw):
    c = _cache(type=1, k_scales=None, v_scales=None)
    a = D.TreeAttentionArgs(type=1, scale=0.25, batch=2, nodes=3, q_heads=4, max_len=32, q=0x10000000, out=0x11000000,
                            lse=0x12000000, q_batch_stride=192, q_node_stride=64, q_head_stride=16, out_batch_stride=192,
                            out_node_stride=64, out_head_stride=16, cache=c, table=0x13000000, table_cols=4, table_stride=4,
                            lens=0x14000000)
    for key, value in kw.items():
        setattr(a.cache if hasattr(D.PagedCache, key) and not hasattr(D.TreeAttentionArgs, key) else a, key, value)
    return a


ATTEND_BAD = [
    dict(type=0), dict(type=2), dict(type=3), dict(scale=float("inf")), dict(scale=float("nan")), dict(nodes=65), dict(q_heads=5),
    dict(batch=65536), dict(q_heads=65538), dict(max_len=(1 << 30) + 1), dict(table_stride=-1), dict(q=None), dict(out=None),
    dict(lse=None), dict(lens=None), dict(table=None), dict(q=0x10000008), dict(out=0x11000002), dict(lse=0x12000002),
    dict(table=0x13000002), dict(tree_mask=0x15000004), dict(node_count=0x15000002), dict(q_node_stride=60), dict(q_head_stride=-16),
    dict(out_head_stride=8), dict(out_node_stride=48), dict(out_batch_stride=128), dict(out=0x10000000), dict(out=0x10000000 + 128),
    dict(dim=8), dict(dim=24), dict(dim=272), dict(place_stride=20), dict(k=A + 2), dict(k=A + 8), dict(k=None),
]


@pytest.mark.parametrize("bad", ATTEND_BAD, ids=lambda b: "-".join(b))
def test_tree_attention_refuses(bad):
    a = _attend(**bad)
    assert rl.lib().red_tree_attention(ctypes.byref(a), None) == INVALID


def test_tree_attention_nothing_to_do():
    f = rl.lib().red_tree_attention
    assert f(None, None) == INVALID
    for kw in (dict(batch=0), dict(nodes=0), dict(q_heads=0)):
        assert f(ctypes.byref(_attend(**kw)), None) == rl.RED_OK


def _verify(**kw):
    a = D.VerifyDraftsArgs(type=0, batch=2, drafts=3, vocab=100, p=A, p_batch_stride=400, p_step_stride=100, q=B,
                           q_batch_stride=300, q_step_stride=100, drafted=C, u=E, r=F, draft_count=None, accepted=G,
                           tokens=0x10000000)
    for key, value in kw.items():
        setattr(a, key, value)
    return a


VERIFY_BAD = [
    dict(type=3), dict(type=5), dict(batch=65536), dict(drafts=(1 << 20) + 1), dict(vocab=0), dict(vocab=(1 << 40) + 1), dict(p=None),
    dict(drafted=None), dict(u=None), dict(r=None), dict(accepted=None), dict(tokens=None), dict(p=A + 2), dict(q=B + 1),
    dict(drafted=C + 4), dict(u=E + 2), dict(r=F + 1), dict(draft_count=2), dict(accepted=G + 2), dict(tokens=0x10000004),
    dict(p_step_stride=-1), dict(p_batch_stride=1 << 60), dict(q_step_stride=-100),
]


@pytest.mark.parametrize("bad", VERIFY_BAD, ids=lambda b: "-".join(b))
def test_verify_drafts_refuses(bad):
    assert rl.lib().red_verify_drafts(ctypes.byref(_verify(**bad)), None) == INVALID


def test_verify_drafts_nothing_to_do():
    assert rl.lib().red_verify_drafts(None, None) == INVALID
    assert rl.lib().red_verify_drafts(ctypes.byref(_verify(batch=0, p=None, r=None)), None) == rl.RED_OK


@pytest.mark.skipif(__import__("torch").cuda.device_count() > 0, reason="only meaningful where no GPU is visible")
def test_valid_arguments_reach_the_device():
    L, ref = rl.lib(), ctypes.byref
    c, k, v = _cache(), _heads(0x10000000, 2, 16), _heads(0x11000000, 2, 16)
    a, dq, dk = _norm(), _heads(0x10000000, 4), _heads(0x11000000, 2)
    for st in (L.red_qk_norm_rope(ref(a), None), L.red_qk_norm_rope_backward(ref(a), ref(dq), ref(dk), None, None, None),
               L.red_cache_write(ref(c), 1, ref(k), ref(v), F, 3, None), L.red_cache_read(ref(c), 2, ref(k), ref(v), F, 3, None),
               L.red_tree_attention(ref(_attend()), None), L.red_verify_drafts(ref(_verify()), None)):
        assert st == rl.RED_ERR_NO_DEVICE
