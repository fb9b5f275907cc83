"""Refusals of the cache and attention entry points: every call here returns
before any HIP call (no GPU needed)."""
import ctypes
import math
import os

import pytest

import mixture_experts_expert_sigmoid_amd as M

pytestmark = pytest.mark.skipif(not os.path.exists(M.LIB_PATH), reason="library not built")
NULL, SHAPE, FORMAT, PARAM, WS = -1, -2, -3, -5, -6
BIG = 1 << 40


def _c(**kw):
    d = dict(fmt=M.MOE_KV_BF16, n_pages=10, page_size=16, n_heads=2, head_dim=128,
             stride_page=4096, stride_head=2048, stride_tok=128, k=256, v=256, k_scale=None,
             v_scale=None)
    d.update(kw)
    return M.MoeKvCache(**d)


def _t(**kw):
    d = dict(n_slots=4, max_pages=8, ld=8, n_pages=10, page_size=16, table=256, len=256, refs=256)
    d.update(kw)
    return M.MoeKvTable(**d)


def _a(**kw):
    d = dict(fmt=M.MOE_KV_BF16, n_heads=8, q=256, q_stride_row=1024, q_stride_head=128, out=256,
             out_stride_row=1024, out_stride_head=128, lse=None, scale=0.1, window=0, n_first=0)
    d.update(kw)
    return M.MoeAttn(**d)


def _ref(x):
    return None if x is None else ctypes.byref(x)


def _decode(c=_c(), t=_t(), a=_a(), n=4, slots=256, err=256, ws=256, nb=BIG):
    return M.lib().moe_attn_decode(_ref(c), _ref(t), slots, n, _ref(a), err, ws, nb, None)


def _prefill(c=_c(), t=_t(), a=_a(), n=4, T=16, slots=256, cu=256, err=256, ws=256, nb=BIG):
    return M.lib().moe_attn_prefill(_ref(c), _ref(t), slots, n, cu, T, _ref(a), err, ws, nb, None)


def _append(c=_c(), t=_t(), n=4, T=16, slots=256, start=256, cu=256, fmt=M.MOE_KV_BF16, k=256,
            kr=256, kh=128, v=256, err=256):
    return M.lib().moe_cache_append(_ref(c), _ref(t), slots, start, cu, n, T, fmt, k, kr, kh, v,
                                    256, 128, err, None)


BAD_CACHE = [
    (None, NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(fmt=3), FORMAT),
    (dict(fmt=-1), FORMAT), (dict(n_pages=0), SHAPE), (dict(page_size=8), SHAPE),
    (dict(page_size=24), SHAPE), (dict(page_size=8192), SHAPE), (dict(n_heads=0), SHAPE),
    (dict(head_dim=96), SHAPE), (dict(head_dim=0), SHAPE), (dict(stride_tok=64), SHAPE),
    (dict(stride_tok=130), SHAPE), (dict(stride_tok=1 << 26), SHAPE),
    (dict(stride_page=-4096), SHAPE), (dict(stride_head=2052), SHAPE), (dict(k=264), PARAM),
    (dict(v=260), PARAM), (dict(k_scale=256), PARAM),
    (dict(fmt=M.MOE_KV_E4M3), NULL),
    (dict(fmt=M.MOE_KV_E4M3, k_scale=256, v_scale=256, stride_tok=136), SHAPE),
]
BAD_TABLE = [
    (None, NULL), (dict(table=None), NULL), (dict(len=None), NULL), (dict(n_slots=0), SHAPE),
    (dict(max_pages=0), SHAPE), (dict(ld=7), SHAPE), (dict(max_pages=1 << 25, ld=1 << 25), SHAPE),
    (dict(page_size=17), SHAPE), (dict(n_pages=0), SHAPE),
]


@pytest.mark.parametrize("call", [_decode, _prefill, _append])
def test_bad_descriptors(call):
    for kw, want in BAD_CACHE:
        assert call(c=None if kw is None else _c(**kw)) == want, kw
    for kw, want in BAD_TABLE:
        assert call(t=None if kw is None else _t(**kw)) == want, kw
    # the table is not this cache's
    assert call(t=_t(n_pages=11)) == SHAPE
    assert call(t=_t(page_size=32)) == SHAPE
    assert call(err=None) == NULL
    assert call(n=-1) == SHAPE and call(n=1 << 20) == SHAPE
    assert call(n=5, slots=None) == SHAPE          # more rows than slots


@pytest.mark.parametrize("call", [_decode, _prefill])
def test_bad_attention_arguments(call):
    for kw, want in [
            (dict(fmt=M.MOE_KV_E4M3), FORMAT), (dict(fmt=M.MOE_KV_F16), FORMAT),
            (dict(n_heads=0), SHAPE), (dict(n_heads=7), SHAPE), (dict(n_heads=2 * 65), SHAPE),
            (dict(q=None), NULL), (dict(out=None), NULL), (dict(q=264), PARAM),
            (dict(out=8), PARAM), (dict(q_stride_row=64), SHAPE), (dict(q_stride_head=132), SHAPE),
            (dict(out_stride_row=-1024), SHAPE), (dict(out_stride_head=64), SHAPE),
            (dict(scale=math.nan), PARAM), (dict(scale=math.inf), PARAM),
            (dict(window=-1), PARAM), (dict(n_first=-1), PARAM)]:
        assert call(a=_a(**kw)) == want, kw
    assert call(a=None) == NULL
    assert call(ws=None) == WS or call is _prefill


def test_workspaces():
    L = M.lib()
    c = _c()
    need = L.moe_attn_decode_workspace_size(ctypes.byref(c), 4, 8)
    assert need > 0 and _decode(nb=need - 1) == WS and _decode(ws=264) == WS
    # few rows: the keys are split, with a workspace; many: none needed
    need = L.moe_attn_prefill_workspace_size(ctypes.byref(c), 1, 16, 8)
    assert need > 0 and _prefill(n=1, T=16, nb=need - 1) == WS
    assert L.moe_attn_prefill_workspace_size(ctypes.byref(c), 1, 20000, 8) == 0
    for f in (lambda *a: L.moe_attn_decode_workspace_size(*a),
              lambda c_, n, h: L.moe_attn_prefill_workspace_size(c_, n, 16, h)):
        assert f(None, 4, 8) == 0 and f(ctypes.byref(c), -1, 8) == 0
        assert f(ctypes.byref(c), 4, 7) == 0
        assert f(ctypes.byref(_c(head_dim=96)), 4, 8) == 0
    t = _t()
    need = L.moe_cache_workspace_size(ctypes.byref(t), 4)
    assert need > 0 and L.moe_cache_workspace_size(None, 4) == 0
    assert L.moe_cache_workspace_size(ctypes.byref(t), -1) == 0
    tr = ctypes.byref(t)
    assert L.moe_cache_grow(tr, 256, 256, 4, 256, 256, 256, need - 1, None) == WS
    assert L.moe_cache_grow(tr, 256, 256, 4, 256, 256, None, BIG, None) == WS
    cs = (M.MoeKvCache * 1)(c)
    assert L.moe_cache_fork(cs, 1, tr, 256, 256, 4, 256, 256, need - 1, None) == WS
    assert L.moe_cache_compact(cs, 1, tr, None, 256, None, BIG, None) == WS


def test_empty_calls_do_nothing():
    assert _decode(n=0, a=_a(q=None, out=None), ws=None) == 0
    assert _prefill(T=0, a=_a(q=None, out=None), cu=None, ws=None) == 0
    assert _append(n=0, T=0, k=None, v=None, start=None, cu=None) == 0
    L, t = M.lib(), _t()
    tr, cs = ctypes.byref(t), (M.MoeKvCache * 1)(_c())
    assert L.moe_cache_grow(tr, None, None, 0, None, 256, None, 0, None) == 0
    assert L.moe_cache_free(tr, None, 0, 256, None) == 0
    assert L.moe_cache_trim(tr, None, 0, 4, 0, 256, None) == 0
    assert L.moe_cache_fork(cs, 1, tr, None, None, 0, 256, None, 0, None) == 0
    assert L.moe_cache_copy_pages(cs, 1, None, None, 0, 256, None) == 0


def test_prefill_and_append_lists():
    assert _prefill(cu=None) == NULL
    assert _prefill(n=0) == SHAPE                   # rows without a sequence
    assert _prefill(T=-1) == SHAPE and _prefill(T=1 << 30) == SHAPE
    assert _append(cu=None) == SHAPE                # T != n
    assert _append(fmt=M.MOE_KV_E4M3) == FORMAT
    assert _append(fmt=M.MOE_KV_F16) == FORMAT      # a bf16 cache
    assert _append(k=None) == NULL and _append(v=None) == NULL and _append(start=None) == NULL
    assert _append(k=264) == PARAM
    assert _append(kr=100) == SHAPE and _append(kh=64) == SHAPE
    assert _append(T=-1) == SHAPE and _append(n=0) == SHAPE


def test_upkeep_refusals():
    L = M.lib()
    c = _c()
    one = (M.MoeKvCache * 1)(c)
    for kw, want in BAD_TABLE + [(dict(refs=None), NULL)]:
        t = None if kw is None else _t(**kw)
        tr = _ref(t)
        assert L.moe_cache_grow(tr, 256, 256, 4, 256, 256, 256, BIG, None) == want, kw
        assert L.moe_cache_free(tr, 256, 4, 256, None) == want, kw
        assert L.moe_cache_trim(tr, 256, 4, 4, 0, 256, None) == want, kw
        assert L.moe_cache_fork(one, 1, tr, 256, 256, 4, 256, 256, BIG, None) == want, kw
        assert L.moe_cache_compact(one, 1, tr, None, 256, 256, BIG, None) == want, kw
    t = _t()
    tr = ctypes.byref(t)
    assert L.moe_cache_trim(tr, 256, 4, 0, 0, 256, None) == PARAM
    assert L.moe_cache_trim(tr, 256, 4, 4, -1, 256, None) == PARAM
    assert L.moe_cache_grow(tr, 256, None, 4, 256, 256, 256, BIG, None) == NULL
    assert L.moe_cache_grow(tr, 256, 256, 4, None, 256, 256, BIG, None) == NULL
    assert L.moe_cache_free(tr, 256, 4, None, None) == NULL
    assert L.moe_cache_free(tr, None, 5, 256, None) == SHAPE
    assert L.moe_cache_fork(one, 1, tr, None, 256, 4, 256, 256, BIG, None) == NULL
    assert L.moe_cache_fork(one, 1, tr, 256, 256, 65536, 256, 256, BIG, None) == SHAPE
    for layers, n, want in [(None, 1, NULL), (one, 0, SHAPE), (one, 1025, SHAPE)]:
        assert L.moe_cache_copy_pages(layers, n, 256, 256, 4, 256, None) == want
    # layers that differ in more than their pointers
    two = (M.MoeKvCache * 2)(c, _c(stride_page=8192))
    assert L.moe_cache_copy_pages(two, 2, 256, 256, 4, 256, None) == SHAPE
    two = (M.MoeKvCache * 2)(c, _c(fmt=M.MOE_KV_F16))
    assert L.moe_cache_copy_pages(two, 2, 256, 256, 4, 256, None) == FORMAT
    assert L.moe_cache_copy_pages(one, 1, 256, None, 4, 256, None) == NULL
    assert L.moe_cache_copy_pages(one, 1, 256, 256, 4, None, None) == NULL
