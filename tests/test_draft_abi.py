"""Refusals of the calls for drafted trees and for latent attention, and the host
side of their bindings: every call here returns before any HIP call (no GPU
needed)."""
import math
import os

import pytest
import torch

import mixture_experts_expert_sigmoid_amd as M
from tests.test_cache_abi import (BAD_CACHE, BAD_TABLE, BIG, FORMAT, NULL, PARAM, SHAPE, WS, _a,
                                  _c, _ref, _t)
from tests.test_kv_host import _i, _OnGpu

pytestmark = pytest.mark.skipif(not os.path.exists(M.LIB_PATH), reason="library not built")


def _lc(**kw):
    d = dict(fmt=M.MOE_KV_BF16, n_pages=10, page_size=16, latent_dim=512, rope_dim=64,
             stride_page=9216, stride_tok=576, c=256, scale=None)
    d.update(kw)
    return M.MoeLatentCache(**d)


def _la(**kw):
    return _a(**{**dict(q_stride_row=8 * 576, q_stride_head=576, out_stride_row=8 * 512,
                        out_stride_head=512), **kw})


def _pa(**kw):
    return _a(**{**dict(q_stride_row=8 * 192, q_stride_head=192), **kw})


def _kr(**kw):
    d = dict(k=256, k_stride_row=1024, k_stride_head=128, k_rope=256, rope_stride_row=64, v=256,
             v_stride_row=1024, v_stride_head=128)
    d.update(kw)
    return M.MoeLatentRows(**d)


def _tree(c=_c(), t=_t(), a=_a(), n=4, T=16, slots=256, cu=256, parent=256, err=256, ws=256,
          nb=BIG):
    return M.lib().moe_attn_tree(_ref(c), _ref(t), slots, n, cu, T, parent, _ref(a), err, ws, nb,
                                 None)


def _latent(c=_lc(), t=_t(), a=_la(), n=4, T=16, slots=256, cu=256, parent=None, err=256, ws=256,
            nb=BIG):
    return M.lib().moe_attn_latent(_ref(c), _ref(t), slots, n, cu, T, parent, _ref(a), err, ws,
                                   nb, None)


def _prompt(kv=_kr(), a=_pa(), n=4, cu_k=256, S=40, cu=256, T=16, ws=256, nb=BIG):
    return M.lib().moe_attn_latent_prompt(_ref(kv), n, cu_k, S, cu, T, _ref(a), ws, nb, None)


def _lappend(c=_lc(), t=_t(), n=4, T=16, slots=256, start=256, cu=256, fmt=M.MOE_KV_BF16, x=256,
             xr=512, r=256, rr=64, err=256):
    return M.lib().moe_latent_append(_ref(c), _ref(t), slots, start, cu, n, T, fmt, x, xr, r, rr,
                                     err, None)


def _keep(c=(_c(),), t=_t(), slots=256, n_draft=256, cu=256, path=256, n_path=16, n=4, err=256,
          layers=None):
    arr = None if c is None else (M.MoeKvCache * len(c))(*c)
    return M.lib().moe_cache_keep(arr, len(c or ()) if layers is None else layers, _ref(t), slots,
                                  n_draft, cu, path, n_path, n, err, None)


BAD_LATENT = [
    (None, NULL), (dict(c=None), NULL), (dict(fmt=3), FORMAT), (dict(fmt=-1), FORMAT),
    (dict(n_pages=0), SHAPE), (dict(page_size=8), SHAPE), (dict(page_size=24), SHAPE),
    (dict(page_size=8192), SHAPE), (dict(latent_dim=128), SHAPE), (dict(latent_dim=0), SHAPE),
    (dict(rope_dim=32), SHAPE), (dict(stride_tok=568), SHAPE), (dict(stride_tok=580), SHAPE),
    (dict(stride_tok=1 << 26), SHAPE), (dict(stride_page=-9216), SHAPE),
    (dict(stride_page=9220), SHAPE), (dict(c=264), PARAM), (dict(scale=256), PARAM),
    (dict(fmt=M.MOE_KV_E4M3), NULL), (dict(fmt=M.MOE_KV_E4M3, scale=256, stride_tok=584), SHAPE),
]
BAD_ATTN = [
    (dict(fmt=M.MOE_KV_E4M3), FORMAT), (dict(n_heads=0), SHAPE), (dict(q=None), NULL),
    (dict(out=None), NULL), (dict(q=264), PARAM), (dict(out=8), PARAM),
    (dict(q_stride_row=64), SHAPE), (dict(q_stride_head=132), SHAPE),
    (dict(out_stride_row=-1024), SHAPE), (dict(out_stride_head=64), SHAPE),
    (dict(scale=math.nan), PARAM), (dict(scale=math.inf), PARAM), (dict(window=-1), PARAM),
    (dict(n_first=-1), PARAM)]


@pytest.mark.parametrize("call,cache,bad", [
    (_tree, _c, BAD_CACHE), (_latent, _lc, BAD_LATENT), (_lappend, _lc, BAD_LATENT)])
def test_bad_descriptors(call, cache, bad):
    for kw, want in bad:
        assert call(c=None if kw is None else cache(**kw)) == want, kw
    for kw, want in BAD_TABLE:
        assert call(t=None if kw is None else _t(**kw)) == want, kw
    assert call(t=_t(n_pages=11)) == SHAPE and call(t=_t(page_size=32)) == SHAPE
    assert call(err=None) == NULL
    assert call(n=-1) == SHAPE and call(n=1 << 20) == SHAPE
    assert call(n=5, slots=None) == SHAPE          # more sequences than slots
    assert call(n=0) == SHAPE                      # rows without a sequence
    assert call(T=-1) == SHAPE and call(T=1 << 31) == SHAPE


@pytest.mark.parametrize("call,attn", [(_tree, _a), (_latent, _la), (_prompt, _pa)])
def test_bad_attention_arguments(call, attn):
    for kw, want in BAD_ATTN:
        assert call(a=attn(**kw)) == want, kw
    assert call(a=None) == NULL
    if call is not _prompt:
        assert call(a=attn(fmt=M.MOE_KV_F16)) == FORMAT          # a bf16 cache
    for heads in ((7, 2 * 65) if call is _tree else (1025,)):
        assert call(a=attn(n_heads=heads)) == SHAPE
    assert call(T=(1 << 31) // 8) == SHAPE                       # rows * heads


def test_lists():
    assert _tree(cu=None) == NULL and _tree(parent=None) == NULL
    assert _latent(cu=None) == SHAPE                             # T != n
    assert _prompt(cu=None) == NULL and _prompt(cu_k=None) == NULL
    assert _prompt(n=0) == SHAPE and _prompt(n=-1) == SHAPE and _prompt(n=1 << 20) == SHAPE
    assert _prompt(S=-1) == SHAPE and _prompt(S=(1 << 28) + 1) == SHAPE and _prompt(T=-1) == SHAPE
    assert _lappend(cu=None) == SHAPE and _lappend(start=None) == NULL
    assert _lappend(fmt=M.MOE_KV_E4M3) == FORMAT and _lappend(fmt=M.MOE_KV_F16) == FORMAT
    assert _lappend(x=None) == NULL and _lappend(r=None) == NULL
    assert _lappend(x=264) == PARAM and _lappend(r=8) == PARAM
    assert _lappend(xr=504) == SHAPE and _lappend(rr=68) == SHAPE
    for kw, want in [(None, NULL), (dict(k=None), NULL), (dict(k_rope=None), NULL),
                     (dict(v=None), NULL), (dict(k=264), PARAM), (dict(v=8), PARAM),
                     (dict(k_rope=24), PARAM), (dict(k_stride_row=120), SHAPE),
                     (dict(k_stride_head=132), SHAPE), (dict(v_stride_row=1 << 25), SHAPE),
                     (dict(v_stride_head=-128), SHAPE), (dict(rope_stride_row=60), SHAPE)]:
        assert _prompt(kv=None if kw is None else _kr(**kw)) == want, kw


def test_keep_refusals():
    for kw, want in BAD_CACHE[1:]:
        assert _keep(c=(_c(**kw),)) == want, kw
    for kw, want in BAD_TABLE + [(dict(refs=None), NULL)]:
        assert _keep(t=None if kw is None else _t(**kw)) == want, kw
    assert _keep(c=None, layers=1) == NULL
    assert _keep(layers=0) == SHAPE and _keep(layers=1025) == SHAPE
    assert _keep(c=(_c(), _c(stride_page=8192))) == SHAPE
    assert _keep(c=(_c(), _c(fmt=M.MOE_KV_F16))) == FORMAT
    assert _keep(n=-1) == SHAPE and _keep(n=1 << 20) == SHAPE
    assert _keep(n=5, slots=None) == SHAPE
    assert _keep(n_path=-1) == SHAPE and _keep(n_path=1 << 31) == SHAPE
    assert _keep(err=None) == NULL
    assert _keep(n_draft=None) == NULL and _keep(cu=None) == NULL and _keep(path=None) == NULL


def test_empty_calls_do_nothing():
    none = dict(q=None, out=None)
    assert _tree(n=0, T=0, a=_a(**none), cu=None, parent=None, ws=None) == 0
    assert _tree(T=0, a=_a(**none), cu=None, parent=None, ws=None) == 0
    assert _latent(n=0, T=0, a=_la(**none), cu=None, ws=None) == 0
    assert _prompt(n=0, T=0, S=0, a=_pa(**none), cu=None, cu_k=None, ws=None,
                   kv=_kr(k=None, v=None, k_rope=None)) == 0
    assert _lappend(n=0, T=0, x=None, r=None, start=None, cu=None) == 0
    assert _keep(n=0, n_draft=None, cu=None, path=None, n_path=0) == 0


def test_workspaces():
    L, c, lc = M.lib(), _c(), _lc()
    need = L.moe_attn_tree_workspace_size(_ref(c), 1, 16, 8)
    assert need > 0 and _tree(n=1, nb=need - 1) == WS and _tree(n=1, ws=264) == WS
    assert _tree(n=1, ws=None) == WS
    need = L.moe_attn_latent_workspace_size(_ref(lc), 4, 16, 8)
    assert need > 0 and _latent(nb=need - 1) == WS and _latent(ws=264) == WS
    assert _latent(ws=None) == WS
    need = L.moe_attn_latent_prompt_workspace_size(1, 16, 8)
    assert need > 0 and _prompt(n=1, nb=need - 1) == WS and _prompt(n=1, ws=None) == WS
    for f, d in ((L.moe_attn_tree_workspace_size, c), (L.moe_attn_latent_workspace_size, lc)):
        assert f(None, 4, 16, 8) == 0 and f(_ref(d), -1, 16, 8) == 0
        assert f(_ref(d), 4, -1, 8) == 0 and f(_ref(d), 4, 1 << 30, 8) == 0
    assert L.moe_attn_tree_workspace_size(_ref(c), 4, 16, 7) == 0
    assert L.moe_attn_latent_workspace_size(_ref(_lc(latent_dim=128)), 4, 16, 8) == 0
    assert L.moe_attn_latent_workspace_size(_ref(lc), 4, 16, 1025) == 0
    assert L.moe_attn_latent_prompt_workspace_size(4, 16, 0) == 0
    assert L.moe_attn_latent_prompt_workspace_size(-1, 16, 8) == 0


def test_a_latent_cache_as_pages():
    """Moved with every value of its tokens, and refused by nothing that moves
    pages; a table that is not its own is."""
    lc, pages = _lc(stride_page=10240, stride_tok=640), M.MoeKvCache()
    L = M.lib()
    assert L.moe_latent_pages(_ref(lc), _ref(pages)) == 0
    assert (pages.n_heads * pages.head_dim, pages.stride_head) == (576, 64)
    assert (pages.k, pages.v, pages.stride_page, pages.stride_tok) == (256, 256, 10240, 640)
    assert _keep(c=(pages,), n=0) == 0 and _keep(c=(pages,), t=_t(n_pages=11)) == SHAPE
    for kw, want in BAD_LATENT:
        assert L.moe_latent_pages(None if kw is None else _ref(_lc(**kw)), _ref(pages)) == want
    assert L.moe_latent_pages(_ref(lc), None) == NULL


# ------------------------------------------------------------- the bindings

def _calls():
    """Every binding with its tensors by name, as a call of them."""
    c, t, lc, b, f = _c(), _t(), _lc(), torch.bfloat16, torch.float32
    q = dict(q=_i(4, 8, 128, dt=b), out=_i(4, 8, 128, dt=b), err=_i(1), ws=_i(1 << 20),
             slots=_i(4), lse=_i(4, 8, dt=f), cu=_i(5))
    yield dict(q, parent=_i(4)), lambda q, out, err, ws, slots, lse, cu, parent: M.moe_attn_tree(
        c, t, q, cu, parent, out, 0.1, err, ws, slots=slots, lse=lse)
    yield dict(q, q=_i(4, 8, 576, dt=b), out=_i(4, 8, 512, dt=b), parent=_i(4)), \
        lambda q, out, err, ws, slots, lse, cu, parent: M.moe_attn_latent(
            lc, t, q, cu, out, 0.1, err, ws, parent=parent, slots=slots, lse=lse)
    yield dict(q=_i(4, 8, 192, dt=b), k=_i(9, 8, 128, dt=b), r=_i(9, 64, dt=b),
               v=_i(9, 8, 128, dt=b), out=_i(4, 8, 128, dt=b), ws=_i(1 << 20),
               lse=_i(4, 8, dt=f), cu=_i(5), cu_k=_i(5)), \
        lambda q, k, r, v, out, ws, lse, cu, cu_k: M.moe_attn_latent_prompt(
            q, k, r, v, cu, cu_k, out, 0.1, ws, lse=lse)
    yield dict(x=_i(4, 512, dt=b), r=_i(4, 64, dt=b), start=_i(4), cu=_i(5), err=_i(1),
               slots=_i(4)), lambda x, r, start, cu, err, slots: M.moe_latent_append(
        lc, t, start, cu, x, r, err, slots=slots)
    yield dict(n_draft=_i(4), cu=_i(5), path=_i(9), err=_i(1), slots=_i(4)), \
        lambda n_draft, cu, path, err, slots: M.moe_cache_keep(
            [c], t, n_draft, cu, path, err, slots=slots)
    yield dict(x=_i(10, 16, 576, dt=torch.float8_e4m3fn), s=_i(1, dt=f)), \
        lambda x, s: M.latent_cache(x, 512, s)


@pytest.mark.parametrize("i", range(6))
def test_host_tensors_are_refused(i):
    """Any one tensor of a call in host memory: refused before the call."""
    tensors, call = list(_calls())[i]
    for bad in tensors:
        kw = {k: x if k == bad else x.as_subclass(_OnGpu) for k, x in tensors.items()}
        with pytest.raises(M.MoeError) as e:
            call(**kw)
        assert e.value.status == -5 and "cpu" in str(e.value), bad


@pytest.mark.parametrize("i,name,shape", [
    (0, "out", (4, 8, 64)), (0, "parent", (3,)), (0, "q", (4, 8, 64)), (0, "lse", (4, 7)),
    (1, "q", (4, 8, 512)), (1, "out", (4, 8, 576)), (1, "out", (4, 7, 512)), (1, "parent", (3,)),
    (2, "q", (4, 8, 128)), (2, "out", (4, 8, 192)), (2, "k", (9, 7, 128)), (2, "v", (8, 8, 128)),
    (2, "r", (9, 128)), (2, "r", (8, 64)), (2, "cu_k", (4,)), (2, "k", (9, 1024)),
    (3, "x", (4, 576)), (3, "r", (3, 64)), (3, "slots", (3,)), (4, "cu", (4,)),
    (4, "slots", (3,)), (5, "x", (10, 16, 500)), (5, "s", (2,)), (5, "x", (16, 576))])
def test_shapes_that_do_not_fit(i, name, shape):
    tensors, call = list(_calls())[i]
    kw = {k: x.as_subclass(_OnGpu) for k, x in tensors.items()}
    kw[name] = _i(*shape, dt=tensors[name].dtype).as_subclass(_OnGpu)
    with pytest.raises(M.MoeError) as e:
        call(**kw)
    assert e.value.status == SHAPE


@pytest.mark.parametrize("i,name,dt,status", [
    (0, "out", torch.float16, SHAPE), (1, "q", torch.float32, SHAPE),
    (2, "v", torch.float16, SHAPE), (2, "r", torch.float32, SHAPE), (3, "r", torch.float16, SHAPE),
    (0, "parent", torch.int64, SHAPE), (4, "path", torch.int64, SHAPE),
    (5, "x", torch.float32, FORMAT), (5, "s", torch.float64, SHAPE)])
def test_types_that_do_not_fit(i, name, dt, status):
    tensors, call = list(_calls())[i]
    kw = {k: x.as_subclass(_OnGpu) for k, x in tensors.items()}
    kw[name] = tensors[name].to(dt).as_subclass(_OnGpu)
    with pytest.raises(M.MoeError) as e:
        call(**kw)
    assert e.value.status == status


def test_strides_of_latent_rows():
    """Rows with gaps keep them; a dimension of one entry has no stride of its own."""
    x = _i(10, 16, 640, dt=torch.bfloat16).as_subclass(_OnGpu)
    d = M.latent_cache(x[:, :, :576], 512)
    assert (d.stride_page, d.stride_tok, d.latent_dim, d.rope_dim) == (10240, 640, 512, 64)
    assert M.latent_cache(x[3:4, :, :576], 512).stride_page == 16 * 576
    with pytest.raises(M.MoeError):
        M.latent_cache(x.transpose(1, 2), 512)
    with pytest.raises(M.MoeError):
        M.latent_cache(x, 1024)
