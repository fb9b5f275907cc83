"""Host side of the cache and attention bindings, without a GPU."""
import gc
import os
import weakref

import pytest
import torch

import mixture_experts_expert_sigmoid_amd as M
from tests.test_cache_abi import _c, _t

needs_lib = pytest.mark.skipif(not os.path.exists(M.LIB_PATH), reason="library not built")


def test_workspaces_stay_when_a_larger_one_is_needed():
    """A captured graph, or work on another stream, may still write to one that
    was handed out."""
    ws = M._Workspace("cpu")
    refs, at = [], set()
    for need in (100, 10, 1000, 1001, 5000):
        buf = ws.get(need)
        assert buf.numel() >= need
        refs.append(weakref.ref(buf))
        at.add(buf.data_ptr())
        del buf
    gc.collect()
    assert all(r() is not None for r in refs)
    assert len(at) == 4 and ws.get(1).numel() >= 5000          # 100, 1000, 2000, 5000
    assert sum(b.numel() for b in ws.buffers) <= 2 * ws.buffers[-1].numel()


class _OnGpu(torch.Tensor):
    """A host tensor that passes for one of the device."""
    is_cuda = True


def _i(*shape, dt=torch.int32):
    return torch.zeros(shape, dtype=dt)


def _calls():
    """Every binding with its tensors by name."""
    c, t, b = _c(), _t(), torch.bfloat16
    q = dict(q=_i(4, 8, 128, dt=b), out=_i(4, 8, 128, dt=b), err=_i(1), ws=_i(1 << 20),
             slots=_i(4), lse=_i(4, 8, dt=torch.float32))
    yield q, lambda q, out, err, ws, slots, lse: M.moe_attn_decode(
        c, t, q, out, 0.1, err, ws, slots=slots, lse=lse)
    yield dict(q, cu=_i(5)), lambda q, out, err, ws, slots, lse, cu: M.moe_attn_prefill(
        c, t, q, cu, out, 0.1, err, ws, slots=slots, lse=lse)
    yield dict(k=_i(4, 2, 128, dt=b), v=_i(4, 2, 128, dt=b), start=_i(4), cu=_i(5), err=_i(1),
               slots=_i(4)), lambda k, v, start, cu, err, slots: M.moe_cache_append(
        c, t, start, cu, k, v, err, slots=slots)
    yield dict(slots=_i(4), new=_i(4), start=_i(4), err=_i(1), ws=_i(1 << 20)), \
        lambda slots, new, start, err, ws: M.moe_cache_grow(t, slots, new, start, err, ws)
    yield dict(slots=_i(4), err=_i(1)), lambda slots, err: M.moe_cache_free(t, slots, err)
    yield dict(slots=_i(4), err=_i(1)), lambda slots, err: M.moe_cache_trim(t, slots, 8, 0, err)
    yield dict(src=_i(2), dst=_i(2), err=_i(1), ws=_i(1 << 20)), \
        lambda src, dst, err, ws: M.moe_cache_fork([c], t, src, dst, err, ws)
    yield dict(n=_i(1), err=_i(1), ws=_i(1 << 20)), \
        lambda n, err, ws: M.moe_cache_compact([c], t, n, err, ws)
    yield dict(src=_i(2), dst=_i(2), err=_i(1)), \
        lambda src, dst, err: M.moe_cache_copy_pages([c], src, dst, err)
    kv = dict(k=_i(10, 2, 16, 128, dt=torch.float8_e4m3fn),
              v=_i(10, 2, 16, 128, dt=torch.float8_e4m3fn),
              ks=_i(2, dt=torch.float32), vs=_i(2, dt=torch.float32))
    yield kv, lambda k, v, ks, vs: M.kv_cache(k, v, ks, vs)
    yield dict(table=_i(4, 8), lens=_i(4), refs=_i(10)), \
        lambda table, lens, refs: M.kv_table(table, lens, 16, 10, refs)


@needs_lib
@pytest.mark.parametrize("i", range(11))
def test_host_tensors_are_refused(i):
    """Any one tensor of a call in host memory: refused before the call."""
    tensors, call = list(_calls())[i]
    for bad in tensors:
        kw = {k: x if k == bad else x.as_subclass(_OnGpu) for k, x in tensors.items()}
        with pytest.raises(M.MoeError) as e:
            call(**kw)
        assert e.value.status == -5 and "cpu" in str(e.value), bad


@needs_lib
def test_error_words_and_workspaces_of_a_wrong_kind():
    for i in (0, 1, 3, 6, 7):
        tensors, call = list(_calls())[i]
        for bad, x in (("err", _i(1, dt=torch.uint8)), ("err", _i(0)),
                       ("ws", _i(1 << 20, 2)[:, 0])):
            kw = {k: t.as_subclass(_OnGpu) for k, t in dict(tensors, **{bad: x}).items()}
            with pytest.raises(M.MoeError) as e:
                call(**kw)
            assert e.value.status == -2, (i, bad)


@needs_lib
def test_upkeep_workspaces_are_aligned():
    L, t, c = M.lib(), _t(), _c()
    big, at = 1 << 40, 264                       # not a multiple of 16
    assert L.moe_cache_grow(t, 256, 256, 4, 256, 256, at, big, None) == -6
    assert L.moe_cache_fork((M.MoeKvCache * 1)(c), 1, t, 256, 256, 4, 256, at, big, None) == -6
    assert L.moe_cache_compact((M.MoeKvCache * 1)(c), 1, t, None, 256, at, big, None) == -6


def test_dimensions_of_one_entry_have_no_stride():
    """One head, or one page, of a cache: k and v that differ only in strides
    that address nothing, or have such below head_dim, are the same layout."""
    b = torch.bfloat16
    k = torch.zeros(6, 16, 64, dtype=b).unsqueeze(1)                # stride(1) = 1024
    v = torch.zeros(6, 16, 1, 64, dtype=b).transpose(1, 2)          # stride(1) = 64
    assert k.stride() != v.stride()
    small = torch.zeros(6 * 1024, dtype=b).as_strided((6, 1, 16, 64), (1024, 1, 64, 1))
    for pair in ((k, v), (v, k), (small, v)):
        c = M.kv_cache(*(x.as_subclass(_OnGpu) for x in pair))
        assert (c.stride_page, c.stride_tok, c.n_heads) == (1024, 64, 1)
        assert c.stride_head >= 64 and c.stride_head % 8 == 0
    one = torch.zeros(2 * 1024, dtype=b).as_strided((1, 2, 16, 64), (1, 1024, 64, 1))
    c = M.kv_cache(one.as_subclass(_OnGpu), torch.zeros(1, 2, 16, 64, dtype=b).as_subclass(_OnGpu))
    assert c.stride_page >= 64 and c.stride_page % 8 == 0
    assert (c.stride_head, c.stride_tok) == (1024, 64)
    k = torch.zeros(6, 2, 16, 64, dtype=b)
    for v in (torch.zeros(6, 2, 17, 64, dtype=b)[:, :, :16],
              torch.zeros(6, 16, 2, 64, dtype=b).transpose(1, 2)):
        with pytest.raises(M.MoeError):
            M.kv_cache(k, v)
