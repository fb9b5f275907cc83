"""Slots that end inside a page that another slot's table names too: moe_cache_keep
may cut a fork's drafted tokens back to there. Nobody's tokens are written over."""
import pytest
import torch

import mixture_experts_expert_sigmoid_amd as M
from tests.test_gpu_cache import _i

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]

PS, W = 16, 576


def _cache(kind):
    sizes = dict(n_layers=2, n_pages=24, page_size=PS, n_slots=6, max_pages=8)
    if kind == "kv":
        return M.KvCache(n_heads=2, head_dim=64, **sizes)
    return M.LatentCache(**sizes)


def _arrays(c):
    return [c.k, c.v] if isinstance(c, M.KvCache) else [c.c]


def _append(c, slots, start, cu, value):
    T = int(cu[-1])
    for i in range(2):
        if isinstance(c, M.KvCache):
            x = torch.full((T, 2, 64), value, dtype=torch.bfloat16, device="cuda")
            c.append(i, slots, start, cu, x, x)
        else:
            x = torch.full((T, W), value, dtype=torch.bfloat16, device="cuda")
            c.append(i, slots, start, cu, x[:, :512], x[:, 512:])


def _tokens(c, slot):
    """[array, layer][token] of a slot, as raw bytes."""
    n = int(c.lens[slot])
    pages = c.table[slot, :-(-n // PS)].long()
    assert int(pages.min()) >= 0
    out = []
    for x in _arrays(c):
        y = x[:, pages]                          # [layer][page]([head])[token][D]
        y = y.transpose(2, 3) if y.dim() == 5 else y
        out.append(y.reshape(2, len(pages) * PS, -1)[:, :n].clone())
    return out


def _alike(a, b):
    return all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(a, b))


@pytest.mark.parametrize("kind", ["kv", "latent"])
def test_growth_of_a_kept_fork(kind):
    """64 tokens of which 24 are drafted, forked: all four pages are shared. Kept to
    42 and 41, both slots end in the third."""
    c = _cache(kind)
    gen = torch.Generator(device="cuda").manual_seed(3)
    for x in _arrays(c):
        x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
    c.grow(_i([0, 4, 5]), _i([64, 20, 64]))
    c.fork(_i([0]), _i([1]))
    c.keep(_i([0, 1]), _i([24, 24]), _i([0, 2, 3]), _i([0, 1, 0]))
    torch.cuda.synchronize()
    assert c.lens.tolist() == [42, 41, 0, 0, 20, 64] and int(c.err_word) == 0
    assert c.table[0, 2] == c.table[1, 2]
    before = {s: _tokens(c, s) for s in (0, 1, 4, 5)}
    state = [x.clone() for x in (c.table, c.lens, c.refs)]
    raw = [x.clone() for x in _arrays(c)]

    # neither may grow there; by no tokens they may
    start = c.grow(_i([0, 1]), _i([5, 30]))
    _append(c, _i([0, 1]), start, _i([0, 5, 35]), 7.0)
    torch.cuda.synchronize()
    assert start.tolist() == [-1, -1]
    assert M.moe_read_device_error(c.err_word) == M.MOE_DEVERR_CACHE_BUSY
    assert all(torch.equal(x, y) for x, y in zip((c.table, c.lens, c.refs), state))
    assert all(torch.equal(x.view(torch.int16), y.view(torch.int16))
               for x, y in zip(_arrays(c), raw))
    c.err_word.zero_()
    assert c.grow(_i([0, 1]), _i([0, 0])).tolist() == [42, 41] and int(c.err_word) == 0

    # others of the list as if they were not in it; a whole shared page is no bar
    c.fork(_i([5]), _i([3]))
    start = c.grow(_i([4, 0, 3, 1]), _i([3, 1, 2, 200]))
    _append(c, _i([4, 0, 3, 1]), start, _i([0, 3, 4, 6, 206]), 9.0)
    torch.cuda.synchronize()
    # 200 more tokens than a row holds: full, whoever shares the page
    assert start.tolist() == [20, -1, 64, -1]
    assert int(c.err_word) == M.MOE_DEVERR_CACHE_BUSY | M.MOE_DEVERR_CACHE_FULL
    for s in (0, 1, 5):
        assert _alike(_tokens(c, s), before[s]), s
    assert all((x[:, 64:] == 9).all() for x in _tokens(c, 3))
    c.err_word.zero_()

    # a fork has a copy of that page, and goes on
    c.fork(_i([0]), _i([2]))
    start = c.grow(_i([2]), _i([30]))
    _append(c, _i([2]), start, _i([0, 30]), 11.0)
    torch.cuda.synchronize()
    assert start.tolist() == [42] and int(c.err_word) == 0
    two = _tokens(c, 2)
    assert all((x[:, 42:] == 11).all() for x in two)
    assert _alike([x[:, :42] for x in two], before[0])
    for s in (0, 1, 5):
        assert _alike(_tokens(c, s), before[s]), s

    # and so does the last slot that has it
    c.free(_i([1]))
    start = c.grow(_i([0]), _i([9]))
    _append(c, _i([0]), start, _i([0, 9]), 13.0)
    torch.cuda.synchronize()
    assert start.tolist() == [42] and int(c.err_word) == 0
    zero = _tokens(c, 0)
    assert all((x[:, 42:] == 13).all() for x in zero)
    assert _alike([x[:, :42] for x in zero], before[0]) and _alike(_tokens(c, 2), two)
