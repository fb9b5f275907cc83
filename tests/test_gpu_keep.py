"""moe_cache_keep and moe_latent_append against plain host simulations, bit for
bit."""
import numpy as np
import pytest
import torch

import mixture_experts_expert_sigmoid_amd as M
from tests.cache_ref import DT
from tests.test_gpu_cache import Sim, _cache, _i, _same

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]


def keep(sim, arrays, slots, n_draft, paths):
    """As the header states it; arrays: [layers][page][head][token][D]."""
    for s, m, path in zip(slots, n_draft, paths):
        if s < 0:
            continue
        if s >= len(sim.t):
            sim.err |= M.MOE_DEVERR_CACHE_PAGE
            continue
        L = sim.len[s]
        C, at = L - m, lambda p: (sim.t[s][p // sim.ps], p % sim.ps)
        if not 0 <= m <= L or any(a >= b for a, b in zip([-1] + path, path + [m])):
            sim.err |= M.MOE_DEVERR_TREE
            continue
        moves = [(at(C + a), at(C + j)) for j, a in enumerate(path) if a != j]
        if any(sim.refs[d] > 1 for _, (d, _) in moves if d >= 0):
            sim.err |= M.MOE_DEVERR_CACHE_BUSY
            continue
        for (a, i), (b, j) in moves:
            if a < 0 or b < 0:
                sim.err |= M.MOE_DEVERR_CACHE_PAGE
                continue
            for x in arrays:
                x[:, b, :, j] = x[:, a, :, i]
        sim.len[s] = C + len(path)
        for e in range(-(-sim.len[s] // sim.ps), -(-L // sim.ps)):
            if sim.t[s][e] >= 0:
                sim.refs[sim.t[s][e]] -= 1
            sim.t[s][e] = -1


def _call(c, slots, n_draft, paths):
    cu = np.concatenate([[0], np.cumsum([len(p) for p in paths])])
    c.keep(_i(slots), _i(n_draft), _i(cu.tolist()), _i([a for p in paths for a in p] + [0]))


def _check(c, sim, host, where):
    _same(c, sim, where)
    for x, y in zip((c.k, c.v), host):
        assert torch.equal(x.view(torch.uint8).cpu(), y.view(torch.uint8)), where


@pytest.mark.parametrize("ps,layers,hkv,D,dtype", [
    (16, 2, 2, 64, "bf16"), (48, 1, 3, 128, "e4m3"), (32, 35, 1, 256, "f16"),
    (16, 3, 8, 128, "bf16")])
def test_paths(ps, layers, hkv, D, dtype):
    """Paths of every kind, turn after turn, with growth between them: places
    that are sources of earlier tokens, pages that end inside, nothing accepted,
    all accepted, single tokens, a slot twice as long as a step's tokens."""
    rng = np.random.default_rng(ps + D)
    S, mp, P = 7, 24, 120
    sc = torch.ones(layers, hkv, device="cuda")
    c = M.KvCache(n_layers=layers, n_pages=P, page_size=ps, n_heads=hkv, head_dim=D, n_slots=S,
                  max_pages=mp, dtype=DT[dtype],
                  **(dict(k_scale=sc, v_scale=sc) if dtype == "e4m3" else {}))
    for x in (c.k, c.v):
        x.view(torch.uint8).copy_(torch.randint(0, 256, x.view(torch.uint8).shape,
                                                device="cuda", dtype=torch.uint8))
    sim = Sim(S, mp, P, ps)
    host = [x.cpu() for x in (c.k, c.v)]
    raw = [x.view(torch.uint8) for x in host]
    for turn in range(6):
        slots = [int(x) for x in rng.permutation(S)]
        new = [int(x) for x in rng.choice([1, 2, 5, 17, 33, 70], S)]
        c.grow(_i(slots), _i(new))
        sim.grow(slots, new)
        paths = []
        for i, m in enumerate(new):
            k = [0, 1, m, m // 2, min(m, 9), m, m - 1][(i + turn) % 7]
            paths.append(sorted(rng.choice(m, k, replace=False).tolist()))
        # 1, 2, 3, ...: every place but the last is the one before's source
        paths[turn % S] = list(range(1, new[turn % S]))
        _call(c, slots, new, paths)
        keep(sim, raw, slots, new, paths)
        _check(c, sim, host, turn)


def test_refusals_leave_the_slot():
    """Paths that are none, lists without a slot, shared pages, pages that are
    not there: only the slot concerned is left as it was."""
    c = _cache(8, 8, 60, 16, layers=2, hkv=2, D=64)
    sim = Sim(8, 8, 60, 16)
    host = [x.cpu() for x in (c.k, c.v)]
    raw = [x.view(torch.uint8) for x in host]
    for step in (([0, 1, 2, 3, 4], [40, 40, 40, 40, 40]), ([0, 1, 2, 3, 4], [12] * 5)):
        c.grow(_i(step[0]), _i(step[1]))
        sim.grow(*step)

    def turn(slots, n_draft, paths, err):
        _call(c, slots, n_draft, paths)
        keep(sim, raw, slots, n_draft, paths)
        assert sim.err == err
        _check(c, sim, host, (slots, paths))
        c.err_word.zero_()
        sim.err = 0

    tree, busy, page = M.MOE_DEVERR_TREE, M.MOE_DEVERR_CACHE_BUSY, M.MOE_DEVERR_CACHE_PAGE
    for bad in ([3, 3], [4, 2], [0, 12], [-1, 4], [1, 1 << 30], list(range(13))):
        turn([0, 1], [12, 12], [bad, []], tree)
        c.grow(_i([1]), _i([12]))
        sim.grow([1], [12])
    turn([0, 1], [53, 12], [[], [2]], tree)              # more than the slot holds
    turn([0, 1], [-1, 0], [[], []], tree)
    turn([-1, 8, 2], [12, 12, 12], [[5], [5], [5, 7]], page)
    # a fork of drafted tokens shares their pages
    c.grow(_i([3]), _i([12]))                            # 64 tokens: four whole pages
    sim.grow([3], [12])
    c.fork(_i([3]), _i([6]))
    for a, b in sim.fork([3], [6]):
        for x in raw:
            x[:, b] = x[:, a]
    turn([3, 4, 6], [24, 12, 24], [[1, 3], [1, 3], [1, 3]], busy)
    turn([3, 6], [24, 24], [[0, 1], [0]], 0)             # nothing is written: given back
    # a page taken out of the table
    c.table[0, 2] = -1
    sim.t[0][2] = -1
    turn([0], [12], [[2, 9, 11]], page)


def test_a_slot_named_twice():
    """Not allowed, and what becomes of that slot is open; but nothing is read or
    written outside its own tokens, other slots are as if it had not been there,
    and no page is given back twice."""
    c = _cache(6, 8, 48, 16, layers=2, hkv=2, D=64)
    sim = Sim(6, 8, 48, 16)
    host = [x.cpu() for x in (c.k, c.v)]
    raw = [x.view(torch.uint8) for x in host]
    new = [60, 60, 60, 60, 60]
    c.grow(_i([0, 1, 2, 3, 4]), _i(new))
    sim.grow([0, 1, 2, 3, 4], new)
    paths = [[1, 5], [0, 30, 31, 58], [2, 4, 40], list(range(0, 60, 3)), [9]]
    _call(c, [0, 2, 2, 2, 4], [40, 60, 45, 60, 20], paths)
    keep(sim, raw, [0, 4], [40, 20], [paths[0], paths[4]])
    assert M.moe_read_device_error(c.err_word) & ~M.MOE_DEVERR_TREE == 0
    other = [0, 1, 3, 4]
    table, refs = c.table.cpu(), c.refs.cpu()
    assert c.lens[other].tolist() == [sim.len[s] for s in other]
    for s in other:
        assert table[s].tolist() == list(sim.t[s])
    mine = {int(e) for e in table[2] if e >= 0} | {e for e in sim.t[2] if e >= 0}
    assert 0 <= int(c.lens[2]) <= 60 and set(refs.tolist()) <= {0, 1}
    for x, y in zip((c.k, c.v), host):
        for p in range(48):
            if p not in mine:
                assert torch.equal(x[:, p].view(torch.uint8).cpu(), y[:, p].view(torch.uint8)), p


def test_list_entries_outside_the_path():
    """cu beyond the path, falling or negative: those entries are left."""
    c = _cache(4, 4, 20, 16, layers=1)
    sim = Sim(4, 4, 20, 16)
    for x in (c, sim):
        x.grow(*(([0, 1, 2, 3], [20] * 4) if x is sim else (_i([0, 1, 2, 3]), _i([20] * 4))))
    path = _i([1, 4, 6, 8])
    for cu, good in [([0, 2, 5, 5, 4], {0: [1, 4]}), ([-1, 2, 3, 1, 4], {1: [6], 3: [4, 6, 8]})]:
        host = [x.cpu() for x in (c.k, c.v)]
        c.keep(_i([0, 1, 2, 3]), _i([10] * 4), _i(cu), path)
        for s, p in good.items():
            keep(sim, [x.view(torch.uint8) for x in host], [s], [10], [p])
        sim.err = M.MOE_DEVERR_TREE
        _check(c, sim, host, cu)


def test_graph():
    """Captured once, with other drafts and paths at each replay, eager calls
    between them."""
    c = _cache(3, 20, 60, 16, layers=2)
    sim = Sim(3, 20, 60, 16)
    host = [x.cpu() for x in (c.k, c.v)]
    raw = [x.view(torch.uint8) for x in host]
    slots, m, cu, path = _i([0, 2, -1]), _i([0] * 3), _i([0] * 4), _i([0] * 64)
    c.keep(slots, m, cu, path)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.keep(slots, m, cu, path)
    for a, b in [([1, 2, 9], []), ([0], [3, 8, 15]), (list(range(16)), [15])]:
        c.grow(_i([0, 2]), _i([20, 16]))
        sim.grow([0, 2], [20, 16])
        m.copy_(_i([20, 16, 0]))
        cu.copy_(_i([0, len(a), len(a) + len(b), len(a) + len(b)]))
        path[:len(a) + len(b)] = _i(a + b)
        g.replay()
        keep(sim, raw, [0, 2], [20, 16], [a, b])
        _check(c, sim, host, (a, b))


# ------------------------------------------------------------ latent rows

def _codes(x, sc):
    """What a cache of this type keeps of 16-bit rows."""
    if sc is None:
        return x
    y = x.float() / sc                   # the fp32 quotient, then the code
    return torch.where(y.isnan(), y, y.clamp(-448, 448)).to(torch.float8_e4m3fn)


# dt, cache, latent_dim, page, rows of each, starts, gaps in the cache's rows, in the inputs'
APPEND = {
    "one_each": ("bf16", "bf16", 512, 16, None, [0, 15, 16, -1, 100], 0, 0),
    "prompts": ("f16", "f16", 256, 48, [0, 1, 47, 200], [3, 0, 1, 70], 0, 8),
    "e4m3": ("bf16", "e4m3", 512, 64, [33, 1, 130], [60, 7, 0], 0, 64),
    "e4m3_f16": ("f16", "e4m3", 256, 16, [5, 64], [0, 11], 16, 0),
    "gaps": ("bf16", "bf16", 512, 16, [7, 30], [9, 2], 24, 16),
    "many": ("bf16", "e4m3", 512, 64, [4000, 5001], [1, 0], 0, 0),
}


@pytest.mark.parametrize("name", list(APPEND))
def test_latent_append(name):
    dt, kv, dc, ps, rows, starts, gap, pad = APPEND[name]
    rng = np.random.default_rng(len(name))
    n = len(starts)
    m = [1] * n if rows is None else rows
    T, W = sum(m), dc + 64
    need = [-(-(max(s, 0) + k) // ps) for s, k in zip(starts, m)]
    P = sum(need) + 2
    tab = np.full((n, max(need) + 1), -1, np.int32)
    order, at = rng.permutation(P), 0
    for i, k in enumerate(need):
        tab[i, :k] = order[at:at + k]
        at += k
    gen = torch.Generator(device="cuda").manual_seed(1)
    pool = torch.randint(0, 256, (P, ps, (W + gap) * (1 if kv == "e4m3" else 2)), generator=gen,
                         device="cuda", dtype=torch.uint8).view(DT[kv])[..., :W]
    full = pool.clone()
    sc = torch.tensor([0.0173], device="cuda") if kv == "e4m3" else None
    new = (3 * torch.randn(T, W + pad, generator=gen, device="cuda")).to(DT[dt])
    new[0, :6] = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), 60000.0])
    c, r = new[:, :dc], new[:, dc:W]
    cache = M.latent_cache(pool, dc, sc)
    table = M.kv_table(torch.from_numpy(tab).cuda(), _i([0] * n), ps, P)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = None if rows is None else _i(np.concatenate([[0], np.cumsum(m)]).tolist())
    M.moe_latent_append(cache, table, _i(starts), cu, c, r, err)
    codes = _codes(new[:, :W], sc)
    at = 0
    for i, (s, k) in enumerate(zip(starts, m)):
        for j in range(k if s >= 0 else 0):
            full[int(tab[i, (s + j) // ps]), (s + j) % ps] = codes[at + j]
        at += k
    torch.cuda.synchronize()
    bits = torch.uint8 if kv == "e4m3" else torch.int16
    got, ref = pool.contiguous().view(bits), full.contiguous().view(bits)
    if kv == "e4m3":                     # one code of a NaN or the other
        nan = (ref & 0x7F) == 0x7F
        assert ((got & 0x7F) == 0x7F)[nan].all()
        got, ref = got[~nan], ref[~nan]
    assert torch.equal(got, ref)
    assert M.moe_read_device_error(err) == 0


def test_latent_append_without_a_page():
    """Tokens without a page, beyond the table or of a slot beyond it: flagged,
    the others written."""
    pool = torch.zeros(3, 16, 320, dtype=torch.bfloat16, device="cuda")
    tab = torch.tensor([[0, -1, 1], [2, 7, -1]], dtype=torch.int32, device="cuda")
    cache, table = M.latent_cache(pool, 256), M.kv_table(tab, _i([0, 0]), 16, 3)
    new = torch.ones(60, 320, dtype=torch.bfloat16, device="cuda")
    for slots, start, cu, filled in [([0], [10], [0, 30], {0: range(10, 16), 1: range(8)}),
                                     ([1], [12], [0, 20], {2: range(12, 16)}),
                                     ([0], [40], [0, 20], {1: range(8, 16)}),
                                     ([2, 1], [0, 3], [0, 4, 7], {2: range(3, 6)})]:
        pool.zero_()
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        k = cu[-1]
        M.moe_latent_append(cache, table, _i(start), _i(cu), new[:k, :256], new[:k, 256:], err,
                            slots=_i(slots))
        want = torch.zeros_like(pool)
        for p, rows in filled.items():
            want[p, list(rows)] = 1
        torch.cuda.synchronize()
        assert torch.equal(pool, want), (slots, start)
        assert M.moe_read_device_error(err) == M.MOE_DEVERR_CACHE_PAGE


@pytest.mark.parametrize("kv,dc,gap", [("bf16", 512, 0), ("e4m3", 256, 16), ("f16", 512, 24)])
def test_pages_of_a_latent_cache_move(kv, dc, gap):
    """fork, compact, copy_pages and keep over a latent cache's array."""
    W, ps, P, S = dc + 64, 16, 24, 5
    es = 1 if kv == "e4m3" else 2
    raw = torch.randint(0, 256, (2, P, ps, (W + gap) * es), device="cuda", dtype=torch.uint8)
    pools = [x.view(DT[kv])[..., :W] for x in raw]
    sc = torch.ones(1, device="cuda") if kv == "e4m3" else None
    caches = [M.moe_latent_pages(M.latent_cache(x, dc, sc)) for x in pools]
    tab, lens, refs = torch.full((S, 4), -1, dtype=torch.int32, device="cuda"), _i([0] * S), \
        _i([0] * P)
    table = M.kv_table(tab, lens, ps, P, refs)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(M.moe_cache_workspace_size(table, 8), dtype=torch.uint8, device="cuda")
    sim = Sim(S, 4, P, ps)
    host = raw.cpu()

    def same(where):
        torch.cuda.synchronize()
        assert tab.tolist() == sim.t and lens.tolist() == sim.len and refs.tolist() == sim.refs
        got = raw.cpu()
        assert torch.equal(got[..., :W * es], host[..., :W * es]), where
        assert M.moe_read_device_error(err) == 0

    M.moe_cache_grow(table, _i([0, 1, 2]), _i([40, 17, 33]), _i([0] * 3), err, ws)
    sim.grow([0, 1, 2], [40, 17, 33])
    M.moe_cache_fork(caches, table, _i([0, 2]), _i([3, 4]), err, ws)
    for a, b in sim.fork([0, 2], [3, 4]):
        host[:, b] = host[:, a]
    same("fork")
    M.moe_cache_keep(caches, table, _i([7, 12]), _i([0, 3, 5]), _i([1, 2, 6, 4, 11]), err,
                     slots=_i([3, 1]))
    # [layers][page][token][bytes] -> with a head axis
    keep(sim, [host[:, :, None]], [3, 1], [7, 12], [[1, 2, 6], [4, 11]])
    same("keep")
    M.moe_cache_free(table, _i([0]), err)
    sim.free([0])
    M.moe_cache_compact(caches, table, None, err, ws)
    moves = sim.compact()[1]
    before = host.clone()
    for a, b in moves:
        host[:, b] = before[:, a]
    same("compact")
    M.moe_cache_copy_pages(caches, _i([0, 1]), _i([20, 21]), err)
    host[:, 20], host[:, 21] = host[:, 0].clone(), host[:, 1].clone()
    same("copy")
