"""Page upkeep and append against a plain host simulation, bit for bit."""
import numpy as np
import pytest
import torch

import mixture_experts_expert_sigmoid_amd as M
from tests.cache_ref import DT

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]


class Sim:
    """The pool's bookkeeping as the header states it, one page at a time."""

    def __init__(self, slots, max_pages, P, ps):
        self.t = [[-1] * max_pages for _ in range(slots)]
        self.len, self.refs, self.ps, self.P, self.mp = [0] * slots, [0] * P, ps, P, max_pages
        self.err = 0

    def _free(self):
        return [p for p in range(self.P) if self.refs[p] == 0]

    def grow(self, slots, new):
        free, start = self._free(), []
        asked = 0
        taken = {}
        for i, (s, a) in enumerate(zip(slots, new)):
            if s < 0:
                start.append(-1)
                continue
            have, want = -(-self.len[s] // self.ps), -(-(self.len[s] + a) // self.ps)
            if want > self.mp:
                self.err |= M.MOE_DEVERR_CACHE_FULL
                start.append(-1)
                continue
            need = want - have
            first = asked
            asked += need
            if need and asked > len(free):
                self.err |= M.MOE_DEVERR_CACHE_FULL
                start.append(-1)
                continue
            for j in range(need):
                taken[free[first + j]] = 1
                self.t[s][have + j] = free[first + j]
            start.append(self.len[s])
            self.len[s] += a
        for p in taken:
            self.refs[p] = 1
        return start

    def free(self, slots):
        for s in slots:
            if s < 0:
                continue
            for j in range(-(-self.len[s] // self.ps)):
                if self.t[s][j] >= 0:
                    self.refs[self.t[s][j]] -= 1
                self.t[s][j] = -1
            self.len[s] = 0

    def trim(self, slots, window, first):
        for s in slots:
            if s < 0:
                continue
            for j in range(self.mp):
                a, b = j * self.ps, (j + 1) * self.ps
                if self.t[s][j] >= 0 and a >= first and b <= self.len[s] - window:
                    self.refs[self.t[s][j]] -= 1
                    self.t[s][j] = -1

    def fork(self, src, dst):
        free, copies, used = self._free(), [], 0
        todo = []
        for a, b in zip(src, dst):
            if a < 0 or b < 0:
                continue
            if self.len[b]:
                self.err |= M.MOE_DEVERR_CACHE_BUSY
                continue
            L = self.len[a]
            row = list(self.t[a])
            if L % self.ps and self.t[a][L // self.ps] >= 0:
                used += 1
                if used > len(free):
                    self.err |= M.MOE_DEVERR_CACHE_FULL
                    continue
                copies.append((row[L // self.ps], free[used - 1]))
                row[L // self.ps] = free[used - 1]
            todo.append((b, L, row))
        for b, L, row in todo:
            for j in range(-(-L // self.ps)):
                self.t[b][j] = row[j]
                if row[j] >= 0:
                    self.refs[row[j]] += 1
            self.len[b] = L
        return copies

    def compact(self):
        U = sum(r > 0 for r in self.refs)
        holes = [p for p in range(U) if self.refs[p] == 0]
        movers = [p for p in range(U, self.P) if self.refs[p] > 0]
        m = dict(zip(movers, holes))
        for a, b in m.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.t = [[m.get(e, e) for e in row] for row in self.t]
        return U, list(m.items())


def _i(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cache(slots, mp, P, ps, layers=2, hkv=2, D=64, dtype=torch.bfloat16, seed=0, fill=True):
    c = M.KvCache(n_layers=layers, n_pages=P, page_size=ps, n_heads=hkv, head_dim=D,
                  n_slots=slots, max_pages=mp, dtype=dtype)
    if fill:
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for x in (c.k, c.v):
            x.view(torch.uint8).copy_(torch.randint(0, 256, x.view(torch.uint8).shape,
                                                    generator=gen, device="cuda",
                                                    dtype=torch.uint8))
    return c


def _same(c, sim, where):
    torch.cuda.synchronize()
    assert c.lens.tolist() == sim.len, where
    assert c.refs.tolist() == sim.refs, where
    assert c.table.tolist() == sim.t, where
    assert M.moe_read_device_error(c.err_word) == sim.err, where


def _moved(c, before, copies):
    k, v = (x.clone() for x in before)
    for a, b in copies:
        k[:, b], v[:, b] = before[0][:, a], before[1][:, a]
    for x, y in ((c.k, k), (c.v, v)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("ps,layers,dtype", [(16, 2, "bf16"), (48, 1, "e4m3"), (64, 33, "f16")])
def test_a_server_s_turns(ps, layers, dtype):
    """Many random turns of grow, fork, trim, free and compact on a small pool
    that runs full now and then: tables, counts, lengths, error bits and page
    contents after every call."""
    rng = np.random.default_rng(ps)
    S, mp, P = 13, 9, 40
    sc = torch.ones(layers, 2, device="cuda")
    c = M.KvCache(n_layers=layers, n_pages=P, page_size=ps, n_heads=2, head_dim=64, n_slots=S,
                  max_pages=mp, dtype=DT[dtype],
                  **(dict(k_scale=sc, v_scale=sc) if dtype == "e4m3" else {}))
    for x in (c.k, c.v):
        x.view(torch.uint8).copy_(torch.randint(0, 256, x.view(torch.uint8).shape,
                                                device="cuda", dtype=torch.uint8))
    sim = Sim(S, mp, P, ps)
    seen = 0
    for turn in range(25):
        slots = [int(x) for x in rng.permutation(S)[:5]]
        if turn % 4 == 3:
            slots[1] = -1
        new = [int(x) for x in rng.choice([0, 1, 3, ps, 2 * ps + 1, 5 * ps], 5)]
        start = c.grow(_i(slots), _i(new))
        want = sim.grow(slots, new)
        _same(c, sim, ("grow", turn))
        assert start.tolist() == want, turn
        if turn % 2:
            c.trim(_i(slots), ps + 3, 2)
            sim.trim(slots, ps + 3, 2)
            _same(c, sim, ("trim", turn))
        empty = [s for s in range(S) if sim.len[s] == 0][:3]
        busy = [s for s in range(S) if sim.len[s]]
        if busy and empty:
            src = [busy[int(x)] for x in rng.integers(0, len(busy), len(empty))]
            dst = list(empty)
            if turn % 5 == 4 and len(busy) > 1:
                src.append(busy[0])
                dst.append(busy[1])           # refused: holds tokens
                src = [s for s in src if s != busy[1]] + [busy[0]] * src.count(busy[1])
            before = c.k.clone(), c.v.clone()
            c.fork(_i(src), _i(dst))
            copies = sim.fork(src, dst)
            _same(c, sim, ("fork", turn))
            _moved(c, before, copies)
        out = [int(x) for x in rng.permutation(S)[:4 if turn % 3 else 7]]
        c.free(_i(out))
        sim.free(out)
        _same(c, sim, ("free", turn))
        if turn % 3 == 2:
            before = c.k.clone(), c.v.clone()
            n = torch.zeros(1, dtype=torch.int32, device="cuda")
            c.compact(n)
            used, copies = sim.compact()
            _same(c, sim, ("compact", turn))
            _moved(c, before, copies)
            assert n.tolist() == [used]
        seen |= sim.err
    assert seen & M.MOE_DEVERR_CACHE_FULL


@pytest.mark.parametrize("P,n", [(70001, 40), (200000, 1500), (9000, 1100)])
def test_grow_and_fork_in_large_pools(P, n):
    """Pools beyond one scan step (and beyond the size whose free pages are
    counted first), lists beyond one workgroup, few free pages at scattered
    places."""
    rng = np.random.default_rng(P)
    mp, ps = 6, 16
    sim = Sim(2 * n, mp, P, ps)
    free = rng.choice(P, 3 * n + 20, replace=False)
    refs = np.ones(P, np.int32)
    refs[free] = 0
    sim.refs = refs.tolist()
    c = _cache(2 * n, mp, P, ps, layers=1, hkv=1, D=64, fill=False)
    c.k.zero_(), c.v.zero_()
    c.refs.copy_(torch.from_numpy(refs))
    slots = [int(x) for x in rng.permutation(n)]
    new = [int(x) for x in rng.integers(0, 40, n)]
    start = c.grow(_i(slots), _i(new))
    want = sim.grow(slots, new)
    _same(c, sim, "grow")
    assert start.tolist() == want
    src, dst = list(range(n)), list(range(n, 2 * n))
    c.fork(_i(src), _i(dst))
    sim.fork(src, dst)
    _same(c, sim, "fork")
    # ask for more than there is: the first that does not fit ends it
    new = [33] * n
    start = c.grow(_i(slots), _i(new))
    want = sim.grow(slots, new)
    _same(c, sim, "full")
    assert start.tolist() == want and -1 in want
    n_used = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.compact(n_used)
    used, _ = sim.compact()
    _same(c, sim, "compact")
    assert n_used.tolist() == [used]


def test_grow_without_a_list_and_empty_calls():
    c = _cache(3, 4, 8, 16, layers=1)
    sim = Sim(3, 4, 8, 16)
    start = c.grow(None, _i([5, 0, 64]))
    assert start.tolist() == sim.grow([0, 1, 2], [5, 0, 64])
    _same(c, sim, "grow")
    # the row is too short: refused, others served
    start = c.grow(None, _i([1, 1, 1]))
    assert start.tolist() == sim.grow([0, 1, 2], [1, 1, 1]) and start.tolist()[2] == -1
    _same(c, sim, "row")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    c.free(none)
    c.trim(none, 4)
    c.fork(none, none)
    _same(c, sim, "empty")
    c.free(_i([0, 1, 2]))
    c.compact()
    sim.free([0, 1, 2])
    _same(c, sim, "all free")


@pytest.mark.parametrize("layout", ["head", "tok", "padded"])
@pytest.mark.parametrize("D,dtype", [(64, "e4m3"), (128, "bf16"), (256, "f16")])
def test_copy_pages(layout, D, dtype):
    P, H, ps = 9, 3, 48
    def make():
        if layout == "head":
            return torch.empty(P, H, ps, D, dtype=DT[dtype], device="cuda")
        if layout == "tok":
            return torch.empty(P, ps, H, D, dtype=DT[dtype], device="cuda").transpose(1, 2)
        return torch.empty(P, H, ps + 2, D + 16, dtype=DT[dtype], device="cuda")[:, :, :ps, :D]
    sc = torch.ones(H, device="cuda")
    kv = []
    for _ in range(2):
        k, v = make(), make()
        for x in (k, v):
            x.view(torch.uint8).copy_(torch.randint(0, 255, x.view(torch.uint8).shape,
                                                    dtype=torch.uint8, device="cuda"))
        kv.append((k, v))
    caches = [M.kv_cache(k, v, *((sc, sc) if dtype == "e4m3" else ())) for k, v in kv]
    want = [[x.clone() for x in p] for p in kv]
    src, dst = [0, 5, -1, 2, 3, 1], [7, 4, 6, -1, 99, 8]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    M.moe_cache_copy_pages(caches, _i(src), _i(dst), err)
    for p in want:
        for x in p:
            for a, b in ((0, 7), (5, 4), (1, 8)):
                x[b] = x[a].clone()
    for p, w in zip(kv, want):
        for x, y in zip(p, w):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert M.moe_read_device_error(err) == M.MOE_DEVERR_CACHE_PAGE


def _codes(x, scale):
    """e4m3fn codes of x / scale: the fp32 quotient saturated, one rounding."""
    q = x.float() / scale[:, None]
    return q.clamp(-448, 448).to(torch.float8_e4m3fn)


@pytest.mark.parametrize("dt,kv", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"),
                                   ("f16", "e4m3")])
@pytest.mark.parametrize("D,layout,how", [(64, "head", "dense"), (128, "tok", "pad"),
                                          (256, "head", "heads")])
def test_append(dt, kv, D, layout, how):
    """Prompts and single tokens, ragged, across page ends, through slots and
    not, with rows that are not written; everything else keeps its bits."""
    rng = np.random.default_rng(D)
    P, H, ps, S, mp = 23, 3, 16, 5, 7
    def make():
        x = torch.randint(0, 255, (P, H, ps, D * (1 if kv == "e4m3" else 2)),
                          dtype=torch.uint8, device="cuda").view(DT[kv])
        return x if layout == "head" else x.transpose(1, 2).contiguous().transpose(1, 2)
    k, v = make(), make()
    sc = [torch.rand(H, device="cuda") * 0.1 + 0.01 for _ in range(2)]
    cache = M.kv_cache(k, v, *(sc if kv == "e4m3" else ()))
    tab = np.full((S, mp), -1, np.int32)
    tab[:, :4] = rng.permutation(P)[:20].reshape(S, 4)
    table = M.kv_table(torch.from_numpy(tab).cuda(), _i([0] * S), ps, P)
    slots, rows, start = [4, 2, -1, 0, 1], [40, 0, 3, 17, 5], [9, 3, 1, 15, -1]
    T = sum(rows)
    shape = {"dense": (T, H, D), "pad": (T, H + 2, D + 8), "heads": (H, T, D)}[how]
    new = []
    for _ in range(2):
        x = torch.from_numpy(rng.standard_normal(shape)).to("cuda", DT[dt]) * 3
        x = x[:, :H, :D] if how == "pad" else x.transpose(0, 1) if how == "heads" else x
        if kv == "e4m3":               # saturation, zeros, NaN
            x[0, 0, 0], x[1, 1, 1], x[2, 2, 2], x[3, 0, 5] = 1000.0, -1000.0, 0.0, float("nan")
            x[4, 0, 6], x[4, 0, 7] = float("inf"), -float("inf")
        new.append(x)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = [x.clone() for x in (k, v)]
    cu = np.concatenate([[0], np.cumsum(rows)])
    for w, x, s in zip(want, new, sc):
        y = _codes(x, s) if kv == "e4m3" else x
        for i in range(5):
            if slots[i] < 0 or start[i] < 0:
                continue
            for j in range(rows[i]):
                p = start[i] + j
                w.view(torch.uint8)[tab[slots[i], p // ps], :, p % ps] = \
                    y[cu[i] + j].contiguous().view(torch.uint8)
    M.moe_cache_append(cache, table, _i(start), _i(cu.tolist()), new[0], new[1], err,
                       slots=_i(slots))
    for x, w in zip((k, v), want):
        assert torch.equal(x.view(torch.uint8), w.view(torch.uint8))
    assert M.moe_read_device_error(err) == 0
    # one token each, no lists; a row beyond its pages is flagged, not written
    start = [0, 1, 63, 64, 500]
    for w, x, s in zip(want, new, sc):
        y = _codes(x[:5], s) if kv == "e4m3" else x[:5]
        for i in range(3):
            w.view(torch.uint8)[tab[i, start[i] // ps], :, start[i] % ps] = \
                y[i].contiguous().view(torch.uint8)
    M.moe_cache_append(cache, table, _i(start), None, new[0][:5], new[1][:5], err)
    for x, w in zip((k, v), want):
        assert torch.equal(x.view(torch.uint8), w.view(torch.uint8))
    assert M.moe_read_device_error(err) == M.MOE_DEVERR_CACHE_PAGE


def test_upkeep_replays_in_a_graph():
    """A turn of grow, append, trim and fork captured once and replayed,
    against the simulation, with eager work between."""
    S, mp, P, ps = 6, 8, 40, 16
    c = _cache(S, mp, P, ps, layers=2)
    sim = Sim(S, mp, P, ps)
    c.grow(_i([0, 1]), _i([20, 33]))
    sim.grow([0, 1], [20, 33])
    slots, new = _i([0, 1]), _i([1, 18])
    start = torch.empty(2, dtype=torch.int32, device="cuda")
    src, dst, gone = _i([1, 0]), _i([4, 5]), _i([4, 5])
    ws = c.workspace(M.moe_cache_workspace_size(c.desc, 4))
    rows = torch.randn(19, 2, 64, device="cuda", dtype=torch.bfloat16)
    cu = _i([0, 1, 19])

    def turn():
        M.moe_cache_free(c.desc, gone, c.err_word)
        M.moe_cache_grow(c.desc, slots, new, start, c.err_word, ws)
        M.moe_cache_append(c.layers[1], c.desc, start, cu, rows, rows, c.err_word, slots=slots)
        M.moe_cache_trim(c.desc, slots, 30, 3, c.err_word)
        M.moe_cache_fork(c.layers, c.desc, src, dst, c.err_word, ws)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        turn()
    for rep in range(4):
        g.replay()
        torch.cuda.synchronize()
        sim.free([4, 5])
        want = sim.grow([0, 1], [1, 18])
        sim.trim([0, 1], 30, 3)
        sim.fork([1, 0], [4, 5])
        assert start.tolist() == want
        _same(c, sim, rep)
        torch.ones(1000, device="cuda").sum().item()
