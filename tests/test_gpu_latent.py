"""moe_attn_latent against a plain 64-bit attention whose values are the first
part of its keys.

Everything that no query sees is NaN in the cache; bars are derived in
cache_ref.attention.
"""
import numpy as np
import pytest
import torch

import mixture_experts_expert_sigmoid_amd as M
from tests.cache_ref import DT, attention, check, visible
from tests.test_gpu_attn import _q
from tests.test_gpu_tree import bushy, chain, sees, star

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]
ROPE = 64


class LatentPool:
    """One layer's latent cache on the GPU, unwritten tokens NaN, and its
    contents in float64 on the host."""

    def __init__(self, rng, *, kv, dc, ps, lens, gap=0, max_pages=None, spare=3, amp=1.0):
        self.kv, self.dc, self.ps, self.lens = kv, dc, ps, list(lens)
        need = [-(-L // ps) for L in self.lens]
        self.P = sum(need) + spare
        mp = max([1] + need) if max_pages is None else max_pages
        order = rng.permutation(self.P)
        self.tab = np.full((len(self.lens), mp), -1, np.int32)
        at = 0
        for i, n in enumerate(need):
            self.tab[i, :n] = order[at:at + n]
            at += n
        W = dc + ROPE
        self.sc = float(np.float32(rng.uniform(0.01, 0.05))) if kv == "e4m3" else None
        x = torch.full((self.P, ps, W + gap), float("nan"))
        self.host = []
        for i, L in enumerate(self.lens):
            y = torch.from_numpy(amp * rng.standard_normal((L, W)).astype(np.float32))
            if self.sc:
                y = (y / self.sc).clamp(-448, 448)
            y = y.to(DT[kv]).float()
            for pg in range(need[i]):
                a, b = pg * ps, min(L, pg * ps + ps)
                x[self.tab[i, pg], :b - a, :W] = y[a:b]
            self.host.append((y.double() * (self.sc or 1.0)).numpy())
        self.c = x.to(DT[kv]).cuda()[..., :W]
        self.table = torch.from_numpy(self.tab).cuda()
        self.len_t = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.scale = torch.tensor([self.sc], device="cuda") if self.sc else None

    def set(self, slot, pos, dims, value):
        raw = torch.tensor([value]).to(DT[self.kv])
        page = int(self.tab[slot, pos // self.ps])
        bits = torch.uint8 if self.kv == "e4m3" else torch.int16
        self.c.view(bits)[page, pos % self.ps, dims] = raw.view(bits).cuda()
        self.host[slot][pos, dims] = raw.double().item() * (self.sc or 1.0)

    def desc(self):
        return (M.latent_cache(self.c, self.dc, self.scale),
                M.kv_table(self.table, self.len_t, self.ps, self.P))

    def keys(self):
        return lambda s: [(self.host[s], self.host[s][:, :self.dc])] if s >= 0 else \
            [(np.zeros((0, self.dc + ROPE)), np.zeros((0, self.dc)))]


def want_of(pool, slots, parents, rows, q, window, first, scale, dt):
    """parents: per entry the tree, or None for rows in their order."""
    C = [(pool.lens[s] if s >= 0 else 0) - m for s, m in zip(slots, rows)]
    see = []
    for s, m, c, par in zip(slots, rows, C, parents):
        L = pool.lens[s] if s >= 0 else 0
        if par is None:
            see.append(visible(np.arange(L - m, L), L, window, first))
        elif c < 0:
            see.append(np.zeros((m, L), bool))
        else:
            see.append(sees(par, c, window, first))
    shape = [np.zeros(m) for m in rows]
    out = reference_latent(pool, slots, shape, C, q, scale, dt, see)
    return out, see


def reference_latent(pool, slots, shape, C, q, scale, dt, see):
    acc, at = [], 0
    for i, s in enumerate(slots):
        m = len(shape[i])
        k, v = pool.keys()(s)[0]
        o, z, bo, bl = _wide(q[at:at + m], k, v, see[i], scale, dt)
        acc.append((o, z, bo, bl))
        at += m
    return [np.concatenate(x, 0) for x in zip(*acc)]


def _wide(q, k, v, see, scale, dt):
    """attention() takes its result's width from q's: values padded to the
    keys' width, the padding cut off."""
    pad = np.zeros((v.shape[0], k.shape[1] - v.shape[1]))
    o, z, bo, bl = attention(q, k, np.concatenate([v, pad], 1), see, scale, dt)
    n = v.shape[1]
    return o[..., :n], z, bo[..., :n], bl


def hide(pool, slots, see):
    for s, ok in zip(slots, see):
        if s < 0 or ok.size == 0:
            continue
        seen = ok.any(0)
        for j in np.nonzero(~seen)[0]:
            pool.set(s, int(j), slice(None), float("nan"))
        for pg in range(-(-pool.lens[s] // pool.ps)):
            if not seen[pg * pool.ps:(pg + 1) * pool.ps].any():
                pool.tab[s, pg] = -1
    pool.table.copy_(torch.from_numpy(pool.tab))


def run(pool, slots, parents, rows, q, window, first, scale, dt, how="dense", one=False):
    cache, table = pool.desc()
    T, H, n, dc = q.shape[0], q.shape[1], len(rows), pool.dc

    def empty(d):
        if how == "pad":
            return torch.full((T, H + 1, d + 8), float("nan"), dtype=DT[dt],
                              device="cuda")[:, :H, :d]
        if how == "heads":
            return torch.full((H, T, d), float("nan"), dtype=DT[dt],
                              device="cuda").transpose(0, 1)
        return torch.full((T, H, d), float("nan"), dtype=DT[dt], device="cuda")
    qd, out = empty(dc + ROPE), empty(dc)
    qd.copy_(torch.from_numpy(q))
    lse = torch.full((T, H), 7.0, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    err = torch.zeros(1, **i32)
    sl = None if slots is None else torch.tensor(slots, **i32)
    cu = None if one else torch.tensor(np.concatenate([[0], np.cumsum(rows)]), **i32)
    par = None if parents is None else torch.tensor(np.concatenate(parents), **i32)
    ws = torch.empty(M.moe_attn_latent_workspace_size(cache, n, T, H), dtype=torch.uint8,
                     device="cuda")
    ws.fill_(0xFF)                       # NaN in whatever is read unwritten
    got = []
    for _ in range(2):
        M.moe_attn_latent(cache, table, qd, cu, out, scale, err, ws, parent=par, window=window,
                          n_first=first, slots=sl, lse=lse)
        torch.cuda.synchronize()
        got.append((out.contiguous().view(torch.int16).clone(), lse.view(torch.int32).clone()))
    # the same inputs give the same bits
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), M.moe_read_device_error(err)


# dt, cache, latent_dim, heads, page, strides, gap, (context, new) of each, tree, window, first
CASES = {
    "first_token": ("bf16", "bf16", 512, 16, 16, "dense", 0, [(0, 1)], None, 0, 0),
    "one_each": ("bf16", "bf16", 512, 128, 16, "pad", 0,
                 [(30, 1), (31, 1), (32, 1), (4, 1), (126, 1), (128, 1), (700, 1)], None, 0, 0),
    "few_heads": ("f16", "f16", 256, 5, 48, "heads", 8, [(99, 1), (0, 1), (999, 1), (47, 1)], None,
                  0, 0),
    "one_head": ("bf16", "bf16", 256, 1, 16, "dense", 0, [(64, 1), (95, 70)], None, 0, 0),
    "prompt": ("bf16", "bf16", 512, 6, 32, "dense", 0, [(0, 77), (0, 1), (0, 33)], None, 0, 0),
    "chunk": ("f16", "f16", 512, 12, 16, "pad", 0, [(200, 19), (63, 40)], None, 0, 0),
    "heads_1000": ("bf16", "bf16", 256, 1000, 16, "dense", 0, [(40, 2), (3, 1)], None, 0, 0),
    "heads_1024": ("f16", "f16", 512, 1024, 16, "heads", 0, [(70, 1)], None, 0, 0),
    "odd_heads": ("bf16", "bf16", 512, 33, 16, "dense", 24, [(50, 2), (300, 3)], None, 0, 0),
    "e4m3": ("bf16", "e4m3", 512, 16, 64, "dense", 0, [(200, 1), (62, 1), (512, 1)], None, 0, 0),
    "e4m3_128": ("bf16", "e4m3", 512, 128, 64, "heads", 16, [(200, 1), (63, 2)], None, 0, 0),
    "e4m3_f16": ("f16", "e4m3", 256, 20, 16, "dense", 0, [(33, 7), (290, 3)], None, 0, 0),
    "split_long": ("bf16", "bf16", 512, 16, 64, "dense", 0, [(20010, 1)], None, 0, 0),
    "split_few": ("f16", "f16", 256, 5, 128, "dense", 0, [(12011, 1), (3001, 2)], None, 0, 0),
    "split_rows": ("bf16", "bf16", 512, 3, 32, "pad", 0, [(15000, 30)], None, 0, 0),
    "split_codes": ("bf16", "e4m3", 256, 1, 16, "dense", 0, [(9000, 3), (14001, 1)], star, 0, 0),
    "split_heads": ("bf16", "bf16", 512, 128, 64, "dense", 0, [(5000, 1), (77, 1)], None, 0, 0),
    "split_e4m3": ("f16", "e4m3", 512, 40, 128, "dense", 0, [(9001, 3), (36, 1)], None, 0, 0),
    "tree": ("bf16", "bf16", 512, 8, 16, "dense", 0, [(30, 8), (0, 33), (63, 64)], bushy, 0, 0),
    "tree_chain": ("f16", "f16", 256, 16, 48, "pad", 0, [(100, 9), (500, 40)], chain, 0, 0),
    "tree_star": ("bf16", "e4m3", 512, 16, 64, "dense", 0, [(47, 40), (16, 3)], star, 0, 0),
    "tree_large": ("bf16", "bf16", 256, 1, 32, "dense", 0, [(77, 256), (1, 255)], bushy, 0, 0),
    "tree_split": ("bf16", "bf16", 512, 16, 64, "dense", 0, [(7011, 13)], bushy, 0, 0),
    "window": ("bf16", "bf16", 512, 8, 16, "dense", 0,
               [(0, 1), (16, 1), (100, 30), (1000, 1), (515, 7)], None, 64, 4),
    "window_1": ("f16", "f16", 256, 4, 32, "dense", 0, [(0, 1), (1, 1), (299, 9)], None, 1, 0),
    "window_first": ("bf16", "bf16", 256, 4, 16, "dense", 0, [(49, 1), (299, 20), (128, 1)], None,
                     40, 100),
    "window_tree": ("bf16", "bf16", 512, 4, 16, "dense", 0, [(6, 60), (300, 40)], chain, 9, 30),
    "window_long": ("bf16", "e4m3", 512, 16, 16, "dense", 0, [(9777, 5)], bushy, 6000, 17),
}


@pytest.mark.parametrize("name", list(CASES))
def test_latent(name):
    dt, kv, dc, H, ps, how, gap, seqs, tree, window, first = CASES[name]
    print(f"[case] latent {name}", flush=True)
    rng = np.random.default_rng(len(name) * 7 + dc)
    rows = [m for _, m in seqs]
    pool = LatentPool(rng, kv=kv, dc=dc, ps=ps, lens=[c + m for c, m in seqs], gap=gap)
    n = len(seqs)
    parents = [None if tree is None else tree(m, i) for i, m in enumerate(rows)]
    q = _q(rng, sum(rows), H, dc + ROPE, dt)
    scale = (dc + ROPE) ** -0.5
    want, see = want_of(pool, range(n), parents, rows, q, window, first, scale, dt)
    hide(pool, range(n), see)
    out, lse, err = run(pool, None, None if tree is None else parents, rows, q, window, first,
                        scale, dt, how, one=tree is None and set(rows) == {1})
    assert err == 0
    check(lse, want[1], want[3], "lse")
    print("  worst error / bar: %.3f" % check(out, want[0], want[2], "out"), flush=True)


@pytest.mark.parametrize("dt,H,wide", [("bf16", 16, 0), ("f16", 64, 700)])
def test_many_sequences(dt, H, wide):
    """More sequences than one launch takes, many of them empty, through a
    table with room for long contexts."""
    rng = np.random.default_rng(9)
    lens = [int(x) for x in rng.integers(0, 60, 300)]
    pool = LatentPool(rng, kv=dt, dc=256, ps=16, lens=lens, max_pages=wide or None)
    q = _q(rng, 300, H, 320, dt)
    want, _ = want_of(pool, range(300), [None] * 300, [1] * 300, q, 0, 0, 0.06, dt)
    out, lse, err = run(pool, None, None, [1] * 300, q, 0, 0, 0.06, dt, one=True)
    assert err == 0
    check(out, want[0], want[2], "out")
    check(lse, want[1], want[3], "lse")
    # the same as a list of rows, some sequences without any
    rows = [int(x) for x in rng.integers(0, 3, 300)]
    T = sum(rows)
    q = _q(rng, T, H, 320, dt)
    want, _ = want_of(pool, range(300), [None] * 300, rows, q, 0, 0, 0.06, dt)
    out, lse, err = run(pool, None, None, rows, q, 0, 0, 0.06, dt)
    assert err == 0
    check(out, want[0], want[2], "out")
    check(lse, want[1], want[3], "lse")


def test_slots_and_rows_without_a_sequence():
    """A permuted list with rows without a sequence, a slot beyond the table
    (flagged), an empty slot, more rows than tokens; rows of q outside the list
    are not written."""
    rng = np.random.default_rng(4)
    pool = LatentPool(rng, kv="bf16", dc=256, ps=16, lens=[70, 0, 200, 5])
    slots, rows = [2, -1, 0, 1, 3], [12, 5, 20, 3, 9]
    q = _q(rng, sum(rows), 4, 320, "bf16")
    want, _ = want_of(pool, slots, [None] * 5, rows, q, 0, 0, 0.06, "bf16")
    out, lse, err = run(pool, slots, None, rows, q, 0, 0, 0.06, "bf16")
    assert err == 0
    check(out, want[0], want[2], "out")
    check(lse, want[1], want[3], "lse")
    parents = [bushy(m, i) for i, m in enumerate(rows)]
    want, _ = want_of(pool, slots, parents, rows, q, 0, 0, 0.06, "bf16")
    out, lse, err = run(pool, slots, parents, rows, q, 0, 0, 0.06, "bf16")
    assert err == 0
    check(out, want[0], want[2], "out")
    # beyond the table
    out, lse, err = run(pool, [9, 0], None, [3, 2], q[:5], 0, 0, 0.06, "bf16")
    assert err == M.MOE_DEVERR_CACHE_PAGE
    assert (out[:3] == 0).all() and (lse[:3] == -np.inf).all() and (lse[3:] > -np.inf).all()
    # rows around the list's
    cache, table = pool.desc()
    i32 = dict(dtype=torch.int32, device="cuda")
    buf = torch.full((40, 4, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((40, 4), 7.0, device="cuda")
    ws = torch.empty(M.moe_attn_latent_workspace_size(cache, 2, 40, 4), dtype=torch.uint8,
                     device="cuda")
    M.moe_attn_latent(cache, table, torch.from_numpy(q[:40]).to("cuda", torch.bfloat16),
                      torch.tensor([10, 14, 30], **i32), buf, 0.06, torch.zeros(1, **i32), ws,
                      lse=lse)
    torch.cuda.synchronize()
    for x in (buf, lse):
        assert (x[:10] == 7).all() and (x[30:] == 7).all() and (x[10:30] != 7).all()


def test_missing_page_is_masked_and_flagged():
    rng = np.random.default_rng(5)
    pool = LatentPool(rng, kv="bf16", dc=512, ps=16, lens=[200, 90])
    pool.tab[0, 3] = -1
    pool.tab[1, 0] = 1 << 20
    pool.table.copy_(torch.from_numpy(pool.tab))
    q = _q(rng, 4, 16, 576, "bf16")
    see = [visible(np.arange(198, 200), 200, 0, 0), visible(np.arange(88, 90), 90, 0, 0)]
    see[0][:, 48:64] = False
    see[1][:, :16] = False
    want = reference_latent(pool, [0, 1], [np.zeros(2)] * 2, None, q, 0.04, "bf16", see)
    out, lse, err = run(pool, None, None, [2, 2], q, 0, 0, 0.04, "bf16")
    assert err == M.MOE_DEVERR_CACHE_PAGE
    check(out, want[0], want[2], "out")
    check(lse, want[1], want[3], "lse")


@pytest.mark.parametrize("kv,H", [("bf16", 16), ("f16", 40), ("e4m3", 16)])
def test_values_that_are_not_finite(kv, H):
    """In latent vectors of drafted leaves, of tokens behind a chunk's rows and
    of the context: they reach the rows that see them and no others."""
    rng = np.random.default_rng(6)
    pool = LatentPool(rng, kv=kv, dc=256, ps=16, lens=[62, 62])
    par = bushy(30)
    leaf = [t for t in range(30) if t not in par]
    bad = [float("nan")] if kv == "e4m3" else [float("inf"), float("-inf"), float("nan")]
    for t, b in zip(leaf, bad):
        pool.set(0, 32 + t, slice(5, 200, 13), b)
        pool.set(0, 32 + t, slice(257, 258), 0.5)
    dt = "bf16" if kv == "bf16" else "f16"
    q = _q(rng, 60, H, 320, dt)
    with np.errstate(invalid="ignore"):
        want, _ = want_of(pool, [0], [par], [30], q[:30], 0, 0, 0.06, dt)
    out, lse, err = run(pool, [0], [par], [30], q[:30], 0, 0, 0.06, dt)
    assert err == 0
    # a row that sees one: its score is not finite either, so all of it is NaN
    hit = np.isnan(want[0]).any((1, 2))
    assert hit.any() and not hit.all()
    check(out[~hit], want[0][~hit], want[2][~hit], "out")
    assert np.isnan(out[hit]).any((1, 2)).all()
    # the newest of a chunk, seen by the last row only
    pool.set(1, 61, slice(7, 8), float("nan"))
    with np.errstate(invalid="ignore"):
        want, _ = want_of(pool, [1], [None], [30], q[30:], 0, 0, 0.06, dt)
    out, lse, err = run(pool, [1], None, [30], q[30:], 0, 0, 0.06, dt)
    check(out[:29], want[0][:29], want[2][:29], "out")
    assert np.isnan(out[29]).all()


def test_infinite_values_of_finite_scores():
    """Latent values whose queries are zero there: scores are NaN (0 times
    infinity) as the formula has them, but rows that do not see them stand."""
    rng = np.random.default_rng(8)
    pool = LatentPool(rng, kv="f16", dc=512, ps=16, lens=[100])
    # infinities in the rotary part: the values are finite
    q = _q(rng, 20, 16, 576, "f16")
    q[..., 512:] = np.abs(q[..., 512:]) + 0.25
    pool.set(0, 95, slice(512, 513), float("-inf"))
    want, _ = want_of(pool, [0], [None], [20], q, 0, 0, 0.04, "f16")
    out, lse, err = run(pool, [0], None, [20], q, 0, 0, 0.04, "f16")
    assert np.isfinite(want[0]).all()
    check(out, want[0], want[2], "out")
    check(lse, want[1], want[3], "lse")


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_scores_that_grow_and_are_large(dt):
    """Maxima that grow tile after tile, and weak keys beside a strong one."""
    rng = np.random.default_rng(10)
    pool = LatentPool(rng, kv=dt, dc=256, ps=16, lens=[900, 500], amp=0.25)
    for j in range(0, 900, 5):           # a rotary part that rises with the position
        pool.set(0, j, slice(256, 320), j / 900 * 4)
    pool.set(1, 3, slice(256, 320), 8.0)
    q = _q(rng, 2, 24, 320, dt, amp=0.3)
    q[..., 256:] = 0.5
    want, _ = want_of(pool, [0, 1], [None] * 2, [1, 1], q, 0, 0, 0.3, dt)
    out, lse, err = run(pool, None, None, [1, 1], q, 0, 0, 0.3, dt, one=True)
    check(out, want[0], want[2], "out")
    check(lse, want[1], want[3], "lse")
    want, _ = want_of(pool, [0, 1], [None] * 2, [1, 1], q, 0, 0, -0.3, dt)
    out, lse, err = run(pool, None, None, [1, 1], q, 0, 0, -0.3, dt, one=True)
    check(out, want[0], want[2], "negative scale")


def test_page_offsets_beyond_32_bits():
    """Pages that lie further apart than 2^32 bytes."""
    rng = np.random.default_rng(11)
    pool = LatentPool(rng, kv="bf16", dc=512, ps=16, lens=[40], spare=1)
    W, far = 576, 1 << 31                # elements
    buf = torch.empty(far * 3 + 16 * W, dtype=torch.bfloat16, device="cuda")
    big = buf.as_strided((4, 16, W), (far, W, 1))
    for p in range(4):
        big[p].copy_(pool.c[p])
    q = _q(rng, 3, 16, 576, "bf16")
    want, _ = want_of(pool, [0], [None], [3], q, 0, 0, 0.04, "bf16")
    pool.c = big
    out, lse, err = run(pool, None, None, [3], q, 0, 0, 0.04, "bf16")
    assert err == 0
    check(out, want[0], want[2], "out")


def test_graph_with_other_lengths():
    """Captured once; replays take the lengths and slots of the time."""
    rng = np.random.default_rng(12)
    pool = LatentPool(rng, kv="bf16", dc=512, ps=16, lens=[700, 40, 333], max_pages=60)
    cache, table = pool.desc()
    i32 = dict(dtype=torch.int32, device="cuda")
    q = _q(rng, 4, 32, 576, "bf16")
    qd = torch.from_numpy(q).to("cuda", torch.bfloat16)
    out, lse = torch.empty(4, 32, 512, dtype=torch.bfloat16, device="cuda"), \
        torch.empty(4, 32, device="cuda")
    err, sl = torch.zeros(1, **i32), torch.tensor([0, 1, 2, -1], **i32)
    ws = torch.empty(M.moe_attn_latent_workspace_size(cache, 4, 4, 32), dtype=torch.uint8,
                     device="cuda")
    call = lambda: M.moe_attn_latent(cache, table, qd, None, out, 0.04, err, ws,  # noqa: E731
                                     slots=sl, lse=lse)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens, slots in [([700, 40, 333], [2, 0, 1, -1]), ([1, 33, 0], [0, 1, 2, -1]),
                        ([699, 8, 300], [-1, 2, 1, 0])]:
        pool.len_t.copy_(torch.tensor(lens))
        sl.copy_(torch.tensor(slots))
        out.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        replayed, z = out.clone(), lse.clone()
        see = [np.broadcast_to(np.arange(pool.lens[s]) < lens[s], (1, pool.lens[s]))
               if s >= 0 else np.zeros((1, 0), bool) for s in slots]
        want = reference_latent(pool, slots, [np.zeros(1)] * 4, None, q, 0.04, "bf16", see)
        check(replayed.double().cpu().numpy(), want[0], want[2], "out")
        check(z.double().cpu().numpy(), want[1], want[3], "lse")
        call()
        torch.cuda.synchronize()
        assert torch.equal(out, replayed)
    assert M.moe_read_device_error(err) == 0
