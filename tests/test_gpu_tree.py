"""moe_attn_tree against a plain 64-bit attention over each row's ancestors.

As in the tests of the prompts, everything that no query sees is NaN in the
cache, and bars are derived in cache_ref.attention.
"""
import numpy as np
import pytest
import torch

import mixture_experts_expert_sigmoid_amd as M
from tests.cache_ref import DT, Pool, attention, check, visible
from tests.test_gpu_attn import _q, _strided

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]


def bushy(m, i=0):
    """Some children of the context, others of earlier tokens."""
    t = np.arange(m)
    f = (t * 0.6180339887498949 + i * 0.7548776662466927) % 1.0
    return np.clip(np.floor(t * (0.4 + 0.7 * f)).astype(int) - 1, -1, t - 1)


def chain(m, i=0):
    return np.arange(m) - 1


def star(m, i=0):
    return np.full(m, -1)


def sees(parents, C, window=0, first=0):
    """Boolean [m, C + m]: which keys each drafted token sees."""
    m = len(parents)
    anc, depth = np.zeros((m, m), bool), np.zeros(m, int)
    for t in range(m):
        a, d = t, -1
        while a >= 0:
            anc[t, a] = True
            a, d = parents[a], d + 1
        depth[t] = d
    ok = np.concatenate([np.ones((m, C), bool), anc], 1)
    if window:
        pk = np.concatenate([np.arange(C), C + depth])
        ok &= ((C + depth)[:, None] - pk < window) | (pk < first)
    return ok


def reference(keys, slots, parents, C, q, hq, window, first, scale, dt, see=None):
    """keys(slot, kv head) -> (k, v) float64 [L, .]; q float64 [T, hq, .]"""
    acc, at = [], 0
    for i, (s, par) in enumerate(zip(slots, parents)):
        m = len(par)
        ok = see[i] if see is not None else sees(par, C[i], window, first)
        heads = keys(s)
        g = hq // len(heads)
        per = [attention(q[at:at + m, h * g:(h + 1) * g], k, v, ok, scale, dt)
               for h, (k, v) in enumerate(heads)]
        # out and its bar take their width from v, which may be part of k
        acc.append([np.concatenate(x, 1) for x in zip(*per)])
        at += m
    return [np.concatenate(x, 0) for x in zip(*acc)]


def pool_keys(pool):
    return lambda s: [(pool.host[s][0][h], pool.host[s][1][h]) for h in range(pool.hkv)] \
        if s >= 0 else [(np.zeros((0, pool.D)),) * 2] * pool.hkv


def hide(pool, slots, C, parents, window, first):
    """NaN into every token that no query sees, and -1 for pages without any
    that one sees."""
    for s, c, par in zip(slots, C, parents):
        if s < 0 or len(par) == 0:
            continue
        seen = sees(par, c, window, first).any(0)
        pool.poison(s, np.nonzero(~seen)[0])
        for pg in range(-(-pool.lens[s] // pool.ps)):
            if not seen[pg * pool.ps:(pg + 1) * pool.ps].any():
                pool.tab[s, pg] = -1
    pool.table.copy_(torch.from_numpy(pool.tab))


def run(pool, slots, parents, q, hq, window, first, scale, dt, how="dense"):
    cache, table = pool.desc(M)
    T, n = q.shape[0], len(parents)
    qd, out = _strided((T, hq, pool.D), dt, how), _strided((T, hq, pool.D), dt, how)
    qd.copy_(torch.from_numpy(q))
    lse = torch.full((T, hq), 7.0, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    err = torch.zeros(1, **i32)
    sl = None if slots is None else torch.tensor(slots, **i32)
    cu = torch.tensor(np.concatenate([[0], np.cumsum([len(p) for p in parents])]), **i32)
    par = torch.tensor(np.concatenate(parents), **i32)
    ws = torch.empty(max(16, M.moe_attn_tree_workspace_size(cache, n, T, hq)), dtype=torch.uint8,
                     device="cuda")
    ws.fill_(0xFF)                       # NaN in whatever is read unwritten
    got = []
    for _ in range(2):
        M.moe_attn_tree(cache, table, qd, cu, par, out, scale, err, ws, window=window,
                        n_first=first, slots=sl, lse=lse)
        torch.cuda.synchronize()
        got.append((out.contiguous().view(torch.int16).clone(), lse.view(torch.int32).clone()))
    # the same inputs give the same bits
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), M.moe_read_device_error(err)


# dt, kv, D, hq, hkv, page, layout, strides, (context, drafted) of each, tree, window, first
CASES = {
    "one_token": ("bf16", "bf16", 128, 8, 2, 16, "head", "dense", [(0, 1), (5, 1)], bushy, 0, 0),
    "small": ("bf16", "bf16", 128, 8, 2, 16, "head", "pad",
              [(30, 8), (31, 1), (64, 5), (0, 33), (63, 64)], bushy, 0, 0),
    "chains": ("f16", "f16", 64, 6, 2, 48, "tok", "heads", [(100, 9), (1000, 64)], chain, 0, 0),
    "stars": ("f16", "f16", 64, 5, 1, 16, "tok", "dense", [(47, 40), (16, 3)], star, 0, 0),
    "largest": ("bf16", "bf16", 64, 2, 2, 32, "head", "dense", [(77, 256), (1, 255)], bushy, 0, 0),
    "deep": ("bf16", "bf16", 128, 1, 1, 16, "head", "dense", [(3, 200)], chain, 0, 0),
    "d256": ("bf16", "bf16", 256, 4, 1, 32, "head", "dense", [(77, 20), (300, 70)], bushy, 0, 0),
    "e4m3": ("bf16", "e4m3", 128, 16, 2, 64, "head", "dense", [(200, 31), (64, 12)], bushy, 0, 0),
    "e4m3_d64": ("f16", "e4m3", 64, 5, 1, 16, "tok", "pad", [(33, 7), (290, 30)], bushy, 0, 0),
    "e4m3_d256": ("f16", "e4m3", 256, 3, 3, 32, "head", "dense", [(150, 130), (31, 9)], bushy, 0,
                  0),
    "split_long": ("bf16", "bf16", 128, 4, 1, 64, "head", "dense", [(20011, 24)], bushy, 0, 0),
    "split_two": ("f16", "e4m3", 128, 16, 2, 128, "tok", "dense", [(9001, 37), (11, 60)], bushy,
                  0, 0),
    "split_many": ("f16", "f16", 256, 5, 1, 128, "head", "dense", [(9011, 2)], bushy, 0, 0),
    "split_many_d64": ("bf16", "bf16", 64, 3, 3, 16, "tok", "pad", [(9500, 7), (77, 3)], bushy, 0,
                       0),
    "split_many_e4m3": ("bf16", "e4m3", 128, 4, 2, 64, "head", "dense", [(15000, 3), (9000, 1)],
                        star, 0, 0),
    "mqa_64": ("bf16", "bf16", 128, 64, 1, 16, "head", "dense", [(95, 11), (400, 3)], bushy, 0, 0),
    "window": ("bf16", "bf16", 128, 8, 2, 16, "head", "dense",
               [(1, 20), (100, 30), (1000, 64), (515, 7)], bushy, 64, 4),
    "window_in_tree": ("f16", "f16", 64, 4, 2, 32, "head", "dense", [(40, 50), (0, 60)], chain, 7,
                       3),
    "window_1": ("bf16", "bf16", 64, 4, 2, 16, "head", "dense", [(20, 9), (300, 17)], bushy, 1, 0),
    "first_in_tree": ("bf16", "bf16", 64, 4, 2, 16, "head", "dense", [(6, 60), (300, 40)], chain,
                      9, 30),
    "window_long": ("bf16", "e4m3", 128, 8, 2, 16, "head", "dense", [(12777, 40)], bushy, 9000,
                    17),
}


@pytest.mark.parametrize("name", list(CASES))
def test_tree(name):
    dt, kv, D, hq, hkv, ps, layout, how, seqs, tree, window, first = CASES[name]
    print(f"[case] tree {name}", flush=True)
    rng = np.random.default_rng(len(name) * 7 + D)
    C = [c for c, _ in seqs]
    pool = Pool(rng, kv=kv, hkv=hkv, D=D, ps=ps, lens=[c + m for c, m in seqs], layout=layout)
    parents = [tree(m, i) for i, (_, m) in enumerate(seqs)]
    n = len(seqs)
    hide(pool, range(n), C, parents, window, first)
    q = _q(rng, sum(m for _, m in seqs), hq, D, dt)
    out, lse, err = run(pool, None, parents, q, hq, window, first, D ** -0.5, dt, how)
    want = reference(pool_keys(pool), range(n), parents, C, q, hq, window, first, D ** -0.5, dt)
    assert err == 0
    check(lse, want[1], want[3], "lse")
    print("  worst error / bar: %.3f" % check(out, want[0], want[2], "out"), flush=True)


def test_chain_is_the_prompt():
    """A tree without branches sees what moe_attn_prefill sees."""
    rng = np.random.default_rng(3)
    pool = Pool(rng, kv="bf16", hkv=2, D=128, ps=16, lens=[500, 90])
    parents = [chain(40), chain(90)]
    q = _q(rng, 130, 8, 128, "bf16")
    out, lse, err = run(pool, None, parents, q, 8, 0, 0, 0.1, "bf16")
    cache, table = pool.desc(M)
    i32 = dict(dtype=torch.int32, device="cuda")
    qd = torch.from_numpy(q).to("cuda", torch.bfloat16)
    o2, l2 = torch.empty_like(qd), torch.empty(130, 8, device="cuda")
    e = torch.zeros(1, **i32)
    ws = torch.empty(max(16, M.moe_attn_prefill_workspace_size(cache, 2, 130, 8)),
                     dtype=torch.uint8, device="cuda")
    M.moe_attn_prefill(cache, table, qd, torch.tensor([0, 40, 130], **i32), o2, 0.1, e, ws, lse=l2)
    want = reference(pool_keys(pool), [0, 1], parents, [460, 0], q, 8, 0, 0, 0.1, "bf16",
                     see=[visible(np.arange(460, 500), 500, 0, 0),
                          visible(np.arange(90), 90, 0, 0)])
    check(out, want[0], want[2], "tree")
    check(o2.double().cpu().numpy(), want[0], want[2], "prompt")
    check(lse, l2.double().cpu().numpy(), 2 * want[3], "lse")
    assert err == 0


def test_slots_and_rows_without_a_sequence():
    """A permuted slot list with a row group without a sequence, a slot beyond
    the table (flagged), an empty slot and one shorter than its tree."""
    rng = np.random.default_rng(4)
    pool = Pool(rng, kv="bf16", hkv=2, D=64, ps=16, lens=[70, 0, 200, 5])
    slots, rows = [2, -1, 0, 9, 1, 3], [12, 5, 20, 4, 3, 6]
    parents = [bushy(m, i) for i, m in enumerate(rows)]
    q = _q(rng, sum(rows), 4, 64, "bf16")
    out, lse, err = run(pool, slots, parents, q, 4, 0, 0, 0.125, "bf16")
    assert err == M.MOE_DEVERR_CACHE_PAGE
    want = reference(pool_keys(pool), [2, 0], [parents[0], parents[2]], [188, 50],
                     np.concatenate([q[:12], q[17:37]]), 4, 0, 0, 0.125, "bf16")
    pick = np.r_[0:12, 17:37]
    check(out[pick], want[0], want[2], "out")
    check(lse[pick], want[1], want[3], "lse")
    rest = np.setdiff1d(np.arange(sum(rows)), pick)
    assert (out[rest] == 0).all() and (lse[rest] == -np.inf).all()


def test_bad_parents_and_large_trees():
    """A parent that does not come before its child: flagged, taken as -1. A
    tree of 257: flagged, its rows empty. Others are as ever."""
    rng = np.random.default_rng(5)
    pool = Pool(rng, kv="bf16", hkv=1, D=64, ps=16, lens=[60, 300, 50])
    good = [bushy(20, 0), bushy(257, 1), bushy(10, 2)]
    q = _q(rng, 287, 2, 64, "bf16")
    out, lse, err = run(pool, None, good, q, 2, 0, 0, 0.125, "bf16")
    assert err == M.MOE_DEVERR_TREE
    assert (out[20:277] == 0).all() and (lse[20:277] == -np.inf).all()
    pick = np.r_[0:20, 277:287]
    want = reference(pool_keys(pool), [0, 2], [good[0], good[2]], [40, 40], q[pick], 2, 0, 0,
                     0.125, "bf16")
    check(out[pick], want[0], want[2], "out")
    for bad in (7, 8, 1 << 30, -2):
        p = bushy(20, 0)
        p[7] = bad
        fixed = p.copy()
        fixed[7] = -1
        out, lse, err = run(pool, [0], [p], q[:20], 2, 0, 0, 0.125, "bf16")
        assert err == M.MOE_DEVERR_TREE
        want = reference(pool_keys(pool), [0], [fixed], [40], q[:20], 2, 0, 0, 0.125, "bf16")
        check(out, want[0], want[2], "out")


@pytest.mark.parametrize("kv", ["f16", "e4m3"])
def test_values_that_are_not_finite(kv):
    """Infinities and NaN in drafted tokens and at the context's end: they
    reach the rows that see them and no others."""
    if kv == "e4m3":
        bad = [float("nan")]
    else:
        bad = [float("inf"), float("-inf"), float("nan")]
    rng = np.random.default_rng(6)
    pool = Pool(rng, kv=kv, hkv=2, D=64, ps=16, lens=[62])
    par = bushy(30)
    leaf = [t for t in range(30) if t not in par][:len(bad)]
    for t, b in zip(leaf, bad):
        pool.poison(0, [32 + t], k=1.0 if kv == "f16" else 0.5, v=b)
    if kv == "e4m3":                     # what the host keeps is the code's value
        for hi, sc in ((0, pool.scales[0]), (1, pool.scales[1])):
            for t in leaf:
                pool.host[0][hi][:, 32 + t] = (0.5 * sc.double().numpy()[:, None] if hi == 0
                                               else np.nan)
    q = _q(rng, 30, 4, 64, "f16")
    out, lse, err = run(pool, None, [par], q, 4, 0, 0, 0.125, "f16")
    with np.errstate(invalid="ignore"):
        want = reference(pool_keys(pool), [0], [par], [32], q, 4, 0, 0, 0.125, "f16")
    assert err == 0
    check(out, want[0], want[2], "out")
    check(lse, want[1], want[3], "lse")


def test_graph_with_other_trees():
    """Captured once; replays take the lengths, trees and rows of the time."""
    rng = np.random.default_rng(7)
    pool = Pool(rng, kv="bf16", hkv=2, D=128, ps=16, lens=[300, 120])
    cache, table = pool.desc(M)
    i32 = dict(dtype=torch.int32, device="cuda")
    T, hq = 48, 8
    q = _q(rng, T, hq, 128, "bf16")
    qd = torch.from_numpy(q).to("cuda", torch.bfloat16)
    out, lse = torch.empty_like(qd), torch.empty(T, hq, device="cuda")
    err, cu, par = torch.zeros(1, **i32), torch.zeros(3, **i32), torch.zeros(T, **i32)
    ws = torch.empty(M.moe_attn_tree_workspace_size(cache, 2, T, hq), dtype=torch.uint8,
                     device="cuda")
    call = lambda: M.moe_attn_tree(cache, table, qd, cu, par, out, 0.1, err, ws,  # noqa: E731
                                   lse=lse)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for a, b, tree in [(40, 8, bushy), (1, 47, chain), (24, 24, star)]:
        parents = [tree(a, 0), tree(b, 1)]
        cu.copy_(torch.tensor([0, a, a + b]))
        par.copy_(torch.tensor(np.concatenate(parents)))
        out.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        want = reference(pool_keys(pool), [0, 1], parents, [300 - a, 120 - b], q, hq, 0, 0, 0.1,
                         "bf16")
        check(out.double().cpu().numpy(), want[0], want[2], "out")
        replayed = out.clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(out, replayed)
    assert M.moe_read_device_error(err) == 0
