"""moe_attn_decode and moe_attn_prefill against a plain 64-bit attention.

Everything that a query does not see is NaN in the cache (unwritten slots of
pages, tokens outside the window, later tokens of a prompt), so any leak
shows. Bars are derived in cache_ref.attention.
"""
import numpy as np
import pytest
import torch

import mixture_experts_expert_sigmoid_amd as M
from tests.cache_ref import DT, Pool, attention, check, visible

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]


def _strided(shape, dt, how):
    """An empty tensor of this shape: dense, with padded rows and heads, or
    with the heads outermost."""
    r, h, d = shape
    if how == "pad":
        return torch.full((r, h + 1, d + 8), float("nan"), dtype=DT[dt], device="cuda")[:, :h, :d]
    if how == "heads":
        return torch.full((h, r, d), float("nan"), dtype=DT[dt], device="cuda").transpose(0, 1)
    return torch.full(shape, float("nan"), dtype=DT[dt], device="cuda")


def _reference(pool, slots, rows, q, hq, window, first, scale, dt):
    """rows: per list entry the number of new tokens; q float64 [T, hq, D]"""
    g = hq // pool.hkv
    out, lse, bo, bl = [], [], [], []
    at = 0
    for s, m in zip(slots, rows):
        L = pool.lens[s] if s >= 0 else 0
        see = visible(np.arange(L - m, L), L, window, first)
        for h in range(pool.hkv):
            if s >= 0:
                k, v = (pool.host[s][i][h] for i in range(2))
            else:
                k = v = np.zeros((0, pool.D))
            r = attention(q[at:at + m, h * g:(h + 1) * g], k, v, see, scale, dt)
            for acc, x in zip((out, lse, bo, bl), r):
                acc.append(x)
        at += m

    def join(parts, per):
        # parts: [seq][head] of [m, g, ...] -> [T, hq, ...]
        seqs = []
        for i in range(0, len(parts), pool.hkv):
            seqs.append(np.concatenate(parts[i:i + pool.hkv], 1))
        return np.concatenate(seqs, 0)
    return tuple(join(x, None) for x in (out, lse, bo, bl))


def _hide(pool, slots, rows, window, first):
    """NaN into every token that no query of the call sees, and -1 into the
    table entries of pages without any seen token."""
    for s, m in zip(slots, rows):
        if s < 0 or pool.lens[s] == 0 or m == 0:
            continue
        L = pool.lens[s]
        seen = visible(np.arange(L - m, L), L, window, first).any(0)
        pool.poison(s, np.nonzero(~seen)[0])
        for pg in range(-(-L // pool.ps)):
            if not seen[pg * pool.ps:(pg + 1) * pool.ps].any():
                pool.tab[s, pg] = -1
    pool.table.copy_(torch.from_numpy(pool.tab))


def _run(kind, pool, slots, rows, q, hq, window, first, scale, dt, how="dense"):
    cache, table = pool.desc(M)
    T, D = q.shape[0], pool.D
    qd = _strided((T, hq, D), dt, how)
    qd.copy_(torch.from_numpy(q))
    out = _strided((T, hq, D), dt, how)
    lse = torch.full((T, hq), 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    sl = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    n = len(rows)
    if kind == "decode":
        ws = torch.empty(M.moe_attn_decode_workspace_size(cache, n, hq), dtype=torch.uint8,
                         device="cuda")
        call = lambda: M.moe_attn_decode(cache, table, qd, out, scale, err, ws,  # noqa: E731
                                         window=window, n_first=first, slots=sl, lse=lse)
    else:
        cu = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32,
                          device="cuda")
        ws = torch.empty(max(16, M.moe_attn_prefill_workspace_size(cache, n, T, hq)),
                         dtype=torch.uint8, device="cuda")
        call = lambda: M.moe_attn_prefill(cache, table, qd, cu, out, scale, err, ws,  # noqa: E731
                                          window=window, n_first=first, slots=sl, lse=lse)
    ws.fill_(0xFF)                       # NaN in whatever is read unwritten
    call()
    torch.cuda.synchronize()
    o1, l1 = out.clone(), lse.clone()
    call()
    torch.cuda.synchronize()
    # the same inputs give the same bits
    assert torch.equal(o1.view(torch.int16), out.contiguous().view(torch.int16).view(o1.shape))
    assert torch.equal(l1.view(torch.int32), lse.view(torch.int32))
    return out.double().cpu().numpy(), lse.double().cpu().numpy(), \
        M.moe_read_device_error(err)


def _q(rng, T, hq, D, dt, amp=1.5):
    return torch.from_numpy(amp * rng.standard_normal((T, hq, D))).to(DT[dt]).double().numpy()


# id: dt, kv, D, hq, hkv, ps, layout, strides, lens, window, first
DECODE = {
    "one_token": ("bf16", "bf16", 128, 8, 2, 16, "head", "dense", [1], 0, 0),
    "short_odd": ("bf16", "bf16", 128, 8, 2, 16, "head", "pad", [31, 32, 33, 5, 127, 129], 0, 0),
    "f16_d64": ("f16", "f16", 64, 6, 2, 48, "tok", "heads", [100, 1, 1000, 47, 48, 49], 0, 0),
    "d256": ("bf16", "bf16", 256, 4, 1, 32, "head", "dense", [77, 300], 0, 0),
    "d256_f16_mha": ("f16", "f16", 256, 2, 2, 16, "tok", "pad", [65, 3], 0, 0),
    "e4m3": ("bf16", "e4m3", 128, 16, 2, 64, "head", "dense", [200, 63, 64, 65, 513], 0, 0),
    "e4m3_f16_d64": ("f16", "e4m3", 64, 5, 1, 16, "tok", "dense", [33, 290], 0, 0),
    "e4m3_d256": ("bf16", "e4m3", 256, 3, 3, 32, "head", "pad", [150, 31], 0, 0),
    "mqa_40": ("bf16", "bf16", 128, 40, 1, 16, "head", "dense", [95, 400], 0, 0),
    "split_long": ("bf16", "bf16", 128, 4, 1, 64, "head", "dense", [20011], 0, 0),
    "split_two": ("f16", "e4m3", 128, 16, 2, 128, "tok", "dense", [9001, 37], 0, 0),
    "window": ("bf16", "bf16", 128, 8, 2, 16, "head", "dense", [1, 16, 17, 100, 1000, 515], 64, 4),
    "window_1": ("f16", "f16", 64, 4, 2, 32, "head", "dense", [1, 2, 300], 1, 0),
    "window_first_big": ("bf16", "bf16", 64, 4, 2, 16, "head", "dense", [50, 300, 129], 40, 100),
    "window_odd": ("bf16", "e4m3", 128, 8, 2, 16, "head", "dense", [2777, 999], 333, 17),
}


@pytest.mark.parametrize("name", list(DECODE))
def test_decode(name):
    dt, kv, D, hq, hkv, ps, layout, how, lens, window, first = DECODE[name]
    print(f"[case] decode {name}", flush=True)
    rng = np.random.default_rng(len(name) * 7 + D)
    pool = Pool(rng, kv=kv, hkv=hkv, D=D, ps=ps, lens=lens, layout=layout)
    n = len(lens)
    rows = [1] * n
    _hide(pool, range(n), rows, window, first)
    q = _q(rng, n, hq, D, dt)
    scale = D ** -0.5
    out, lse, err = _run("decode", pool, None, rows, q, hq, window, first, scale, dt, how)
    want = _reference(pool, range(n), rows, q, hq, window, first, scale, dt)
    assert err == 0
    check(lse, want[1], want[3], "lse")
    print("  worst error / bar: %.3f" % check(out, want[0], want[2], "out"), flush=True)


def test_decode_slots_and_empty_rows():
    """A batch through a slot list: permuted, with rows without a sequence, a
    slot of length zero, and one beyond the table (flagged)."""
    rng = np.random.default_rng(3)
    lens = [40, 0, 300, 17]
    pool = Pool(rng, kv="bf16", hkv=2, D=128, ps=16, lens=lens)
    slots = [3, -1, 0, 1, 2, -1]
    q = _q(rng, len(slots), 8, 128, "bf16")
    out, lse, err = _run("decode", pool, slots, [1] * 6, q, 8, 0, 0, 0.1, "bf16")
    want = _reference(pool, slots, [1] * 6, q, 8, 0, 0, 0.1, "bf16")
    # _reference skips a query at position -1 by its empty mask
    assert err == 0
    check(out, want[0], want[2], "out")
    check(lse, want[1], want[3], "lse")
    assert np.all(out[[1, 3, 5]] == 0) and np.all(np.isneginf(lse[[1, 3, 5]]))
    out2, lse2, err = _run("decode", pool, [3, 9, 0, 1, 2, -1], [1] * 6, q, 8, 0, 0, 0.1, "bf16")
    assert err == M.MOE_DEVERR_CACHE_PAGE
    assert np.array_equal(out, out2) and np.array_equal(lse, lse2)


def test_decode_many_sequences():
    """More sequences than one launch takes."""
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.integers(0, 70, 1100)]
    pool = Pool(rng, kv="f16", hkv=1, D=64, ps=16, lens=lens)
    q = _q(rng, len(lens), 2, 64, "f16")
    rows = [1] * len(lens)
    out, lse, err = _run("decode", pool, None, rows, q, 2, 0, 0, 0.125, "f16")
    want = _reference(pool, range(len(lens)), rows, q, 2, 0, 0, 0.125, "f16")
    assert err == 0
    check(out, want[0], want[2], "out")
    check(lse, want[1], want[3], "lse")


# Enough (sequence, key-value head, 16 query heads) pairs that each is one
# wave's work: lens are n random lengths up to the given one and one long one.
MANY = {
    "d64": ("f16", "f16", 64, 12, 4, 16, "pad", 400, 60, 3001, 0, 0),
    "d64_e4m3": ("bf16", "e4m3", 64, 8, 8, 32, "heads", 200, 50, 2000, 0, 0),
    "d128": ("bf16", "bf16", 128, 16, 8, 16, "dense", 140, 70, 5000, 0, 0),
    "d128_e4m3_window": ("f16", "e4m3", 128, 8, 8, 16, "pad", 140, 300, 900, 50, 5),
    "d128_64_heads_share": ("bf16", "bf16", 128, 128, 2, 16, "dense", 130, 40, 1500, 0, 0),
    "d256": ("bf16", "bf16", 256, 6, 2, 16, "dense", 260, 40, 1800, 0, 0),
    "d256_e4m3": ("f16", "e4m3", 256, 8, 4, 16, "heads", 260, 40, 700, 30, 0),
}


@pytest.mark.parametrize("name", list(MANY))
def test_decode_many_pairs(name):
    dt, kv, D, hq, hkv, ps, how, n, top, long, window, first = MANY[name]
    print(f"[case] decode many {name}", flush=True)
    rng = np.random.default_rng(len(name) * 11 + D)
    lens = [int(x) for x in rng.integers(1, top, n)]
    lens[n // 3] = long
    pool = Pool(rng, kv=kv, hkv=hkv, D=D, ps=ps, lens=lens)
    rows = [1] * n
    _hide(pool, range(n), rows, window, first)
    q = _q(rng, n, hq, D, dt)
    scale = D ** -0.5
    out, lse, err = _run("decode", pool, None, rows, q, hq, window, first, scale, dt, how)
    want = _reference(pool, range(n), rows, q, hq, window, first, scale, dt)
    assert err == 0
    check(lse, want[1], want[3], "lse")
    print("  worst error / bar: %.3f" % check(out, want[0], want[2], "out"), flush=True)


def test_decode_missing_page_is_masked_and_flagged():
    rng = np.random.default_rng(5)
    pool = Pool(rng, kv="bf16", hkv=2, D=128, ps=16, lens=[100])
    q = _q(rng, 1, 4, 128, "bf16")
    for bad in (-1, pool.P, 1 << 30):
        tab = pool.tab.copy()
        tab[0, 2] = bad
        pool.table.copy_(torch.from_numpy(tab))
        out, lse, err = _run("decode", pool, None, [1], q, 4, 0, 0, 0.1, "bf16")
        assert err == M.MOE_DEVERR_CACHE_PAGE
        see = np.ones((1, 100), bool)
        see[0, 32:48] = False
        for h in range(2):
            w = attention(q[:, 2 * h:2 * h + 2], pool.host[0][0][h], pool.host[0][1][h], see,
                          0.1, "bf16")
            check(out[:, 2 * h:2 * h + 2], w[0], w[2], "out")


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("dt,kv", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3")])
def test_values_not_finite(kind, dt, kv):
    """Visible infinities and NaN enter as the formula says; scores of minus
    infinity take no part; large scores do not overflow."""
    rng = np.random.default_rng(6)
    L, D = 90, 128
    pool = Pool(rng, kv=kv, hkv=1, D=D, ps=16, lens=[L, L, L], amp=1.0)
    q = _q(rng, 3, 2, D, dt, amp=30.0)
    q[1] /= 32                           # every probability well above underflow
    if kv != "e4m3":
        pool.v[int(pool.tab[1, 50 // 16]), 0, 50 % 16, 7] = float("inf")
        pool.host[1][1][0, 50, 7] = np.inf
        # slot 2: keys of -inf along a positive query component: score -inf
        q[2, :, 0] = 3.0
        pool.k[int(pool.tab[2, 20 // 16]), 0, 20 % 16, 0] = -float("inf")
        pool.host[2][0][0, 20, 0] = -np.inf
    out, lse, err = _run(kind, pool, None, [1, 1, 1], q, 2, 0, 0, 0.3, dt)
    with np.errstate(invalid="ignore"):
        for i in range(3):
            see = np.ones((1, L), bool)
            if kv != "e4m3" and i == 2:
                see[0, 20] = False
            w = attention(q[i:i + 1], pool.host[i][0][0], pool.host[i][1][0], see, 0.3, dt)
            bar = np.where(np.isfinite(w[2]), w[2], 1.0)
            check(out[i:i + 1], w[0], bar, ("out", i))
            check(lse[i:i + 1], w[1], w[3], ("lse", i))


# id: dt, kv, D, hq, hkv, ps, layout, strides, lens, rows, window, first
PREFILL = {
    "one_token": ("bf16", "bf16", 128, 8, 2, 16, "head", "dense", [1], [1], 0, 0),
    "prompt_37": ("bf16", "bf16", 128, 8, 2, 16, "head", "pad", [37], [37], 0, 0),
    "ragged": ("f16", "f16", 64, 6, 2, 48, "tok", "heads", [100, 1, 260, 47, 64],
               [100, 1, 260, 0, 64], 0, 0),
    "chunk": ("bf16", "bf16", 128, 8, 1, 16, "head", "dense", [300, 129, 64], [33, 64, 1], 0, 0),
    "d256": ("bf16", "bf16", 256, 4, 2, 32, "head", "dense", [77, 130], [77, 20], 0, 0),
    "d256_e4m3": ("f16", "e4m3", 256, 3, 3, 16, "tok", "dense", [90], [70], 0, 0),
    "e4m3": ("bf16", "e4m3", 128, 8, 2, 64, "head", "dense", [200, 65], [200, 2], 0, 0),
    "e4m3_d64": ("f16", "e4m3", 64, 10, 2, 16, "head", "pad", [150, 63], [150, 63], 0, 0),
    "mha": ("bf16", "bf16", 64, 3, 3, 16, "head", "dense", [300], [300], 0, 0),
    "mqa_40": ("bf16", "bf16", 128, 40, 1, 16, "head", "dense", [66], [13], 0, 0),
    "split": ("bf16", "bf16", 128, 4, 1, 64, "head", "dense", [5003], [9], 0, 0),
    "split_two": ("f16", "e4m3", 128, 4, 2, 128, "tok", "dense", [3001, 700], [3, 40], 0, 0),
    "window": ("bf16", "bf16", 128, 8, 2, 16, "head", "dense", [400, 33], [400, 33], 64, 4),
    "window_chunk": ("f16", "f16", 64, 4, 2, 32, "head", "dense", [1000, 517], [130, 65], 100, 17),
    "window_1": ("bf16", "bf16", 64, 2, 1, 16, "head", "dense", [140], [140], 1, 0),
    "window_first_big": ("bf16", "e4m3", 64, 4, 2, 16, "head", "dense", [300], [300], 40, 150),
    "more_rows_than_len": ("bf16", "bf16", 128, 4, 2, 16, "head", "dense", [20], [50], 0, 0),
}


@pytest.mark.parametrize("name", list(PREFILL))
def test_prefill(name):
    dt, kv, D, hq, hkv, ps, layout, how, lens, rows, window, first = PREFILL[name]
    print(f"[case] prefill {name}", flush=True)
    rng = np.random.default_rng(len(name) * 11 + D)
    pool = Pool(rng, kv=kv, hkv=hkv, D=D, ps=ps, lens=lens, layout=layout)
    n = len(lens)
    _hide(pool, range(n), rows, window, first)
    q = _q(rng, sum(rows), hq, D, dt)
    scale = D ** -0.5
    out, lse, err = _run("prefill", pool, None, rows, q, hq, window, first, scale, dt, how)
    want = _reference(pool, range(n), rows, q, hq, window, first, scale, dt)
    assert err == 0
    check(lse, want[1], want[3], "lse")
    print("  worst error / bar: %.3f" % check(out, want[0], want[2], "out"), flush=True)


# The same calls over tables with room for long contexts: what the table can
# hold decides whether keys are split and joined.
@pytest.mark.parametrize("kind,name", [("decode", n) for n in DECODE] +
                         [("prefill", n) for n in PREFILL])
def test_wide_tables(kind, name):
    print(f"[case] wide {kind} {name}", flush=True)
    if kind == "decode":
        dt, kv, D, hq, hkv, ps, layout, how, lens, window, first = DECODE[name]
        rows = [1] * len(lens)
    else:
        dt, kv, D, hq, hkv, ps, layout, how, lens, rows, window, first = PREFILL[name]
    rng = np.random.default_rng(len(name) * 5 + D)
    pool = Pool(rng, kv=kv, hkv=hkv, D=D, ps=ps, lens=lens, layout=layout,
                max_pages=1 + 32768 // ps)
    _hide(pool, range(len(lens)), rows, window, first)
    q = _q(rng, sum(rows), hq, D, dt)
    out, lse, err = _run(kind, pool, None, rows, q, hq, window, first, D ** -0.5, dt, how)
    want = _reference(pool, range(len(lens)), rows, q, hq, window, first, D ** -0.5, dt)
    assert err == 0
    check(lse, want[1], want[3], "lse")
    print("  worst error / bar: %.3f" % check(out, want[0], want[2], "out"), flush=True)


@pytest.mark.parametrize("dt,kv,D", [("bf16", "bf16", 128), ("f16", "f16", 64),
                                     ("bf16", "e4m3", 128), ("bf16", "bf16", 256)])
@pytest.mark.parametrize("window", [0, 24])
def test_prefill_later_tokens_do_not_leak(dt, kv, D, window):
    """NaN (and infinite, where the type has them) keys and values at some
    tokens of a prompt: rows that do not see them keep their exact results,
    rows that see them get NaN where the formula does."""
    rng = np.random.default_rng(8)
    L, hq, hkv = 150, 4, 2
    pool = Pool(rng, kv=kv, hkv=hkv, D=D, ps=16, lens=[L])
    pool.poison(0, [70], k=0.25, v=float("nan"))
    pool.poison(0, [101])
    if kv != "e4m3":
        pool.poison(0, [90], k=0.5, v=float("inf"))
    q = _q(rng, L, hq, D, dt)
    out, lse, err = _run("prefill", pool, None, [L], q, hq, window, 3 if window else 0, 0.1, dt)
    with np.errstate(invalid="ignore"):
        want = _reference(pool, [0], [L], q, hq, window, 3 if window else 0, 0.1, dt)
    assert err == 0
    bar = np.where(np.isfinite(want[2]), want[2], 1.0)
    check(out, want[0], bar, "out")
    assert np.isfinite(out[:70]).all()


def test_prefill_slots_and_rows_without_a_sequence():
    rng = np.random.default_rng(9)
    pool = Pool(rng, kv="bf16", hkv=2, D=128, ps=16, lens=[40, 0, 200])
    slots, rows = [2, -1, 0, 1], [30, 5, 40, 3]
    q = _q(rng, sum(rows), 4, 128, "bf16")
    out, lse, err = _run("prefill", pool, slots, rows, q, 4, 0, 0, 0.1, "bf16")
    want = _reference(pool, slots, rows, q, 4, 0, 0, 0.1, "bf16")
    assert err == 0
    check(out, want[0], want[2], "out")
    check(lse, want[1], want[3], "lse")
    assert np.all(out[30:35] == 0) and np.all(out[75:] == 0)


def test_prefill_missing_page_is_masked_and_flagged():
    rng = np.random.default_rng(10)
    pool = Pool(rng, kv="bf16", hkv=1, D=128, ps=16, lens=[100])
    q = _q(rng, 60, 2, 128, "bf16")
    tab = pool.tab.copy()
    tab[0, 2] = -1
    pool.table.copy_(torch.from_numpy(tab))
    out, lse, err = _run("prefill", pool, None, [60], q, 2, 0, 0, 0.1, "bf16")
    assert err == M.MOE_DEVERR_CACHE_PAGE
    see = visible(np.arange(40, 100), 100, 0, 0)
    see[:, 32:48] = False
    w = attention(q, pool.host[0][0][0], pool.host[0][1][0], see, 0.1, "bf16")
    check(out, w[0], w[2], "out")


def test_decode_equals_prefill_of_one_row():
    """The two entry points compute the same function."""
    rng = np.random.default_rng(11)
    lens = [513, 100]
    pool = Pool(rng, kv="bf16", hkv=2, D=128, ps=16, lens=lens)
    q = _q(rng, 2, 8, 128, "bf16")
    want = _reference(pool, [0, 1], [1, 1], q, 8, 50, 4, 0.1, "bf16")
    a = _run("decode", pool, None, [1, 1], q, 8, 50, 4, 0.1, "bf16")
    b = _run("prefill", pool, None, [1, 1], q, 8, 50, 4, 0.1, "bf16")
    assert np.all(np.abs(a[0] - b[0]) <= 2 * want[2])
    assert np.all(np.abs(a[1] - b[1]) <= 2 * want[3])


def test_page_offsets_beyond_32_bits():
    """Pages whose byte offset passes 2^32 (a page stride of 64 MiB)."""
    rng = np.random.default_rng(12)
    D, ps, P, stride = 128, 16, 80, 1 << 25           # elements
    flat = torch.zeros(P * stride + 4096, dtype=torch.bfloat16, device="cuda")
    flat2 = torch.zeros_like(flat)
    k = flat.as_strided((P, 1, ps, D), (stride, ps * D, D, 1))
    v = flat2.as_strided((P, 1, ps, D), (stride, ps * D, D, 1))
    small = Pool(rng, kv="bf16", hkv=1, D=D, ps=ps, lens=[P * ps - 3], spare=0)
    k.copy_(small.k)
    v.copy_(small.v)
    small.k, small.v = k, v
    q = _q(rng, 5, 2, D, "bf16")
    want = _reference(small, [0], [5], q, 2, 0, 0, 0.1, "bf16")
    out, lse, err = _run("prefill", small, None, [5], q, 2, 0, 0, 0.1, "bf16")
    assert err == 0
    check(out, want[0], want[2], "prefill")
    out, lse, err = _run("decode", small, None, [1], q[4:], 2, 0, 0, 0.1, "bf16")
    check(out, want[0][4:], want[2][4:], "decode")


def test_attention_replays_in_a_graph_and_on_a_stream():
    """Captured once, replayed with lengths, queries and cache contents
    changed in place and eager work in between; each replay equals the eager
    call. Then the same on a stream of its own."""
    rng = np.random.default_rng(13)
    lens = [300, 41, 1000]
    pool = Pool(rng, kv="bf16", hkv=2, D=128, ps=16, lens=lens)
    cache, table = pool.desc(M)
    q = torch.from_numpy(_q(rng, 3, 8, 128, "bf16")).to("cuda", torch.bfloat16)
    qp = torch.from_numpy(_q(rng, 60, 8, 128, "bf16")).to("cuda", torch.bfloat16)
    cu = torch.tensor([0, 20, 25, 60], dtype=torch.int32, device="cuda")
    out, outp = torch.empty_like(q), torch.empty_like(qp)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(M.moe_attn_decode_workspace_size(cache, 3, 8), dtype=torch.uint8,
                     device="cuda")
    wsp = torch.empty(max(16, M.moe_attn_prefill_workspace_size(cache, 3, 60, 8)),
                      dtype=torch.uint8, device="cuda")

    def step(stream=None):
        M.moe_attn_decode(cache, table, q, out, 0.1, err, ws, stream=stream)
        M.moe_attn_prefill(cache, table, qp, cu, outp, 0.1, err, wsp, stream=stream)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for rep in range(4):
        pool.len_t.copy_(torch.tensor([300 - rep, 41 - 5 * rep, 1000 - 100 * rep],
                                      dtype=torch.int32))
        q.copy_(torch.roll(q, 1, 0))
        out.fill_(float("nan"))
        outp.fill_(float("nan"))
        ws.fill_(0xFF)
        wsp.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        got = out.clone(), outp.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], outp), rep
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out.zero_()
    s.wait_stream(torch.cuda.current_stream())
    step(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(got[0], out) and torch.equal(got[1], outp)
    assert M.moe_read_device_error(err) == 0
