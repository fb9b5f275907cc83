"""Infinite latent values, which are keys and values at once: a row to which such a
key gives a score of -infinity is as without it, one to which it gives infinity is
NaN, wherever the key lies -- in a tile of keys that all rows see, or in one of which
some see a part."""
import numpy as np
import pytest
import torch

from tests.cache_ref import check, visible
from tests.test_gpu_attn import _q
from tests.test_gpu_latent import LatentPool, _wide, bushy, run, sees

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]

# dt, latent_dim, heads, (context, new rows) of each, tree, window, first
CASES = {
    "one": ("bf16", 512, 16, [(500, 1)], None, 0, 0),
    "one_long": ("bf16", 512, 8, [(9000, 1)], None, 0, 0),
    "batch": ("f16", 512, 24, [(96, 1), (333, 1), (64, 1), (1500, 1)], None, 0, 0),
    "short_vectors": ("f16", 256, 16, [(700, 1), (200, 1)], None, 0, 0),
    "chunk": ("bf16", 256, 6, [(400, 37)], None, 0, 0),
    "chunk_f16": ("f16", 512, 8, [(150, 50), (40, 3)], None, 0, 0),
    "tree": ("bf16", 512, 16, [(300, 20)], "bushy", 0, 0),
    "window": ("f16", 256, 4, [(900, 12)], None, 300, 20),
}


def places(C, L, window, first):
    """Of keys that every row sees: the first one, one on either side of a tile's
    edge, deep ones, the newest of the context."""
    at = [j for j in (0, 31, 32, C // 2, C - 40, C - 1) if 0 <= j < C]
    if window:
        at = [j for j in at if j < first or j > L - window] + [first - 1, C - 7]
    return sorted(set(at))


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("sign", [1, -1])
def test_where_it_lies(name, sign):
    dt, dc, H, seqs, tree, window, first = CASES[name]
    rng = np.random.default_rng(len(name) + 40)
    lens = [C + m for C, m in seqs]
    rows = [m for _, m in seqs]
    q = _q(rng, sum(rows), H, dc + 64, dt)
    dim, scale = 77, 0.04 * sign
    # even heads: -infinity in dimension `dim` of the scaled score; odd ones: +infinity
    q[..., dim] = np.where(np.arange(H) % 2 == 0, -sign, sign) * (np.abs(q[..., dim]) + 0.25)
    par = [bushy(m, i) for i, m in enumerate(rows)] if tree else None
    see = [sees(par[i], C, window, first) if tree else
           visible(np.arange(C, C + m), C + m, window, first) for i, (C, m) in enumerate(seqs)]
    even = np.arange(0, H, 2)
    every = [places(C, C + m, window, first) for C, m in seqs]
    # one place after the other, then all of them
    turns = [[[e[min(t, len(e) - 1)]] for e in every] for t in range(max(map(len, every)))]
    turns.append(every)
    for turn in turns:
        pool = LatentPool(np.random.default_rng(len(name)), kv=dt, dc=dc, ps=16, lens=lens)
        got_at, want = 0, []
        for s, keys in enumerate(turn):
            ok = see[s].copy()
            assert ok[:, keys].all()
            ok[:, keys] = False
            host = pool.host[s]
            want.append(_wide(q[got_at:got_at + rows[s]][:, even], host, host[:, :dc], ok, scale, dt))
            got_at += rows[s]
            for j in keys:
                pool.set(s, j, slice(dim, dim + 1), float("inf"))
        out, lse, err = run(pool, None, par, rows, q, window, first, scale, dt,
                            one=all(m == 1 for m in rows) and not tree)
        o, z, bo, bl = [np.concatenate(x, 0) for x in zip(*want)]
        assert err == 0
        check(out[:, even], o, bo, (turn, "out"))
        check(lse[:, even], z, bl, (turn, "lse"))
        assert np.isnan(out[:, 1::2]).all(), turn


@pytest.mark.parametrize("C,H", [(70, 16), (700, 16), (40, 3)])
def test_no_other_key(C, H):
    """Rows all of whose keys are such: 0 and -infinity, in one part or several."""
    rng = np.random.default_rng(C)
    pool = LatentPool(rng, kv="f16", dc=512, ps=16, lens=[C])
    for j in range(C):
        pool.set(0, j, slice(5, 6), float("inf"))
    q = _q(rng, 1, H, 576, "f16")
    q[..., 5] = -np.abs(q[..., 5]) - 0.25
    out, lse, err = run(pool, None, None, [1], q, 0, 0, 0.05, "f16", one=True)
    assert err == 0 and (out == 0).all() and (lse == -np.inf).all()
