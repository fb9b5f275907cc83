"""Plain 64-bit references of the cache and attention operators, and the
bars their outputs are held to (test infrastructure)."""
from __future__ import annotations

import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
# largest relative error of one rounding to the type: half the spacing of
# numbers with 8 and 11 significant bits (1 + 2^-8 lies midway between the
# bf16 numbers 1 and 1 + 2^-7)
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def visible(pos, L, window, first):
    """Boolean [len(pos), L]: which keys 0..L-1 a query at each position sees."""
    p, j = np.asarray(pos)[:, None], np.arange(L)[None, :]
    ok = j <= p
    if window:
        ok &= (p - j < window) | (j < first)
    return ok


def attention(q, k, v, see, scale, dt):
    """q [m, g, D], k and v [L, D] float64, see [m, L] -> out [m, g, D],
    lse [m, g], and the bars of both.

    Bars. delta bounds a score's error: the fp32 sums of D exact products
    (16-bit operands) and the scaling and base change after them, at most
    (D + 16) 2^-23 of the sum of magnitudes; e^delta is the relative error of
    a probability. A probability is rounded once to the type (u), the result
    once (u); statistics and sums add a few 2^-20 at most. f16 probabilities
    below 2^-14 have an absolute error of 2^-25 each."""
    m, g, D = q.shape
    L = k.shape[0]
    u = UNIT[dt]
    out, lse = np.zeros((m, g, D)), np.full((m, g), -np.inf)
    bo, bl = np.zeros((m, g, D)), np.zeros((m, g))
    for i in range(m):
        idx = np.nonzero(see[i])[0]
        if len(idx) == 0:
            continue
        kk, vv = k[idx], v[idx]
        s = scale * (q[i] @ kk.T)                       # [g, n]
        mag = abs(scale) * (np.abs(q[i]) @ np.abs(kk).T)
        mx = s.max(1, keepdims=True)
        if not np.isfinite(mx).all() and (mx == -np.inf).all():
            continue
        p = np.exp(s - mx)
        z = p.sum(1, keepdims=True)
        p /= z
        out[i] = p @ vv
        lse[i] = (mx + np.log(z))[:, 0]
        delta = (D + 16) * 2.0 ** -23 * mag.max(1, keepdims=True)
        a = p @ np.abs(vv)
        bo[i] = u * np.abs(out[i]) + (u + 2 * delta + 2.0 ** -20) * a
        if dt == "f16":
            bo[i] += 2.0 ** -25 * (1 + np.abs(vv).sum(0))
        else:
            bo[i] += 2.0 ** -126
        bl[i] = (delta[:, 0] + 2.0 ** -21 * (1 + np.abs(lse[i]) + np.abs(mx[:, 0])))
    return out, lse, bo, bl


class Pool:
    """One layer's cache on the GPU with everything unwritten NaN, and its
    contents in float64 on the host. `seqs`: per slot a list of positions that
    hold tokens (others of the slot keep NaN)."""

    def __init__(self, rng, *, kv, hkv, D, ps, lens, layout="head", max_pages=None,
                 spare=3, amp=1.0):
        self.kv, self.hkv, self.D, self.ps, self.lens = kv, hkv, D, ps, list(lens)
        need = [-(-L // ps) for L in self.lens]
        self.P = P = sum(need) + spare
        mp = max([1] + need) if max_pages is None else max_pages
        order = rng.permutation(P)
        self.tab = np.full((len(self.lens), mp), -1, np.int32)
        at = 0
        for i, n in enumerate(need):
            self.tab[i, :n] = order[at:at + n]
            at += n
        shape = (P, hkv, ps, D) if layout == "head" else (P, ps, hkv, D)
        self.scales = (None, None)
        vals = []
        for _ in range(2):
            x = torch.full(shape, float("nan"), dtype=torch.float32)
            x = x if layout == "head" else x.transpose(1, 2)
            vals.append(x)
        if kv == "e4m3":
            self.scales = tuple(torch.from_numpy(rng.uniform(0.01, 0.05, hkv).astype(np.float32))
                                for _ in range(2))
        self.host = []                       # per slot: (k, v) float64 [hkv, L, D]
        for i, L in enumerate(self.lens):
            kv_ = []
            for x, sc in zip(vals, self.scales):
                y = torch.from_numpy(amp * rng.standard_normal((hkv, L, D)).astype(np.float32))
                if sc is not None:
                    y = (y / sc[:, None, None]).clamp(-448, 448)
                y = y.to(DT[kv]).float()
                for pg in range(need[i]):
                    a, b = pg * ps, min(L, pg * ps + ps)
                    x[self.tab[i, pg], :, :b - a] = y[:, a:b]
                y = y.double()
                kv_.append((y if sc is None else y * sc[:, None, None].double()).numpy())
            self.host.append(kv_)
        self.k, self.v = (self._dev(x) for x in vals)
        self.table = torch.from_numpy(self.tab).cuda()
        self.len_t = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.ks, self.vs = (None if s is None else s.cuda() for s in self.scales)

    def _dev(self, x):
        # .to keeps the strides of a dense tensor
        return x.to(DT[self.kv]).cuda()

    def poison(self, slot, positions, k=float("nan"), v=float("nan")):
        """Writes k and v values into these positions of a slot, host copy too."""
        for x, val, hi in ((self.k, k, 0), (self.v, v, 1)):
            raw = torch.tensor([val]).to(DT[self.kv])
            for j in positions:
                pg = int(self.tab[slot, j // self.ps])
                x.view(torch.uint8 if self.kv == "e4m3" else x.dtype)[pg, :, j % self.ps] = \
                    raw.view(torch.uint8 if self.kv == "e4m3" else raw.dtype).cuda()
                self.host[slot][hi][:, j] = raw.double().item()

    def desc(self, M):
        return (M.kv_cache(self.k, self.v, self.ks, self.vs),
                M.kv_table(self.table, self.len_t, self.ps, self.P))


def check(got, want, bar, what):
    """Every element within its bar; infinities and NaN in the same places."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, what
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), (what, "NaN")
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)]), (what, "inf")
    err = np.abs(got[fin] - want[fin]) / np.maximum(bar[fin], 1e-300)
    worst = float(err.max()) if err.size else 0.0
    assert worst <= 1.0, (what, worst)
    return worst
