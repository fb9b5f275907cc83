"""Attention over contexts so long that one workgroup or wave passes more than
64 units of keys: the lookups of pages renewed inside the loops, pairs ended,
taken whole and started by one workgroup, missing pages far inside."""
import numpy as np
import pytest
import torch

import mixture_experts_expert_sigmoid_amd as M
from tests.cache_ref import DT
from tests.test_gpu_attn import _q
from tests.test_gpu_cache import _i

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]


def _truth(q, k, v, see, scale, dt):
    """cache_ref.attention with its bars, for one sequence and key-value head, on
    the GPU: q [m, g, D], k and v [L, D], see [m, L], all float64."""
    u = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dt]
    m, g, D = q.shape
    rows = q.reshape(m * g, D)
    mask = see.repeat_interleave(g, 0)
    kt = k.t().contiguous()
    s = (scale * (rows @ kt)).masked_fill(~mask, -torch.inf)
    mag = (abs(scale) * (rows.abs() @ kt.abs())).masked_fill(~mask, 0).amax(1, keepdim=True)
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    out = p @ v
    delta = (D + 16) * 2.0 ** -23 * mag
    bo = u * out.abs() + (u + 2 * delta + 2.0 ** -20) * (p @ v.abs())
    bo += 2.0 ** -25 * (1 + mask.double() @ v.abs()) if dt == "f16" else 2.0 ** -126
    bl = delta[:, 0] + 2.0 ** -21 * (1 + lse.abs() + s.amax(1).abs())
    return tuple(x.reshape(m, g, *x.shape[1:]) for x in (out, lse, bo, bl))


# Lengths that give a workgroup (or a wave by itself: "wave") over 64 units of
# keys: page lookups are renewed in the loop, and a workgroup ends one pair,
# takes others whole and starts another. id: dt, kv, D, hkv, g, n, lo, hi,
# window, first
LONG = {
    "bf16_d128": ("bf16", "bf16", 128, 8, 2, 60, 4000, 20000, 0, 0),
    "e4m3_d128": ("f16", "e4m3", 128, 8, 3, 60, 4000, 20000, 0, 0),
    "f16_d64": ("f16", "f16", 64, 8, 2, 80, 3000, 22000, 0, 0),
    "bf16_d256": ("bf16", "bf16", 256, 4, 2, 40, 4000, 26000, 0, 0),
    "window_d128": ("bf16", "bf16", 128, 8, 2, 60, 9500, 30000, 10007, 100),
    "wave_bf16_d128": ("bf16", "bf16", 128, 16, 1, 80, 2000, 7000, 0, 0),
    "wave_e4m3_d64": ("bf16", "e4m3", 64, 16, 2, 110, 1500, 9000, 0, 0),
    "wave_window_f16_d64": ("f16", "f16", 64, 16, 1, 110, 2300, 9000, 4005, 33),
}


class _Shared:
    """Slots whose rows name the pages of one pool in different order, so that
    long contexts take little memory; NaN is in a page that no row may read."""

    def __init__(self, seed, kv, D, hkv, lens, ps, pages, window=0, first=0, rows=1, drop=()):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.kv, self.lens, self.ps = kv, lens, ps
        shape = (pages + 1, hkv, ps, D)
        sc = torch.rand(2, hkv, generator=gen, device="cuda") * 0.02 + 0.02
        self.sc = (sc[0].contiguous(), sc[1].contiguous()) if kv == "e4m3" else (None, None)
        kvs = []
        for s in self.sc:
            x = torch.randn(shape, generator=gen, device="cuda")
            x[pages] = float("nan")
            kvs.append((x if s is None else x / s[:, None, None]).to(DT[kv]))
        self.k, self.v = kvs
        self.pages = pages
        need = [-(-L // ps) for L in lens]
        tab = torch.full((len(lens), max(need)), pages, dtype=torch.int64)
        at = torch.arange(max(need))
        for i, m in enumerate(need):
            tab[i, :m] = ((at * (2 * i + 1) + 31 * i) % pages)[:m]
            lo = lens[i] - rows - window + 1 if window else 0
            # pages that no row sees hold NaN
            dead = (at[:m] * ps >= first) & (at[:m] * ps + ps <= lo)
            tab[i, :m][dead] = pages
        for i, j in drop:
            tab[i, j] = -1
        self.tab = tab.cuda()
        self.cache = M.kv_cache(self.k, self.v, *self.sc)
        self.table = M.kv_table(self.tab.int(), _i(lens), ps, pages + 1)

    def head(self, i, h):
        """float64 K and V of a slot's head, zero where there is no page, and
        which keys have one"""
        pg = self.tab[i, :-(-self.lens[i] // self.ps)]
        ok = (pg >= 0) & (pg < self.pages)
        out = []
        for x, s in zip((self.k, self.v), self.sc):
            y = x.view(torch.uint8)[:, h][pg.clamp_min(0)].view(x.dtype) if self.kv == "e4m3" \
                else x[:, h][pg.clamp_min(0)]
            y = y.double() * (1.0 if s is None else s[h].double())
            y = torch.where(ok[:, None, None], y, torch.zeros((), dtype=y.dtype, device="cuda"))
            out.append(y.reshape(-1, y.shape[-1])[:self.lens[i]])
        return out[0], out[1], ok.repeat_interleave(self.ps)[:self.lens[i]]


def _against(sh, n, m, q, out, lse, hkv, window, first, scale, dt):
    g = q.shape[1] // hkv
    worst = 0.0
    for i in range(n):
        L = sh.lens[i]
        p = torch.arange(L - m, L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")
        see = j <= p
        if window:
            see &= (p - j < window) | (j < first)
        for h in range(hkv):
            k, v, ok = sh.head(i, h)
            at = slice(i * m, i * m + m), slice(h * g, h * g + g)
            w = _truth(q[at].double(), k, v, see & ok, scale, dt)
            eo = ((out[at].double() - w[0]).abs() / w[2]).max()
            el = ((lse[at].double() - w[1]).abs() / w[3]).max()
            both = torch.stack([eo, el]).cpu()
            assert bool((both <= 1).all()), (i, h, both.tolist())     # NaN fails
            worst = max(worst, float(both.max()))
    print("  worst error / bar: %.3f" % worst, flush=True)


@pytest.mark.parametrize("name", list(LONG))
def test_decode_over_many_units(name):
    dt, kv, D, hkv, g, n, lo, hi, window, first = LONG[name]
    print(f"[case] decode long {name}", flush=True)
    rng = np.random.default_rng(len(name) + D)
    lens = [int(x) for x in rng.integers(lo, hi, n)]
    lens[n // 2], lens[-1] = hi, 33
    drop = [(n // 2, -(-hi // 32) - 3), (n // 2, -(-hi // 32) - 90), (1, 5)]
    sh = _Shared(n, kv, D, hkv, lens, 32, 1000, window, first,
                 drop=drop if window == 0 else drop[:1])
    q = torch.from_numpy(_q(rng, n, hkv * g, D, dt)).to("cuda", DT[dt])
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((M.moe_attn_decode_workspace_size(sh.cache, n, hkv * g),), 255,
                    dtype=torch.uint8, device="cuda")
    M.moe_attn_decode(sh.cache, sh.table, q, out, D ** -0.5, err, ws, window=window,
                      n_first=first, lse=lse)
    assert M.moe_read_device_error(err) == M.MOE_DEVERR_CACHE_PAGE     # of the dropped ones
    _against(sh, n, 1, q, out, lse, hkv, window, first, D ** -0.5, dt)


@pytest.mark.parametrize("dt,kv,D,hkv,g,window,first", [
    ("bf16", "bf16", 128, 4, 8, 0, 0), ("f16", "f16", 64, 4, 8, 0, 0),
    ("bf16", "e4m3", 128, 8, 4, 5001, 100), ("bf16", "bf16", 256, 8, 4, 0, 0),
    ("f16", "e4m3", 64, 4, 8, 0, 0)])
def test_prefill_over_many_tiles(dt, kv, D, hkv, g, window, first):
    """Enough rows that no tile's keys are split, over more than 64 tiles of
    keys, with a page missing beyond them."""
    n, m = 2, 801
    print(f"[case] prefill long {dt} {kv} {D}", flush=True)
    rng = np.random.default_rng(D + g)
    lens = [5203, 9009]
    drop = [(0, 5203 // 32 - 40), (1, 9009 // 32 - 30), (1, 9009 // 32 - 31)]
    sh = _Shared(3, kv, D, hkv, lens, 32, 400, window, first, rows=m, drop=drop)
    q = torch.from_numpy(_q(rng, n * m, hkv * g, D, dt)).to("cuda", DT[dt])
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert M.moe_attn_prefill_workspace_size(sh.cache, n, n * m, hkv * g) == 0
    M.moe_attn_prefill(sh.cache, sh.table, q, _i([0, m, 2 * m]), out, D ** -0.5, err, None,
                       window=window, n_first=first, lse=lse)
    assert M.moe_read_device_error(err) == M.MOE_DEVERR_CACHE_PAGE
    _against(sh, n, m, q, out, lse, hkv, window, first, D ** -0.5, dt)
