"""Turns of a server with drafted trees, calls of the cache objects as they are
used together: prompts, then trees appended, attended and kept, single tokens
between them, a captured turn, upkeep. Every attention call within its bound of
64 bits from the rows as they were handed to the cache."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import mixture_experts_expert_sigmoid_amd as M
from tests.test_gpu_cache import _i

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]
F8 = torch.float8_e4m3fn


def sees(C, m, parents, window, first):
    """[m][C + m] booleans of a slot's newest rows: an order (parents None) or a
    tree."""
    see = np.zeros((m, C + m), bool)
    depth = []
    for t in range(m):
        a = t - 1 if parents is None else parents[t]
        depth.append(depth[a] + 1 if a >= 0 else 0)
        at = np.concatenate([np.arange(C), C + np.array(depth)])      # positions of keys
        on = np.zeros(C + m, bool)
        on[:C] = True
        while a >= 0:
            on[C + a] = True
            a = a - 1 if parents is None else parents[a]
        on[C + t] = True
        near = (C + depth[t] - at[:on.size] < window) | (at[:on.size] < first) if window else True
        see[t, :at.size] = on[:at.size] & near
    return torch.from_numpy(see).cuda()


def bound_check(q, k, v, see, scale, out, dt, where):
    """One head: rows q over keys k and values v (64 bits). P and the result are
    rounded to the row's type, half a step each; with eps the type's spacing that is
    eps / 2 + eps / 2 of the largest visible |v|, and a twentieth more for fp32
    sums and exponentials."""
    x = (q.double() @ k.double().t()) * scale
    p = torch.softmax(x.masked_fill(~see, -torch.inf), -1)
    want = p @ v.double()
    most = (v.double().abs().amax(1)[None] * see).amax()
    err = float((out.double() - want).abs().max() / most)
    assert err <= 1.05 * torch.finfo(dt).eps, (where, err)


class Keys:
    """k and v of [layer][slot] as handed to the cache; what an e4m3 cache keeps."""

    def __init__(self, scale=None):
        self.rows, self.scale = {}, scale

    def kept(self, x):
        if self.scale is None:
            return x.double()
        # the nearest codes: 448 at most
        return ((x.double() / self.scale).clamp(-448, 448).float().to(F8).double() * self.scale)

    def add(self, slots, cu, xs):
        for i, s in enumerate(slots):
            new = [self.kept(x[cu[i]:cu[i + 1]]) for x in xs]
            old = self.rows.get(s)
            self.rows[s] = new if old is None else [torch.cat(p) for p in zip(old, new)]

    def keep(self, slots, rows, paths):
        for s, m, path in zip(slots, rows, paths):
            self.rows[s] = [torch.cat([x[:len(x) - m], x[[len(x) - m + a for a in path]]])
                            for x in self.rows[s]]


def trees(rng, n):
    out = []
    for i in range(n):
        m = int(rng.choice([1, 2, 7, 13, 30, 64]))
        out.append([int(rng.integers(-1, t)) if t else -1 for t in range(m)])
    return out


def path_in(rng, parents):
    """A way down from a child of the context, or none."""
    path, at = [], -1
    while True:
        below = [t for t, a in enumerate(parents) if a == at]
        if not below or rng.random() < 0.15:
            return path
        at = below[int(rng.integers(len(below)))]
        path.append(at)


def cu_of(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(int).tolist()


@pytest.mark.parametrize("dt,kv,D,hq,hkv,ps,window,first", [
    (torch.bfloat16, torch.bfloat16, 128, 8, 2, 16, 0, 0),
    (torch.float16, torch.float16, 64, 6, 6, 48, 70, 5),
    (torch.bfloat16, F8, 256, 8, 1, 32, 40, 0)])
def test_turns_of_keys_and_values(dt, kv, D, hq, hkv, ps, window, first):
    rng = np.random.default_rng(D + ps)
    gen = torch.Generator(device="cuda").manual_seed(ps)
    S, layers, scale = 5, 2, D ** -0.5
    sc = torch.full((layers, hkv), 1 / 64, device="cuda") if kv == F8 else None
    c = M.KvCache(n_layers=layers, n_pages=200, page_size=ps, n_heads=hkv, head_dim=D, n_slots=S,
                  max_pages=40, dtype=kv, k_scale=sc, v_scale=sc)
    host = [Keys(1 / 64 if kv == F8 else None) for _ in range(layers)]
    slots = [3, 0, 4, 1]

    def turn(rows, parents=None, where=""):
        cu = cu_of(rows)
        start = c.grow(_i(slots), _i(rows))
        for l in range(layers):
            q, k, v = (torch.randn(cu[-1], h, D, generator=gen, device="cuda").to(dt)
                       for h in (hq, hkv, hkv))
            c.append(l, _i(slots), start, _i(cu), k, v)
            host[l].add(slots, cu, (k, v))
            kw = dict(window=window, n_first=first)
            if parents:
                out = c.tree(l, _i(slots), q, _i(cu), _i(sum(parents, [])), scale, **kw)
            elif max(rows) == 1:
                out = c.decode(l, _i(slots), q, scale, **kw)
            else:
                out = c.prefill(l, _i(slots), q, _i(cu), scale, **kw)
            for i, s in enumerate(slots):
                ks, vs = host[l].rows[s]
                see = sees(len(ks) - rows[i], rows[i], parents[i] if parents else None, window,
                           first)
                for h in range(hq):
                    bound_check(q[cu[i]:cu[i + 1], h], ks[:, h * hkv // hq].contiguous(),
                                vs[:, h * hkv // hq].contiguous(), see, scale,
                                out[cu[i]:cu[i + 1], h], dt, (where, l, s, h))

    turn([33, 1, 90, 17], where="prompts")
    for t in range(5):
        tr = trees(rng, len(slots))
        paths = [path_in(rng, p) for p in tr]
        rows = [len(p) for p in tr]
        turn(rows, tr, f"tree {t}")
        c.keep(_i(slots), _i(rows), _i(cu_of([len(p) for p in paths])), _i(sum(paths, []) + [0]))
        for h in host:
            h.keep(slots, rows, paths)
        turn([1] * 4, where=f"one {t}")
        if t == 2:
            c.compact()
        assert c.lens[slots].tolist() == [len(host[0].rows[s][0]) for s in slots]
    assert M.moe_read_device_error(c.err_word) == 0
    c.free(_i(slots))
    assert int(c.refs.abs().sum()) == 0


@pytest.mark.parametrize("dt,kv,dc,H,ps,window,first", [
    (torch.bfloat16, torch.bfloat16, 512, 16, 16, 0, 0),
    (torch.float16, torch.float16, 256, 5, 48, 70, 5),
    (torch.bfloat16, F8, 512, 8, 64, 40, 0)])
def test_turns_of_latent_vectors(dt, kv, dc, H, ps, window, first):
    rng = np.random.default_rng(dc + ps)
    gen = torch.Generator(device="cuda").manual_seed(ps)
    S, layers, scale = 5, 2, 192 ** -0.5
    sc = torch.full((layers,), 1 / 64, device="cuda") if kv == F8 else None
    c = M.LatentCache(n_layers=layers, n_pages=200, page_size=ps, latent_dim=dc, n_slots=S,
                      max_pages=40, dtype=kv, scale=sc)
    host = [Keys(1 / 64 if kv == F8 else None) for _ in range(layers)]
    slots = [3, 0, 4, 1]
    side = torch.cuda.Stream()

    def turn(rows, parents=None, where="", one=False):
        cu = cu_of(rows)
        start = c.grow(_i(slots), _i(rows))
        for l in range(layers):
            q = torch.randn(cu[-1], H, dc + 64, generator=gen, device="cuda").to(dt)
            x = torch.randn(cu[-1], dc + 64, generator=gen, device="cuda").to(dt)
            cud, par = _i(cu), _i(sum(parents, [])) if parents else None
            # on a stream of its own, as a server with several would
            side.wait_stream(torch.cuda.current_stream())
            c.append(l, _i(slots), start, cud, x[:, :dc], x[:, dc:], stream=side)
            out = c.attend(l, _i(slots), q, None if one else cud, scale, parent=par,
                           window=window, n_first=first, stream=side)
            torch.cuda.current_stream().wait_stream(side)
            host[l].add(slots, cu, (x,))
            for i, s in enumerate(slots):
                ks, = host[l].rows[s]
                see = sees(len(ks) - rows[i], rows[i], parents[i] if parents else None, window,
                           first)
                for h in range(H):
                    bound_check(q[cu[i]:cu[i + 1], h], ks, ks[:, :dc].contiguous(), see, scale,
                                out[cu[i]:cu[i + 1], h], dt, (where, l, s, h))

    turn([33, 1, 90, 17], where="prompts")
    for t in range(5):
        tr = trees(rng, len(slots))
        paths = [path_in(rng, p) for p in tr]
        rows = [len(p) for p in tr]
        turn(rows, tr, f"tree {t}")
        c.keep(_i(slots), _i(rows), _i(cu_of([len(p) for p in paths])), _i(sum(paths, []) + [0]))
        for h in host:
            h.keep(slots, rows, paths)
        turn([1] * 4, where=f"one {t}", one=True)
        if t == 1:                               # slot 2 continues the third sequence
            c.fork(_i([4]), _i([2]))
            for h in host:
                h.rows[2] = list(h.rows[4])
            slots[1] = 2
        if t == 2:
            c.compact()
        assert c.lens[slots].tolist() == [len(host[0].rows[s][0]) for s in slots]
    assert M.moe_read_device_error(c.err_word) == 0
    c.free(_i([0, 1, 2, 3, 4]))
    assert int(c.refs.abs().sum()) == 0


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_expanded_and_absorbed_agree(dt):
    """A prompt's attention over rows expanded from the latent vectors, and the same
    rows through the cache with queries that took up Wk; the values' product with
    Wv comes after. Exact products in 64 bits stand between them."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    H, dc, D, rows, ctx, scale = 4, 512, 128, [37, 1, 70], [0, 65, 30], 192 ** -0.5
    eps = torch.finfo(dt).eps

    def rand(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dt)

    wk, wv = rand(H, D, dc, std=dc ** -0.5), rand(H, D, dc, std=dc ** -0.5)
    cu, cu_k = cu_of(rows), cu_of([a + b for a, b in zip(rows, ctx)])
    c, r = rand(cu_k[-1], dc), rand(cu_k[-1], 64)
    qn, qr = rand(cu[-1], H, D), rand(cu[-1], H, 64)
    cache = M.LatentCache(n_layers=1, n_pages=40, page_size=16, n_slots=3, max_pages=12, dtype=dt)
    sl = _i([0, 1, 2])
    start = cache.grow(sl, _i([a + b for a, b in zip(rows, ctx)]))
    cache.append(0, sl, start, _i(cu_k), c, r)
    up = torch.stack([c.double() @ wk[h].double().t() for h in range(H)], 1)
    k = up.to(dt)
    v = torch.stack([c.double() @ wv[h].double().t() for h in range(H)], 1).to(dt)
    qc = torch.stack([qn[:, h].double() @ wk[h].double() for h in range(H)], 1).to(dt)
    wide = cache.prompt(torch.cat([qn, qr], -1), k, r, v, _i(cu), _i(cu_k), scale)
    thin = cache.attend(0, sl, torch.cat([qc, qr], -1), _i(cu), scale)
    thin = torch.stack([thin[:, h].double() @ wv[h].double().t() for h in range(H)], 1)
    for i in range(3):
        at = slice(cu_k[i], cu_k[i + 1])
        see = sees(ctx[i], rows[i], None, 0, 0)
        for h in range(H):
            q = qn[cu[i]:cu[i + 1], h].double()
            x = (q @ up[at, h].t() + qr[cu[i]:cu[i + 1], h].double() @ r[at].double().t()) * scale
            p = torch.softmax(x.masked_fill(~see, -torch.inf), -1)
            cv = c[at].double() @ wv[h].double().t()
            want = p @ cv
            # Rounding k (or q') by half a step moves a score by up to eps / 2 of the
            # sum of the products' magnitudes, and a weighted mean by twice the
            # largest move of a score times the largest value; then P, the values and
            # the result, half a step each.
            mag = (q.abs() @ up[at, h].abs().t()) * scale
            magc = (qc[cu[i]:cu[i + 1], h].double().abs() @ c[at].double().abs().t()) * scale
            most = cv.abs().max()
            err = (wide[cu[i]:cu[i + 1], h].double() - want).abs().max()
            assert err <= 1.05 * eps * most * (mag.max() + 1.5), (i, h, "expanded")
            # here the sum's rounding comes before Wv: |Wv| |c| for each value
            wide_c = (wv[h].double().abs().sum(1) * c[at].double().abs().max()).max()
            err = (thin[cu[i]:cu[i + 1], h] - want).abs().max()
            assert err <= 1.05 * eps * (most * magc.max() + wide_c), (i, h, "absorbed")
    assert M.moe_read_device_error(cache.err_word) == 0


def test_captured_turns():
    """A turn of a tree in a graph: append, attention and keep of both caches,
    replayed with other drafts, other paths and eager work between; every replay is
    the eager turn, bit for bit, pages and all."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    rng = np.random.default_rng(9)
    n, m, most = 3, 12, 12

    def caches():
        a = M.KvCache(n_layers=1, n_pages=60, page_size=16, n_heads=2, head_dim=64, n_slots=n,
                      max_pages=16)
        b = M.LatentCache(n_layers=1, n_pages=60, page_size=16, n_slots=n, max_pages=16)
        for x in (a.k, a.v, b.c):
            x.zero_()
        return a, b

    sl, cu = _i(range(n)), _i(cu_of([m] * n))
    inp = dict(q=(n * m, 4, 64), k=(n * m, 2, 64), v=(n * m, 2, 64), ql=(n * m, 16, 576),
               c=(n * m, 512), r=(n * m, 64))
    inp = {k: torch.zeros(s, dtype=torch.bfloat16, device="cuda") for k, s in inp.items()}
    new, parent = _i([m] * n), _i([-1] * (n * m))
    cu_path, path = _i([0] * (n + 1)), _i([0] * (n * most))

    def turn(a, b):
        out = []
        for c in (a, b):
            start = c.grow(sl, new)
            if c is a:
                c.append(0, sl, start, cu, inp["k"], inp["v"])
                out.append(c.tree(0, sl, inp["q"], cu, parent, 0.125))
            else:
                c.append(0, sl, start, cu, inp["c"], inp["r"])
                out.append(c.attend(0, sl, inp["ql"], cu, 0.07, parent=parent))
            c.keep(sl, new, cu_path, path)
        return out

    def draw():
        for x in inp.values():
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        tr = [[int(rng.integers(-1, t)) if t else -1 for t in range(m)] for _ in range(n)]
        paths = [path_in(rng, p) for p in tr]
        parent.copy_(_i(sum(tr, [])))
        cu_path.copy_(_i(cu_of([len(p) for p in paths])))
        flat = sum(paths, [])
        path.copy_(_i(flat + [0] * (n * most - len(flat))))

    eager, graphed = caches(), caches()
    draw()
    turn(*eager)
    turn(*graphed)                                # workspaces are there before the capture
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = turn(*graphed)
    for rep in range(4):
        draw()
        want = turn(*eager)
        g.replay()
        torch.cuda.synchronize()
        for w, x in zip(want, got):
            assert torch.equal(w, x), rep
        for e, x in zip(eager, graphed):
            for name in ("table", "lens", "refs", "err_word"):
                assert torch.equal(getattr(e, name), getattr(x, name)), (rep, name)
        assert torch.equal(eager[0].k, graphed[0].k) and torch.equal(eager[0].v, graphed[0].v)
        assert torch.equal(eager[1].c, graphed[1].c)
        assert M.moe_read_device_error(eager[0].err_word) == 0


def test_two_streams():
    """Calls in flight on two streams at once, each with a workspace of its own, and
    two graphs that share one, replayed in turn: the results of calls by themselves."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    n, m, L = 3, 9, 2000
    a = M.KvCache(n_layers=1, n_pages=400, page_size=16, n_heads=2, head_dim=128, n_slots=n,
                  max_pages=130)
    b = M.LatentCache(n_layers=1, n_pages=400, page_size=16, n_slots=n, max_pages=130)
    for x in (a.k, a.v, b.c):
        x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
    sl, cu, parent = _i(range(n)), _i(cu_of([m] * n)), _i([-1, 0, 0, 1, 2, 2, 4, 5, 5] * n)
    for c in (a, b):
        c.grow(sl, _i([L] * n))
    q = torch.randn(n * m, 8, 128, generator=gen, device="cuda").bfloat16()
    ql = torch.randn(n * m, 16, 576, generator=gen, device="cuda").bfloat16()
    ws = [torch.empty(1 << 27, dtype=torch.uint8, device="cuda") for _ in range(4)]
    outs = [torch.empty_like(q) for _ in range(2)] + [
        torch.empty(n * m, 16, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def call(i, w):
        if i < 2:
            M.moe_attn_tree(a.layers[0], a.desc, q, cu, parent, outs[i], 0.09, a.err_word, w)
        else:
            M.moe_attn_latent(b.layers[0], b.desc, ql, cu, outs[i], 0.07, b.err_word, w,
                              parent=parent)

    for i in range(4):
        call(i, ws[i])
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                call(i, ws[i])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want))
    graphs = []
    for i in (0, 2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i, ws[0])
        graphs.append(g)
    for _ in range(3):
        outs[0].zero_()
        outs[2].zero_()
        ws[0].fill_(0xFF)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[2], want[2])
    assert M.moe_read_device_error(a.err_word) == 0 and M.moe_read_device_error(b.err_word) == 0


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_example(kv):
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "paged_decoder.py")
    spec = importlib.util.spec_from_file_location("paged_decoder", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    dec, text, _ = ex.session(kv, check=True, steps=8)
    have = [len(text[s]) for s in (1, 2, 4)]
    kept = ex.drafted(dec, text, [1, 2, 4], 6)
    assert kept >= 18 and sum(len(text[s]) for s in (1, 2, 4)) == sum(have) + kept
    assert 0.0 < dec.dense.worst <= 1.0
