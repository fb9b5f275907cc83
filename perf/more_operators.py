"""Cases of two further kinds of attention over paged caches, and of what they
need beside them: drafted tokens that form a tree, and keys and values that
are one shared latent vector a token.

A case names one operator (`op`):
  tree     attention of a tree of drafted tokens over a key-value cache
  keep     the accepted path of each tree moved to the front of the drafted
           tokens, in every layer, and the pages past it given back
  write    new latent vectors and rotary keys written into a latent cache
  latent   absorbed attention over a latent cache: single tokens, the newest
           tokens of a sequence, trees of drafted ones
  prompt   expanded attention of prompts: keys and values of each head in
           dense rows, the rotary part of the keys shared by the heads

Lengths and trees follow a fixed pattern of the case (`_lens`, `_parents`),
so a case's work does not depend on the seed; values, page order and queries
do.
"""
import math
import random

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
_SIZE = {"bf16": 2, "f16": 2, "e4m3": 1}
ROPE = 64                    # rotary values of a latent cache's keys
NOPE = 128                   # other values of an expanded head's keys, and its values


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one user's eight drafted tokens: the smallest call, latency
        dict(name="tree_one", op="tree", dt="bf16", kv="bf16", n=1, hq=32, hkv=8, d=128, ps=16,
             lo=777, hi=777, mlo=8, mhi=8, window=0, first=0),
        # a server's batch, ragged contexts and trees
        dict(name="tree_batch", op="tree", dt="bf16", kv="bf16", n=48, hq=32, hkv=8, d=128, ps=64,
             lo=201, hi=4001, mlo=9, mhi=33, window=0, first=0),
        # large trees over two long contexts in an 8-bit cache
        dict(name="tree_long", op="tree", dt="bf16", kv="e4m3", n=2, hq=64, hkv=8, d=128, ps=64,
             lo=50003, hi=60001, mlo=41, mhi=61, window=0, first=0),
        # the end of a drafted step of a small batch, few layers: latency
        dict(name="keep_step", op="keep", kv="bf16", n=16, hkv=8, d=128, ps=16, layers=4,
             lo=100, hi=400, mlo=12, mhi=16, most=5),
        # the same of a large batch and large trees
        dict(name="keep_many", op="keep", kv="bf16", n=256, hkv=8, d=128, ps=16, layers=8,
             lo=17, hi=90, mlo=40, mhi=64, most=12),
        # one token of each sequence of a batch
        dict(name="write_step", op="write", dt="bf16", kv="bf16", n=64, dc=512, ps=64,
             lo=200, hi=4000, mlo=1, mhi=1),
        # prompts into an 8-bit cache
        dict(name="write_prompts", op="write", dt="bf16", kv="e4m3", n=8, dc=512, ps=64,
             lo=0, hi=900, mlo=500, mhi=8001),
        # one user, the heads of one of several GPUs: latency
        dict(name="latent_one", op="latent", dt="bf16", kv="bf16", n=1, hq=16, dc=512, ps=16,
             lo=776, hi=776, mlo=1, mhi=1, tree=False, window=0, first=0),
        # a server's batch of single tokens, all heads on this GPU
        dict(name="latent_batch", op="latent", dt="bf16", kv="bf16", n=64, hq=128, dc=512, ps=64,
             lo=200, hi=4000, mlo=1, mhi=1, tree=False, window=0, first=0),
        # drafted trees over long contexts in an 8-bit cache
        dict(name="latent_tree", op="latent", dt="bf16", kv="e4m3", n=3, hq=64, dc=512, ps=64,
             lo=20003, hi=40001, mlo=5, mhi=13, tree=True, window=0, first=0),
        # a few short prompts: latency
        dict(name="prompt_short", op="prompt", dt="bf16", n=3, hq=16, lo=0, hi=0, mlo=17, mhi=130,
             window=0, first=0),
        # a long prompt: the largest
        dict(name="prompt_long", op="prompt", dt="bf16", n=1, hq=32, lo=0, hi=0, mlo=6001,
             mhi=6001, window=0, first=0),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "keep", "write", "latent", "latent", "latent", "prompt",
                     "prompt"])
    dt = rng.choice(["bf16", "f16"])
    kv = rng.choice([dt, dt, "e4m3"])
    ps = rng.choice([16, 32, 64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128, 128, 256])
    window = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
    first = rng.choice([0, 4, 17]) if window else 0
    if op == "tree":
        g = rng.choice([1, 2, 4, 5, 8, 16])
        n, mhi = _log(rng, 1, 96), _log(rng, 1, 128)
        hi = _log(rng, 16, 60000)
        # query and key pairs in all, padded, and the cache's size
        while n * hkv * g * mhi * hi * d > 60_000_000_000 or n * hkv * hi * d > 110_000_000:
            if n > 1:
                n //= 2
            elif hi > 3000:
                hi //= 2
            else:
                mhi = (mhi + 1) // 2
        return dict(op=op, dt=dt, kv=kv, n=n, hq=hkv * g, hkv=hkv, d=d, ps=ps,
                    lo=rng.randint(0, hi), hi=hi, mlo=rng.randint(1, mhi), mhi=mhi,
                    window=window, first=first)
    if op == "keep":
        n, mhi = _log(rng, 1, 256), _log(rng, 4, 64)
        hi = _log(rng, 4, 400)
        layers = rng.randint(1, 8)
        while n * (hi + mhi + ps) * hkv * d * layers > 300_000_000:
            if layers > 1:
                layers -= 1
            else:
                n = (n + 1) // 2
        return dict(op=op, kv=rng.choice(["bf16", "f16"]), n=n, hkv=hkv, d=d, ps=ps,
                    layers=layers, lo=rng.randint(0, hi), hi=hi, mlo=rng.randint(4, mhi),
                    mhi=mhi, most=rng.randint(0, 12))
    dc = rng.choice([256, 512, 512])
    if op == "write":
        n = _log(rng, 1, 256)
        mhi = _log(rng, 1, max(2, min(8192, 30000 // n)))
        hi = rng.randint(0, 2000)
        return dict(op=op, dt=dt, kv=kv, n=n, dc=dc, ps=ps, lo=rng.randint(0, hi), hi=hi,
                    mlo=rng.randint(1, mhi), mhi=mhi)
    if op == "latent":
        hq = rng.choice([1, 4, 5, 8, 16, 32, 64, 128])
        mhi = rng.choice([1, 1, 1, _log(rng, 2, 64)])
        n, hi = _log(rng, 1, 192), _log(rng, 16, 60000)
        while n * hq * mhi * hi > 60_000_000 or n * hi > 500_000:
            if n > 1:
                n //= 2
            elif hi > 3000:
                hi //= 2
            else:
                mhi = (mhi + 1) // 2
        return dict(op=op, dt=dt, kv=kv, n=n, hq=hq, dc=dc, ps=ps, lo=rng.randint(0, hi), hi=hi,
                    mlo=rng.randint(1, mhi), mhi=mhi, tree=rng.random() < 0.5, window=window,
                    first=first)
    hq = rng.choice([1, 3, 8, 16, 32])
    n, mhi = _log(rng, 1, 16), _log(rng, 1, 6000)
    hi = rng.choice([0, 0, _log(rng, 1, 8000)])
    while n * hq * mhi * (mhi + hi) > 1_000_000_000:
        if n > 1:
            n //= 2
        else:
            mhi, hi = (mhi + 1) // 2, hi // 2
    return dict(op=op, dt=dt, n=n, hq=hq, lo=rng.randint(0, hi), hi=hi,
                mlo=rng.randint(1, mhi), mhi=mhi, window=window, first=first)


# ------------------------------------------------------------ case geometry

def _lens(n, lo, hi):
    """n lengths in lo..hi, the last hi, spread evenly and out of order."""
    f = (np.arange(1, n + 1) * 0.6180339887498949) % 1.0
    v = (lo + np.floor(f * (hi - lo + 1))).astype(np.int64)
    v[-1] = hi
    return v


def _parents(m, i):
    """The tree of m drafted tokens of sequence i: some children of the
    context, the others of earlier tokens, chains and bushes mixed."""
    t = np.arange(m)
    f = (t * 0.6180339887498949 + i * 0.7548776662466927) % 1.0
    p = np.floor(t * (0.45 + 0.6 * f)).astype(np.int64) - 1
    return np.clip(p, -1, t - 1)


def _ancestors(p):
    """[m, m] truth values: token t's row has itself and its ancestors."""
    m = len(p)
    a = np.eye(m, dtype=bool)
    for t in range(m):
        if p[t] >= 0:
            a[t] |= a[p[t]]
    return a


def _geometry(c):
    """(tokens before, new tokens of each sequence)"""
    return _lens(c["n"], c["lo"], c["hi"]), _lens(c["n"], c["mlo"], c["mhi"])


def _ceil(a, b):
    return -(-a // b)


def _is_tree(c):
    return c["op"] == "tree" or c.get("tree", False)


def _sees(c, i, C, m):
    """[m, C + m] truth values: which keys the new tokens of sequence i see."""
    anc = _ancestors(_parents(m, i)) if _is_tree(c) else np.tril(np.ones((m, m), bool))
    depth = anc.sum(1) - 1
    see = np.concatenate([np.ones((m, C), bool), anc], 1)
    if c["window"]:
        pos_k = np.concatenate([np.arange(C), C + depth])
        see &= ((C + depth)[:, None] - pos_k < c["window"]) | (pos_k < c["first"])
    return see


def _visible(c):
    """Visible (query, key) pairs, and the keys that any query sees."""
    pairs = keys = 0
    for i, (C, m) in enumerate(zip(*(x.tolist() for x in _geometry(c)))):
        if c["window"] or _is_tree(c):
            see = _sees(c, i, C, m)
            pairs += int(see.sum())
            keys += int(see.any(0).sum())
        else:
            pairs += m * C + m * (m + 1) // 2
            keys += C + m
    return pairs, keys


def work(c):
    C, m = _geometry(c)
    t = int(m.sum())
    op = c["op"]
    if op == "tree":
        pairs, keys = _visible(c)
        return {"bytes": keys * 2 * c["hkv"] * c["d"] * _SIZE[c["kv"]] +
                t * c["hq"] * (2 * c["d"] * 2 + 4), "flops": 4 * pairs * c["hq"] * c["d"]}
    if op == "latent":
        pairs, keys = _visible(c)
        return {"bytes": keys * (c["dc"] + ROPE) * _SIZE[c["kv"]] +
                t * c["hq"] * ((2 * c["dc"] + ROPE) * 2 + 4),
                "flops": 2 * pairs * c["hq"] * (2 * c["dc"] + ROPE)}
    if op == "prompt":
        pairs, keys = _visible(c)
        return {"bytes": keys * (c["hq"] * 2 * NOPE + ROPE) * 2 +
                t * c["hq"] * ((2 * NOPE + ROPE) * 2 + 4),
                "flops": 2 * pairs * c["hq"] * (2 * NOPE + ROPE)}
    if op == "write":
        return {"bytes": t * (c["dc"] + ROPE) * (2 + _SIZE[c["kv"]]), "flops": 0}
    moved = sum(sum(1 for j, a in enumerate(p) if a != j) for p in _paths(c))
    return {"bytes": moved * c["layers"] * 4 * c["hkv"] * c["d"] * _SIZE[c["kv"]] +
            4 * (3 * c["n"] + sum(len(p) for p in _paths(c))), "flops": 0}


def _paths(c):
    """The accepted tokens of each sequence, ascending: none to `most`. What
    is moved is never moved onto another one's place, so that a pass does its
    whole work on a state that a pass before it has run on."""
    out = []
    for i, m in enumerate(_geometry(c)[1].tolist()):
        k = min((i * 5 + 3) % (c["most"] + 1), m // 2)
        if i % 2 and k:
            p = [0] + np.linspace(k, m - 1, k - 1).astype(int).tolist()
        else:
            p = np.linspace(k, m - 1, k).astype(int).tolist()
        out.append(p)
    return out


# -------------------------------------------------------------- page layouts

def _layout(seed, lens, ps, spare):
    """Tables of shuffled pages for these lengths: (table, pages)."""
    r = np.random.RandomState(seed % (1 << 31))
    need = _ceil(lens, ps)
    total = int(need.sum())
    order = r.permutation(total + spare)
    table = np.full((len(lens), max(int(need.max()), 1)), -1, np.int32)
    at = 0
    for i, k in enumerate(need.tolist()):
        table[i, :k] = order[at:at + k]
        at += k
    return table, total + spare


# ------------------------------------------------------------------ prepare

def _randn(gen, shape, dt, scale=1.0):
    if dt == "e4m3":
        # values / scale, in slices: the 32-bit draw of a long cache is large
        out = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
        flat = out.view(-1)
        step = 1 << 26
        for a in range(0, flat.numel(), step):
            m = min(step, flat.numel() - a)
            flat[a:a + m] = (torch.randn(m, generator=gen, device="cuda") / scale).to(
                torch.float8_e4m3fn)
        return out
    return torch.randn(shape, generator=gen, device="cuda", dtype=_DT[dt])


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to("cuda")  # noqa: E731
    i32 = lambda a: dev(np.asarray(a, np.int32))  # noqa: E731
    s, op = dict(c), c["op"]
    C, m = _geometry(c)
    cu = np.concatenate([[0], np.cumsum(m)])
    t = int(cu[-1])
    s["cu"], s["max_m"], s["max_len"] = i32(cu), int(m.max()), int((C + m).max())
    s["before"] = i32(C)
    if op == "prompt":
        cuk = np.concatenate([[0], np.cumsum(C + m)])
        s["cu_k"] = i32(cuk)
        # the rows as a layer's products leave them: a head's keys and values
        # in one row, the shared rotary part behind the latent vector
        kv = _randn(gen, (int(cuk[-1]), c["hq"], 2 * NOPE), c["dt"])
        s["k"], s["v"] = kv[..., :NOPE], kv[..., NOPE:]
        s["k_rope"] = _randn(gen, (int(cuk[-1]), ROPE), c["dt"])
        s["q"] = 1.5 * _randn(gen, (t, c["hq"], NOPE + ROPE), c["dt"])
        s["out"] = torch.empty(t, c["hq"], NOPE, dtype=_DT[c["dt"]], device="cuda")
        s["lse"] = torch.empty(t, c["hq"], device="cuda")
        s["scale"] = (NOPE + ROPE) ** -0.5
    else:
        table, pages = _layout(seed, C + m, c["ps"], 5)
        if c.get("window", 0):
            # pages that no query of this call sees have been given back
            pg = np.arange(table.shape[1])[None, :] * c["ps"]
            gone = (pg >= c["first"]) & (pg + c["ps"] - 1 < (C - c["window"])[:, None])
            table[gone] = -1
        s["table"], s["lens"] = dev(table), i32(C + m)
        s["pages"] = pages
    if op in ("tree", "latent"):
        d = c["d"] if op == "tree" else c["dc"] + ROPE
        dv = c["d"] if op == "tree" else c["dc"]
        s["q"] = 1.5 * _randn(gen, (t, c["hq"], d), c["dt"])
        s["out"] = torch.empty(t, c["hq"], dv, dtype=_DT[c["dt"]], device="cuda")
        s["lse"] = torch.empty(t, c["hq"], device="cuda")
        s["scale"] = d ** -0.5
        s["parent"] = None
        if _is_tree(c):
            s["parent"] = i32(np.concatenate([_parents(k, i) for i, k in enumerate(m.tolist())]))
        s["max_depth"] = max(int(_ancestors(_parents(k, i)).sum(1).max())
                             for i, k in enumerate(m.tolist())) if _is_tree(c) else s["max_m"]
    if op == "tree":
        shape, sc = (pages, c["hkv"], c["ps"], c["d"]), 0.02
        s["k"], s["v"] = _randn(gen, shape, c["kv"], sc), _randn(gen, shape, c["kv"], sc)
        s["ks"] = s["vs"] = None
        if c["kv"] == "e4m3":
            s["ks"] = sc * (0.5 + torch.rand(c["hkv"], generator=gen, device="cuda"))
            s["vs"] = sc * (0.5 + torch.rand(c["hkv"], generator=gen, device="cuda"))
    if op in ("latent", "write"):
        sc = 0.02
        s["c"] = _randn(gen, (pages, c["ps"], c["dc"] + ROPE), c["kv"], sc)
        s["cs"] = None
        if c["kv"] == "e4m3":
            s["cs"] = sc * (0.5 + torch.rand(1, generator=gen, device="cuda"))
    if op == "write":
        # the two parts of one product's rows
        new = _randn(gen, (t, c["dc"] + ROPE), c["dt"])
        s["c_new"], s["rope_new"] = new[:, :c["dc"]], new[:, c["dc"]:]
    if op == "keep":
        paths = _paths(c)
        s["path"] = i32([a for p in paths for a in p] + [0])
        s["cu_path"] = i32(np.concatenate([[0], np.cumsum([len(p) for p in paths])]))
        s["n_path"], s["n_draft"] = sum(len(p) for p in paths), i32(m)
        refs = np.zeros(pages, np.int32)
        refs[table[table >= 0]] = 1
        s["refs"] = dev(refs)
        s["table0"], s["refs0"], s["lens0"] = (s[k].clone() for k in ("table", "refs", "lens"))
        shape = (c["layers"], pages, c["hkv"], c["ps"], c["d"])
        s["k"], s["v"] = _randn(gen, shape, c["kv"]), _randn(gen, shape, c["kv"])
    if own:
        _own_handles(s)
    return s


def _own_handles(s):
    """Descriptors and workspaces, as a serving program keeps them."""
    import mixture_experts_expert_sigmoid_amd as M
    op, ws = s["op"], 0
    s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op != "prompt":
        s["tab"] = M.kv_table(s["table"], s["lens"], s["ps"], s["pages"], refs=s.get("refs"))
    if op == "keep":
        s["caches"] = [M.kv_cache(s["k"][i], s["v"][i]) for i in range(s["layers"])]
    if op == "tree":
        s["cache"] = M.kv_cache(s["k"], s["v"], s["ks"], s["vs"])
        ws = M.moe_attn_tree_workspace_size(s["cache"], s["n"], s["q"].shape[0], s["hq"])
    if op in ("latent", "write"):
        s["cache"] = M.latent_cache(s["c"], s["dc"], s["cs"])
    if op == "latent":
        ws = M.moe_attn_latent_workspace_size(s["cache"], s["n"], s["q"].shape[0], s["hq"])
    if op == "prompt":
        ws = M.moe_attn_latent_prompt_workspace_size(s["n"], s["q"].shape[0], s["hq"])
    s["ws"] = torch.empty(max(ws, 1), dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------------- run

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import mixture_experts_expert_sigmoid_amd as M
    op = s["op"]
    if op == "tree":
        M.moe_attn_tree(s["cache"], s["tab"], s["q"], s["cu"], s["parent"], s["out"], s["scale"],
                        s["err"], s["ws"], window=s["window"], n_first=s["first"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "latent":
        M.moe_attn_latent(s["cache"], s["tab"], s["q"], None if s["mhi"] == 1 else s["cu"],
                          s["out"], s["scale"], s["err"], s["ws"], parent=s["parent"],
                          window=s["window"], n_first=s["first"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "prompt":
        M.moe_attn_latent_prompt(s["q"], s["k"], s["k_rope"], s["v"], s["cu"], s["cu_k"],
                                 s["out"], s["scale"], s["ws"], window=s["window"],
                                 n_first=s["first"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "write":
        M.moe_latent_append(s["cache"], s["tab"], s["before"], s["cu"], s["c_new"],
                            s["rope_new"], s["err"])
        return {"c": s["c"]}
    _rewind(s)
    M.moe_cache_keep(s["caches"], s["tab"], s["n_draft"], s["cu_path"], s["path"], s["err"])
    return _pool(s)


def _rewind(s):
    """The tables as prepare made them, so that every pass has the drafted
    tokens before it."""
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    s["lens"].copy_(s["lens0"])


def _pool(s):
    return {k: s[k] for k in ("table", "refs", "lens", "k", "v")}


def _run_plain(s):
    op = s["op"]
    if op in ("tree", "latent", "prompt"):
        return _plain_attention(s)
    if op == "write":
        return _plain_write(s)
    _rewind(s)
    return _plain_keep(s)


def _f32(x, sc):
    y = x.float()
    return y if sc is None else y * sc


def _keys_values(s, pos, ok):
    """Keys and values of positions pos [n, L] in 32 bits, zero where not ok:
    [n, heads, L, d] each, and where there are any."""
    zero = torch.zeros((), device=pos.device)
    if s["op"] == "prompt":
        at = (s["cu_k"].long()[:-1, None] + pos).clamp_max(s["k"].shape[0] - 1)
        k = torch.cat([s["k"][at].float(),
                       s["k_rope"][at].float()[:, :, None].expand(-1, -1, s["hq"], -1)], 3)
        v = s["v"][at].float()
        k, v = (torch.where(ok[:, :, None, None], y, zero).transpose(1, 2).contiguous()
                for y in (k, v))
        return k, v, ok
    page = torch.gather(s["table"].long(), 1, (pos // s["ps"]).clamp_max(s["table"].shape[1] - 1))
    ok = ok & (page >= 0)
    pick = lambda x, at: (x.view(torch.uint8)[at].view(x.dtype)  # noqa: E731
                          if x.dtype == torch.float8_e4m3fn else x[at])
    if s["op"] == "latent":
        rows = _f32(pick(s["c"], (page.clamp_min(0), pos % s["ps"])), s["cs"])
        rows = torch.where(ok[:, :, None], rows, zero)[:, None]
        return rows, rows[..., :s["dc"]], ok
    at = (page.clamp_min(0), slice(None), pos % s["ps"])
    k, v = (torch.where(ok[:, :, None, None],
                        _f32(pick(x, at), None if sc is None else sc[:, None]),
                        zero).transpose(1, 2).contiguous()
            for x, sc in ((s["k"], s["ks"]), (s["v"], s["vs"])))
    return k, v, ok


def _tree_masks(s, at, m):
    """Of rows `at` [n, mm] of the batch: [n, mm, mm] which new tokens are a
    row's own or its ancestors, and the rows' depths."""
    n, mm = at.shape
    dev = at.device
    t = torch.arange(mm, device=dev)
    if s["parent"] is None:
        return (t[None, :] <= t[:, None]).expand(n, -1, -1), t.expand(n, -1)
    up = torch.where(t < m[:, None], s["parent"].long()[at], -1)
    anc = torch.eye(mm, dtype=torch.bool, device=dev).expand(n, -1, -1).clone()
    for _ in range(s["max_depth"] - 1):        # one generation further each time
        anc |= torch.nn.functional.one_hot(up.clamp_min(0), mm).bool() & (up >= 0)[:, :, None]
        up = torch.where(up >= 0, torch.gather(torch.where(t < m[:, None], s["parent"].long()[at],
                                                           -1), 1, up.clamp_min(0)), -1)
    return anc, anc.sum(-1) - 1


def _plain_attention(s):
    n, hq, mm, dev = s["n"], s["hq"], s["max_m"], s["q"].device
    hkv = s["hkv"] if s["op"] == "tree" else hq if s["op"] == "prompt" else 1
    g = hq // hkv
    cu, C = s["cu"].long(), s["before"].long()
    m = cu[1:] - cu[:-1]
    pos = torch.arange(s["max_len"], device=dev).expand(n, -1)
    k, v, ok = _keys_values(s, pos, pos < (C + m)[:, None])
    t = torch.arange(mm, device=dev).expand(n, -1)
    at = (cu[:-1, None] + t).clamp_max(s["q"].shape[0] - 1)
    q = s["q"].float()[at].view(n, mm, hkv, g, -1).permute(0, 2, 3, 1, 4).reshape(
        n, hkv, g * mm, -1)
    new = pos - C[:, None]                                   # which new token a key is
    if s["op"] == "prompt" or s["parent"] is None:
        p, pk = C[:, None] + t, pos
        see = ok[:, None, :] & (pos[:, None, :] <= p[:, :, None])
    else:
        anc, depth = _tree_masks(s, at, m)
        p = C[:, None] + depth
        own_key = new.clamp(0, mm - 1)
        pk = torch.where(new >= 0, C[:, None] + torch.gather(depth, 1, own_key), pos)
        up = torch.gather(anc, 2, own_key[:, None, :].expand(-1, mm, -1))
        see = ok[:, None, :] & (up | (new < 0)[:, None, :])
    if s["window"]:
        see = see & ((p[:, :, None] - pk[:, None, :] < s["window"]) |
                     (pk[:, None, :] < s["first"]))
    scores = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(s["scale"])
    scores = torch.where(see[:, None, None], scores.view(n, hkv, g, mm, -1),
                         torch.full((), -math.inf, device=dev))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    w = torch.exp(scores - top)
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.view(n, hkv, g * mm, -1), v).view(n, hkv, g, mm, -1)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = (torch.log(total) + top)[..., 0]
    row = torch.repeat_interleave(torch.arange(n, device=dev), m, output_size=s["q"].shape[0])
    col = torch.arange(s["q"].shape[0], device=dev) - cu[row]
    o = o.permute(0, 3, 1, 2, 4)[row, col].reshape(len(row), hq, -1)
    return {"out": o.to(s["q"].dtype), "lse": lse.permute(0, 3, 1, 2)[row, col].reshape(-1, hq)}


def _plain_write(s):
    cu = s["cu"].long()
    t = s["c_new"].shape[0]
    row = torch.repeat_interleave(torch.arange(s["n"], device=cu.device), cu[1:] - cu[:-1],
                                  output_size=t)
    pos = s["before"].long()[row] + torch.arange(t, device=cu.device) - cu[row]
    page = s["table"].long()[row, pos // s["ps"]]
    y = torch.cat([s["c_new"], s["rope_new"]], 1).float()
    if s["cs"] is not None:
        y = (y / s["cs"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        s["c"].view(torch.uint8)[page, pos % s["ps"]] = y.view(torch.uint8)
    else:
        s["c"][page, pos % s["ps"]] = y.to(s["c"].dtype)
    return {"c": s["c"]}


def _plain_keep(s):
    table, refs, lens, ps = s["table"], s["refs"], s["lens"], s["ps"]
    dev = table.device
    cu = s["cu_path"].long()
    k = cu[1:] - cu[:-1]
    row = torch.repeat_interleave(torch.arange(s["n"], device=dev), k, output_size=s["n_path"])
    j = torch.arange(s["n_path"], device=dev) - cu[row]
    C = (lens - s["n_draft"]).long()
    src, dst = C[row] + s["path"].long()[:s["n_path"]], C[row] + j
    ps_, pd = table.long()[row, src // ps], table.long()[row, dst // ps]
    for x in (s["k"], s["v"]):
        x[:, pd, :, dst % ps] = x[:, ps_, :, src % ps]
    lens.copy_(C + k)
    gone = torch.arange(table.shape[1], device=dev) >= ((C + k + ps - 1) // ps)[:, None]
    gone &= table >= 0
    refs.index_add_(0, table.clamp_min(0).reshape(-1).long(), -gone.reshape(-1).int())
    table.copy_(torch.where(gone, -1, table))
    return _pool(s)


# -------------------------------------------------------------------- exact

def exact(c, seed):
    """The definitions in 64 bits, one sequence (and head) after another."""
    s = prepare(c, seed)
    if c["op"] in ("tree", "latent", "prompt"):
        return _exact_attention(c, s)
    return _exact_write(c, s) if c["op"] == "write" else _exact_keep(c, s)


def _exact_rows(c, s, i, L, h):
    """Keys and values of the L tokens of sequence i for query head h."""
    if c["op"] == "prompt":
        a = int(s["cu_k"][i])
        return (torch.cat([s["k"][a:a + L, h], s["k_rope"][a:a + L]], 1).double(),
                s["v"][a:a + L, h].double())
    pages = s["table"][i, :_ceil(L, c["ps"])].clamp_min(0).long()
    take = lambda x: x.view(torch.uint8)[pages].view(x.dtype)  # noqa: E731
    if c["op"] == "latent":
        x = (take(s["c"]) if c["kv"] == "e4m3" else s["c"][pages]).double()
        x = x.reshape(-1, c["dc"] + ROPE)[:L]
        if s["cs"] is not None:
            x = x * s["cs"].double()
        return x, x[:, :c["dc"]]
    h = h // (c["hq"] // c["hkv"])
    both = []
    for x, sc in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        y = (x.view(torch.uint8)[pages, h].view(x.dtype) if c["kv"] == "e4m3"
             else x[pages, h]).double().reshape(-1, c["d"])[:L]
        both.append(y if sc is None else y * sc[h].double())
    return both


def _exact_attention(c, s):
    outs, lses = [], []
    at = 0
    # heads that share their keys and values
    share = {"tree": c["hq"] // c.get("hkv", 1), "latent": c["hq"], "prompt": 1}[c["op"]]
    for i, (C, m) in enumerate(zip(*(x.tolist() for x in _geometry(c)))):
        plain = not c["window"] and not _is_tree(c)
        see = None if plain else torch.from_numpy(_sees(c, i, C, m)).cuda()
        o = torch.zeros_like(s["out"][at:at + m], dtype=torch.float64)
        z = torch.zeros(m, c["hq"], dtype=torch.float64, device="cuda")
        j = torch.arange(C + m, device="cuda")
        for h in range(0, c["hq"], share):
            k, v = _exact_rows(c, s, i, C + m, h)
            step = max(1, (1 << 27) // ((C + m) * share))
            for a in range(0, m, step):
                b = min(m, a + step)
                q = s["q"][at + a:at + b, h:h + share].double()
                w = torch.mm(q.reshape(-1, q.shape[2]), k.t()) * s["scale"]
                rows = (j <= C + torch.arange(a, b, device="cuda")[:, None]) if plain else see[a:b]
                w = w.view(b - a, share, -1).masked_fill(~rows[:, None], -math.inf)
                z[a:b, h:h + share] = torch.logsumexp(w, -1)
                w = torch.exp(w - z[a:b, h:h + share, None])
                o[a:b, h:h + share] = torch.mm(w.view(-1, C + m), v).view(b - a, share, -1)
        outs.append(o)
        lses.append(z)
        at += m
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_write(c, s):
    C, m = _geometry(c)
    table = s["table"].cpu().numpy()
    x = s["c"].double()
    new = torch.cat([s["c_new"].double(), s["rope_new"].double()], 1)
    if s["cs"] is not None:
        new = (new / s["cs"].double()).clamp(-448.0, 448.0)
    at = 0
    for i, (L, q) in enumerate(zip(C.tolist(), m.tolist())):
        pos = np.arange(L, L + q)
        page = torch.from_numpy(table[i, pos // c["ps"]].astype(np.int64)).cuda()
        x[page, torch.from_numpy(pos % c["ps"]).cuda()] = new[at:at + q]
        at += q
    return {"c": x}


def _exact_keep(c, s):
    table, refs, lens = (s[k].cpu().tolist() for k in ("table", "refs", "lens"))
    k, v, ps = s["k"].double(), s["v"].double(), c["ps"]
    fr, to = [], []
    for i, (C, path) in enumerate(zip(_geometry(c)[0].tolist(), _paths(c))):
        for j, a in enumerate(path):
            fr.append((table[i][(C + a) // ps], (C + a) % ps))
            to.append((table[i][(C + j) // ps], (C + j) % ps))
        lens[i] = C + len(path)
        for e in range(len(table[i])):
            if e * ps >= lens[i] and table[i][e] >= 0:
                refs[table[i][e]] -= 1
                table[i][e] = -1
    if fr:
        fp, ft = (torch.tensor(x, device="cuda") for x in zip(*fr))
        tp, tt = (torch.tensor(x, device="cuda") for x in zip(*to))
        for x in (k, v):
            x[:, tp, :, tt] = x[:, fp, :, ft]
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"table": t(table), "refs": t(refs), "lens": t(lens), "k": k, "v": v}


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(case, work(case))
