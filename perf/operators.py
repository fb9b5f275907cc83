"""Cases of the cache and attention operators: a paged key-value cache, the
attention that reads it, and the upkeep of its pages.

A case names one operator (`op`):
  decode   attention of one new token per sequence over the pages
  prefill  attention of a prompt, or of the next chunk of one, over the pages
  append   new keys and values written into the pages
  turn     one turn of the pages between two steps of a server: finished
           sequences freed, passed pages trimmed, the next tokens' pages
           taken, running sequences forked
  compact  the used pages moved to the front of the pool

Lengths follow a fixed pattern of the case (`_lens`), so a case's work does
not depend on the seed; values, page order and queries do.
"""
import math
import random

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
_SIZE = {"bf16": 2, "f16": 2, "e4m3": 1}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one user, a few hundred tokens in: the smallest call, latency
        dict(name="decode_one", op="decode", dt="bf16", kv="bf16", n=1, hq=32, hkv=8, d=128,
             ps=16, lo=777, hi=777, window=0, first=0),
        # an ordinary batch of a server, ragged lengths
        dict(name="decode_batch", op="decode", dt="bf16", kv="bf16", n=64, hq=32, hkv=8, d=128,
             ps=64, lo=201, hi=4001, window=0, first=0),
        # two very long contexts in an 8-bit cache: few rows, a long axis
        dict(name="decode_long", op="decode", dt="bf16", kv="e4m3", n=2, hq=64, hkv=8, d=128,
             ps=64, lo=100003, hi=130001, window=0, first=0),
        # a large batch behind a sliding window with first tokens kept, the
        # pages in between given back
        dict(name="decode_window", op="decode", dt="f16", kv="f16", n=192, hq=64, hkv=8, d=64,
             ps=32, lo=60, hi=30011, window=1024, first=4),
        # one short prompt: latency
        dict(name="prefill_short", op="prefill", dt="bf16", kv="bf16", n=1, hq=32, hkv=8, d=128,
             ps=16, lo=37, hi=37, qlo=37, qhi=37, window=0, first=0),
        # a ragged batch of prompts of a layer with a window
        dict(name="prefill_window", op="prefill", dt="f16", kv="f16", n=7, hq=32, hkv=4, d=64,
             ps=32, lo=130, hi=3001, qlo=130, qhi=3001, window=512, first=4),
        # the next chunk of two long prompts over an 8-bit cache
        dict(name="prefill_chunk", op="prefill", dt="bf16", kv="e4m3", n=2, hq=32, hkv=8, d=128,
             ps=64, lo=16001, hi=24013, qlo=500, qhi=509, window=0, first=0),
        # one long prompt, full causal attention: the largest
        dict(name="prefill_long", op="prefill", dt="bf16", kv="bf16", n=1, hq=32, hkv=8, d=128,
             ps=64, lo=11999, hi=11999, qlo=11999, qhi=11999, window=0, first=0),
        # one token of each sequence of a batch
        dict(name="append_step", op="append", dt="bf16", kv="bf16", n=64, hkv=8, d=128, ps=64,
             lo=200, hi=4000, mlo=1, mhi=1),
        # prompts into an 8-bit cache
        dict(name="append_prompts", op="append", dt="bf16", kv="e4m3", n=8, hkv=8, d=128, ps=64,
             lo=0, hi=900, mlo=500, mhi=8001),
        # one turn of a server of 96 slots, four layers
        dict(name="pages_turn", op="turn", kv="bf16", n=96, hkv=4, d=128, ps=16, layers=4,
             pages=4096, lo=17, hi=600, window=256, first=4, forks=12),
        # a half-empty pool of four layers compacted
        dict(name="pages_compact", op="compact", kv="bf16", n=48, hkv=8, d=128, ps=64, layers=4,
             pages=2048, lo=40, hi=2600),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "append", "turn", "compact"])
    dt = rng.choice(["bf16", "f16"])
    kv = rng.choice([dt, dt, "e4m3"])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 5, 8, 16])
    d = rng.choice([64, 128, 128, 256])
    ps = rng.choice([16, 32, 64, 128])
    window = rng.choice([0, 0, _log(rng, 16, 4096)])
    first = rng.choice([0, 4, 17]) if window else 0
    row = hkv * d
    if op == "decode":
        n = _log(rng, 1, 256)
        # as many tokens in all as the largest listed batch holds
        hi = _log(rng, 16, max(17, min(130000, (1 << 28) // (n * row * max(1, g // 2)))))
        return dict(op=op, dt=dt, kv=kv, n=n, hq=hkv * g, hkv=hkv, d=d, ps=ps,
                    lo=rng.randint(1, hi), hi=hi, window=window, first=first)
    if op == "prefill":
        n = _log(rng, 1, 16)
        qhi = _log(rng, 1, 4096)
        hi = qhi + rng.choice([0, 0, _log(rng, 1, 20000)])
        # query and key pairs in all, padded to the longest
        while n * hkv * g * qhi * hi * max(1, d // 128) > 2_000_000_000:
            if n > 1:
                n = n // 2
            else:
                qhi, hi = (qhi + 1) // 2, (hi + 1) // 2
        qlo = rng.randint(1, qhi)
        return dict(op=op, dt=dt, kv=kv, n=n, hq=hkv * g, hkv=hkv, d=d, ps=ps,
                    lo=max(qlo, hi - (qhi - qlo)), hi=hi, qlo=qlo, qhi=qhi,
                    window=window, first=first)
    if op == "append":
        n = _log(rng, 1, 256)
        mhi = _log(rng, 1, max(2, min(8192, 30000 // n)))
        hi = rng.randint(0, 2000)
        return dict(op=op, dt=dt, kv=kv, n=n, hkv=hkv, d=d, ps=ps, lo=rng.randint(0, hi), hi=hi,
                    mlo=rng.randint(1, mhi), mhi=mhi)
    layers = rng.randint(1, 4)
    n = _log(rng, 8, 96)
    lo = rng.randint(1, 100)
    hi = lo + _log(rng, 16, 1500)
    need = 2 * (n + 8) * (hi // ps + 3)
    pages = max(64, need)
    while layers * pages * row * ps > (1 << 29):        # at most the listed pool
        if layers > 1:
            layers -= 1
        elif hkv > 1:
            hkv //= 2
        else:
            d = 64
            break
        row = hkv * d
    c = dict(op=op, kv=rng.choice(["bf16", "f16"]), n=n, hkv=hkv, d=d, ps=ps, layers=layers,
             pages=pages, lo=lo, hi=hi)
    if op == "turn":
        c.update(window=rng.choice([64, 256, 1000]), first=rng.choice([0, 4]),
                 forks=rng.randint(1, max(1, n // 4)))
    return c


# ------------------------------------------------------------ case geometry

def _lens(n, lo, hi):
    """n lengths in lo..hi, the last hi, spread evenly and out of order."""
    f = (np.arange(1, n + 1) * 0.6180339887498949) % 1.0
    v = (lo + np.floor(f * (hi - lo + 1))).astype(np.int64)
    v[-1] = hi
    return v


def _geometry(c):
    """(lengths, new tokens of each sequence)"""
    lens = _lens(c["n"], c["lo"], c["hi"])
    if c["op"] == "decode":
        return lens, np.ones_like(lens)
    if c["op"] == "prefill":
        m = np.minimum(_lens(c["n"], c["qlo"], c["qhi"]), lens)
        return np.maximum(lens, m), m
    if c["op"] == "append":
        return lens, _lens(c["n"], c["mlo"], c["mhi"])
    return lens, None


def _ceil(a, b):
    return -(-a // b)


def _visible(lens, m, window, first):
    """Visible (query, key) pairs, and the keys that any query sees."""
    pairs = keys = 0
    for L, q in zip(lens.tolist(), m.tolist()):
        p = np.arange(L - q, L, dtype=np.int64)
        if window:
            pairs += int((np.minimum(p + 1, window) +
                          np.minimum(first, np.maximum(p + 1 - window, 0))).sum())
            lo = max(0, int(p[0]) + 1 - window) if q else L
            keys += L - lo + min(first, lo)
        else:
            pairs += int((p + 1).sum())
            keys += L
    return pairs, keys


def work(c):
    lens, m = _geometry(c)
    if c["op"] in ("decode", "prefill"):
        pairs, keys = _visible(lens, m, c["window"], c["first"])
        t = int(m.sum())
        return {"bytes": keys * 2 * c["hkv"] * c["d"] * _SIZE[c["kv"]] +
                t * c["hq"] * (2 * c["d"] * 2 + 4),
                "flops": 4 * pairs * c["hq"] * c["d"]}
    if c["op"] == "append":
        t = int(m.sum())
        return {"bytes": t * 2 * c["hkv"] * c["d"] * (2 + _SIZE[c["kv"]]), "flops": 0}
    page = 2 * c["layers"] * c["hkv"] * c["ps"] * c["d"] * _SIZE[c["kv"]]
    plan = _plan(c, 0)
    small = 8 * plan["table"].size + 8 * plan["refs"].size
    if c["op"] == "turn":
        moved = int((plan["lens_fork"] % c["ps"] != 0).sum())
    else:
        used = int((plan["refs"] > 0).sum())
        moved = int((plan["refs"][used:] > 0).sum())
    return {"bytes": small + 2 * page * moved, "flops": 0}


# -------------------------------------------------------------- page layouts

def _layout(seed, lens, ps, spare):
    """Tables of shuffled pages for these lengths: (table, pages)."""
    r = np.random.RandomState(seed % (1 << 31))
    need = _ceil(lens, ps)
    total = int(need.sum())
    order = r.permutation(total + spare)
    mp = int(need.max()) if len(need) else 0
    table = np.full((len(lens), max(mp, 1)), -1, np.int32)
    at = 0
    for i, k in enumerate(need.tolist()):
        table[i, :k] = order[at:at + k]
        at += k
    return table, total + spare


def _plan(c, seed):
    """A pool in use, for the cases of page upkeep: tables, lengths and
    reference counts; a third of the slots finish, the first `forks` of the
    rest are forked into empty slots after them."""
    n, ps, P = c["n"], c["ps"], c["pages"]
    r = np.random.RandomState(seed % (1 << 31))
    lens = _lens(n, c["lo"], c["hi"])
    forks = c.get("forks", 0)
    mp = _ceil(c["hi"] + 2 * ps, ps)
    table = np.full((n + forks, mp), -1, np.int32)
    refs = np.zeros(P, np.int32)
    # the pool's first part is half in use, as after many requests; what is
    # used where differs by the seed, how many pages are used where does not
    need = _ceil(lens, ps)
    total = int(need.sum())
    span = min(P, 2 * total)
    if c["op"] == "compact":                  # half of them beyond `total`
        back = total // 2 if span - total >= total // 2 else span - total
        keep = r.permutation(total)[:total - back]
        far = total + r.permutation(span - total)[:back]
        order = r.permutation(np.concatenate([keep, far]))
    else:
        order = r.permutation(span)[:total]
    at = 0
    for i, k in enumerate(need.tolist()):
        table[i, :k] = order[at:at + k]
        at += k
    refs[order[:at]] = 1
    lens_all = np.zeros(n + forks, np.int32)
    lens_all[:n] = lens
    done = np.arange(2, n, 3, dtype=np.int32)
    live = np.setdiff1d(np.arange(n, dtype=np.int32), done)
    new = np.where(np.arange(len(live)) % 7 == 3, ps + 5, 1).astype(np.int32)
    src = live[np.arange(forks) % len(live)] if forks else np.zeros(0, np.int32)
    dst = np.arange(n, n + forks, dtype=np.int32)
    at_src = np.searchsorted(live, src)
    return dict(table=table, refs=refs, lens=lens_all, done=done, live=live, new=new,
                src=src.astype(np.int32), dst=dst,
                lens_fork=lens[src] + new[at_src] if forks else np.zeros(0, np.int64),
                moves=int((refs[total:] > 0).sum()))


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
    s = dict(c)
    if c["op"] in ("turn", "compact"):
        p = _plan(c, seed)
        for k in ("table", "refs", "lens", "done", "live", "new", "src", "dst"):
            s[k] = dev(p[k])
        s["moves"] = p["moves"]
        s["table0"], s["refs0"], s["lens0"] = (s[k].clone() for k in ("table", "refs", "lens"))
        shape = (c["layers"], c["pages"], c["hkv"], c["ps"], c["d"])
        s["k"] = _randn(gen, shape, c["kv"])
        s["v"] = _randn(gen, shape, c["kv"])
        s["start"] = torch.zeros(len(p["live"]), dtype=torch.int32, device="cuda")
        s["n_used"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    else:
        lens, m = _geometry(c)
        hold = lens + m if c["op"] == "append" else lens
        table, pages = _layout(seed, hold, c["ps"], 5)
        if c["window"] if "window" in c else 0:
            # pages that no query of this call sees have been given back
            first_q = lens - m
            pg = np.arange(table.shape[1])[None, :] * c["ps"]
            gone = (pg >= c["first"]) & (pg + c["ps"] - 1 < (first_q - c["window"])[:, None])
            table[gone] = -1
        shape = (pages, c["hkv"], c["ps"], c["d"])
        sc = 0.02
        s["k"] = _randn(gen, shape, c["kv"], sc)
        s["v"] = _randn(gen, shape, c["kv"], sc)
        if c["kv"] == "e4m3":
            s["ks"] = sc * (0.5 + torch.rand(c["hkv"], generator=gen, device="cuda"))
            s["vs"] = sc * (0.5 + torch.rand(c["hkv"], generator=gen, device="cuda"))
        else:
            s["ks"] = s["vs"] = None
        s["table"] = dev(table)
        s["lens"] = dev(lens.astype(np.int32))
        cu = np.concatenate([[0], np.cumsum(m)]).astype(np.int32)
        s["cu"] = dev(cu)
        t = int(cu[-1])
        s["max_len"], s["max_m"] = int(hold.max()), int(m.max())
        if c["op"] == "append":
            s["start"] = s["lens"].clone()
            s["k_new"] = torch.randn(t, c["hkv"], c["d"], generator=gen, device="cuda",
                                     dtype=_DT[c["dt"]])
            s["v_new"] = torch.randn(t, c["hkv"], c["d"], generator=gen, device="cuda",
                                     dtype=_DT[c["dt"]])
        else:
            s["q"] = 1.5 * torch.randn(t, c["hq"], c["d"], generator=gen, device="cuda",
                                       dtype=_DT[c["dt"]])
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(t, c["hq"], device="cuda")
            s["scale"] = c["d"] ** -0.5
    if own:
        _own_handles(s)
    return s


def _own_handles(s):
    """Descriptors and workspaces, as a serving program keeps them."""
    import mixture_experts_expert_sigmoid_amd as M
    s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    op = s["op"]
    ws = 0
    if op in ("turn", "compact"):
        s["caches"] = [M.kv_cache(s["k"][i], s["v"][i]) for i in range(s["layers"])]
        s["tab"] = M.kv_table(s["table"], s["lens"], s["ps"], s["pages"], refs=s["refs"])
        ws = M.moe_cache_workspace_size(s["tab"], s["table"].shape[0])
    else:
        s["cache"] = M.kv_cache(s["k"], s["v"], s["ks"], s["vs"])
        s["tab"] = M.kv_table(s["table"], s["lens"], s["ps"], s["k"].shape[0])
        if op == "decode":
            ws = M.moe_attn_decode_workspace_size(s["cache"], s["n"], s["hq"])
        elif op == "prefill":
            ws = M.moe_attn_prefill_workspace_size(s["cache"], s["n"], s["q"].shape[0], s["hq"])
    s["ws"] = torch.empty(max(ws, 1), dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------------- run

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import mixture_experts_expert_sigmoid_amd as M
    op = s["op"]
    if op == "decode":
        M.moe_attn_decode(s["cache"], s["tab"], s["q"], s["out"], s["scale"], s["err"], s["ws"],
                          window=s["window"], n_first=s["first"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "prefill":
        M.moe_attn_prefill(s["cache"], s["tab"], s["q"], s["cu"], s["out"], s["scale"], s["err"],
                           s["ws"], window=s["window"], n_first=s["first"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "append":
        M.moe_cache_append(s["cache"], s["tab"], s["start"], s["cu"], s["k_new"], s["v_new"],
                           s["err"])
        return {"k": s["k"], "v": s["v"]}
    _rewind(s)
    if op == "turn":
        M.moe_cache_free(s["tab"], s["done"], s["err"])
        M.moe_cache_trim(s["tab"], s["live"], s["window"], s["first"], s["err"])
        M.moe_cache_grow(s["tab"], s["live"], s["new"], s["start"], s["err"], s["ws"])
        M.moe_cache_fork(s["caches"], s["tab"], s["src"], s["dst"], s["err"], s["ws"])
        return _pool_outputs(s)
    M.moe_cache_compact(s["caches"], s["tab"], s["n_used"], s["err"], s["ws"])
    return _pool_outputs(s)


def _rewind(s):
    """The pool's tables as prepare made them: a pass does its whole work on
    a state that a pass before it has run on (the pages' contents that a pass
    moves are still where it takes them from)."""
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    s["lens"].copy_(s["lens0"])


def _pool_outputs(s):
    o = {k: s[k] for k in ("table", "refs", "lens", "k", "v")}
    o["n"] = s["start"] if s["op"] == "turn" else s["n_used"]
    return o


def _run_plain(s):
    op = s["op"]
    if op == "decode":
        return _plain_decode(s)
    if op == "prefill":
        return _plain_prefill(s)
    if op == "append":
        return _plain_append(s)
    _rewind(s)
    return _plain_turn(s) if op == "turn" else _plain_compact(s)


def _gather(s, pos, ok):
    """K and V of positions pos [n, L] in 32 bits, zero where not ok:
    [n, hkv, L, d] each."""
    ps = s["ps"]
    page = torch.gather(s["table"].long(), 1, (pos // ps).clamp(0, s["table"].shape[1] - 1))
    ok = ok & (page >= 0)
    at = (page.clamp_min(0), slice(None), pos % ps)
    both = []
    for x, sc in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        raw = x.view(torch.uint8)[at].view(x.dtype) if x.dtype == torch.float8_e4m3fn else x[at]
        y = raw.float()                                     # [n, L, hkv, d]
        if sc is not None:
            y = y * sc[:, None]
        y = torch.where(ok[:, :, None, None], y, torch.zeros((), device=y.device))
        both.append(y.transpose(1, 2).contiguous())
    return both[0], both[1], ok


def _softmax_av(scores, mask, v):
    """softmax over the masked scores times v, and the log-sum-exp."""
    scores = torch.where(mask, scores, torch.full((), -math.inf, device=scores.device))
    m = scores.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    p = torch.exp(scores - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o, (torch.log(total) + m)[..., 0]


def _plain_decode(s):
    n, hq, hkv, d = s["n"], s["hq"], s["hkv"], s["d"]
    dev = s["q"].device
    lens = s["lens"].long()
    if s["window"]:
        w = min(s["window"], s["max_len"])
        lo = (lens - s["window"]).clamp_min(0)
        head = torch.arange(s["first"], device=dev).expand(n, -1)
        tail = lens[:, None] - w + torch.arange(w, device=dev)
        pos = torch.cat([head, tail], 1)
        ok = torch.cat([head < lo[:, None], tail >= 0], 1)
    else:
        pos = torch.arange(s["max_len"], device=dev).expand(n, -1)
        ok = pos < lens[:, None]
    k, v, ok = _gather(s, pos.clamp_min(0), ok)
    q = s["q"].float().view(n, hkv, hq // hkv, d)
    scores = torch.matmul(q, k.transpose(2, 3).contiguous()) * s["scale"]
    o, lse = _softmax_av(scores, ok[:, None, None, :], v)
    return {"out": o.reshape(n, hq, d).to(s["q"].dtype), "lse": lse.reshape(n, hq)}


def _plain_prefill(s):
    n, hq, hkv, d = s["n"], s["hq"], s["hkv"], s["d"]
    g, mm, dev = hq // hkv, s["max_m"], s["q"].device
    lens, cu = s["lens"].long(), s["cu"].long()
    m = cu[1:] - cu[:-1]
    pos = torch.arange(s["max_len"], device=dev).expand(n, -1)
    k, v, ok = _gather(s, pos, pos < lens[:, None])
    t = torch.arange(mm, device=dev).expand(n, -1)
    at = (cu[:-1, None] + t).clamp_max(s["q"].shape[0] - 1)
    q = s["q"].float()[at].view(n, mm, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, g * mm, d)
    p = (lens - m)[:, None] + t
    see = ok[:, None, :] & (pos[:, None, :] <= p[:, :, None])
    if s["window"]:
        see &= (p[:, :, None] - pos[:, None, :] < s["window"]) | (pos[:, None, :] < s["first"])
    scores = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(s["scale"])
    o, lse = _softmax_av(scores.view(n, hkv, g, mm, -1), see[:, None, None], v[:, :, None])
    row = torch.repeat_interleave(torch.arange(n, device=dev), m, output_size=s["q"].shape[0])
    col = torch.arange(s["q"].shape[0], device=dev) - cu[row]
    o = o.permute(0, 3, 1, 2, 4)[row, col].reshape(-1, hq, d)
    return {"out": o.to(s["q"].dtype), "lse": lse.permute(0, 3, 1, 2)[row, col].reshape(-1, hq)}


def _plain_append(s):
    cu = s["cu"].long()
    t = s["k_new"].shape[0]
    row = torch.repeat_interleave(torch.arange(s["n"], device=cu.device), cu[1:] - cu[:-1],
                                  output_size=t)
    pos = s["start"].long()[row] + torch.arange(t, device=cu.device) - cu[row]
    page = s["table"].long()[row, pos // s["ps"]]
    for x, new, sc in ((s["k"], s["k_new"], s["ks"]), (s["v"], s["v_new"], s["vs"])):
        y = new.float()
        if sc is not None:
            y = (y / sc[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            x.view(torch.uint8)[page, :, pos % s["ps"]] = y.view(torch.uint8)
        else:
            x[page, :, pos % s["ps"]] = y.to(x.dtype)
    return {"k": s["k"], "v": s["v"]}


def _drop(refs, pages, held):
    refs.index_add_(0, pages.clamp_min(0).reshape(-1).long(), -held.reshape(-1).to(refs.dtype))


def _put(x, at, values, ok):
    """x.view(-1)[at] = values where ok, by a last element that is thrown away."""
    flat = torch.cat([x.reshape(-1), x.new_zeros(1)])
    flat[torch.where(ok, at, torch.full((), flat.numel() - 1, device=at.device)).reshape(-1)] = \
        values.reshape(-1).to(x.dtype)
    x.copy_(flat[:-1].view_as(x))


def _plain_turn(s):
    table, refs, lens, ps = s["table"], s["refs"], s["lens"], s["ps"]
    mp, dev = table.shape[1], table.device
    done, live = s["done"].long(), s["live"].long()
    # free
    rows = table[done]
    _drop(refs, rows, rows >= 0)
    table[done] = -1
    lens[done] = 0
    # trim
    rows = table[live]
    pg = torch.arange(mp, device=dev) * ps
    dead = (rows >= 0) & (pg >= s["first"]) & (pg + ps - 1 < lens[live][:, None] - s["window"])
    _drop(refs, rows, dead)
    table[live] = torch.where(dead, -1, rows)
    # grow: the lowest free pages, in the order of the slots (the pool holds them)
    old = lens[live].long()
    s["start"].copy_(old)
    have = (old + ps - 1) // ps
    need = (old + s["new"] + ps - 1) // ps - have
    free = torch.sort((refs > 0).int(), stable=True).indices
    j = torch.arange(mp, device=dev)
    ok = j < need[:, None]
    page = free[((torch.cumsum(need, 0) - need)[:, None] + j).clamp_max(free.numel() - 1)]
    _put(table, live[:, None] * mp + have[:, None] + j, page, ok)
    _put(refs, page, torch.ones_like(page), ok)
    lens[live] += s["new"]
    # fork: shared pages, a copy of the last one where it is partly filled
    src, dst = s["src"].long(), s["dst"].long()
    n = lens[src].long()
    part = n % ps != 0
    last = n // ps
    free = torch.sort((refs > 0).int(), stable=True).indices
    page = free[torch.cumsum(part.long(), 0) - part.long()]
    rows = table[src]
    own_page = part[:, None] & (torch.arange(mp, device=dev) == last[:, None])
    from_page = torch.gather(rows, 1, last.clamp_max(mp - 1)[:, None])[:, 0].long()
    _drop(refs, rows, -((rows >= 0) & ~own_page).int())
    _put(refs, page, torch.ones_like(page), part)
    table[dst] = torch.where(own_page, page[:, None].int(), rows)
    lens[dst] = lens[src]
    to = torch.where(part, page, from_page.clamp_min(0))
    fr = from_page.clamp_min(0)
    for x in (s["k"], s["v"]):
        x[:, to] = x[:, fr]
    return _pool_outputs(s)


def _plain_compact(s):
    table, refs = s["table"], s["refs"]
    P = refs.numel()
    used = refs > 0
    total = used.sum()
    idx = torch.arange(P, device=refs.device)
    hole = ~used & (idx < total)
    mover = used & (idx >= total)
    k = s["moves"]
    to = torch.sort((~hole).int(), stable=True).indices[:k]
    fr = torch.sort((~mover).int(), stable=True).indices[:k]
    for x in (s["k"], s["v"]):
        x[:, to] = x[:, fr]
    remap = idx.int()
    remap[fr] = to.int()
    refs[to] = refs[fr]
    refs[fr] = 0
    table.copy_(torch.where(table >= 0, remap[table.clamp_min(0).long()], table))
    s["n_used"].copy_(total)
    return _pool_outputs(s)


# -------------------------------------------------------------------- exact

def exact(c, seed):
    """The definitions in 64 bits, one sequence (or page) after another."""
    s = prepare(c, seed)
    if c["op"] in ("decode", "prefill"):
        return _exact_attention(c, s)
    if c["op"] == "append":
        return _exact_append(c, s)
    return _exact_pages(c, s)


def _exact_attention(c, s):
    lens, m = _geometry(c)
    g, d, ps = c["hq"] // c["hkv"], c["d"], c["ps"]
    table = s["table"].cpu().numpy()
    outs, lses = [], []
    at = 0
    for i, (L, q) in enumerate(zip(lens.tolist(), m.tolist())):
        pages = torch.from_numpy(np.maximum(table[i, :_ceil(L, ps)], 0).astype(np.int64)).cuda()
        o = torch.zeros(q, c["hq"], d, dtype=torch.float64, device="cuda")
        z = torch.zeros(q, c["hq"], dtype=torch.float64, device="cuda")
        j = torch.arange(L, device="cuda")
        for h in range(c["hkv"]):
            kk, vv = ((x.view(torch.uint8)[pages, h].view(x.dtype)
                       if x.dtype == torch.float8_e4m3fn else x[pages, h])
                      .double().reshape(-1, d)[:L] for x in (s["k"], s["v"]))
            if s["ks"] is not None:
                kk, vv = kk * s["ks"][h].double(), vv * s["vs"][h].double()
            step = max(1, (1 << 27) // (L * g))
            for a in range(0, q, step):
                b = min(q, a + step)
                p = torch.arange(L - q + a, L - q + b, device="cuda")[:, None]
                see = j <= p
                if c["window"]:
                    see &= (j > p - c["window"]) | (j < c["first"])
                rows = s["q"][at + a:at + b, h * g:(h + 1) * g].double()
                w = torch.mm(rows.reshape(-1, d), kk.t()) * s["scale"]
                w = w.view(b - a, g, L).masked_fill(~see[:, None], -math.inf)
                z[a:b, h * g:(h + 1) * g] = torch.logsumexp(w, -1)
                w = torch.exp(w - z[a:b, h * g:(h + 1) * g, None])
                o[a:b, h * g:(h + 1) * g] = torch.mm(w.view(-1, L), vv).view(b - a, g, d)
        outs.append(o)
        lses.append(z)
        at += q
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_append(c, s):
    lens, m = _geometry(c)
    table = s["table"].cpu().numpy()
    out = {}
    for name in ("k", "v"):
        x = s[name].double()
        new = s[name + "_new"].double()
        sc = s[name + "s"]
        if sc is not None:
            new = (new / sc.double()[:, None]).clamp(-448.0, 448.0)
        at = 0
        for i, (L, q) in enumerate(zip(lens.tolist(), m.tolist())):
            pos = np.arange(L, L + q)
            page = torch.from_numpy(table[i, pos // c["ps"]].astype(np.int64)).cuda()
            x[page, :, torch.from_numpy(pos % c["ps"]).cuda()] = new[at:at + q]
            at += q
        out[name] = x
    return out


def _exact_pages(c, s):
    table, refs, lens = (s[k].cpu().tolist() for k in ("table", "refs", "lens"))
    k, v, ps = s["k"].double(), s["v"].double(), c["ps"]
    if c["op"] == "turn":
        for i in s["done"].tolist():
            for e in table[i]:
                if e >= 0:
                    refs[e] -= 1
            table[i] = [-1] * len(table[i])
            lens[i] = 0
        for i in s["live"].tolist():
            for a, e in enumerate(table[i]):
                if e >= 0 and a * ps >= c["first"] and a * ps + ps <= lens[i] - c["window"]:
                    refs[e] -= 1
                    table[i][a] = -1
        start = []
        for i, new in zip(s["live"].tolist(), s["new"].tolist()):
            start.append(lens[i])
            for a in range(_ceil(lens[i], ps), _ceil(lens[i] + new, ps)):
                table[i][a] = refs.index(0)
                refs[table[i][a]] = 1
            lens[i] += new
        for i, j in zip(s["src"].tolist(), s["dst"].tolist()):
            table[j], lens[j] = list(table[i]), lens[i]
            if lens[i] % ps:
                a = lens[i] // ps
                e = refs.index(0)
                k[:, e], v[:, e] = k[:, table[i][a]], v[:, table[i][a]]
                table[j][a], refs[e] = e, 0
            for e in table[j]:
                if e >= 0:
                    refs[e] += 1
        last = start
    else:
        used = [e for e in range(len(refs)) if refs[e] > 0]
        n = len(used)
        to = [e for e in range(n) if refs[e] == 0]
        fr = [e for e in used if e >= n]
        new = dict(zip(fr, to))
        k[:, to], v[:, to] = k[:, fr], v[:, fr]
        for a, b in new.items():
            refs[b], refs[a] = refs[a], 0
        table = [[new.get(e, e) for e in row] for row in table]
        last = [n]
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"table": t(table), "refs": t(refs), "lens": t(lens), "k": k, "v": v, "n": t(last)}


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(i)) for i in range(6)]:
        print(case, work(case))
