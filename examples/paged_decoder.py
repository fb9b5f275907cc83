"""A small decoder served from a paged key-value cache.

Random weights; each layer is attention over the cache (moe_cache_append,
moe_attn_prefill, moe_attn_decode) followed by a routed mixture of experts
(moe_forward). The session runs the cache's calls as a server would: prompts of
different lengths in one batch, a second chunk of one of them, a fork that
continues one sequence twice, single-token steps with pages that the window has
passed returned to the pool, a sequence that ends, and a compaction with more
steps after it.

    python examples/paged_decoder.py [--kv e4m3] [--check]

--check recomputes every attention call densely in 64 bits from the keys and
values as they were handed to the cache.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import mixture_experts_expert_sigmoid_amd as M  # noqa: E402

LAYERS, H, HQ, HKV, D, VOCAB = 3, 256, 8, 2, 64, 500
EXPERTS, TOP_K, INNER = 16, 4, 256
WINDOW, FIRST = 96, 4
PAGE, PAGES, SLOTS = 16, 64, 6


def _norm(x):
    x = x.float()
    return (x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Layer:
    def __init__(self, gen):
        def w(*shape, std):
            return (torch.randn(*shape, generator=gen, device="cuda") * std).bfloat16()
        self.qkv = w((HQ + 2 * HKV) * D, H, std=H ** -0.5)
        self.o = w(H, HQ * D, std=(HQ * D) ** -0.5)
        self.gate = w(EXPERTS, H, std=H ** -0.5)
        self.experts = M.MoeModule(
            fmt=M.MOE_W_BF16, H=H, I=INNER, num_experts_global=EXPERTS, top_k=TOP_K,
            w13_q=w(EXPERTS, 2 * INNER, H, std=H ** -0.5),
            w2_q=w(EXPERTS, H, INNER, std=INNER ** -0.5))


class Dense:
    """Keys and values of every slot as handed to the cache, and attention over
    them in 64 bits. The bound: P is rounded to bf16 and so is the result, each
    by a factor within 1 +- 2^-8, and an average of V is at most max |V|; a
    twentieth more covers the fp32 sums and exponentials."""

    def __init__(self, scales):
        self.kv, self.scales, self.worst = {}, scales, 0.0

    def add(self, layer, slots, cu, k, v):
        for i, s in enumerate(slots):
            kv = []
            for x, sc in zip((k, v), self.scales):
                x = x[cu[i]:cu[i + 1]]
                if sc is not None:               # what the cache keeps of it
                    c = (x.float() / sc[layer][:, None]).clamp(-448, 448)
                    x = c.to(torch.float8_e4m3fn).double() * sc[layer][:, None].double()
                kv.append(x.double())
            old = self.kv.get((layer, s))
            self.kv[layer, s] = kv if old is None else [torch.cat(p) for p in zip(old, kv)]

    def check(self, layer, slots, cu, q, out):
        for i, s in enumerate(slots):
            k, v = self.kv[layer, s]
            L, m = k.shape[0], cu[i + 1] - cu[i]
            j = torch.arange(L, device="cuda")
            p = torch.arange(L - m, L, device="cuda")[:, None]
            see = (j <= p) & ((p - j < WINDOW) | (j < FIRST))
            for h in range(HQ):
                kh, vh = k[:, h // (HQ // HKV)].contiguous(), v[:, h // (HQ // HKV)].contiguous()
                x = (q[cu[i]:cu[i + 1], h].double()[:, None, :] * kh).sum(-1) * D ** -0.5
                y = torch.softmax(x.masked_fill(~see, -torch.inf), -1) @ vh
                err = (out[cu[i]:cu[i + 1], h].double() - y).abs().max()
                self.worst = max(self.worst, float(err / (1.05 * 2 ** -7 * vh.abs().max())))


class Decoder:
    def __init__(self, kv="bf16", check=False, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.embed = torch.randn(VOCAB, H, generator=gen, device="cuda").bfloat16()
        self.head = torch.randn(VOCAB, H, generator=gen, device="cuda").bfloat16()
        self.layers = [Layer(gen) for _ in range(LAYERS)]
        scale = None
        if kv == "e4m3":
            scale = torch.full((LAYERS, HKV), 4.5 / 448, device="cuda")
        self.cache = M.KvCache(
            n_layers=LAYERS, n_pages=PAGES, page_size=PAGE, n_heads=HKV, head_dim=D,
            n_slots=SLOTS, max_pages=32, k_scale=scale, v_scale=scale,
            dtype=torch.float8_e4m3fn if kv == "e4m3" else torch.bfloat16)
        self.dense = Dense((scale, scale)) if check else None
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def _i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def step(self, slots, tokens):
        """tokens: a list of new tokens for each slot. Returns the logits after
        the last of each."""
        rows = [len(t) for t in tokens]
        cu = [0]
        for m in rows:
            cu.append(cu[-1] + m)
        sl, cu_d = self._i32(slots), self._i32(cu)
        start = self.cache.grow(sl, self._i32(rows))
        x = self.embed[torch.tensor(sum(tokens, []), device="cuda")]
        for i, layer in enumerate(self.layers):
            q, k, v = (_norm(x) @ layer.qkv.t()).view(-1, HQ + 2 * HKV, D).split([HQ, HKV, HKV], 1)
            self.cache.append(i, sl, start, cu_d, k, v)
            if max(rows) == 1:
                y = self.cache.decode(i, sl, q, D ** -0.5, window=WINDOW, n_first=FIRST)
            else:
                y = self.cache.prefill(i, sl, q, cu_d, D ** -0.5, window=WINDOW, n_first=FIRST)
            if self.dense:
                self.dense.add(i, slots, cu, k, v)
                self.dense.check(i, slots, cu, q, y)
            x = x + y.reshape(-1, HQ * D) @ layer.o.t()
            z = _norm(x)
            out = layer.experts.forward(z, (z @ layer.gate.t()).float())
            self.err |= out["err_word"]
            x = x + out["out"].bfloat16()
        last = torch.tensor(cu[1:], device="cuda") - 1
        return (_norm(x[last]) @ self.head.t()).float()

    def trim(self, slots):
        self.cache.trim(self._i32(slots), WINDOW, FIRST)

    def fork(self, src, dst):
        self.cache.fork(self._i32([src]), self._i32([dst]))
        if self.dense:
            for i in range(LAYERS):
                self.dense.kv[i, dst] = list(self.dense.kv[i, src])

    def free(self, slot):
        self.cache.free(self._i32([slot]))
        if self.dense:
            for i in range(LAYERS):
                del self.dense.kv[i, slot]


def session(kv="bf16", check=False, steps=40):
    """Returns the decoder, the continuations by slot and the pages in use
    after each part of the session."""
    dec = Decoder(kv, check)
    gen = torch.Generator().manual_seed(1)

    def prompt(n):
        return torch.randint(0, VOCAB, (n,), generator=gen).tolist()

    used = {}

    def note(what):
        used[what] = int((dec.cache.refs > 0).sum())

    slots = [0, 1, 2]
    logits = dec.step(slots, [prompt(70), prompt(33), prompt(150)])
    note("prompts")
    logits[2] = dec.step([2], [prompt(41)])[0]       # a later chunk of the third
    dec.fork(2, 4)
    note("fork")
    top = logits.topk(2).indices.tolist()            # the fork takes the second best
    slots, tokens = [0, 1, 2, 4], [top[0][0], top[1][0], top[2][0], top[2][1]]
    text = {s: [t] for s, t in zip(slots, tokens)}

    def run(n):
        for _ in range(n):
            lg = dec.step(slots, [[text[s][-1]] for s in slots])
            for s, t in zip(slots, lg.argmax(-1).tolist()):
                text[s].append(t)
            dec.trim(slots)

    run(steps)
    note("steps")
    dec.free(0)
    slots.remove(0)
    note("free")
    dec.cache.compact()
    n = used["free"]
    used["highest page after compaction"] = int(torch.nonzero(dec.cache.refs).max())
    assert used["highest page after compaction"] == n - 1
    run(steps // 4)
    errors = M.moe_read_device_error(dec.cache.err_word) | M.moe_read_device_error(dec.err)
    if errors:
        raise RuntimeError(f"error word {errors:#x}")
    return dec, text, used


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--kv", choices=["bf16", "e4m3"], default="bf16")
    ap.add_argument("--check", action="store_true")
    args = ap.parse_args()
    decoder, text, used = session(args.kv, args.check)
    for s, t in text.items():
        print(f"slot {s}: {len(t)} tokens, {t[:12]} ...")
    print("pages in use:", used)
    if args.check:
        print(f"worst attention error / bound: {decoder.dense.worst:.3f}")
