"""moe_attn_latent_prompt against a plain 64-bit attention over rows."""
import numpy as np
import pytest
import torch

import mixture_experts_expert_sigmoid_amd as M
from tests.cache_ref import DT, attention, check, visible
from tests.test_gpu_attn import _q

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]
D, R = 128, 64


class Rows:
    """Keys and values of n sequences on the GPU, NaN around and between them,
    and in float64 on the host."""

    def __init__(self, rng, dt, H, lens, how="dense", extra=5):
        S = sum(lens) + extra
        self.dt, self.H, self.lens, self.S = dt, H, lens, S
        self.cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        x = {"k": rng.standard_normal((S, H, D)), "v": rng.standard_normal((S, H, D)),
             "r": rng.standard_normal((S, R))}
        self.host = {n: torch.from_numpy(y).to(DT[dt]).double() for n, y in x.items()}
        for y in self.host.values():
            y[self.cu[-1]:] = float("nan")       # rows behind the last sequence
        nan = float("nan")
        kw = dict(dtype=DT[dt], device="cuda")
        if how == "joint":               # as one product's rows: a head's keys and values
            kv = torch.full((S, H, 2 * D), nan, **kw)
            self.k, self.v = kv[..., :D], kv[..., D:]
            self.r = torch.full((S, 512 + R), nan, **kw)[:, 512:]
        elif how == "heads":
            self.k, self.v = (torch.full((H, S, D + 8), nan, **kw).transpose(0, 1)[..., :D]
                              for _ in range(2))
            self.r = torch.full((S, R + 8), nan, **kw)[:, :R]
        else:
            self.k, self.v = (torch.full((S, H, D), nan, **kw) for _ in range(2))
            self.r = torch.full((S, R), nan, **kw)
        self.upload()

    def upload(self):
        for n in "kvr":
            getattr(self, n).copy_(self.host[n])

    def keys(self, i, h):
        a, b = self.cu[i], self.cu[i + 1]
        k = np.concatenate([self.host["k"][a:b, h].numpy(), self.host["r"][a:b].numpy()], 1)
        return k, self.host["v"][a:b, h].numpy()


def want_of(rows, m, q, window, first, scale, see=None):
    acc, at = [], 0
    for i, (L, n) in enumerate(zip(rows.lens, m)):
        ok = visible(np.arange(L - n, L), L, window, first) if see is None else see[i]
        per = []
        for h in range(rows.H):
            k, v = rows.keys(i, h)
            v = np.concatenate([v, np.zeros((L, R))], 1)
            o, z, bo, bl = attention(q[at:at + n, h:h + 1], k, v, ok, scale, rows.dt)
            per.append((o[..., :D], z, bo[..., :D], bl))
        acc.append([np.concatenate(x, 1) for x in zip(*per)])
        at += n
    return [np.concatenate(x, 0) for x in zip(*acc)]


def run(rows, m, q, window, first, scale, how="dense"):
    T, H, dt = q.shape[0], rows.H, rows.dt

    def empty(d):
        if how == "heads":
            return torch.full((H, T, d), float("nan"), dtype=DT[dt], device="cuda").transpose(0, 1)
        if how == "pad":
            return torch.full((T, H + 1, d + 8), float("nan"), dtype=DT[dt],
                              device="cuda")[:, :H, :d]
        return torch.full((T, H, d), float("nan"), dtype=DT[dt], device="cuda")
    qd, out = empty(D + R), empty(D)
    qd.copy_(torch.from_numpy(q))
    lse = torch.full((T, H), 7.0, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    cu_q = torch.tensor(np.concatenate([[0], np.cumsum(m)]), **i32)
    cu_k = torch.tensor(rows.cu, **i32)
    ws = torch.empty(max(16, M.moe_attn_latent_prompt_workspace_size(len(m), T, H)),
                     dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    got = []
    for _ in range(2):
        M.moe_attn_latent_prompt(qd, rows.k, rows.r, rows.v, cu_q, cu_k, out, scale, ws,
                                 window=window, n_first=first, lse=lse)
        torch.cuda.synchronize()
        got.append((out.contiguous().view(torch.int16).clone(), lse.view(torch.int32).clone()))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


# dt, heads, strides of rows, of q, (keys, new) of each, window, first
CASES = {
    "one_token": ("bf16", 4, "dense", "dense", [(1, 1)], 0, 0),
    "short": ("bf16", 3, "joint", "pad", [(37, 37), (1, 1), (16, 16), (129, 129)], 0, 0),
    "f16": ("f16", 5, "heads", "heads", [(200, 200), (65, 65)], 0, 0),
    "chunks": ("bf16", 2, "joint", "dense", [(300, 19), (1000, 1), (64, 64), (500, 130)], 0, 0),
    "empty": ("f16", 2, "dense", "dense", [(0, 0), (50, 50), (0, 0), (40, 0), (7, 7)], 0, 0),
    "more_rows_than_keys": ("bf16", 2, "dense", "dense", [(20, 33), (0, 5), (100, 100)], 0, 0),
    "split": ("bf16", 1, "joint", "dense", [(9000, 40)], 0, 0),
    "split_f16": ("f16", 2, "dense", "pad", [(5003, 150), (70, 70)], 0, 0),
    "window": ("bf16", 2, "joint", "dense", [(700, 700), (40, 40), (1200, 33)], 64, 4),
    "window_odd": ("f16", 2, "dense", "dense", [(777, 300), (333, 333)], 101, 17),
    "window_1": ("bf16", 1, "dense", "dense", [(90, 90)], 1, 0),
    "window_first_big": ("bf16", 1, "dense", "dense", [(400, 400)], 40, 100),
    "many": ("bf16", 1, "dense", "dense", [(i % 7, i % 7) for i in range(90)], 0, 0),
}


@pytest.mark.parametrize("name", list(CASES))
def test_prompt(name):
    dt, H, rhow, how, seqs, window, first = CASES[name]
    print(f"[case] prompt {name}", flush=True)
    rng = np.random.default_rng(len(name) * 7 + H)
    rows = Rows(rng, dt, H, [k for k, _ in seqs], rhow)
    m = [n for _, n in seqs]
    q = _q(rng, sum(m), H, D + R, dt)
    scale = (D + R) ** -0.5
    out, lse = run(rows, m, q, window, first, scale, how)
    want = want_of(rows, m, q, window, first, scale)
    check(lse, want[1], want[3], "lse")
    print("  worst error / bar: %.3f" % check(out, want[0], want[2], "out"), flush=True)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_values_that_are_not_finite(dt):
    """Infinities and NaN in later tokens: they reach the rows that see them and
    no others."""
    rng = np.random.default_rng(5)
    rows = Rows(rng, dt, 2, [150, 60])
    for j, x in [(140, float("inf")), (141, float("-inf")), (145, float("nan")), (149, 1e5)]:
        rows.host["v"][j, 0, 3:90:7] = x
    rows.host["v"][150 + 59, 1, 5] = float("nan")
    rows.host["k"][150 + 58, 0, 5] = float("inf")
    rows.host["v"] = rows.host["v"].to(DT[dt]).double()
    rows.upload()
    q = _q(rng, 210, 2, D + R, dt)
    out, lse = run(rows, [150, 60], q, 0, 0, 0.07)
    with np.errstate(invalid="ignore"):
        want = want_of(rows, [150, 60], q, 0, 0, 0.07)
    odd = np.zeros(210, bool)
    odd[[208, 209]] = True               # a key that is not finite: NaN, or out of the sum
    check(out[~odd], want[0][~odd], want[2][~odd], "out")
    check(lse[~odd], want[1][~odd], want[3][~odd], "lse")


def test_rows_outside_the_lists_and_graph():
    """Rows of q around the list's are not written; a captured call takes the
    lengths of the time."""
    rng = np.random.default_rng(6)
    rows = Rows(rng, "bf16", 3, [90, 70])
    q = _q(rng, 200, 3, D + R, "bf16")
    qd = torch.from_numpy(q).to("cuda", torch.bfloat16)
    out = torch.full((200, 3, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((200, 3), 7.0, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    cu_q, cu_k = torch.tensor([20, 110, 180], **i32), torch.tensor([0, 90, 160], **i32)
    ws = torch.empty(max(16, M.moe_attn_latent_prompt_workspace_size(2, 200, 3)),
                     dtype=torch.uint8, device="cuda")
    call = lambda: M.moe_attn_latent_prompt(qd, rows.k, rows.r, rows.v, cu_q, cu_k,  # noqa: E731
                                            out, 0.07, ws, lse=lse)
    call()
    want = want_of(rows, [90, 70], q[20:180], 0, 0, 0.07)
    torch.cuda.synchronize()
    check(out[20:180].double().cpu().numpy(), want[0], want[2], "out")
    for x in (out, lse):
        assert (x[:20] == 7).all() and (x[180:] == 7).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for m, lens in [([50, 60], [80, 60]), ([1, 0], [3, 100]), ([90, 70], [90, 70])]:
        cu_q.copy_(torch.tensor([20, 20 + m[0], 20 + sum(m)]))
        cu_k.copy_(torch.tensor([0, lens[0], sum(lens)]))
        out.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        replayed = out.clone()
        call()
        torch.cuda.synchronize()
        assert torch.equal(out, replayed)
        part = Rows.__new__(Rows)
        part.dt, part.H, part.lens = "bf16", 3, lens
        part.cu, part.host = np.array([0, lens[0], sum(lens)]), rows.host
        want = want_of(part, m, q[20:20 + sum(m)], 0, 0, 0.07)
        check(replayed[20:20 + sum(m)].double().cpu().numpy(), want[0], want[2], "out")


def test_no_keys_and_no_rows():
    """Calls without a key, and sequences without keys or rows among others."""
    i32 = dict(dtype=torch.int32, device="cuda")
    b = dict(dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(16, M.moe_attn_latent_prompt_workspace_size(4, 80, 3)),
                     dtype=torch.uint8, device="cuda")
    q, out = torch.randn(3, 3, 192, **b), torch.full((3, 3, 128), 7.0, **b)
    lse = torch.full((3, 3), 7.0, device="cuda")
    none = torch.empty(0, 3, 128, **b)
    M.moe_attn_latent_prompt(q, none, torch.empty(0, 64, **b), none,
                             torch.tensor([0, 1, 3], **i32), torch.tensor([0, 0, 0], **i32), out,
                             0.07, ws, lse=lse)
    assert (out == 0).all() and (lse == -np.inf).all()
    rng = np.random.default_rng(8)
    rows = Rows(rng, "bf16", 3, [5, 0, 70, 9])
    q = _q(rng, 75, 3, D + R, "bf16")
    out, lse = run(rows, [5, 3, 67, 0], q, 0, 0, 0.07)
    want = want_of(rows, [5, 3, 67, 0], q, 0, 0, 0.07)
    check(out, want[0], want[2], "out")
    check(lse, want[1], want[3], "lse")
    assert (out[5:8] == 0).all() and (lse[5:8] == -np.inf).all()
