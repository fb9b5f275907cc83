"""Batches without a sequence or a row: the workspace they ask for, and the calls of
the cache objects, which ask for it first."""
import os
import subprocess
import sys

import pytest
import torch

import mixture_experts_expert_sigmoid_amd as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SIZES = {
    "decode": "L.moe_attn_decode_workspace_size(kv, 0, 8)",
    "prefill": "L.moe_attn_prefill_workspace_size(kv, 0, 0, 8)",
    "prefill, no rows": "L.moe_attn_prefill_workspace_size(kv, 3, 0, 8)",
    "tree": "L.moe_attn_tree_workspace_size(kv, 0, 0, 8)",
    "tree, no rows": "L.moe_attn_tree_workspace_size(kv, 3, 0, 8)",
    "latent": "L.moe_attn_latent_workspace_size(lat, 0, 0, 8)",
    "prompt": "L.moe_attn_latent_prompt_workspace_size(0, 0, 8)",
    "prompt, no rows": "L.moe_attn_latent_prompt_workspace_size(3, 0, 8)",
    "cache": "L.moe_cache_workspace_size(t, 0)",
    "gate": "L.moe_gate_route_workspace_size(0, 256, 64, 2)",
    "permute": "L.moe_permute_workspace_size(0, 8, 64)",
}
# in a process of its own, which a fault on the host ends; the last name is the case
CODE = """
import ctypes, sys
sys.path.insert(0, {root!r})
import mixture_experts_expert_sigmoid_amd as M
from tests.test_cache_abi import _c, _t
from tests.test_draft_abi import _lc
L, t, lat = M.lib(), ctypes.byref(_t()), ctypes.byref(_lc())
kv = ctypes.byref(_c(head_dim={dim}, stride_page=8192, stride_head=4096, stride_tok={dim}))
for name, call in {sizes!r}.items():
    print(name, flush=True)
    assert eval(call) >= 0
"""


@pytest.mark.skipif(not os.path.exists(M.LIB_PATH), reason="library not built")
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_sizes(dim):
    code = CODE.format(root=ROOT, sizes=SIZES, dim=dim)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stdout, r.stderr[-500:])
    assert r.stdout.splitlines() == list(SIZES)


def _empty(*shape, dt=torch.bfloat16):
    return torch.empty(shape, dtype=dt, device="cuda")


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_calls(dim):
    """No sequences at all, and sequences without a row."""
    kv = M.KvCache(n_layers=1, n_pages=4, page_size=16, n_heads=2, head_dim=dim, n_slots=3,
                   max_pages=2)
    lat = M.LatentCache(n_layers=1, n_pages=4, page_size=16, n_slots=3, max_pages=2)
    for n in (0, 3):
        slots = torch.arange(n, dtype=torch.int32, device="cuda")
        cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
        none = _empty(0, dt=torch.int32)
        q, x = _empty(0, 8, dim), _empty(0, 2, dim)
        for c in (kv, lat):
            assert c.grow(slots, cu[:n]).tolist() == [0] * n
            c.keep(slots, cu[:n], cu, none)
        kv.append(0, slots, cu[:n], cu, x, x)
        outs = [kv.prefill(0, slots, q, cu, 0.1), kv.tree(0, slots, q, cu, none, 0.1)]
        lat.append(0, slots, cu[:n], cu, _empty(0, 512), _empty(0, 64))
        ql, qp = _empty(0, 8, 576), _empty(0, 8, 192)
        outs += [lat.attend(0, slots, ql, cu, 0.1), lat.attend(0, slots, ql, cu, 0.1, parent=none),
                 lat.prompt(qp, _empty(0, 8, 128), _empty(0, 64), _empty(0, 8, 128), cu, cu, 0.1),
                 lat.prompt(qp, _empty(5, 8, 128), _empty(5, 64), _empty(5, 8, 128), cu, cu, 0.1)]
        if n == 0:
            outs += [kv.decode(0, slots, q, 0.1), lat.attend(0, slots, ql, None, 0.1)]
        assert all(y.shape[0] == 0 for y in outs)
    torch.cuda.synchronize()
    for c in (kv, lat):
        assert M.moe_read_device_error(c.err_word) == 0 and c.lens.tolist() == [0] * 3
