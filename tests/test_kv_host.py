"""Host side of the cache and attention bindings, without a GPU."""
import gc
import weakref

import mixture_experts_expert_sigmoid_amd as M


def test_workspaces_stay_when_a_larger_one_is_needed():
    """A captured graph, or work on another stream, may still write to one that
    was handed out."""
    ws = M._Workspace("cpu")
    refs, at = [], set()
    for need in (100, 10, 1000, 1001, 5000):
        buf = ws.get(need)
        assert buf.numel() >= need
        refs.append(weakref.ref(buf))
        at.add(buf.data_ptr())
        del buf
    gc.collect()
    assert all(r() is not None for r in refs)
    assert len(at) == 4 and ws.get(1).numel() >= 5000          # 100, 1000, 2000, 5000
    assert sum(b.numel() for b in ws.buffers) <= 2 * ws.buffers[-1].numel()
