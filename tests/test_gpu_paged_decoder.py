"""The paged decoder example: every attention call within its bound of a dense
recomputation, through prompts, chunks, forks, trims, frees and a compaction."""
import importlib.util
import os

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_session(kv):
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "paged_decoder.py")
    spec = importlib.util.spec_from_file_location("paged_decoder", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    print(f"[case] paged decoder {kv}", flush=True)
    dec, text, used = ex.session(kv, check=True)
    assert 0.0 < dec.dense.worst <= 1.0
    assert sorted(text) == [0, 1, 2, 4]
    assert len(text[0]) == 41 and all(len(text[s]) == 51 for s in (1, 2, 4))
    # 5 + 3 + 10 pages of 16; 191 tokens fill 12, the last of them half: copied
    assert used["prompts"] == 18 and used["fork"] == 21
    # a slot keeps its first page and at most 7 that 96 tokens reach into
    assert used["steps"] <= 4 * 8 and used["free"] < used["steps"]
    table, refs = dec.cache.table.cpu(), dec.cache.refs.cpu()
    ids, count = table[table >= 0].unique(return_counts=True)
    assert torch.equal(refs[ids].long(), count) and int(refs.sum()) == int(count.sum())
