"""Loads that end at a bound carry their whole offset in the lane.

The bound of a raw buffer load is compared with the lane's offset; the scalar
offset is added to the address, and where it exceeds the bound the comparison does
not say what is read. The attention over dense rows (moe_attn_latent_prompt) ends
each sequence by that bound, and over a latent cache it makes zeros of keys without
a page, so the offset of a row may not be partly a scalar. Read off the assembly of
the kernels as they are built, without a GPU."""
import os
import re
import subprocess

import pytest

from mixture_experts_expert_sigmoid_amd import build as B

LOAD = re.compile(r"^\s*buffer_load_dwordx4 v\d+, s\[\d+:\d+\], (\S+) offen lds", re.M)


@pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="no hipcc")
@pytest.mark.parametrize("source", ["attn_dense_128", "attn_latent_256"])
def test_no_scalar_offset(source, tmp_path):
    out = tmp_path / "out.s"
    subprocess.run([B.HIPCC, *B.FLAGS, "--cuda-device-only", "-S",
                    os.path.join(B.CSRC, source + ".hip"), "-o", str(out)], check=True)
    scalar = LOAD.findall(out.read_text())
    assert len(scalar) > 20, "the loads look otherwise"
    assert set(scalar) == {"0"}, sorted(set(scalar))
