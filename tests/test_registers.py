"""The vector registers that the attention kernels need beyond a lane's own: what is
spilled goes through memory in loops that are bound by their instructions."""
import os
import re
import subprocess

import pytest

from token_indexed_ffn_amd import build as B


@pytest.mark.parametrize("source", ["attn.hip", "attn_f32.hip", "attn_decode.hip"])
def test_attention_kernels_keep_their_vector_registers(source, tmp_path):
    try:
        hipcc = B.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    out = tmp_path / "listing.s"
    r = subprocess.run([hipcc] + B.compile_flags() + ["-S", "--cuda-device-only", os.path.join(B.CSRC, source), "-o", str(out)],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    # the kernels' metadata: names and spills in one order
    text = out.read_text()
    names = re.findall(r"^\s+\.symbol:\s+(\S+)\.kd", text, re.M)
    spills = [int(n) for n in re.findall(r"^\s+\.vgpr_spill_count:\s+(\d+)", text, re.M)]
    assert len(names) == len(spills) > 0
    # one of the fp32 forward of wide heads, in its end
    assert all(n <= 1 for n in spills), {k: n for k, n in zip(names, spills) if n}
