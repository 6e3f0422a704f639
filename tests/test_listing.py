"""The assembly of the kernels that load into LDS from inline asm.

The compiler keeps the wait states that gfx950 asks for between its own
instructions, but does not look into inline asm.  A memory instruction may read
a scalar register five wait states after a vector instruction wrote it
(v_readlane, v_readfirstlane: a spilled descriptor word, say), and M0 one wait
state after a scalar instruction wrote it; an earlier read takes the old value,
a wild address.  So the listing is searched for a load that comes too early."""
import os
import re
import subprocess

import pytest

from token_indexed_ffn_amd import build as B


def too_early(listing):
    """(loads into LDS, those that read a scalar register too soon)."""
    lines = [x.strip() for x in listing.split("\n")]
    loads, bad = 0, []
    for i, line in enumerate(lines):
        if not re.match(r"(global_load_lds_dword|buffer_load_dword\S* .*\blds$)", line):
            continue
        loads += 1
        regs = re.search(r"s\[(\d+):(\d+)\]", line)
        regs = set(range(int(regs.group(1)), int(regs.group(2)) + 1)) if regs else set()
        states = 0
        for k in range(i - 1, -1, -1):
            x = lines[k]
            if not x or x.startswith((";", ".")) or x.endswith(":"):
                continue
            vector = re.match(r"v_read\w*lane_b32 (?:s(\d+)|(m0))\b", x)
            if vector and (vector.group(2) or int(vector.group(1)) in regs) or re.match(r"s_\w+ m0\b", x) and states < 1:
                bad.append((i, x, line))
            states += 1 + (int(x.split()[1], 0) if x.startswith("s_nop") else 0)
            if states >= 5:
                break
    return loads, bad


def test_too_early_finds_a_load_that_is():
    wait = "\tv_readlane_b32 s5, v1, 3\n\ts_nop {}\n\tbuffer_load_dwordx4 v2, s[4:7], 0 offen lds\n"
    assert too_early(wait.format(4)) == (1, [])
    assert len(too_early(wait.format(3))[1]) == 1
    assert len(too_early("\ts_mov_b32 m0, s3\n\tglobal_load_lds_dwordx4 v[2:3], off\n")[1]) == 1
    assert too_early("\ts_mov_b32 m0, s3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 v[2:3], off\n") == (1, [])


@pytest.mark.parametrize("source", ["attn.hip", "attn_f32.hip", "gemm.hip"])
def test_loads_into_lds_keep_their_wait_states(source, tmp_path):
    try:
        hipcc = B.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    out = tmp_path / "listing.s"
    r = subprocess.run([hipcc] + B.compile_flags() + ["-S", "--cuda-device-only", os.path.join(B.CSRC, source), "-o", str(out)],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    loads, bad = too_early(out.read_text())
    assert loads > 0 and not bad, bad[:3]
