"""Two builds of the library in one process, each loaded as the binding loads it: neither calls
the other's functions."""
import os
import shutil
import subprocess
import sys

from token_indexed_ffn_amd import _lib as L

PROGRAM = """
import ctypes, sys
import torch   # the HIP runtime
for path in sys.argv[1:]:
    lib = ctypes.CDLL(path, mode=ctypes.RTLD_GLOBAL)
    lib.staple_status_string.restype = ctypes.c_char_p
    assert lib.staple_status_string(0)
print("loaded")
"""


def test_a_second_build_binds_to_itself(tmp_path):
    other = tmp_path / "libstaple.so"
    shutil.copy(L.LIB_PATH, other)
    # every binding at once, and what the loader says of each
    env = dict(os.environ, LD_BIND_NOW="1", LD_DEBUG="bindings")
    r = subprocess.run([sys.executable, "-c", PROGRAM, str(other), L.LIB_PATH], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "loaded" in r.stdout, r.stderr[-2000:]
    ours = [x for x in r.stderr.splitlines() if f"binding file {L.LIB_PATH} " in x]
    assert ours
    crossed = [x for x in ours if f" to {other} " in x]
    assert not crossed, f"{len(crossed)} of {len(ours)}: {crossed[0]}"
