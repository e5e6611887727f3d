"""Lists of many tensors clipped by a thread with a stack of 192 KB, on the CPU: the list is refused for an
overlap, which is found after all of its places have been looked at."""
import os
import subprocess
import sys

import pytest

import reconstruction_lact_chunk_amd as zm

pytestmark = pytest.mark.skipif(not os.path.exists(zm.LIB_PATH),
                                reason="libzmttt.so not built (run the build first)")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import ctypes, sys, threading
sys.path.insert(0, {root!r})
import reconstruction_lact_chunk_amd as zm
lib, out = zm.load_library(), []

def run(count):
    rows = [zm.Tensor((1 << 20) + 64 * i, (1 << 30) + 64 * i, 8, zm.F32, 0) for i in range(count)]
    rows[0].y = rows[-1].y + 4
    t = (zm.Tensor * count)(*rows)
    p = ctypes.c_void_p(1 << 40)
    out.append(lib.zm_clip_grads(t, count, 1.0, p, ctypes.c_void_p(1 << 41), 1 << 30, None))

threading.stack_size(192 << 10)
for count in (3, 511, 512, 8192):
    th = threading.Thread(target=run, args=(count,))
    th.start()
    th.join()
print(out)
"""


def test_many_tensors_on_a_small_stack():
    r = subprocess.run([sys.executable, "-c", PROGRAM.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, f"{r.returncode}: {r.stderr[-2000:]}"
    assert r.stdout.split("\n")[-2] == str([zm.ERR_INVALID_ARG] * 4), r.stdout
