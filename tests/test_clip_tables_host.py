"""The tables of tensors that zm_grad_norm and zm_clip_grads hand to their kernels, on the host: the
entry points built with launchers that look at the tables in the kernels' place.  The most that the
header allows (tensors of 2^36 elements, the same one in every place of a table) has to be counted
without an overflow."""
import os
import shutil
import subprocess

import pytest

from reconstruction_lact_chunk_amd import build_lib

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="no hipcc")

PROGRAM = r"""
#include "grad_api.cpp"
#include <stdio.h>
#include <vector>
namespace zm {
static int64_t want, tensors, blocks;
static int bad;
void set_last_error(const char*, ...) {}
static void look(const ClipTable& t) {
  int64_t at = 0;
  for (int i = 0; i < t.count; ++i) {
    if ((int64_t)t.first[i] != at) bad = 1;
    at += clip_pieces(t.n[i], t.f32[i >> 5] >> (i & 31) & 1);
  }
  if ((int64_t)t.first[t.count] != at) bad = 2;
  const int b = clip_blocks(t.first[t.count]);
  if (b < 1 || b > kClipBlocks || b > at) bad = 3;
  tensors += t.count;
  blocks += b;
  want += at;
}
hipError_t launch_grad_squares(const ClipTable& t, double*, hipStream_t) { look(t); return hipSuccess; }
hipError_t launch_grad_norm(const double*, int slots, float*, hipStream_t) { if (slots != blocks) bad = 4; return hipSuccess; }
hipError_t launch_grad_scale(const ClipTable& t, const double*, int slots, float, float*, hipStream_t) {
  look(t);
  return hipSuccess;
}
}
int main() {
  for (int count : {1, 127, 128, 129, 1000}) {
    for (int64_t n : {(int64_t)1, (int64_t)4096, (int64_t)4097, (int64_t)1 << 36}) {
      std::vector<zm_tensor> t;
      for (int i = 0; i < count; ++i) t.push_back(zm_tensor{(void*)0x1000, nullptr, n, n >> 36 || i % 9 ? ZM_F32 : ZM_BF16, 0});
      zm::tensors = zm::blocks = zm::want = 0;
      const int s = zm_grad_norm(t.data(), count, (float*)0x2000, (void*)((size_t)1 << 50), (size_t)1 << 40, nullptr);
      size_t need;
      zm_grad_norm_workspace_size(count, &need);
      if (s != ZM_OK || zm::bad || zm::tensors != count || (size_t)zm::blocks * 8 > need) {
        printf("count %d n %lld: status %d, bad %d, %lld tensors\n", count, (long long)n, s, zm::bad, (long long)zm::tensors);
        return 1;
      }
    }
  }
  return 0;
}
"""


def test_tables_of_the_largest_tensors(tmp_path):
    src, exe = tmp_path / "tables.cpp", tmp_path / "tables"
    src.write_text(PROGRAM)
    cmd = [HIPCC, "-std=c++17", "-O1", f"-I{build_lib.INCLUDE}", f"-I{build_lib.CSRC}", f"--offload-arch={build_lib.ARCH}",
           "-x", "hip", "--offload-host-only", str(src), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
