// The global norm of many tensors and their clipping by it (grad_clip.hip).
#pragma once

#include "zm_internal.h"

namespace zm {

// Tensors of one launch: its arguments hold them, so that no table has to be copied to the
// device (a captured launch keeps it); 3.6 KB of the 4 KB of arguments.
constexpr int kClipTensors = 128;
constexpr int kClipPieceBytes = 16 * 1024;      // of one type's elements, a step of a workgroup
constexpr int kClipBlocks = 4 * kTargetWgs;     // workgroups of a launch at most, each with a partial sum

struct ClipTable {
  const void* x[kClipTensors];
  void* y[kClipTensors];
  int64_t n[kClipTensors];
  uint32_t first[kClipTensors + 1];  // pieces before a tensor's; the last: all
  uint32_t f32[kClipTensors / 32];
  int32_t count;
};
constexpr int64_t clip_pieces(int64_t n, bool f32) {
  // from the 16-byte word of the first element on
  return n > 0 ? (n * (f32 ? 4 : 2) + 14) / kClipPieceBytes + 1 : 0;
}
inline int clip_blocks(int64_t pieces) { return (int)(pieces < kClipBlocks ? pieces : kClipBlocks); }

// The table's sum of squares into clip_blocks(pieces) partial sums.
hipError_t launch_grad_squares(const ClipTable& t, double* part, hipStream_t st);
// The norm from all `count` partial sums.
hipError_t launch_grad_norm(const double* part, int count, float* norm, hipStream_t st);
// y = x min(1, max_norm / (norm + 1e-6)) over the table, and with `norm` the norm itself.
hipError_t launch_grad_scale(const ClipTable& t, const double* part, int count, float max_norm, float* norm,
                             hipStream_t st);

}  // namespace zm
