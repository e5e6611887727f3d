// Launchers of the operators around a streamed token sequence: layer norm
// (layer_norm.hip), multi-axis rotary positions (rotary.hip) and both on the heads
// of q and k (norm_rotary.hip).
#pragma once

#include "zm_internal.h"

namespace zm {

// ---- layer norm ---------------------------------------------------------------
constexpr int kMaxNormWidth = 8192;
// Workgroups of the backward, each with a partial sum of the parameter
// gradients: at least 16 rows to one, and at most four to a compute unit.
inline int norm_slots(int64_t n) {
  const int64_t s = ceil_div(n, 16);
  return (int)(s > 4 * kTargetWgs ? 4 * kTargetWgs : s);
}
hipError_t launch_layer_norm(const void* x, int64_t ldx, const float* gamma, const float* beta,
                             float eps, void* y, int64_t ldy, float* stats, int width, int64_t n,
                             bool f32, hipStream_t st);
// part: norm_slots(n) x 2 x width floats (dgamma, dbeta), unused if both are null.
hipError_t launch_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                      const float* gamma, const float* stats, void* dx,
                                      int64_t lddx, float* dgamma, float* dbeta, float* part,
                                      int width, int64_t n, bool f32, hipStream_t st);

// ---- rotary positions -----------------------------------------------------------
constexpr int kMaxAxes = 4;
struct RotaryTensor {
  const void* x;
  void* y;
  int64_t ldx, ldy;
  int heads;
};
struct RotaryArgs {
  RotaryTensor q, k;
  const void* pos;       // int32 or fp32 [n][axes]
  const float* freqs;    // [pairs]
  int64_t n;
  int d, pairs, axes, layout;
  int first[kMaxAxes + 1];  // axis a owns pairs first[a] .. first[a + 1] - 1
  bool f32, pos_f32, inverse;
};
hipError_t launch_rotary(const RotaryArgs& a, hipStream_t st);

// ---- heads normalised and rotated -------------------------------------------------
struct NormRotaryArgs {
  RotaryArgs r;             // forward: x to y; backward: x and the gradient's rows, below
  const float* gamma[2];    // of q, k: [d] or null (ones)
  const float* beta[2];     // or null (zeros)
  float eps;
  bool layer;               // layer norm, else RMS norm
  // backward
  const void* dy[2];        // gradients of the rotated rows, strides r.q.ldy, r.k.ldy
  void* dx[2];
  int64_t lddx[2];
  float* part;              // norm_rotary_slots(..) x 4 x d: sums for gamma q, beta q, gamma k, beta k
  bool params;              // some of dparam is wanted
  float* dparam[4];         // those sums, each may be null
};
// Workgroups of the backward at most, each with a partial sum of the parameter gradients.
constexpr int kNormRotarySlots = 4 * kTargetWgs;
inline int64_t norm_rotary_slots(int64_t n, int heads) {
  const int64_t s = n * heads;
  return s < kNormRotarySlots ? s : kNormRotarySlots;
}
hipError_t launch_norm_rotary(const NormRotaryArgs& a, hipStream_t st);
hipError_t launch_norm_rotary_backward(const NormRotaryArgs& a, hipStream_t st);

}  // namespace zm
