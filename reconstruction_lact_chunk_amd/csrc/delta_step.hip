// One token of each sequence (delta_rule.h): with w = a S k per row of S,
//   u = b (v - a S k),  S' = a S + u k^T,  o = scale S' q = scale (a S q + u (k.q)).
// Bound by the states' traffic: a row is read once and written once, both dots
// with k and q are taken on the way in.  16 lanes hold a row (D / 16 columns a
// lane), so a wave covers 4 rows at a time and the dots end in 4 exchanges.  256
// sequences, 8 heads of 128 (272 MB): 54 us a call over changing states, 5 TB/s, and 41 us where
// the same ones come again, part of them from cache; one sequence 4.5 us, a launch.
#include "delta_rule.h"

namespace zm {

namespace {

constexpr int kStepRows = 8;  // rows of a 16-lane group: 32 a wave

__device__ __forceinline__ float tok(const uint16_t* p) { return __uint_as_float((unsigned)*p << 16); }
__device__ __forceinline__ float tok(const float* p) { return *p; }
__device__ __forceinline__ void put(uint16_t* p, float x) { *p = to_bf16(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }

// One wave per (sequence, head, 32 rows): blockIdx.x enumerates them in that order.
template <int D, bool F32>
__global__ __launch_bounds__(64) void k_delta_step(DeltaStepArgs a) {
  using T = typename Tok<F32>::T;
  constexpr int E = D / 16, PART = D / 32;
  const int rb = blockIdx.x % PART;
  const int64_t sh = blockIdx.x / PART;
  const int h = (int)(sh % a.heads);
  const int64_t seq = sh / a.heads;
  const int grp = threadIdx.x >> 4, c = threadIdx.x & 15;
  const int hk = h / (a.heads / a.heads_k);
  const T* const kp = (const T*)a.k.p + seq * a.k.ld + hk * D;
  const T* const qp = (const T*)a.q.p + seq * a.q.ld + hk * D;
  float k[E], q[E], kq = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int col = 4 * c + 64 * (e / 4) + e % 4;
    k[e] = tok(kp + col);
    q[e] = tok(qp + col);
    kq = fmaf(k[e], q[e], kq);
  }
#pragma unroll
  for (int x = 1; x < 16; x *= 2) kq += __shfl_xor(kq, x, 64);
  const float al = expf(a.g[seq * a.heads + h]), b = a.beta[seq * a.heads + h];
  float* const sp = a.state + (seq * a.heads + h) * (int64_t)D * D;
  f32x4 s[kStepRows][E / 4];
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const int row = 32 * rb + 4 * i + grp;
#pragma unroll
    for (int e = 0; e < E / 4; ++e) s[i][e] = *(const f32x4*)(sp + (int64_t)row * D + 4 * c + 64 * e);
  }
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const int row = 32 * rb + 4 * i + grp;
    float dk = 0.f, dq = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float x = s[i][e / 4][e % 4] * al;
      s[i][e / 4][e % 4] = x;
      dk = fmaf(x, k[e], dk);
      dq = fmaf(x, q[e], dq);
    }
#pragma unroll
    for (int x = 1; x < 16; x *= 2) {
      dk += __shfl_xor(dk, x, 64);
      dq += __shfl_xor(dq, x, 64);
    }
    const float u = b * (tok((const T*)a.v.p + seq * a.v.ld + h * D + row) - dk);
#pragma unroll
    for (int e = 0; e < E; ++e) s[i][e / 4][e % 4] = fmaf(u, k[e], s[i][e / 4][e % 4]);
#pragma unroll
    for (int e = 0; e < E / 4; ++e) *(f32x4*)(sp + (int64_t)row * D + 4 * c + 64 * e) = s[i][e];
    if (c == 0) put((T*)a.o + seq * a.ld_o + h * D + row, a.scale * fmaf(u, kq, dq));
  }
}

}  // namespace

hipError_t launch_delta_step(const DeltaStepArgs& a, hipStream_t st) {
  if (a.n_seq == 0) return hipSuccess;
  const dim3 grid((unsigned)((int64_t)a.n_seq * a.heads * (a.d / 32))), blk(64);
  if (a.d == 128) {
    if (a.f32) hipLaunchKernelGGL((k_delta_step<128, true>), grid, blk, 0, st, a);
    else hipLaunchKernelGGL((k_delta_step<128, false>), grid, blk, 0, st, a);
  } else {
    if (a.f32) hipLaunchKernelGGL((k_delta_step<64, true>), grid, blk, 0, st, a);
    else hipLaunchKernelGGL((k_delta_step<64, false>), grid, blk, 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace zm
