// One token of each sequence (linear_attn.h): S' = a S + v k^T, o = scale S' q.
// Bound by the states' traffic: a row is read once and written once, its dot with q is
// taken on the way.  16 lanes hold a row (D / 16 columns a lane), so a wave covers 4 rows
// at a time and a dot ends in 4 exchanges.  256 sequences, 8 heads of 128 (272 MB): 54 us a call over
// changing states, 5 TB/s, and 41 us where the same ones come again, part of them from cache;
// one sequence 4.5 us, a launch.
#include "linear_attn.h"

namespace zm {

namespace {

constexpr int kStepRows = 8;  // rows of a 16-lane group: 32 a wave

__device__ __forceinline__ float tok(const uint16_t* p) { return __uint_as_float((unsigned)*p << 16); }
__device__ __forceinline__ float tok(const float* p) { return *p; }
__device__ __forceinline__ void put(uint16_t* p, float x) { *p = to_bf16(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }

// One wave per (sequence, head, 32 rows): blockIdx.x enumerates them in that order.
template <int D, bool F32>
__global__ __launch_bounds__(64) void k_linear_step(LinStepArgs a) {
  using T = typename Tok<F32>::T;
  constexpr int E = D / 16, PART = D / 32;
  const int rb = blockIdx.x % PART;
  const int64_t sh = blockIdx.x / PART;
  const int h = (int)(sh % a.heads);
  const int64_t seq = sh / a.heads;
  const int grp = threadIdx.x >> 4, c = threadIdx.x & 15;
  const int hk = h / (a.heads / a.heads_k);
  float* const sp = a.state + ((seq * a.heads + h) * D + 32 * rb + grp) * (int64_t)D + 4 * c;
  f32x4 s[kStepRows][E / 4];
#pragma unroll
  for (int i = 0; i < kStepRows; ++i)
#pragma unroll
    for (int e = 0; e < E / 4; ++e) s[i][e] = *(const f32x4*)(sp + 4 * i * D + 64 * e);
  const T* const kp = (const T*)a.k.p + seq * a.k.ld + hk * D;
  const T* const qp = (const T*)a.q.p + seq * a.q.ld + hk * D;
  const T* const vp = (const T*)a.v.p + seq * a.v.ld + h * D + 32 * rb + grp;
  float k[E], q[E], v[kStepRows];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int col = 4 * c + 64 * (e / 4) + e % 4;
    k[e] = tok(kp + col);
    q[e] = tok(qp + col);
  }
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) v[i] = tok(vp + 4 * i);
  const float al = a.g ? expf(a.g[seq * a.ld_g + h]) : 1.f;
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    float dq = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float x = fmaf(v[i], k[e], s[i][e / 4][e % 4] * al);
      s[i][e / 4][e % 4] = x;
      dq = fmaf(x, q[e], dq);
    }
#pragma unroll
    for (int x = 1; x < 16; x *= 2) dq += __shfl_xor(dq, x, 64);
#pragma unroll
    for (int e = 0; e < E / 4; ++e) *(f32x4*)(sp + 4 * i * D + 64 * e) = s[i][e];
    if (c == 0) put((T*)a.o + seq * a.ld_o + h * D + 32 * rb + 4 * i + grp, a.scale * dq);
  }
}

}  // namespace

hipError_t launch_linear_step(const LinStepArgs& a, int d, bool f32, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.n_seq * a.heads * (d / 32))), blk(64);
  if (d == 128) {
    if (f32) hipLaunchKernelGGL((k_linear_step<128, true>), grid, blk, 0, st, a);
    else hipLaunchKernelGGL((k_linear_step<128, false>), grid, blk, 0, st, a);
  } else {
    if (f32) hipLaunchKernelGGL((k_linear_step<64, true>), grid, blk, 0, st, a);
    else hipLaunchKernelGGL((k_linear_step<64, false>), grid, blk, 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace zm
