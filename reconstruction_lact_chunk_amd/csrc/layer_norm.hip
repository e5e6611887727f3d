// Layer norm of token rows and its gradient:
//   mu = mean(x), v = mean((x - mu)^2), r = 1 / sqrt(v + eps), xh = (x - mu) r,
//   y = xh gamma + beta;
//   a = dy gamma, dx = r (a - mean(a) - xh mean(a xh)),
//   dgamma = sum over rows of dy xh, dbeta = sum over rows of dy.
// Both are bound by memory (8 and 14 operations an element).  A row is loaded
// once into the registers of WPR waves (16-byte pieces, piece p of a lane at
// element E (lane + 64 WPR p)), so the variance is the mean of the squared
// distances from the mean and not a difference of two large sums.
#include "seq_ops.h"

namespace zm {

namespace {

constexpr int kNormWaves = 4;  // waves of a workgroup
// Workgroups of the forward pass: 4 to a compute unit go over the rows, gamma and beta
// in registers and the next row read ahead.  40001 fp32 rows of 2048 (655 MB): 121 us,
// 5.4 TB/s; 127 with gamma and beta by single loads, and so 128 with 8 workgroups, 133
// with 6, 192 with one to every two rows, 220 with that and both read for every row.
// 1374 bf16 rows of 1024: 4.3 us, about what an empty launch takes.
constexpr int64_t kMaxNormBlocks = kTargetWgs * 4;

template <typename T>
struct Piece;
template <>
struct Piece<uint16_t> {
  static constexpr int E = 8;
  typedef u32x4 Raw;
  static __device__ __forceinline__ void load(const uint16_t* p, float* v) {
    unpack(*(const u32x4*)p, v);
  }
  static __device__ __forceinline__ void unpack(u32x4 w, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16lo(w[i]);
      v[2 * i + 1] = bf16hi(w[i]);
    }
  }
  static __device__ __forceinline__ void store(uint16_t* p, const float* v) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    *(u32x4*)p = w;
  }
};
template <>
struct Piece<float> {
  static constexpr int E = 4;
  typedef f32x4 Raw;
  static __device__ __forceinline__ void load(const float* p, float* v) {
    unpack(*(const f32x4*)p, v);
  }
  static __device__ __forceinline__ void unpack(f32x4 w, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = w[i];
  }
  static __device__ __forceinline__ void store(float* p, const float* v) {
    *(f32x4*)p = f32x4{v[0], v[1], v[2], v[3]};
  }
};

// E elements of a vector from c on, or `other` without one and past its end.
template <int E>
__device__ __forceinline__ void load_or(const float* p, int c, int width, float other, float* v) {
  f32x4 w[E / 4];
#pragma unroll
  for (int i = 0; i < E / 4; ++i) w[i] = f32x4{other, other, other, other};
  if (p && c < width) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) w[i] = *(const f32x4*)(p + c + 4 * i);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = w[e / 4][e % 4];
}

// Sum over the WPR waves of a row, the same bits in every lane.  red: one
// float per wave, of two buffers that alternate from call to call, so that one
// barrier a call is enough.
template <int WPR>
__device__ __forceinline__ float row_sum(float s, float* red) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) s += __shfl_xor(s, m, 64);
  if constexpr (WPR > 1) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[w] = s;
    __syncthreads();
    const int w0 = w / WPR * WPR;
    s = red[w0];
#pragma unroll
    for (int i = 1; i < WPR; ++i) s += red[w0 + i];
  }
  return s;
}

template <typename T, int WPR, int NP>
__global__ __launch_bounds__(64 * kNormWaves) void k_layer_norm(
    const T* x, int64_t ldx, const float* __restrict__ gamma,
    const float* __restrict__ beta, float eps, T* y, int64_t ldy, float* __restrict__ stats,
    int width, int64_t n) {
  constexpr int E = Piece<T>::E, RPG = kNormWaves / WPR;
  typedef typename Piece<T>::Raw Raw;
  __shared__ float red[4][kNormWaves];
  const int lane = threadIdx.x % (64 * WPR), row = threadIdx.x / (64 * WPR);
  const float inv = 1.f / (float)width;
  const int64_t step = (int64_t)gridDim.x * RPG;
  int64_t t0 = (int64_t)blockIdx.x * RPG;
  Raw raw[NP];
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = E * (lane + 64 * WPR * p);
      if (t < n && c < width) raw[p] = *(const Raw*)(x + t * ldx + c);
    }
  };
  fetch(t0 + row);
  float gm[NP][E], bt[NP][E];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int c = E * (lane + 64 * WPR * p);
    load_or<E>(gamma, c, width, 1.f, gm[p]);
    load_or<E>(beta, c, width, 0.f, bt[p]);
  }
  int turn = 0;
  for (; t0 < n; t0 += step, turn ^= 2) {
    const int64_t t = t0 + row;  // a wave past the rows still meets the barriers
    float v[NP][E];
    float s = 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      if (t < n && E * (lane + 64 * WPR * p) < width) {
        Piece<T>::unpack(raw[p], v[p]);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) v[p][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) s += v[p][e];
    }
    fetch(t + step);
    const float mean = row_sum<WPR>(s, red[turn]) * inv;
    s = 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const bool in = E * (lane + 64 * WPR * p) < width;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        v[p][e] -= mean;
        if (in) s = fmaf(v[p][e], v[p][e], s);
      }
    }
    const float r = 1.f / sqrtf(row_sum<WPR>(s, red[turn + 1]) * inv + eps);
    if (t >= n) continue;
    if (stats && lane == 0) {
      stats[t] = mean;
      stats[n + t] = r;
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = E * (lane + 64 * WPR * p);
      if (c >= width) break;
#pragma unroll
      for (int e = 0; e < E; ++e) v[p][e] = fmaf(v[p][e] * r, gm[p][e], bt[p][e]);
      Piece<T>::store(y + t * ldy + c, v[p]);
    }
  }
}

// A workgroup takes every gridDim-th group of kNormWaves / WPR rows and keeps
// its lanes' columns of dgamma and dbeta in registers over all of them; at the
// end its waves add theirs in order through LDS and the sums go to the
// workgroup's slot, which k_norm_param_sum adds in order (no atomics).  137400 bf16 rows
// of 1024 (844 MB): 153 us, 5.5 TB/s, and 5 us for the sum of the slots; 40001 fp32 rows of 2048
// (983 MB) 209 us, 4.7 TB/s.  A row has a wave at least, so narrow ones are far from the memory's
// rate: 1200000 bf16 rows of 64 take 408 us (forward 330), 1.1 TB/s, 300000 of 256 132 us (89).
template <typename T, int WPR, int NP>
__global__ __launch_bounds__(64 * kNormWaves) void k_layer_norm_backward(
    const T* dy, int64_t lddy, const T* x, int64_t ldx, const float* __restrict__ gamma,
    const float* __restrict__ stats, T* dx, int64_t lddx, float* __restrict__ part, int width,
    int64_t n) {
  constexpr int E = Piece<T>::E, RPG = kNormWaves / WPR;
  extern __shared__ float sums[];  // 2 x width, with part and several rows to a workgroup
  __shared__ float red[4][kNormWaves];
  const int lane = threadIdx.x % (64 * WPR), row = threadIdx.x / (64 * WPR);
  float dg[NP][E] = {}, db[NP][E] = {}, gm[NP][E];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int c = E * (lane + 64 * WPR * p);
    load_or<E>(gamma, c, width, 1.f, gm[p]);
  }
  const float inv = 1.f / (float)width;
  int turn = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * RPG; t0 < n; t0 += (int64_t)gridDim.x * RPG, turn ^= 2) {
    const int64_t t = t0 + row;
    const bool live = t < n;
    float xh[NP][E], a[NP][E];
    const float mean = live ? stats[t] : 0.f, r = live ? stats[n + t] : 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = E * (lane + 64 * WPR * p);
      if (live && c < width) {
        Piece<T>::load(x + t * ldx + c, xh[p]);
        Piece<T>::load(dy + t * lddy + c, a[p]);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          xh[p][e] = mean;
          a[p][e] = 0.f;
        }
      }
    }
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        xh[p][e] = (xh[p][e] - mean) * r;
        dg[p][e] = fmaf(a[p][e], xh[p][e], dg[p][e]);
        db[p][e] += a[p][e];
        a[p][e] *= gm[p][e];
        s0 += a[p][e];
        s1 = fmaf(a[p][e], xh[p][e], s1);
      }
    s0 = row_sum<WPR>(s0, red[turn]) * inv;
    s1 = row_sum<WPR>(s1, red[turn + 1]) * inv;
    if (!live) continue;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = E * (lane + 64 * WPR * p);
      if (c >= width) break;
#pragma unroll
      for (int e = 0; e < E; ++e) a[p][e] = r * (a[p][e] - s0 - xh[p][e] * s1);
      Piece<T>::store(dx + t * lddx + c, a[p]);
    }
  }
  if (!part) return;
  float* const out = part + (int64_t)blockIdx.x * 2 * width;
  if constexpr (RPG == 1) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int c = E * (lane + 64 * WPR * p);
      if (c >= width) break;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        out[c + e] = dg[p][e];
        out[width + c + e] = db[p][e];
      }
    }
    return;
  }
#pragma unroll
  for (int w = 0; w < RPG; ++w) {
    if (w == row) {
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int c = E * (lane + 64 * WPR * p);
        if (c >= width) break;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          sums[c + e] = (w ? sums[c + e] : 0.f) + dg[p][e];
          sums[width + c + e] = (w ? sums[width + c + e] : 0.f) + db[p][e];
        }
      }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < 2 * width; c += 64 * kNormWaves) out[c] = sums[c];
}

// dgamma | dbeta from the slots: 16 columns x 64 groups of slots a workgroup, each
// group's slots in order and then the groups in order.
__global__ __launch_bounds__(1024) void k_norm_param_sum(const float* __restrict__ part, int slots,
                                                         int width, float* __restrict__ dgamma,
                                                         float* __restrict__ dbeta) {
  __shared__ float red[64][17];
  const int col = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + col;  // 2 * width is a multiple of 16
  float s = 0.f;
#pragma unroll 4
  for (int i = grp; i < slots; i += 64) s += part[(int64_t)i * 2 * width + c];
  red[grp][col] = s;
  __syncthreads();
  if (grp < 8) {
    s = red[8 * grp][col];
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[8 * grp + i][col];
    red[8 * grp][col] = s;
  }
  __syncthreads();
  if (grp) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) s += red[8 * i][col];
  float* const out = c < width ? dgamma : dbeta;
  if (out) out[c < width ? c : c - width] = s;
}

template <typename T, int WPR, int NP>
hipError_t norm_launch(const void* x, int64_t ldx, const float* gamma, const float* beta, float eps,
                       void* y, int64_t ldy, float* stats, int width, int64_t n, hipStream_t st) {
  int64_t blocks = ceil_div(n, kNormWaves / WPR);
  if (blocks > kMaxNormBlocks) blocks = kMaxNormBlocks;
  hipLaunchKernelGGL((k_layer_norm<T, WPR, NP>), dim3((unsigned)blocks), dim3(64 * kNormWaves), 0, st, (const T*)x, ldx, gamma, beta, eps, (T*)y, ldy,
                     stats, width, n);
  return hipGetLastError();
}

template <typename T, int WPR, int NP>
hipError_t norm_backward_launch(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                const float* gamma, const float* stats, void* dx, int64_t lddx,
                                float* part, int width, int64_t n, hipStream_t st) {
  hipLaunchKernelGGL((k_layer_norm_backward<T, WPR, NP>), dim3(norm_slots(n)),
                     dim3(64 * kNormWaves), part && WPR < kNormWaves ? 2 * width * sizeof(float) : 0, st, (const T*)dy,
                     lddy, (const T*)x, ldx, gamma, stats, (T*)dx, lddx, part, width, n);
  return hipGetLastError();
}

// Waves and pieces to a row: one wave up to 4 pieces a lane, then more waves.
#define ZM_NORM_SHAPE(F, T, ...)                                         \
  do {                                                                   \
    const int pieces = (width + 64 * Piece<T>::E - 1) / (64 * Piece<T>::E); \
    if (pieces <= 1) return F<T, 1, 1>(__VA_ARGS__);                     \
    if (pieces <= 2) return F<T, 1, 2>(__VA_ARGS__);                     \
    if (pieces <= 4) return F<T, 1, 4>(__VA_ARGS__);                     \
    if (pieces <= 8) return F<T, 2, 4>(__VA_ARGS__);                     \
    if (pieces <= 16) return F<T, 4, 4>(__VA_ARGS__);                    \
    return F<T, 4, 8>(__VA_ARGS__);                                      \
  } while (0)

hipError_t norm_backward_any(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                             const float* gamma, const float* stats, void* dx, int64_t lddx,
                             float* part, int width, int64_t n, bool f32, hipStream_t st) {
  if (f32)
    ZM_NORM_SHAPE(norm_backward_launch, float, dy, lddy, x, ldx, gamma, stats, dx, lddx, part,
                  width, n, st);
  ZM_NORM_SHAPE(norm_backward_launch, uint16_t, dy, lddy, x, ldx, gamma, stats, dx, lddx, part,
                width, n, st);
}

}  // namespace

hipError_t launch_layer_norm(const void* x, int64_t ldx, const float* gamma, const float* beta,
                             float eps, void* y, int64_t ldy, float* stats, int width, int64_t n,
                             bool f32, hipStream_t st) {
  if (n == 0) return hipSuccess;
  if (f32) ZM_NORM_SHAPE(norm_launch, float, x, ldx, gamma, beta, eps, y, ldy, stats, width, n, st);
  ZM_NORM_SHAPE(norm_launch, uint16_t, x, ldx, gamma, beta, eps, y, ldy, stats, width, n, st);
}

hipError_t launch_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                      const float* gamma, const float* stats, void* dx,
                                      int64_t lddx, float* dgamma, float* dbeta, float* part,
                                      int width, int64_t n, bool f32, hipStream_t st) {
  const bool params = dgamma || dbeta;
  if (n > 0) {
    const hipError_t e = norm_backward_any(dy, lddy, x, ldx, gamma, stats, dx, lddx,
                                           params ? part : nullptr, width, n, f32, st);
    if (e != hipSuccess) return e;
  }
  if (!params) return hipSuccess;
  hipLaunchKernelGGL(k_norm_param_sum, dim3(2 * width / 16), dim3(1024), 0, st, part,
                     n > 0 ? norm_slots(n) : 0, width, dgamma, dbeta);
  return hipGetLastError();
}

}  // namespace zm
