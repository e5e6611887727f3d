// The heads of q and k normalised and rotated by their positions (rotary.hip) in one pass,
// and the gradient.  Per head x of d elements:
//   r = 1 / sqrt(mean((x - mu)^2) + eps),  xh = (x - mu) r  (mu = mean(x), or 0: RMS norm),
//   y = R (xh gamma + beta),
//   u = R^T dy,  a = u gamma,  dx = r (a - xh mean(a xh) [- mean(a)]),
//   dgamma = sum over tokens and heads of u xh,  dbeta of u.
// Bound by memory: q and k are read once (the gradient: with dy) and written once; the
// statistics are formed again in the gradient.  A group of V pairs is a lane's, so that a
// head's row lies in the registers of a power of two of lanes and its sums take
// few exchanges; the angles of a lane's pairs are formed once for all heads of a token.
// 54,960 fp32 tokens of 20 heads of 64: 139 us, 4.1 TB/s; gradient of 137,400 bf16 tokens of 16 heads
// of 128: 338 us, 5.0 TB/s; one frame of 1374 tokens 8 us from the caches and 9 from memory, loads,
// angles and exchanges one after the other.  Stores past the caches gave 3 to 5% for 8 + 8 heads and
// whole rotations (that gradient 328 us) and cost 3 to 30% for other heads and sections (those fp32
// tokens 151 us): not taken.
#include "rotary_dev.h"

namespace zm {

namespace {

constexpr int64_t kMaxBlocks = 1 << 20;  // more tokens than these take are looped over

template <int W>
struct Which {
  static constexpr int value = W;  // 0 q, 1 k
};

struct Plan {
  int groups;      // V-pair groups of a row: rotated ones, then the unrotated tail
  int turned;      // rotated ones among them
  int lanes;       // of a row, a power of two
  int heads_each;  // heads of one thread
};

// Sum over the `lanes` lanes of a row, the same bits in each.
__device__ __forceinline__ float dpp_add(float x, int moved) { return x + __int_as_float(moved); }
__device__ __forceinline__ float row_sum(float x, int lanes) {
  // exchanges within four, eight and sixteen lanes do not pass through LDS
  if (lanes > 1) x = dpp_add(x, __builtin_amdgcn_mov_dpp(__float_as_int(x), 0xb1, 0xf, 0xf, true));   // 1 0 3 2
  if (lanes > 2) x = dpp_add(x, __builtin_amdgcn_mov_dpp(__float_as_int(x), 0x4e, 0xf, 0xf, true));   // 2 3 0 1
  if (lanes > 4) x = dpp_add(x, __builtin_amdgcn_mov_dpp(__float_as_int(x), 0x141, 0xf, 0xf, true));  // half mirrored
  if (lanes > 8) x = dpp_add(x, __builtin_amdgcn_mov_dpp(__float_as_int(x), 0x140, 0xf, 0xf, true));  // mirrored
  if (lanes > 16) x += __shfl_xor(x, 16, 64);
  if (lanes > 32) x += __shfl_xor(x, 32, 64);
  return x;
}

// A lane's NG groups of a row: elements c0 .. + V and c1 .. + V of each.
template <typename T, int V, int NG>
struct Row {
  Vec<T, V> e[NG][2];
  __device__ __forceinline__ void load(const T* p, const int (*c)[2], const bool* in) {
#pragma unroll
    for (int i = 0; i < NG; ++i)
      if (in[i])
#pragma unroll
        for (int s = 0; s < 2; ++s) e[i][s] = load_v<T, V>(p + c[i][s]);
  }
  __device__ __forceinline__ void get(float (*x)[2][V], const bool* in) const {
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < V; ++j) x[i][s][j] = in[i] ? to_f(e[i][s].e[j]) : 0.f;
  }
};
template <typename T, int V, int NG>
__device__ __forceinline__ void put_row(T* p, const float (*x)[2][V], const int (*c)[2], const bool* in) {
#pragma unroll
  for (int i = 0; i < NG; ++i)
    if (in[i])
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        Vec<T, V> v;
#pragma unroll
        for (int j = 0; j < V; ++j) v.e[j] = from_f<T>(x[i][s][j]);
        store_v<T, V>(p + c[i][s], v);
      }
}
template <int V, int NG>
__device__ __forceinline__ void get_param(float (*x)[2][V], const float* p, float other, const int (*c)[2], const bool* in) {
#pragma unroll
  for (int i = 0; i < NG; ++i)
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (p && in[i]) {
        const Vec<float, V> v = load_v<float, V>(p + c[i][s]);
#pragma unroll
        for (int j = 0; j < V; ++j) x[i][s][j] = v.e[j];
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) x[i][s][j] = other;
      }
    }
}

// (x - mu) in x, and r.
template <int V, int NG>
__device__ __forceinline__ float normalise(float (*x)[2][V], bool layer, float inv, float eps, const bool* in, int lanes) {
  if (layer) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) s += x[i][k][j];
    const float mu = row_sum(s, lanes) * inv;
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) x[i][k][j] = in[i] ? x[i][k][j] - mu : 0.f;
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NG; ++i)
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) s = fmaf(x[i][k][j], x[i][k][j], s);
  return 1.f / sqrtf(row_sum(s, lanes) * inv + eps);
}

template <typename T, int V, bool ADJ, int NG>
__global__ __launch_bounds__(256) void k_norm_rotary(NormRotaryArgs a, Plan pl) {
  const RotaryArgs& r = a.r;
  const int row = threadIdx.x / pl.lanes, lane = threadIdx.x - row * pl.lanes, rows = 256 / pl.lanes;
  int c[NG][2];
  bool in[NG], turn[NG];
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const int grp = lane + i * pl.lanes;
    in[i] = grp < pl.groups;
    turn[i] = grp < pl.turned;
    rotary_runs<V, ADJ>(r, pl.turned, in[i] ? grp : 0, c[i][0], c[i][1]);
  }
  const int all = r.q.heads + r.k.heads, h0 = blockIdx.y * pl.heads_each;
  const int h1 = h0 + pl.heads_each < all ? h0 + pl.heads_each : all;
  const float inv = 1.f / (float)r.d;
  for (int64_t t = (int64_t)blockIdx.x * rows + row; t < r.n; t += (int64_t)gridDim.x * rows) {
    auto src = [&](int h) {
      return h < r.q.heads ? (const T*)r.q.x + t * r.q.ldx + (int64_t)h * r.d
                           : (const T*)r.k.x + t * r.k.ldx + (int64_t)(h - r.q.heads) * r.d;
    };
    // the first head's elements are on their way while the angles are formed
    Row<T, V, NG> next;
    next.load(src(h0), c, in);
    float co[NG][V], si[NG][V], gm[NG][2][V], bt[NG][2][V];
#pragma unroll
    for (int i = 0; i < NG; ++i)
      if (turn[i]) rotary_angles<V>(r, t, (lane + i * pl.lanes) * V, co[i], si[i]);
    for (int h = h0; h < h1; ++h) {
      const int which = h >= r.q.heads;
      if (h == h0 || h == r.q.heads) {
        get_param<V, NG>(gm, a.gamma[which], 1.f, c, in);
        get_param<V, NG>(bt, a.beta[which], 0.f, c, in);
      }
      float x[NG][2][V];
      next.get(x, in);
      if (h + 1 < h1) next.load(src(h + 1), c, in);
      const float s = normalise<V, NG>(x, a.layer, inv, a.eps, in, pl.lanes);
#pragma unroll
      for (int i = 0; i < NG; ++i) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int j = 0; j < V; ++j) x[i][k][j] = fmaf(x[i][k][j] * s, gm[i][k][j], bt[i][k][j]);
        if (turn[i]) rotary_turn<V, ADJ>(x[i][0], x[i][1], co[i], si[i]);
      }
      T* const y = which ? (T*)r.k.y + t * r.k.ldy + (int64_t)(h - r.q.heads) * r.d
                         : (T*)r.q.y + t * r.q.ldy + (int64_t)h * r.d;
      put_row<T, V, NG>(y, x, c, in);
    }
  }
}

// Workgroups go over the tokens and keep their lanes' columns of dgamma and dbeta in
// registers; at the end the lanes of the same columns add theirs, then the waves in order
// through LDS, and the sums go to the workgroup's slot, which k_norm_rotary_params adds in
// order (no atomics).
template <typename T, int V, bool ADJ, int NG>
__global__ __launch_bounds__(256, V == 4 ? 4 : 1) void k_norm_rotary_backward(NormRotaryArgs a, Plan pl) {
  const RotaryArgs& r = a.r;
  extern __shared__ float sums[];  // [4 waves][4][d], with params
  const int row = threadIdx.x / pl.lanes, lane = threadIdx.x - row * pl.lanes, rows = 256 / pl.lanes;
  int c[NG][2];
  bool in[NG], turn[NG];
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    const int grp = lane + i * pl.lanes;
    in[i] = grp < pl.groups;
    turn[i] = grp < pl.turned;
    rotary_runs<V, ADJ>(r, pl.turned, in[i] ? grp : 0, c[i][0], c[i][1]);
  }
  const int all = r.q.heads + r.k.heads, h0 = blockIdx.y * pl.heads_each;
  const int h1 = h0 + pl.heads_each < all ? h0 + pl.heads_each : all;
  const float inv = 1.f / (float)r.d;
  float dg[2][NG][2][V] = {}, db[2][NG][2][V] = {};
  for (int64_t t = (int64_t)blockIdx.x * rows + row; t < r.n; t += (int64_t)gridDim.x * rows) {
    float co[NG][V], si[NG][V];
    auto heads = [&](auto which, int from, int to) {  // heads from .. to - 1 of q or k
      constexpr int W = decltype(which)::value;
      if (from >= to) return;
      const RotaryTensor& m = W ? r.k : r.q;
      const T* const xp = (const T*)m.x + t * m.ldx;
      const T* const yp = (const T*)a.dy[W] + t * m.ldy;
      T* const dp = (T*)a.dx[W] + t * a.lddx[W];
      Row<T, V, NG> nx, ny;
      nx.load(xp + (int64_t)from * r.d, c, in);
      ny.load(yp + (int64_t)from * r.d, c, in);
      float gm[NG][2][V];
      get_param<V, NG>(gm, a.gamma[W], 1.f, c, in);
      if (!W || h0 >= r.q.heads) {  // once to a token
#pragma unroll
        for (int i = 0; i < NG; ++i)
          if (turn[i]) rotary_angles<V>(r, t, (lane + i * pl.lanes) * V, co[i], si[i]);
      }
      for (int h = from; h < to; ++h) {
        float x[NG][2][V], u[NG][2][V];
        nx.get(x, in);
        ny.get(u, in);
        if (h + 1 < to) {
          nx.load(xp + (int64_t)(h + 1) * r.d, c, in);
          ny.load(yp + (int64_t)(h + 1) * r.d, c, in);
        }
        const float s = normalise<V, NG>(x, a.layer, inv, a.eps, in, pl.lanes);
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          if (turn[i]) rotary_turn<V, ADJ>(u[i][0], u[i][1], co[i], si[i]);
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) {
              x[i][k][j] *= s;
              dg[W][i][k][j] = fmaf(u[i][k][j], x[i][k][j], dg[W][i][k][j]);
              db[W][i][k][j] += u[i][k][j];
              u[i][k][j] *= gm[i][k][j];
              s0 += u[i][k][j];
              s1 = fmaf(u[i][k][j], x[i][k][j], s1);
            }
        }
        s0 = a.layer ? row_sum(s0, pl.lanes) * inv : 0.f;
        s1 = row_sum(s1, pl.lanes) * inv;
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) u[i][k][j] = s * (u[i][k][j] - s0 - x[i][k][j] * s1);
        put_row<T, V, NG>(dp + (int64_t)h * r.d, u, c, in);
      }
    };
    const int hq = r.q.heads;
    heads(Which<0>{}, h0, h1 < hq ? h1 : hq);
    heads(Which<1>{}, (h0 > hq ? h0 : hq) - hq, h1 - hq);
  }
  if (!a.params) return;
  const int w = threadIdx.x >> 6;
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float x = dg[which][i][k][j], y = db[which][i][k][j];
          for (int m = pl.lanes; m < 64; m *= 2) {
            x += __shfl_xor(x, m, 64);
            y += __shfl_xor(y, m, 64);
          }
          if ((threadIdx.x & 63) < pl.lanes && in[i]) {
            sums[(w * 4 + 2 * which) * r.d + c[i][k] + j] = x;
            sums[(w * 4 + 2 * which + 1) * r.d + c[i][k] + j] = y;
          }
        }
  __syncthreads();
  float* const out = a.part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 4 * r.d;
  for (int i = threadIdx.x; i < 4 * r.d; i += 256) {
    float s = sums[i];
#pragma unroll
    for (int k = 1; k < 4; ++k) s += sums[k * 4 * r.d + i];
    out[i] = s;
  }
}

// The parameter gradients from the slots: 16 columns x 64 groups of slots a workgroup, each
// group's slots in order and then the groups in order.
__global__ __launch_bounds__(1024) void k_norm_rotary_params(NormRotaryArgs a, int slots) {
  __shared__ float red[64][17];
  const int col = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const int d = a.r.d, c = blockIdx.x * 16 + col;  // 4 d is a multiple of 32
  float s = 0.f;
#pragma unroll 4
  for (int i = grp; i < slots; i += 64) s += a.part[(int64_t)i * 4 * d + c];
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
  const int which = c / d;
  float* out = a.dparam[0];
  if (which == 1) out = a.dparam[1];
  if (which == 2) out = a.dparam[2];
  if (which == 3) out = a.dparam[3];
  if (out) out[c - which * d] = s;
}

template <int V>
Plan plan_of(const RotaryArgs& r) {
  Plan pl;
  pl.turned = r.pairs / V;
  pl.groups = r.d / (2 * V);
  pl.lanes = 1;
  while (pl.lanes < pl.groups && pl.lanes < 64) pl.lanes *= 2;
  pl.heads_each = 0;
  return pl;
}

template <typename T, int V, bool ADJ, int NG>
hipError_t forward_launch(const NormRotaryArgs& a, hipStream_t st) {
  Plan pl = plan_of<V>(a.r);
  const int all = a.r.q.heads + a.r.k.heads;
  // Threads for four waves on each SIMD, as far as the heads can be split: a thread with
  // many heads forms its angles once, one with few starts sooner (one frame from memory: 8.9 us, for eight
  // waves 10.1, for two 8.7, for one 10.0).
  const int64_t want = (int64_t)kTargetWgs * 4 * 4 * 64;
  int64_t splits = ceil_div(want, a.r.n * pl.lanes);
  if (splits > all) splits = all;
  pl.heads_each = (int)ceil_div(all, splits);
  int64_t blocks = ceil_div(a.r.n, 256 / pl.lanes);
  if (blocks > kMaxBlocks) blocks = kMaxBlocks;
  hipLaunchKernelGGL((k_norm_rotary<T, V, ADJ, NG>), dim3((unsigned)blocks, (unsigned)ceil_div(all, pl.heads_each)),
                     dim3(256), 0, st, a, pl);
  return hipGetLastError();
}

template <typename T, int V, bool ADJ, int NG>
hipError_t backward_launch(const NormRotaryArgs& a, hipStream_t st) {
  Plan pl = plan_of<V>(a.r);
  const int all = a.r.q.heads + a.r.k.heads;
  // as many workgroups as there are slots: first by tokens, then by heads
  int64_t blocks = ceil_div(a.r.n, 256 / pl.lanes);
  if (blocks > kNormRotarySlots) blocks = kNormRotarySlots;
  int64_t splits = kNormRotarySlots / blocks;
  if (splits > all) splits = all;
  pl.heads_each = (int)ceil_div(all, splits);
  const unsigned y = (unsigned)ceil_div(all, pl.heads_each);
  hipLaunchKernelGGL((k_norm_rotary_backward<T, V, ADJ, NG>), dim3((unsigned)blocks, y), dim3(256),
                     a.params ? 16 * a.r.d * sizeof(float) : 0, st, a, pl);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.params) return e;
  hipLaunchKernelGGL(k_norm_rotary_params, dim3(4 * a.r.d / 16), dim3(1024), 0, st, a, (int)(blocks * y));
  return hipGetLastError();
}

// Runs of 4 pairs where they fit, else of one: a lane then has one group, or two where a
// head has more than 64 pairs.  Runs of 8 (bf16, 8 + 8 heads of 128, us against runs of 4): one
// frame 10.2 and 8.9, 100 frames 213 and 211, gradients of one frame 30 and 17, of 8 frames 63 and 51, of 100
// frames 323 and 316.
#define ZM_NORM_ROTARY(F, T)                                                                           \
  do {                                                                                                 \
    const bool adj = a.r.layout == 1;                                                                  \
    if (rotary_fits(a.r, 4)) return adj ? F<T, 4, true, 1>(a, st) : F<T, 4, false, 1>(a, st);          \
    if (a.r.d <= 128) return adj ? F<T, 1, true, 1>(a, st) : F<T, 1, false, 1>(a, st);                 \
    return adj ? F<T, 1, true, 2>(a, st) : F<T, 1, false, 2>(a, st);                                   \
  } while (0)

}  // namespace

hipError_t launch_norm_rotary(const NormRotaryArgs& a, hipStream_t st) {
  if (a.r.n == 0) return hipSuccess;
  if (a.r.f32) ZM_NORM_ROTARY(forward_launch, float);
  ZM_NORM_ROTARY(forward_launch, uint16_t);
}

hipError_t launch_norm_rotary_backward(const NormRotaryArgs& a, hipStream_t st) {
  if (a.r.n == 0) {
    if (!a.params) return hipSuccess;
    hipLaunchKernelGGL(k_norm_rotary_params, dim3(4 * a.r.d / 16), dim3(1024), 0, st, a, 0);
    return hipGetLastError();
  }
  if (a.r.f32) ZM_NORM_ROTARY(backward_launch, float);
  ZM_NORM_ROTARY(backward_launch, uint16_t);
}

}  // namespace zm
