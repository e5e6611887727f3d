// Gradients of linear attention with decays (linear_attn.h): one pass from the last chunk
// of a segment to the first for dk and dv, one from the first to the last for dq and dg.
#include "linear_attn.h"

namespace zm {

namespace {

// Sum over the four lane groups of a column.
__device__ __forceinline__ float group_sum(float x) {
  x += __shfl_xor(x, 16, 64);
  return x + __shfl_xor(x, 32, 64);
}

// Sum of the lanes before, and of all up to this one, of 16.
__device__ __forceinline__ float prefix16(float x, int c) {
#pragma unroll
  for (int m = 1; m < 16; m *= 2) {
    const float o = __shfl_up(x, m, 16);
    if (c >= m) x += o;
  }
  return x;
}

// An output element with its factor times the same element of a token tensor's row in
// memory or LDS, summed over the wave's columns.
template <int D, bool F32>
__device__ __forceinline__ float dot_row(const f32x4* o, const typename Tok<F32>::T* row) {
  constexpr int CT = LinCfg<D, F32>::CT;
  float s = 0.f;
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    float x[4];
    if constexpr (F32) {
      const f32x4 v = *(const f32x4*)(row + 4 * ct);
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] = v[r];
    } else {
      const u32x2 v = *(const u32x2*)(row + 4 * ct);
      x[0] = bf16lo(v[0]);
      x[1] = bf16hi(v[0]);
      x[2] = bf16lo(v[1]);
      x[3] = bf16hi(v[1]);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) s = fmaf(o[ct][r], x[r], s);
  }
  return s;
}

// ---- dk, dv --------------------------------------------------------------------
// One workgroup to a (segment, head), four waves each for dv (state D) and dk (D^T).
// The dk waves leave D^T at the chunk's end for the other pass.
template <int D, bool F32>
__global__ __launch_bounds__(512) void k_linear_dkdv(LinArgs a) {
  using C = LinCfg<D, F32>;
  using T = typename Tok<F32>::T;
  __shared__ __attribute__((aligned(16))) uint16_t lds[4 * C::TILE + 2 * C::TRI];
  __shared__ LinFactors fac;
  __shared__ float crossing[kLinWaves][64], going[kLinWaves][64];
  const int h = blockIdx.x % a.heads;
  const LinSeg sg = lin_seg(a.sq, blockIdx.x / a.heads);
  if (sg.count < 0) return;
  const int wave = threadIdx.x >> 6, side = wave >> 2, w = wave & 3;  // side 1: dk
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int hk = h / (a.heads / a.heads_k);
  uint16_t* const q = lds;
  uint16_t* const k = q + C::TILE;
  uint16_t* const v = k + C::TILE;
  uint16_t* const od = v + C::TILE;
  uint16_t* const tri = od + C::TILE + side * C::TRI;
  const uint16_t* const ta = side ? v : k;
  const uint16_t* const tb = side ? od : q;
  const uint16_t* const tc = side ? q : od;
  LinState<D, F32> st;
  const int64_t own = ((int64_t)sg.seq * a.heads + h) * D * D;
  const float* const from = sg.flags != 3 ? a.part[1] + ((int64_t)sg.slot * a.heads + h) * D * D
                            : a.dstate_out ? a.dstate_out + own : nullptr;
  if (!from) st.zero();
  else if (side) st.template load<true>(from, w, g, c);
  else st.template load<false>(from, w, g, c);
  const int n = (sg.count + C::CH - 1) / C::CH;
  if (n > 0) {
    const T* const qp = (const T*)a.q.p + (int64_t)sg.tok * a.q.ld + hk * D;
    const T* const kp = (const T*)a.k.p + (int64_t)sg.tok * a.k.ld + hk * D;
    const T* const vp = (const T*)a.v.p + (int64_t)sg.tok * a.v.ld + h * D;
    const T* const dp = (const T*)a.d_o.p + (int64_t)sg.tok * a.d_o.ld + h * D;
    const float* const gp = a.g ? a.g + (int64_t)sg.tok * a.ld_g + h : nullptr;
    // a half of the waves fetches q and k, the other v and dO
    const LinTokens t0 = side ? a.v : a.q, t1 = side ? a.d_o : a.k;
    const T* const p0 = side ? vp : qp;
    const T* const p1 = side ? dp : kp;
    LinFetch<D, F32, 256> f0, f1;
    float gl = 0.f;
    auto fetch = [&](int j) {
      const int at = j * C::CH, count = sg.count - at < C::CH ? sg.count - at : C::CH;
      f0.load(p0 + (int64_t)at * t0.ld, t0.ld, count);
      f1.load(p1 + (int64_t)at * t1.ld, t1.ld, count);
      gl = gp && lane < count ? gp[(int64_t)(at + lane) * a.ld_g] : 0.f;
      return count;
    };
    int next = fetch(n - 1);
    for (int j = n - 1; j >= 0; --j) {
      const int count = next;
      const int64_t tok0 = (int64_t)sg.tok + (int64_t)j * C::CH;
      if (wave == 3) lin_factors<true>(&fac, gl, a.scale);
      f0.store(side ? v : q, count);
      f1.store(side ? od : k, count);
      __syncthreads();
      if (j > 0) next = fetch(j - 1);
      // wave w the source tokens of row tile w
      float cross[C::IT] = {};
      for (int jt = w; jt < 2 * C::TS; jt += kLinWaves) {
        const int ts = jt >> 1;
        float before[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int it = 0; it < C::IT; ++it) {
          if (!lin_in<D, F32, true>(it, ts)) continue;
          const f32x4 x = lin_gate<true>(lin_tri<D, F32>(ta, tb, it, jt, g, c), &fac, a.scale, it, jt, g, c);
          lin_put(tri, C::FRAGS, lin_frag<D, F32, true>(it, ts), jt, lane, x);
          if (side && a.flow) {
            // of source i's row of X, what comes from tokens before t = 16 it + c, if t <= i
            const f32x4 y = lin_tri<D, F32>(k, q, it, jt, g, c);
            float sum = 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float p = prefix16(x[r] * y[r], c);
              const float up = __shfl_up(p, 1, 16);
              const float pre = before[r] + (c ? up : 0.f);
              if (token_row(jt, 4 * g) + r >= 16 * it + c) sum += pre;
              before[r] += __shfl(p, 15, 16);
            }
            cross[it] += group_sum(sum);
          }
        }
      }
      LinOut<D, F32> out;
      out.read(st, ta, &fac, g, c);
      if (a.flow) {
        if (side) {
          float* const dump = a.d_dump + (((int64_t)sg.chunk0 + j) * a.heads + h) * D * D + w * (C::MT * C::CT * 256) + 4 * lane;
#pragma unroll
          for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
            for (int ct = 0; ct < C::CT; ++ct) *(f32x4*)(dump + (mt * C::CT + ct) * 256) = st.m[mt][ct];
          if (g == 0)
#pragma unroll
            for (int it = 0; it < C::IT; ++it) crossing[w][16 * it + c] = cross[it];
        } else {
#pragma unroll
          for (int it = 0; it < C::IT; ++it) {
            const int row = 16 * it + c < count ? 16 * it + c : count - 1;
            const float s = group_sum(dot_row<D, F32>(out.o[it], vp + ((int64_t)j * C::CH + row) * a.v.ld + lin_col0<D>(w, g)));
            if (g == 0) going[w][16 * it + c] = 16 * it + c < count ? s : 0.f;
          }
        }
      }
      st.scale(fac.last);
      __syncthreads();
      lin_tokens<D, F32, true, true>(&out, st, tri, tb, tc, &fac, w, lane, g, c);
      if (!side) {
        out.store((T*)a.dv + tok0 * a.ld_dv + h * D, a.ld_dv, count, w, g, c);
      } else if (a.dk_part) {
        out.store(a.dk_part + (tok0 * a.heads + h) * D, (int64_t)a.heads * D, count, w, g, c);
      } else {
        out.store((T*)a.dk + tok0 * a.ld_dk + hk * D, a.ld_dk, count, w, g, c);
      }
      if (a.flow && wave == 0) {
        float x = 0.f, y = 0.f;
        if (lane < C::CH)
#pragma unroll
          for (int i = 0; i < kLinWaves; ++i) {
            x += crossing[i][lane];
            y += going[i][lane];
          }
        float all = y;
#pragma unroll
        for (int m = 1; m < 64; m *= 2) {
          const float o = __shfl_up(all, m, 64);
          if (lane >= m) all += o;
        }
        const float up = __shfl_up(all, 1, 64);
        if (lane < count) a.flow[(tok0 + lane) * a.heads + h] = x + (lane ? up : 0.f);
      }
      __syncthreads();
    }
  }
  if ((sg.flags & 1) && a.dstate_in && !side) st.store(a.dstate_in + own, w, g, c);
}

// ---- dq, dg ----------------------------------------------------------------------
template <int D, bool F32>
__global__ __launch_bounds__(256, D == 128 && F32 ? 1 : 2) void k_linear_dq(LinArgs a) {
  using C = LinCfg<D, F32>;
  using T = typename Tok<F32>::T;
  __shared__ __attribute__((aligned(16))) uint16_t lds[3 * C::TILE + C::TRI];
  __shared__ LinFactors fac;
  __shared__ float coming[kLinWaves][64], through[kLinWaves];
  const int h = blockIdx.x % a.heads;
  const LinSeg sg = lin_seg(a.sq, blockIdx.x / a.heads);
  if (sg.count <= 0) return;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int hk = h / (a.heads / a.heads_k);
  uint16_t* const od = lds;
  uint16_t* const v = od + C::TILE;
  uint16_t* const k = v + C::TILE;
  uint16_t* const tri = k + C::TILE;
  LinState<D, F32> st;
  const int64_t own = ((int64_t)sg.seq * a.heads + h) * D * D;
  if (sg.flags != 3) st.template load<true>(a.part[0] + ((int64_t)sg.slot * a.heads + h) * D * D, w, g, c);
  else if (a.state_in) st.template load<true>(a.state_in + own, w, g, c);
  else st.zero();
  const int n = (sg.count + C::CH - 1) / C::CH;
  const T* const qp = (const T*)a.q.p + (int64_t)sg.tok * a.q.ld + hk * D;
  const T* const kp = (const T*)a.k.p + (int64_t)sg.tok * a.k.ld + hk * D;
  const T* const vp = (const T*)a.v.p + (int64_t)sg.tok * a.v.ld + h * D;
  const T* const dp = (const T*)a.d_o.p + (int64_t)sg.tok * a.d_o.ld + h * D;
  const float* const gp = a.g ? a.g + (int64_t)sg.tok * a.ld_g + h : nullptr;
  LinFetch<D, F32, 256> fd, fv, fk;
  float gl = 0.f;
  auto fetch = [&](int j) {
    const int t0 = j * C::CH, count = sg.count - t0 < C::CH ? sg.count - t0 : C::CH;
    fd.load(dp + (int64_t)t0 * a.d_o.ld, a.d_o.ld, count);
    fv.load(vp + (int64_t)t0 * a.v.ld, a.v.ld, count);
    fk.load(kp + (int64_t)t0 * a.k.ld, a.k.ld, count);
    gl = gp && lane < count ? gp[(int64_t)(t0 + lane) * a.ld_g] : 0.f;
    return count;
  };
  int next = fetch(0);
  for (int j = 0; j < n; ++j) {
    const int count = next;
    const int64_t tok0 = (int64_t)sg.tok + (int64_t)j * C::CH;
    if (w == 3) lin_factors<false>(&fac, gl, a.scale);
    fd.store(od, count);
    fv.store(v, count);
    fk.store(k, count);
    __syncthreads();
    if (j + 1 < n) next = fetch(j + 1);
    for (int t = w; t < 2 * C::FRAGS; t += kLinWaves) {
      const int f = t >> 1;
      const int it = C::CH == 32 || f < 2 ? f : 2 + (f - 2) / 2, ts = C::CH == 32 || f < 2 ? 0 : (f - 2) & 1;
      const int jt = 2 * ts + (t & 1);
      const f32x4 x = lin_gate<false>(lin_tri<D, F32>(od, v, it, jt, g, c), &fac, a.scale, it, jt, g, c);
      lin_put(tri, C::FRAGS, f, jt, lane, x);
    }
    LinOut<D, F32> out;
    out.read(st, od, &fac, g, c);
    if (a.flow) {
      const float* const dump = a.d_dump + (((int64_t)sg.chunk0 + j) * a.heads + h) * D * D + w * (C::MT * C::CT * 256) + 4 * lane;
      float e = 0.f;
#pragma unroll
      for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
        for (int ct = 0; ct < C::CT; ++ct) {
          const f32x4 x = *(const f32x4*)(dump + (mt * C::CT + ct) * 256);
#pragma unroll
          for (int r = 0; r < 4; ++r) e = fmaf(st.m[mt][ct][r], x[r], e);
        }
#pragma unroll
      for (int m = 1; m < 64; m *= 2) e += __shfl_xor(e, m, 64);
      if (lane == 0) through[w] = e;
#pragma unroll
      for (int it = 0; it < C::IT; ++it) {
        const int row = 16 * it + c < count ? 16 * it + c : count - 1;
        const float s = group_sum(dot_row<D, F32>(out.o[it], qp + ((int64_t)j * C::CH + row) * a.q.ld + lin_col0<D>(w, g)));
        if (g == 0) coming[w][16 * it + c] = 16 * it + c < count ? s : 0.f;
      }
    }
    st.scale(fac.last);
    __syncthreads();
    lin_tokens<D, F32, false, true>(&out, st, tri, v, k, &fac, w, lane, g, c);
    if (a.o_part) out.store(a.o_part + (tok0 * a.heads + h) * D, (int64_t)a.heads * D, count, w, g, c);
    else out.store((T*)a.o + tok0 * a.ld_o + hk * D, a.ld_o, count, w, g, c);
    if (a.flow && w == 0) {
      float x = 0.f, e = 0.f;
#pragma unroll
      for (int i = 0; i < kLinWaves; ++i) {
        x += lane < C::CH ? coming[i][lane] : 0.f;
        e += through[i];
      }
#pragma unroll
      for (int m = 1; m < 64; m *= 2) {
        const float o = __shfl_down(x, m, 64);
        if (lane + m < 64) x += o;
      }
      const float d = lane < count ? a.flow[(tok0 + lane) * a.heads + h] + x + e * fac.last : 0.f;
      if (a.ld_g) {
        if (lane < count) a.dg[(tok0 + lane) * a.heads + h] = d;
      } else {
        float s = d;
#pragma unroll
        for (int m = 1; m < 64; m *= 2) s += __shfl_xor(s, m, 64);
        if (lane == 0) a.dg[((int64_t)sg.chunk0 + j) * a.heads + h] = s;
      }
    }
    __syncthreads();
  }
}

// ---- sums ------------------------------------------------------------------------
// Eight elements a thread: the value heads of a key head in order.  Rows outside the
// sequences are left as they are.
template <typename T>
__global__ __launch_bounds__(256) void k_linear_groups(const float* x, T* y, int64_t ldy, LinSeqs sq, int heads,
                                                       int heads_k, int d) {
  const int per = heads_k * d / 8, rep = heads / heads_k;
  const int2 range = lin_range(sq);
  const int64_t all = (int64_t)(range.y - range.x) * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
    const int64_t t = range.x + i / per;
    const int col = 8 * (int)(i % per), hk = col / d, e = col % d;
    const float* const p = x + (t * heads + (int64_t)hk * rep) * d + e;
    float s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = p[j];
    for (int r = 1; r < rep; ++r)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] += p[(int64_t)r * d + j];
    T* const to = y + t * ldy + col;
    if constexpr (sizeof(T) == 4) {
      *(f32x4*)to = f32x4{s[0], s[1], s[2], s[3]};
      *(f32x4*)(to + 4) = f32x4{s[4], s[5], s[6], s[7]};
    } else {
      *(u32x4*)to = u32x4{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]), pack_bf16x2(s[4], s[5]),
                          pack_bf16x2(s[6], s[7])};
    }
  }
}

// A workgroup to a head; the chunks' sums in 64 bits, always in the same order.
__global__ __launch_bounds__(256) void k_linear_decay_sum(const float* sums, LinSeqs sq, int heads, float* dg) {
  __shared__ double red[4];
  const int2 range = sq.segs || sq.n_seq == 0 ? int2{0, 0} : lin_range(sq);
  const int chunks = sq.segs ? sq.of_seq[sq.n_seq + 1].x : lin_chunks(sq, range.y - range.x);
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < chunks; i += 256) s += (double)sums[i * heads + blockIdx.x];
#pragma unroll
  for (int m = 1; m < 64; m *= 2) s += __shfl_xor(s, m, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) dg[blockIdx.x] = (float)(red[0] + red[1] + red[2] + red[3]);
}

template <int D>
hipError_t dkdv_any(const LinArgs& a, bool f32, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.sq.n_segs * a.heads)), blk(512);
  if (f32) hipLaunchKernelGGL((k_linear_dkdv<D, true>), grid, blk, 0, st, a);
  else hipLaunchKernelGGL((k_linear_dkdv<D, false>), grid, blk, 0, st, a);
  return hipGetLastError();
}

template <int D>
hipError_t dq_any(const LinArgs& a, bool f32, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.sq.n_segs * a.heads)), blk(256);
  if (f32) hipLaunchKernelGGL((k_linear_dq<D, true>), grid, blk, 0, st, a);
  else hipLaunchKernelGGL((k_linear_dq<D, false>), grid, blk, 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_dkdv(const LinArgs& a, int d, bool f32, hipStream_t st) {
  return d == 128 ? dkdv_any<128>(a, f32, st) : dkdv_any<64>(a, f32, st);
}

hipError_t launch_linear_dq(const LinArgs& a, int d, bool f32, hipStream_t st) {
  return d == 128 ? dq_any<128>(a, f32, st) : dq_any<64>(a, f32, st);
}

hipError_t launch_linear_groups(const float* x, void* y, int64_t ld_y, const LinArgs& a, int d, bool f32,
                                hipStream_t st) {
  int64_t blocks = ceil_div((int64_t)a.sq.n * (a.heads_k * d / 8), 256);
  if (blocks > 8 * kTargetWgs) blocks = 8 * kTargetWgs;
  if (f32) hipLaunchKernelGGL((k_linear_groups<float>), dim3((unsigned)blocks), dim3(256), 0, st, x, (float*)y, ld_y,
                              a.sq, a.heads, a.heads_k, d);
  else hipLaunchKernelGGL((k_linear_groups<uint16_t>), dim3((unsigned)blocks), dim3(256), 0, st, x, (uint16_t*)y, ld_y,
                          a.sq, a.heads, a.heads_k, d);
  return hipGetLastError();
}

hipError_t launch_linear_decay_sum(const float* sums, const LinSeqs& s, int heads, float* dg, hipStream_t st) {
  hipLaunchKernelGGL(k_linear_decay_sum, dim3(heads), dim3(256), 0, st, sums, s, heads, dg);
  return hipGetLastError();
}

}  // namespace zm
