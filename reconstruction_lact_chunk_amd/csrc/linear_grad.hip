// Gradients of linear attention with decays (linear_attn.h): one pass from the last chunk
// of a segment to the first for dk and dv, one from the first to the last for dq and dg.
#include "linear_attn.h"

#include <type_traits>

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

// A lane's four outputs of a token times the same elements of a token tensor: in memory, or in
// a tile.
__device__ __forceinline__ float dot4(const f32x4& o, const f32x4& v) {
  return o[0] * v[0] + o[1] * v[1] + o[2] * v[2] + o[3] * v[3];
}
__device__ __forceinline__ float dot4(const f32x4& o, const u32x2& v) {
  return o[0] * bf16lo(v[0]) + o[1] * bf16hi(v[0]) + o[2] * bf16lo(v[1]) + o[3] * bf16hi(v[1]);
}
template <int D, bool F32>
__device__ __forceinline__ float dot4(const f32x4& o, const uint16_t* tile, int row, int w, int g) {
  using C = LinCfg<D, F32>;
  float s = 0.f;
#pragma unroll
  for (int k = C::NT - 1; k >= 0; --k)
    s += dot4(o, *(const u32x2*)(tile + k * C::PART + lin_at<D, F32>(row, 2 * w + (g >> 1)) + 4 * (g & 1)));
  return s;
}

// ---- dk, dv --------------------------------------------------------------------
// One workgroup to a (segment, head), D / 16 waves each for dv (state D) and dk (D^T).
// The dk waves leave D^T at the chunk's end for the other pass.
template <int D, bool F32>
__global__ __launch_bounds__(8 * D) void k_linear_dkdv(LinArgs a) {
  using C = LinCfg<D, F32>;
  using T = typename Tok<F32>::T;
  __shared__ __attribute__((aligned(16))) uint16_t lds[4 * C::TILE + 2 * C::TRI];
  __shared__ LinFactors fac[2];
  __shared__ float next_decays[64];
  __shared__ float crossing[4][64], going[C::WAVES][64];
  const int h = blockIdx.x % a.heads;
  const LinSeg sg = lin_seg(a.sq, blockIdx.x / a.heads);
  if (sg.count < 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), side = wave / C::WAVES, w = wave % C::WAVES;  // side 1: dk
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
    LinFetch<D, F32> f0, f1;
    auto tokens = [&](int j) { return sg.count - j * C::CH < C::CH ? sg.count - j * C::CH : C::CH; };
    auto decay = [&](int j) {
      return gp && lane < tokens(j) ? gp[(int64_t)(j * C::CH + lane) * a.ld_g] : 0.f;
    };
    auto fetch = [&](int j) {
      const int64_t at = (int64_t)j * C::CH;
      f0.load(p0 + at * t0.ld, (unsigned)t0.ld, tokens(j));
      f1.load(p1 + at * t1.ld, (unsigned)t1.ld, tokens(j));
    };
    const bool mine = wave == 2 * C::WAVES - 1;  // the factors are this wave's, a chunk ahead
    float gl = 0.f;
    fetch(n - 1);
    if (mine) {
      lin_factors<true>(fac + ((n - 1) & 1), nullptr, decay(n - 1), tokens(n - 1), a.scale);
      if (n > 1) gl = decay(n - 2);
    }
    for (int j = n - 1; j >= 0; --j) {
      const int count = tokens(j);
      const int64_t tok0 = (int64_t)sg.tok + (int64_t)j * C::CH;
      if (mine) next_decays[lane] = gl;
      f0.store(side ? v : q);
      f1.store(side ? od : k);
      __syncthreads();
      const LinFactors* const f = fac + (j & 1);
      const int flags = f->flags;
      if (mine && j > 0) lin_factors<true>(fac + (~j & 1), f, next_decays[lane], tokens(j - 1), a.scale);
      if (j > 0) fetch(j - 1);
      if (flags & kLinScale) st.scale(f->pre);
      auto chunk = [&](auto gated) {
        constexpr bool GATED = decltype(gated)::value;
        // wave w < 2 TS the source tokens of row tile w
        float cross[C::IT] = {};
        if (w < 2 * C::TS) {
          const int jt = w, ts = jt >> 1;
          const LinLane l(lane);
          const int g = l.g, c = l.c;
          float before[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int it = 0; it < C::IT; ++it) {
            if (!lin_in<D, F32, true>(it, ts)) continue;
            const f32x4 x = lin_gate<true, GATED>(lin_tri<D, F32>(ta, tb, it, jt, g, c), f, a.scale, it, jt, g, c);
            lin_put(tri, C::FRAGS, lin_frag<D, F32, true>(it, ts), jt, l.lane, x);
            if (side && a.flow) {
              // of source i's row of X, what comes from tokens before t = 16 it + c, if t <= i
              const f32x4 y = lin_tri<D, F32>(k, q, it, jt, g, c);
              const float up = GATED ? 1.f : f->up[16 * it + c];
              float sum = 0.f;
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const float p = prefix16(x[r] * y[r] * up, c);
                const float left = __shfl_up(p, 1, 16);
                if (token_row(jt, 4 * g) + r >= 16 * it + c) sum += before[r] + (c ? left : 0.f);
                before[r] += __shfl(p, 15, 16);
              }
              cross[it] += group_sum(sum);
            }
          }
        }
        LinOut<D, F32> out;
        {
          const LinLane l(lane);
          out.read(st, ta, l.g, l.c);
        }
        if (a.flow) {
          const LinLane l(lane);
          const int g = l.g, c = l.c;
          if (side) {
            if (w == 0 && lane == 0) a.d_exp[((int64_t)sg.chunk0 + j) * a.heads + h] = f->s;
            float* const dump =
                a.d_dump + (((int64_t)sg.chunk0 + j) * a.heads + h) * D * D + w * (C::MT * 256) + 4 * l.lane;
#pragma unroll
            for (int mt = 0; mt < C::MT; ++mt) *(f32x4*)(dump + mt * 256) = st.m[mt];
            if (w < 4 && g == 0)
#pragma unroll
              for (int it = 0; it < C::IT; ++it) crossing[w][16 * it + c] = cross[it];
          } else {
#pragma unroll
            for (int it = 0; it < C::IT; ++it) {
              const int t = 16 * it + c;
              const float x = group_sum(dot4<D, F32>(out.o[it], v, t, w, g));
              if (g == 0) going[w][t] = t < count ? x * f->up[t] : 0.f;
            }
          }
        }
        if (GATED) {
          out.scale(f, c);
          st.scale(f->last);
        }
        __syncthreads();
        const LinLane lt(lane);
        lin_tokens<D, F32, true, true>(&out, st, tri, tb, tc, f, w, lt.lane, lt.g, lt.c);
        const LinLane l(lane);
        if (!GATED) out.scale(f, l.c);
        if (!side) {
          out.store((T*)a.dv + tok0 * a.ld_dv + h * D, (unsigned)a.ld_dv, count, w, l.g, l.c);
        } else if (a.dk_part) {
          out.store(a.dk_part + (tok0 * a.heads + h) * D, (unsigned)(a.heads * D), count, w, l.g, l.c);
        } else {
          out.store((T*)a.dk + tok0 * a.ld_dk + hk * D, (unsigned)a.ld_dk, count, w, l.g, l.c);
        }
      };
      if (flags & kLinGated) chunk(LinBool<true>{});
      else chunk(LinBool<false>{});
      if (a.flow && wave == 0) {
        float x = 0.f, y = 0.f;
        if (lane < C::CH) {
#pragma unroll
          for (int i = 0; i < 4; ++i) x += crossing[i][lane];
#pragma unroll
          for (int i = 0; i < C::WAVES; ++i) y += going[i][lane];
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
      gl = mine && j > 1 ? decay(j - 2) : 0.f;
      __syncthreads();
    }
    st.scale(fac[0].end);
  }
  if ((sg.flags & 1) && a.dstate_in && !side) st.store(a.dstate_in + own, w, g, c);
}

// ---- dq, dg ----------------------------------------------------------------------
template <int D, bool F32>
__global__ __launch_bounds__(4 * D, F32 ? 2 : D == 64 ? 3 : 4) void k_linear_dq(LinArgs a) {
  using C = LinCfg<D, F32>;
  using T = typename Tok<F32>::T;
  using Four = std::conditional_t<F32, f32x4, u32x2>;
  __shared__ __attribute__((aligned(16))) uint16_t lds[3 * C::TILE + C::TRI];
  __shared__ LinFactors fac[2];
  __shared__ float next_decays[64];
  __shared__ float coming[C::WAVES][64], through[C::WAVES];
  const int h = blockIdx.x % a.heads;
  const LinSeg sg = lin_seg(a.sq, blockIdx.x / a.heads);
  if (sg.count <= 0) return;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
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
  LinFetch<D, F32> fd, fv, fk;
  auto tokens = [&](int j) { return sg.count - j * C::CH < C::CH ? sg.count - j * C::CH : C::CH; };
  auto decay = [&](int j) {
    return gp && lane < tokens(j) ? gp[(int64_t)(j * C::CH + lane) * a.ld_g] : 0.f;
  };
  auto fetch = [&](int j) {
    const int64_t t0 = (int64_t)j * C::CH;
    const LinLane l(lane);
    if constexpr (F32) {
      fd.load(dp + t0 * a.d_o.ld, (unsigned)a.d_o.ld, tokens(j));
      fv.load(vp + t0 * a.v.ld, (unsigned)a.v.ld, tokens(j));
      fk.load(kp + t0 * a.k.ld, (unsigned)a.k.ld, tokens(j));
    } else {
      lin_load<D>(od, dp + t0 * a.d_o.ld, (unsigned)a.d_o.ld, tokens(j), w, l.lane);
      lin_load<D>(v, vp + t0 * a.v.ld, (unsigned)a.v.ld, tokens(j), w, l.lane);
      lin_load<D>(k, kp + t0 * a.k.ld, (unsigned)a.k.ld, tokens(j), w, l.lane);
    }
  };
  const bool mine = w == C::WAVES - 1;  // the factors are this wave's, a chunk ahead
  float gl = 0.f;
  fetch(0);
  if (mine) {
    lin_factors<false>(fac, nullptr, decay(0), tokens(0), a.scale);
    if (n > 1) gl = decay(1);
  }
  for (int j = 0; j < n; ++j) {
    const int count = tokens(j);
    const int64_t tok0 = (int64_t)sg.tok + (int64_t)j * C::CH;
    if (mine) next_decays[lane] = gl;
    if constexpr (F32) {
      fd.store(od);
      fv.store(v);
      fk.store(k);
    } else {
      lin_wait_loads();
    }
    __syncthreads();
    const LinFactors* const f = fac + (j & 1);
    const int flags = f->flags;
    if (mine && j + 1 < n) lin_factors<false>(fac + (~j & 1), f, next_decays[lane], tokens(j + 1), a.scale);
    if (F32 && j + 1 < n) fetch(j + 1);
    if (flags & kLinScale) st.scale(f->pre);
    auto chunk = [&](auto gated) {
      constexpr bool GATED = decltype(gated)::value;
      // q's elements of a lane's outputs are on their way meanwhile
      Four qe[C::IT];
      if (a.flow) {
        const LinLane l(lane);
#pragma unroll
        for (int it = 0; it < C::IT; ++it) {
          const int row = 16 * it + l.c < count ? 16 * it + l.c : count - 1;
          qe[it] = *(const Four*)(qp + ((int64_t)j * C::CH + row) * a.q.ld + 16 * w + 4 * l.g);
        }
      }
      for (int t = w; t < 2 * C::FRAGS; t += C::WAVES) {
        const LinLane l(lane);
        const int fr = t >> 1;
        const int it = C::CH == 32 || fr < 2 ? fr : 2 + (fr - 2) / 2, ts = C::CH == 32 || fr < 2 ? 0 : (fr - 2) & 1;
        const int jt = 2 * ts + (t & 1);
        const f32x4 x =
            lin_gate<false, GATED>(lin_tri<D, F32>(od, v, it, jt, l.g, l.c), f, a.scale, it, jt, l.g, l.c);
        lin_put(tri, C::FRAGS, fr, jt, l.lane, x);
      }
      LinOut<D, F32> out;
      {
        const LinLane l(lane);
        out.read(st, od, l.g, l.c);
      }
      if (a.flow) {
        const LinLane l(lane);
        const float* const dump =
            a.d_dump + (((int64_t)sg.chunk0 + j) * a.heads + h) * D * D + w * (C::MT * 256) + 4 * l.lane;
        float e = 0.f;
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) {
          const f32x4 x = *(const f32x4*)(dump + mt * 256);
#pragma unroll
          for (int r = 0; r < 4; ++r) e = fmaf(st.m[mt][r], x[r], e);
        }
#pragma unroll
        for (int m = 1; m < 64; m *= 2) e += __shfl_xor(e, m, 64);
        if (lane == 0) through[w] = e;
#pragma unroll
        for (int it = 0; it < C::IT; ++it) {
          const float x = group_sum(dot4(out.o[it], qe[it]));
          if (l.g == 0) coming[w][16 * it + l.c] = 16 * it + l.c < count ? x * f->up[16 * it + l.c] : 0.f;
        }
      }
      if (GATED) {
        out.scale(f, c);
        st.scale(f->last);
      }
      __syncthreads();
      const LinLane lt(lane);
      lin_tokens<D, F32, false, true>(&out, st, tri, v, k, f, w, lt.lane, lt.g, lt.c);
      const LinLane l(lane);
      if (!GATED) out.scale(f, l.c);
      if (a.o_part) out.store(a.o_part + (tok0 * a.heads + h) * D, (unsigned)(a.heads * D), count, w, l.g, l.c);
      else out.store((T*)a.o + tok0 * a.ld_o + hk * D, (unsigned)a.ld_o, count, w, l.g, l.c);
    };
    if (flags & kLinGated) chunk(LinBool<true>{});
    else chunk(LinBool<false>{});
    if (a.flow && w == 0) {
      float x = 0.f, e = 0.f;
#pragma unroll
      for (int i = 0; i < C::WAVES; ++i) {
        x += lane < C::CH ? coming[i][lane] : 0.f;
        e += through[i];
      }
#pragma unroll
      for (int m = 1; m < 64; m *= 2) {
        const float o = __shfl_down(x, m, 64);
        if (lane + m < 64) x += o;
      }
      // M at the chunk's start, D at its end and the decay between
      const double power = f->s + a.d_exp[((int64_t)sg.chunk0 + j) * a.heads + h] + f->cs[63];
      const float d = lane < count ? a.flow[(tok0 + lane) * a.heads + h] + x + e * exp2_wide(power) : 0.f;
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
    if (!F32 && j + 1 < n) fetch(j + 1);
    gl = mine && j + 2 < n ? decay(j + 2) : 0.f;
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
  const dim3 grid((unsigned)((int64_t)a.sq.n_segs * a.heads)), blk(8 * D);
  if (f32) hipLaunchKernelGGL((k_linear_dkdv<D, true>), grid, blk, 0, st, a);
  else hipLaunchKernelGGL((k_linear_dkdv<D, false>), grid, blk, 0, st, a);
  return hipGetLastError();
}

template <int D>
hipError_t dq_any(const LinArgs& a, bool f32, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.sq.n_segs * a.heads)), blk(4 * D);
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
