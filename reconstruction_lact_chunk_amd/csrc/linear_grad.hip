// Gradients of linear attention with decays (linear_attn.h): what segments add to the states
// and their gradients, one pass from the last chunk of a segment to the first for dk and dv,
// one from the first to the last for dq and dg.
#include "linear_attn.h"

#include <type_traits>

namespace zm {

namespace {

// Sum over the four lane groups of a column.
__device__ __forceinline__ float group_sum(float x) {
  x += __shfl_xor(x, 16, 64);
  return x + __shfl_xor(x, 32, 64);
}
// Within 16 lanes: of the lanes before, and of all.
__device__ __forceinline__ float from_left(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x111, 0xf, 0xf, false));
}
__device__ __forceinline__ float row16_sum(float x) {  // rotated by 8, 4, 2, 1
  x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x128, 0xf, 0xf, true));
  x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x124, 0xf, 0xf, true));
  x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x122, 0xf, 0xf, true));
  return x + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x121, 0xf, 0xf, true));
}

// A lane's four outputs of a token times the same elements of a token tensor.
__device__ __forceinline__ float dot4(const f32x4& o, const f32x4& v) {
  return o[0] * v[0] + o[1] * v[1] + o[2] * v[2] + o[3] * v[3];
}
__device__ __forceinline__ float dot4(const f32x4& o, const u32x2& v) {
  return o[0] * bf16lo(v[0]) + o[1] * bf16hi(v[0]) + o[2] * bf16lo(v[1]) + o[3] * bf16hi(v[1]);
}
template <bool F32>
using Four = std::conditional_t<F32, f32x4, u32x2>;

// ---- what a segment adds, and dg within the chunks -----------------------------------
// One workgroup to a (segment, head), all of q, k, v, dO read once: M and D of the segment (the
// state's part at its end, the gradient's at its start), and per chunk
//   sum over i >= t > j of X_ij,  X_ij = T_ij (dO_i.v_j),
// from both triangles: units of two 16 x 16 tiles, columns j in prefix sums over a row's lanes,
// then sums over the rows i.  A row's sum over columns 0..31 counts for all t in 32..i.
// 10,992 tokens of 8 heads of 128, bf16: 54 us; 4123 fp32 tokens of 6 heads of 64 17 us.
// Two workgroups of d = 128 to a compute unit fit with 46 registers spilled: a frame's whole gradient 60.6 us
// against 56.8, of 60 frames 1187 against 1164, of 40 packed sequences 938 against 952.
template <int D, bool F32>
__global__ __launch_bounds__(4 * D, F32 || D == 128 ? 2 : 4) void k_linear_grad_states(LinArgs a) {
  using C = LinCfg<D, F32>;
  using T = typename Tok<F32>::T;
  constexpr int UNITS = C::CH == 64 ? 6 : 2;
  __shared__ __attribute__((aligned(16))) uint16_t lds[4 * C::TILE];
  __shared__ LinFactors fac[2];
  __shared__ __attribute__((aligned(16))) float to_end[2][64], to_start[2][64];  // of V in M, of dO in D
  __shared__ __attribute__((aligned(16))) float rows[64], crossing[UNITS][32], next_decays[64];
  const int h = blockIdx.x % a.heads;
  const LinSeg sg = lin_seg(a.sq, blockIdx.x / a.heads);
  const bool need_m = !(sg.flags & 2), need_d = !(sg.flags & 1);
  if (sg.count <= 0 || !(need_m || need_d || a.flow)) return;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int hk = h / (a.heads / a.heads_k);
  uint16_t* const q = lds;
  uint16_t* const k = q + C::TILE;
  uint16_t* const v = k + C::TILE;
  uint16_t* const od = v + C::TILE;
  const T* const qp = (const T*)a.q.p + (int64_t)sg.tok * a.q.ld + hk * D;
  const T* const kp = (const T*)a.k.p + (int64_t)sg.tok * a.k.ld + hk * D;
  const T* const vp = (const T*)a.v.p + (int64_t)sg.tok * a.v.ld + h * D;
  const T* const dp = (const T*)a.d_o.p + (int64_t)sg.tok * a.d_o.ld + h * D;
  const float* const gp = a.g ? a.g + (int64_t)sg.tok * a.ld_g + h : nullptr;
  const int n = (sg.count + C::CH - 1) / C::CH;
  LinState<D, F32> m, d;
  m.zero();
  d.zero();
  LinFetch<D, F32> fq, fk, fv, fd;
  auto tokens = [&](int j) { return sg.count - j * C::CH < C::CH ? sg.count - j * C::CH : C::CH; };
  auto decay = [&](int j) {
    return gp && lane < tokens(j) ? gp[(int64_t)(j * C::CH + lane) * a.ld_g] : 0.f;
  };
  auto fetch = [&](int j) {
    const int64_t t0 = (int64_t)j * C::CH;
    if constexpr (F32) {
      fq.load(qp + t0 * a.q.ld, (unsigned)a.q.ld, tokens(j));
      fk.load(kp + t0 * a.k.ld, (unsigned)a.k.ld, tokens(j));
      fv.load(vp + t0 * a.v.ld, (unsigned)a.v.ld, tokens(j));
      fd.load(dp + t0 * a.d_o.ld, (unsigned)a.d_o.ld, tokens(j));
    } else {
      const LinLane l(lane);
      lin_load<D>(q, qp + t0 * a.q.ld, (unsigned)a.q.ld, tokens(j), w, l.lane);
      lin_load<D>(k, kp + t0 * a.k.ld, (unsigned)a.k.ld, tokens(j), w, l.lane);
      lin_load<D>(v, vp + t0 * a.v.ld, (unsigned)a.v.ld, tokens(j), w, l.lane);
      lin_load<D>(od, dp + t0 * a.d_o.ld, (unsigned)a.d_o.ld, tokens(j), w, l.lane);
    }
  };
  // the factors of chunk j (one wave): T's as for the pass from the last chunk to the first
  auto factors = [&](int j, float gl) {
    LinFactors* const f = fac + (j & 1);
    const double before = j > 0 ? fac[~j & 1].sum : 0.0;
    lin_factors<true>(f, nullptr, gl, tokens(j), a.scale);
    const bool in = lane < tokens(j);
    to_end[j & 1][lane] = in ? f->up[lane] : 0.f;
    to_start[j & 1][lane] = in ? a.scale * exp2_wide(before + f->cs[lane]) : 0.f;
    if (lane == 0) f->sum += before;
  };
  const bool mine = w == C::WAVES - 1;
  float gl = 0.f;
  fetch(0);
  if (mine) {
    factors(0, decay(0));
    if (n > 1) gl = decay(1);
  }
  for (int j = 0; j < n; ++j) {
    const int count = tokens(j);
    if (mine) next_decays[lane] = gl;
    if constexpr (F32) {
      fq.store(q);
      fk.store(k);
      fv.store(v);
      fd.store(od);
    } else {
      lin_wait_loads();
    }
    __syncthreads();
    const LinFactors* const f = fac + (j & 1);
    if (mine && j + 1 < n) factors(j + 1, next_decays[lane]);
    if (F32 && j + 1 < n) fetch(j + 1);
    if (a.flow) {
      auto cross = [&](auto gated) {
        constexpr bool GATED = decltype(gated)::value;
        for (int u = w; u < UNITS; u += C::WAVES) {
          const LinLane l(lane);
          const int jt = u < 2 ? u : 2 + ((u - 2) >> 1), pair = u < 2 ? 0 : (u - 2) & 1;
          const int src = token_row(jt, 4 * l.g);
          float before[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int it = 2 * pair + i;
            const f32x4 x = lin_gate<true, GATED>(lin_tri<D, F32>(v, od, it, jt, l.g, l.c), f, a.scale, it, jt, l.g, l.c);
            const f32x4 y = lin_tri<D, F32>(k, q, it, jt, l.g, l.c);
            const float up = GATED ? 1.f : f->up[16 * it + l.c];
            float sum = 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float z = x[r] * y[r] * up, p = lin_prefix16(z);
              if (src + r >= 16 * it + l.c) sum += before[r] + from_left(p);
              before[r] += row16_sum(z);
            }
            sum = group_sum(sum);
            if (l.g == 0) crossing[u][16 * i + l.c] = sum;
          }
          if (pair == 0 && l.c == 0) *(f32x4*)(rows + src) = f32x4{before[0], before[1], before[2], before[3]};
        }
      };
      if (f->flags & kLinGated) cross(LinBool<true>{});
      else cross(LinBool<false>{});
    }
    if (need_m) {
      m.scale(f->last);
      const LinLane l(lane);
      lin_tokens<D, F32, false, false>(nullptr, m, nullptr, k, v, to_end[j & 1], w, l.lane, l.g, l.c);
    }
    if (need_d) {
      const LinLane l(lane);
      lin_tokens<D, F32, true, false>(nullptr, d, nullptr, q, od, to_start[j & 1], w, l.lane, l.g, l.c);
    }
    __syncthreads();
    if (!F32 && j + 1 < n) fetch(j + 1);
    gl = mine && j + 2 < n ? decay(j + 2) : 0.f;
    if (a.flow && w == 0) {
      float x = 0.f;
      if constexpr (C::CH == 64) {
        // rows from the last one down in the lanes' order: prefix sums are sums over i >= t
        const float below = lin_prefix(lane < 32 ? rows[63 - lane] : 0.f);
        const int t = 63 - lane;
        x = t < 32 ? crossing[0][t] + crossing[1][t] + crossing[2][t] + crossing[4][t]
                   : crossing[3][t - 32] + crossing[5][t - 32] + below;
        if (t < count) a.flow[((int64_t)sg.tok + (int64_t)j * C::CH + t) * a.heads + h] = x;
      } else {
        x = lane < 32 ? crossing[0][lane] + crossing[1][lane] : 0.f;
        if (lane < count) a.flow[((int64_t)sg.tok + (int64_t)j * C::CH + lane) * a.heads + h] = x;
      }
    }
  }
  const LinLane l(lane);
  const int64_t dd = (int64_t)D * D;
  if (need_m) m.store(a.part[0] + ((int64_t)(sg.slot + 1) * a.heads + h) * dd, w, l.g, l.c);
  if (need_d) d.store(a.part[1] + ((int64_t)(sg.slot - 1) * a.heads + h) * dd, w, l.g, l.c);
  if (mine && lane == 0) {
    const float2 all = lin_exp2_parts(fac[(n - 1) & 1].sum);
    if (need_m) a.decay[0][(int64_t)sg.slot * a.heads + h] = all;
    if (need_d) a.decay[1][(int64_t)sg.slot * a.heads + h] = all;
  }
}

// ---- dk, dv --------------------------------------------------------------------
// One workgroup to a (segment, head, side): SIDE 0 dv (state D) with dg's part to the chunk's
// end, 1 dk (D^T), which leaves D^T at the chunks' ends for the pass that follows.  Two sides in one
// workgroup took 113 us for the 10,992 tokens, side by side 84 (5 us a chunk and compute unit, as
// the outputs'; D^T is 90 MB of its 144 MB of writes; 3.1 TB/s).
template <int D, bool F32, int SIDE>
__device__ __forceinline__ void back_pass(const LinArgs& a, const LinSeg& sg, int h, uint16_t* lds, LinFactors* fac,
                                          float (*going)[64], float* next_decays) {
  using C = LinCfg<D, F32>;
  using T = typename Tok<F32>::T;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  const int hk = h / (a.heads / a.heads_k);
  uint16_t* const ta = lds;
  uint16_t* const tb = ta + C::TILE;
  uint16_t* const tc = tb + C::TILE;
  uint16_t* const tri = tc + C::TILE;
  LinState<D, F32> st;
  const int64_t own = ((int64_t)sg.seq * a.heads + h) * D * D;
  const float* const from = sg.flags != 3 ? a.part[1] + ((int64_t)sg.slot * a.heads + h) * D * D
                            : a.dstate_out ? a.dstate_out + own : nullptr;
  const int n = (sg.count + C::CH - 1) / C::CH;
  const LinTokens at = SIDE ? a.v : a.k, bt = SIDE ? a.d_o : a.q, ct = SIDE ? a.q : a.d_o;
  const T* const ap = (const T*)at.p + (int64_t)sg.tok * at.ld + (SIDE ? h : hk) * D;
  const T* const bp = (const T*)bt.p + (int64_t)sg.tok * bt.ld + (SIDE ? h : hk) * D;
  const T* const cp = (const T*)ct.p + (int64_t)sg.tok * ct.ld + (SIDE ? hk : h) * D;
  const T* const vp = (const T*)a.v.p + (int64_t)sg.tok * a.v.ld + h * D;
  const float* const gp = a.g ? a.g + (int64_t)sg.tok * a.ld_g + h : nullptr;
  LinFetch<D, F32> fa, fb, fc;
  auto tokens = [&](int j) { return sg.count - j * C::CH < C::CH ? sg.count - j * C::CH : C::CH; };
  auto decay = [&](int j) {
    return gp && lane < tokens(j) ? gp[(int64_t)(j * C::CH + lane) * a.ld_g] : 0.f;
  };
  auto fetch = [&](int j) {
    const int64_t t0 = (int64_t)j * C::CH;
    if constexpr (F32) {
      fa.load(ap + t0 * at.ld, (unsigned)at.ld, tokens(j));
      fb.load(bp + t0 * bt.ld, (unsigned)bt.ld, tokens(j));
      fc.load(cp + t0 * ct.ld, (unsigned)ct.ld, tokens(j));
    } else {
      const LinLane l(lane);
      lin_load<D>(ta, ap + t0 * at.ld, (unsigned)at.ld, tokens(j), w, l.lane);
      lin_load<D>(tb, bp + t0 * bt.ld, (unsigned)bt.ld, tokens(j), w, l.lane);
      lin_load<D>(tc, cp + t0 * ct.ld, (unsigned)ct.ld, tokens(j), w, l.lane);
    }
  };
  const bool mine = w == C::WAVES - 1;  // the factors are this wave's, a chunk ahead
  float gl = 0.f;
  if (n > 0) fetch(n - 1);
  {
    const LinLane l(lane);
    if (!from) st.zero();
    else st.template load<SIDE != 0>(from, w, l.g, l.c);
  }
  if (n > 0 && mine) {
    lin_factors<true>(fac + ((n - 1) & 1), nullptr, decay(n - 1), tokens(n - 1), a.scale);
    if (n > 1) gl = decay(n - 2);
  }
  for (int j = n - 1; j >= 0; --j) {
    const int count = tokens(j);
    const int64_t tok0 = (int64_t)sg.tok + (int64_t)j * C::CH;
    if (mine) next_decays[lane] = gl;
    if constexpr (F32) {
      fa.store(ta);
      fb.store(tb);
      fc.store(tc);
    } else {
      lin_wait_loads();
    }
    __syncthreads();
    const LinFactors* const f = fac + (j & 1);
    const int flags = f->flags;
    if (mine && j > 0) lin_factors<true>(fac + (~j & 1), f, next_decays[lane], tokens(j - 1), a.scale);
    if (F32 && j > 0) fetch(j - 1);
    if (flags & kLinScale) st.scale(f->pre);
    auto chunk = [&](auto gated) {
      constexpr bool GATED = decltype(gated)::value;
      // v's elements of a lane's outputs are on their way meanwhile
      Four<F32> ve[C::IT];
      if (SIDE == 0 && a.flow) {
        const LinLane l(lane);
#pragma unroll
        for (int it = 0; it < C::IT; ++it) {
          const int row = 16 * it + l.c < count ? 16 * it + l.c : count - 1;
          ve[it] = *(const Four<F32>*)(vp + ((int64_t)j * C::CH + row) * a.v.ld + 16 * w + 4 * l.g);
        }
      }
      if (SIDE == 1 && a.flow) {
        const LinLane l(lane);
        if (w == 0 && lane == 0) a.d_exp[((int64_t)sg.chunk0 + j) * a.heads + h] = f->s;
        float* const dump = a.d_dump + (((int64_t)sg.chunk0 + j) * a.heads + h) * D * D + w * (C::MT * 256) + 4 * l.lane;
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) *(f32x4*)(dump + mt * 256) = st.m[mt];
      }
      for (int t = w; t < 2 * C::FRAGS; t += C::WAVES) {
        const LinLane l(lane);
        const int fr = t >> 1;
        const int it = C::CH == 32 ? fr : fr < 4 ? fr >> 1 : fr - 2, ts = C::CH == 32 ? 0 : fr < 4 ? fr & 1 : 1;
        const int jt = 2 * ts + (t & 1);
        const f32x4 x = lin_gate<true, GATED>(lin_tri<D, F32>(ta, tb, it, jt, l.g, l.c), f, a.scale, it, jt, l.g, l.c);
        lin_put(tri, C::FRAGS, fr, jt, l.lane, x);
      }
      LinOut<D, F32> out;
      {
        const LinLane l(lane);
        out.read(st, ta, l.g, l.c);
      }
      if (SIDE == 0 && a.flow) {
        const LinLane l(lane);
#pragma unroll
        for (int it = 0; it < C::IT; ++it) {
          const int t = 16 * it + l.c;
          const float x = group_sum(dot4(out.o[it], ve[it]));
          if (l.g == 0) going[w][t] = t < count ? x * f->up[t] : 0.f;
        }
      }
      if (GATED) {
        const LinLane l(lane);
        out.scale(f, l.c);
        st.scale(f->last);
      }
      __syncthreads();
      const LinLane lt(lane);
      lin_tokens<D, F32, true, true>(&out, st, tri, tb, tc, f->dn, w, lt.lane, lt.g, lt.c);
      const LinLane l(lane);
      if (!GATED) out.scale(f, l.c);
      if (SIDE == 0) {
        out.store((T*)a.dv + tok0 * a.ld_dv + h * D, (unsigned)a.ld_dv, count, w, l.g, l.c);
      } else if (a.dk_part) {
        out.store(a.dk_part + (tok0 * a.heads + h) * D, (unsigned)(a.heads * D), count, w, l.g, l.c);
      } else {
        out.store((T*)a.dk + tok0 * a.ld_dk + hk * D, (unsigned)a.ld_dk, count, w, l.g, l.c);
      }
    };
    if (flags & kLinGated) chunk(LinBool<true>{});
    else chunk(LinBool<false>{});
    if (SIDE == 0 && a.flow && w == 0) {
      float y = 0.f;
      if (lane < C::CH)
#pragma unroll
        for (int i = 0; i < C::WAVES; ++i) y += going[i][lane];
      const float up = __shfl_up(lin_prefix(y), 1, 64);  // of the tokens before
      if (lane < count) a.flow[(tok0 + lane) * a.heads + h] += lane ? up : 0.f;
    }
    __syncthreads();
    if (!F32 && j > 0) fetch(j - 1);
    gl = mine && j > 1 ? decay(j - 2) : 0.f;
  }
  if (SIDE == 0 && (sg.flags & 1) && a.dstate_in) {
    const LinLane l(lane);
    if (n > 0) st.scale(fac[0].end);
    st.store(a.dstate_in + own, w, l.g, l.c);
  }
}

template <int D, bool F32>
__global__ __launch_bounds__(4 * D, F32 ? 2 : D == 64 ? 3 : 4) void k_linear_dkdv(LinArgs a, int side) {
  using C = LinCfg<D, F32>;
  __shared__ __attribute__((aligned(16))) uint16_t lds[3 * C::TILE + C::TRI];
  __shared__ LinFactors fac[2];
  __shared__ float going[C::WAVES][64], next_decays[64];
  const int h = blockIdx.x % a.heads;
  const LinSeg sg = lin_seg(a.sq, blockIdx.x / a.heads);
  if (sg.count < 0) return;
  if (side + blockIdx.y == 0) back_pass<D, F32, 0>(a, sg, h, lds, fac, going, next_decays);
  else if (sg.count > 0) back_pass<D, F32, 1>(a, sg, h, lds, fac, going, next_decays);
}

// ---- dq, dg ----------------------------------------------------------------------
// As the outputs, with M^T; dg is put together here.  55 us for the 10,992 tokens, 2.5 TB/s.
template <int D, bool F32>
__global__ __launch_bounds__(4 * D, F32 ? 2 : D == 64 ? 3 : 4) void k_linear_dq(LinArgs a) {
  using C = LinCfg<D, F32>;
  using T = typename Tok<F32>::T;
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
      // q's elements of a lane's outputs and D^T are on their way meanwhile
      f32x4 de[C::MT];
      Four<F32> qe[C::IT];
      double d_exp = 0.0;
      if (a.flow) {
        const LinLane l(lane);
        d_exp = a.d_exp[((int64_t)sg.chunk0 + j) * a.heads + h];
#pragma unroll
        for (int it = 0; it < C::IT; ++it) {
          const int row = 16 * it + l.c < count ? 16 * it + l.c : count - 1;
          qe[it] = *(const Four<F32>*)(qp + ((int64_t)j * C::CH + row) * a.q.ld + 16 * w + 4 * l.g);
        }
        const float* const dump =
            a.d_dump + (((int64_t)sg.chunk0 + j) * a.heads + h) * D * D + w * (C::MT * 256) + 4 * l.lane;
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) de[mt] = *(const f32x4*)(dump + mt * 256);
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
      if (a.flow) {
        // M at the chunk's start, D at its end and the decay between.  Both are held less powers of
        // up to 2^60, so each takes half of the exponent before they meet: their product with neither could
        // be past fp32's range where the sum is not.
        const float half = exp2_wide(0.5 * (f->s + d_exp + f->cs[63]));
        float e = 0.f;
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
          for (int r = 0; r < 4; ++r) e = fmaf(st.m[mt][r] * half, de[mt][r] * half, e);
        e = lin_prefix(e);
        if (lane == 63) through[w] = e;
      }
      LinOut<D, F32> out;
      {
        const LinLane l(lane);
        out.read(st, od, l.g, l.c);
      }
      if (a.flow) {
        const LinLane l(lane);
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
      lin_tokens<D, F32, false, true>(&out, st, tri, v, k, f->dn, w, lt.lane, lt.g, lt.c);
      const LinLane l(lane);
      if (!GATED) out.scale(f, l.c);
      if (a.o_part) out.store(a.o_part + (tok0 * a.heads + h) * D, (unsigned)(a.heads * D), count, w, l.g, l.c);
      else out.store((T*)a.o + tok0 * a.ld_o + hk * D, (unsigned)a.ld_o, count, w, l.g, l.c);
    };
    if (flags & kLinGated) chunk(LinBool<true>{});
    else chunk(LinBool<false>{});
    if (a.flow && w == 0) {
      // tokens from the last one down in the lanes' order: prefix sums are sums over i >= t
      const int t = 63 - lane;
      float x = 0.f, e = 0.f;
#pragma unroll
      for (int i = 0; i < C::WAVES; ++i) {
        x += t < C::CH ? coming[i][t] : 0.f;
        e += through[i];
      }
      x = lin_prefix(x);
      const float d = t < count ? a.flow[(tok0 + t) * a.heads + h] + x + e : 0.f;
      if (a.ld_g) {
        if (t < count) a.dg[(tok0 + t) * a.heads + h] = d;
      } else {
        const float s = lin_prefix(d);
        if (lane == 63) a.dg[((int64_t)sg.chunk0 + j) * a.heads + h] = s;
      }
    }
    __syncthreads();
    if (!F32 && j + 1 < n) fetch(j + 1);
    gl = mine && j + 2 < n ? decay(j + 2) : 0.f;
  }
}

// ---- sums ------------------------------------------------------------------------
// dg [heads]: a workgroup to a head, the chunks' sums in 64 bits, always in the same order.
__device__ __forceinline__ void decay_sum(const float* sums, const LinSeqs& sq, int heads, int h, float* dg) {
  __shared__ double red[4];
  const int chunks = lin_all(sq).z;
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < chunks; i += 256) s += (double)sums[i * heads + h];
#pragma unroll
  for (int m = 1; m < 64; m *= 2) s += __shfl_xor(s, m, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) dg[h] = (float)(red[0] + red[1] + red[2] + red[3]);
}
__global__ __launch_bounds__(256) void k_linear_decay_sum(const float* sums, LinSeqs sq, int heads, float* dg) {
  decay_sum(sums, sq, heads, blockIdx.x, dg);
}

// Eight elements a thread: the value heads of a key head in order, blockIdx.y 0 dq, 1 dk.
// Rows outside the sequences are left as they are.  Workgroups past `blocks` form dg [heads].
template <typename T>
__global__ __launch_bounds__(256) void k_linear_groups(LinArgs a, int d, int blocks, float* dg) {
  if ((int)blockIdx.x >= blocks) {
    if (blockIdx.y == 0) decay_sum(a.dg, a.sq, a.heads, blockIdx.x - blocks, dg);
    return;
  }
  const int heads = a.heads, per = a.heads_k * d / 8, rep = heads / a.heads_k;
  const float* const x = blockIdx.y ? a.dk_part : a.o_part;
  T* const y = (T*)(blockIdx.y ? a.dk : a.o);
  const int64_t ldy = blockIdx.y ? a.ld_dk : a.ld_o;
  const int4 range = lin_all(a.sq);
  const int64_t all = (int64_t)(range.y - range.x) * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)blocks * 256) {
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

template <int D>
hipError_t grad_states_any(const LinArgs& a, bool f32, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.sq.n_segs * a.heads)), blk(4 * D);
  if (f32) hipLaunchKernelGGL((k_linear_grad_states<D, true>), grid, blk, 0, st, a);
  else hipLaunchKernelGGL((k_linear_grad_states<D, false>), grid, blk, 0, st, a);
  return hipGetLastError();
}

template <int D>
hipError_t dkdv_any(const LinArgs& a, bool f32, hipStream_t st) {
  const unsigned blocks = (unsigned)((int64_t)a.sq.n_segs * a.heads);
  auto sides = [&](int first, int count) {
    const dim3 grid(blocks, count), blk(4 * D);
    if (f32) hipLaunchKernelGGL((k_linear_dkdv<D, true>), grid, blk, 0, st, a, first);
    else hipLaunchKernelGGL((k_linear_dkdv<D, false>), grid, blk, 0, st, a, first);
    return hipGetLastError();
  };
  // Of a sequence in one segment both sides start from dstate_out, and side 0 ends with
  // dstate_in.  Where that is the same array side 1 is a launch before side 0's; not where the
  // only sequence is known to be cut: its segments start from part[1].  Whole gradients, in place and apart:
  // one frame whose offsets are on the device 65 and 56 us, 8 frames 212 and 200.
  const bool cut = !a.sq.offsets && a.sq.n > a.sq.seg_tokens;
  if (!a.dstate_in || a.dstate_in != a.dstate_out || cut) return sides(0, 2);
  const hipError_t e = sides(1, 1);
  return e != hipSuccess ? e : sides(0, 1);
}

template <int D>
hipError_t dq_any(const LinArgs& a, bool f32, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.sq.n_segs * a.heads)), blk(4 * D);
  if (f32) hipLaunchKernelGGL((k_linear_dq<D, true>), grid, blk, 0, st, a);
  else hipLaunchKernelGGL((k_linear_dq<D, false>), grid, blk, 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_grad_states(const LinArgs& a, int d, bool f32, hipStream_t st) {
  return d == 128 ? grad_states_any<128>(a, f32, st) : grad_states_any<64>(a, f32, st);
}

hipError_t launch_linear_dkdv(const LinArgs& a, int d, bool f32, hipStream_t st) {
  return d == 128 ? dkdv_any<128>(a, f32, st) : dkdv_any<64>(a, f32, st);
}

hipError_t launch_linear_dq(const LinArgs& a, int d, bool f32, hipStream_t st) {
  return d == 128 ? dq_any<128>(a, f32, st) : dq_any<64>(a, f32, st);
}

hipError_t launch_linear_groups(const LinArgs& a, int d, bool f32, float* dg, hipStream_t st) {
  int64_t blocks = ceil_div((int64_t)a.sq.n * (a.heads_k * d / 8), 256);
  if (blocks > 4 * kTargetWgs) blocks = 4 * kTargetWgs;
  const dim3 grid((unsigned)blocks + (dg ? a.heads : 0), 2);
  if (f32) hipLaunchKernelGGL((k_linear_groups<float>), grid, dim3(256), 0, st, a, d, (int)blocks, dg);
  else hipLaunchKernelGGL((k_linear_groups<uint16_t>), grid, dim3(256), 0, st, a, d, (int)blocks, dg);
  return hipGetLastError();
}

hipError_t launch_linear_decay_sum(const float* sums, const LinSeqs& s, int heads, float* dg, hipStream_t st) {
  hipLaunchKernelGGL(k_linear_decay_sum, dim3(heads), dim3(256), 0, st, sums, s, heads, dg);
  return hipGetLastError();
}

}  // namespace zm
