// fp32 tokens: the chunks of a segment in order, one workgroup per (segment, head),
// each wave 32 columns of M (d_v) and all its rows (delta_rule.h).  A wave's columns need
// nothing from the other waves but the operands they share: K and Q, read from
// LDS in rows and, for K^T, through the transposing read; T and P, read as
// operand tiles.  M, R and U stay in registers: each is the result of one product
// and the right operand of the next.  Columns 2 c and 2 c + 1 of a wave belong to
// lane c's two column tiles, so tokens go in and out as pairs.  Bound by the latency
// of a chunk's chain of products, one wave on each SIMD: 1374 tokens, 8 heads of 128 in
// segments of 2 chunks 38 us, 17 more for the triangles' kernel.
#include "delta_scan.h"

namespace zm {

namespace {

// MODE 0: outputs and the last state.  MODE 1 (backward): M at every chunk's start
// and U instead of the outputs.  MODE 2: the segment's transition: blocks of the
// first `heads` columns run the values from a zero state, the others no values
// from the identity, so M_end = N M_start + B.
enum { kOutputs = 0, kKeep = 1, kTransition = 2 };

template <int D, int MODE>
__global__ __launch_bounds__(2 * D, 1) void k_delta_scan(DeltaArgs a, DeltaScanArgs sa) {
  using C = ScanCfg<D, true>;
  constexpr int NT = C::NT, KS = D / 32, MT = D / 16;
  __shared__ __attribute__((aligned(16))) uint16_t lds[(MODE == kOutputs ? 2 : 1) * NT * C::TILE];
  uint16_t* const kl = lds;
  uint16_t* const ql = lds + NT * C::TILE;  // kOutputs only
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  int blk = blockIdx.x;
  const int h = blk % a.heads;
  blk /= a.heads;
  const bool unit = MODE == kTransition && (blk & 1);
  const int si = MODE == kTransition ? blk >> 1 : blk;
  const int4 sg = delta_seg(a.sq, si);
  if (sg.y < 0) return;
  // nothing follows the last segment; its N serves the way back
  if (MODE == kTransition && (sg.w & 2) && !(unit && sa.both)) return;
  const int hk = h / (a.heads / a.heads_k);
  const int dv = 32 * (threadIdx.x >> 6) + 2 * c;  // of the lane's pair of columns

  f32x4 m[MT][2];
  const int64_t dd = (int64_t)D * D;
  const float* init = nullptr;
  if (MODE != kTransition) {
    if (sa.seg_start) init = sa.seg_start + ((int64_t)si * a.heads + h) * dd;
    else if (sa.state_in) init = sa.state_in + ((int64_t)sg.z * a.heads + h) * dd;
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int ct = 0; ct < 2; ++ct) {
      const int dk = dim_row(mt, 4 * g);
      if (init) {
        m[mt][ct] = *(const f32x4*)(init + (int64_t)(dv + ct) * D + dk);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) m[mt][ct][r] = unit && dk + r == dv + ct ? 1.f : 0.f;
      }
    }

  for (int j = 0; j < sg.y; ++j) {
    const int ci = sg.x + j;
    const int4 ch = delta_chunk(a.sq, ci);
    const int count = ch.y;
    const int64_t slot = (int64_t)ci * a.heads + h;
    const uint16_t* const tf = a.t_frags + slot * 3 * kTriFrags * kFragElems;
    const uint16_t* const pf = a.p_frags + slot * 3 * kTriFrags * kFragElems;
    const float* const rows = a.rows + slot * 3 * kChunk;
    __syncthreads();
    stage<D>(kl, (const float*)a.k.p + (int64_t)ch.x * a.k.ld + hk * D, a.k.ld, count);
    if (MODE == kOutputs)
      stage<D>(ql, (const float*)a.q.p + (int64_t)ch.x * a.q.ld + hk * D, a.q.ld, count);
    __syncthreads();

    if (MODE == kKeep) {
      float* const mo = sa.m_out + slot * dd;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          *(f32x2*)(mo + (dv >> 5) * D * 32 + dim_row(mt, 4 * g + r) * 32 + (dv & 31)) =
              f32x2{m[mt][0][r], m[mt][1][r]};
    }

    // K M and Q M
    f32x4 km[4][2], qm[4][2];
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) km[it][ct] = qm[it][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      Parts<3> b[2];
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) b[ct] = split_tiles<3>(m[2 * s][ct], m[2 * s + 1][ct]);
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int row = token_row(it, c), col = 32 * s + 8 * g;
        const auto ka = lds_row<D, true>(kl, row, col);
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) mma<2>(km[it][ct], ka, b[ct]);
        if (MODE == kOutputs) {
          const auto qa = lds_row<D, true>(ql, row, col);
#pragma unroll
          for (int ct = 0; ct < 2; ++ct) mma<2>(qm[it][ct], qa, b[ct]);
        }
      }
    }
    // X = beta o (V - gam o K M), in km
    const float* const vp = (const float*)a.v.p + (int64_t)ch.x * a.v.ld + h * D + dv;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int t0 = token_row(it, 4 * g);
      const f32x4 gm = *(const f32x4*)(rows + t0), be = *(const f32x4*)(rows + 2 * kChunk + t0);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        f32x2 v = {0.f, 0.f};
        if (!unit && t0 + r < count) v = *(const f32x2*)(vp + (int64_t)(t0 + r) * a.v.ld);
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) km[it][ct][r] = be[r] * fmaf(-gm[r], km[it][ct][r], v[ct]);
      }
    }
    // U = T X
    f32x4 u[4][2];
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) u[it][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ts = 0; ts < 2; ++ts) {
      Parts<3> b[2];
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) b[ct] = split_tiles<3>(km[2 * ts][ct], km[2 * ts + 1][ct]);
#pragma unroll
      for (int it = 2 * ts; it < 4; ++it) {
        const auto ta = frag<3>(tf, low_frag(it, ts), lane);
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) mma<2>(u[it][ct], ta, b[ct]);
      }
    }
    if (MODE == kKeep) {
      float* const uo = sa.u_out + slot * kChunk * D + (dv >> 5) * kChunk * 32 + (dv & 31);
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = token_row(it, 4 * g + r);
          if (t < count)
            *(f32x2*)(uo + t * 32) = f32x2{u[it][0][r], u[it][1][r]};
        }
    }
    if (MODE == kOutputs) {
      // O = scale gam o (Q M) + P U
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const f32x4 gm = *(const f32x4*)(rows + token_row(it, 4 * g));
#pragma unroll
        for (int ct = 0; ct < 2; ++ct)
#pragma unroll
          for (int r = 0; r < 4; ++r) qm[it][ct][r] *= a.scale * gm[r];
      }
#pragma unroll
      for (int ts = 0; ts < 2; ++ts) {
        Parts<3> b[2];
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) b[ct] = split_tiles<3>(u[2 * ts][ct], u[2 * ts + 1][ct]);
#pragma unroll
        for (int it = 2 * ts; it < 4; ++it) {
          const auto pa = frag<3>(pf, low_frag(it, ts), lane);
#pragma unroll
          for (int ct = 0; ct < 2; ++ct) mma<2>(qm[it][ct], pa, b[ct]);
        }
      }
      float* const op = (float*)sa.o + (int64_t)ch.x * sa.ld_o + h * D + dv;
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = token_row(it, 4 * g + r);
          if (t < count) *(f32x2*)(op + (int64_t)t * sa.ld_o) = f32x2{qm[it][0][r], qm[it][1][r]};
        }
    }
    // M <- gam_C M + K^T (dec o U)
    const float gl = rows[kChunk - 1];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int ct = 0; ct < 2; ++ct)
#pragma unroll
        for (int r = 0; r < 4; ++r) m[mt][ct][r] *= gl;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const f32x4 de = *(const f32x4*)(rows + kChunk + token_row(it, 4 * g));
#pragma unroll
      for (int ct = 0; ct < 2; ++ct)
#pragma unroll
        for (int r = 0; r < 4; ++r) u[it][ct][r] *= de[r];
    }
#pragma unroll
    for (int ts = 0; ts < 2; ++ts) {
      Parts<3> b[2];
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) b[ct] = split_tiles<3>(u[2 * ts][ct], u[2 * ts + 1][ct]);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const auto ka = lds_col<D, true>(kl, mt, ts, g, c);
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) mma<2>(m[mt][ct], ka, b[ct]);
      }
    }
  }

  float* out = nullptr;
  if (MODE == kTransition)
    out = sa.trans + ((int64_t)si * a.heads + h) * (sa.both ? 3 : 2) * dd + (unit ? 2 : 1) * dd;
  if (unit) {  // N for the join, and its transpose for the one on the way back
    if (sa.both) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int ct = 0; ct < 2; ++ct)
          *(f32x4*)(out + join_n<D>(dv + ct, dim_row(mt, 4 * g))) = m[mt][ct];
    }
    out -= 2 * dd;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *(f32x2*)(out + join_n<D>(dim_row(mt, 4 * g + r), dv)) = f32x2{m[mt][0][r], m[mt][1][r]};
    return;
  }
  if (MODE != kTransition && (sg.w & 2) && sa.state_out) out = sa.state_out + ((int64_t)sg.z * a.heads + h) * dd;
  if (out) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int ct = 0; ct < 2; ++ct)
        *(f32x4*)(out + (MODE == kTransition ? join_b<D>(dv + ct, mt, g)
                                             : (dv + ct) * D + dim_row(mt, 4 * g))) = m[mt][ct];
  }
}

// The states at the segments' starts, M <- N M + B along each sequence, or (REV) the
// gradients at the segments' ends, M <- N^T M + E from its last segment back.  The
// blocks of a sequence's first (last) segment go through all of its segments, one
// for each 16 columns of a head; wave w forms rows dim_row(w, .).  Each step is one
// product that waits for the step before, so all else is out of the way: N's rows
// are loaded three steps ahead, M passes between the waves through LDS, and the
// product takes both in fp32 (v_mfma_f32_16x16x4_f32, row 8 g + e of a 32-row step in
// slot g of instruction e): twice the time on the matrix cores of bf16 parts, but
// splitting N's rows, once for every 16 columns, took as long.  N lies as it is
// loaded: by rows each load touched sixteen lines and a step took 2.4 us instead of 1.8.
template <int D, bool REV>
__global__ __launch_bounds__(4 * D) void k_delta_join(DeltaArgs a, DeltaJoinArgs ja) {
  constexpr int KS = D / 32, SL = D / 16;
  __shared__ __attribute__((aligned(16))) f32x4 mp[2][SL][64];
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  // the blocks of one segment and head 8 apart: on one XCD, whose L2 holds N for them
  const int unit = 8 * (blockIdx.x / (8 * SL)) + blockIdx.x % 8;
  const int dv = 16 * (blockIdx.x / 8 % SL) + c;
  const int h = unit % a.heads;
  int si = unit / a.heads;
  if (si >= a.sq.n_segs) return;
  const int4 sg = delta_seg(a.sq, si);
  if (sg.y < 0 || !(sg.w & (REV ? 2 : 1))) return;
  const int64_t dd = (int64_t)D * D;
  const int64_t col = (int64_t)dv * D + dim_row(w, 4 * g);
  int turn = 0;
  f32x4 m = {0.f, 0.f, 0.f, 0.f};
  if (ja.init) m = *(const f32x4*)(ja.init + ((int64_t)sg.z * a.heads + h) * dd + col);
  // N's rows and what is added, kAhead segments ahead
  constexpr int kAhead = 3;
  f32x4 raw[kAhead][2 * KS], add[kAhead];
  auto load = [&](int slot, int sj) {
    const int64_t at = (int64_t)sj * a.heads + h;
    const float* const nn = ja.trans + at * ja.stride * dd;
    add[slot] = *(const f32x4*)((REV ? ja.e + at * dd : nn + dd) + join_b<D>(dv, w, g));
    const float* const r = nn + (REV ? 2 * dd : 0) + (w * SL * 64 + lane) * 4;
#pragma unroll
    for (int s = 0; s < SL; ++s) raw[slot][s] = *(const f32x4*)(r + s * 256);
  };
  constexpr int kStep = REV ? -1 : 1;
  int left = sg.w >> 2;  // segments to go: one product fewer
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (left > i + 1) load(i, si + kStep * i);
  while (true) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      *(f32x4*)(ja.to + ((int64_t)si * a.heads + h) * dd + col) = m;
      if (--left <= 0) return;
      si += kStep;
      f32x4(*const buf)[64] = mp[turn];
      turn ^= 1;
      buf[w][lane] = m;
      lds_barrier();  // the other buffer's readers are past it too
      f32x4 acc[KS];
#pragma unroll
      for (int s = 0; s < KS; ++s) acc[s] = f32x4{0.f, 0.f, 0.f, 0.f};
      acc[0] = add[i];
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int s = 0; s < KS; ++s)
            acc[s] = __builtin_amdgcn_mfma_f32_16x16x4f32(raw[i][2 * s + e][r], buf[2 * s + e][lane][r],
                                                          acc[s], 0, 0, 0);
      if (left > kAhead) load(i, si + kStep * kAhead - kStep);
      m = acc[0] + acc[1];
#pragma unroll
      for (int s = 2; s < KS; ++s) m += acc[s];
    }
  }
}

template <int D>
hipError_t scan_any(const DeltaArgs& a, const DeltaScanArgs& s, hipStream_t st) {
  const int64_t blocks = (int64_t)a.sq.n_segs * a.heads;
  const dim3 grid((unsigned)blocks), twice((unsigned)(2 * blocks)), blk(2 * D);
  if (s.trans) hipLaunchKernelGGL((k_delta_scan<D, kTransition>), twice, blk, 0, st, a, s);
  else if (s.m_out) hipLaunchKernelGGL((k_delta_scan<D, kKeep>), grid, blk, 0, st, a, s);
  else hipLaunchKernelGGL((k_delta_scan<D, kOutputs>), grid, blk, 0, st, a, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_scan(const DeltaArgs& a, const DeltaScanArgs& s, hipStream_t st) {
  return a.d == 128 ? scan_any<128>(a, s, st) : scan_any<64>(a, s, st);
}

hipError_t launch_delta_join(const DeltaArgs& a, const DeltaJoinArgs& j, hipStream_t st) {
  const int64_t units = (int64_t)a.sq.n_segs * a.heads;
  const dim3 grid((unsigned)(8 * ceil_div(units, 8) * (a.d / 16))), blk(4 * a.d);
  if (a.d == 128) {
    if (j.e) hipLaunchKernelGGL((k_delta_join<128, true>), grid, blk, 0, st, a, j);
    else hipLaunchKernelGGL((k_delta_join<128, false>), grid, blk, 0, st, a, j);
  } else {
    if (j.e) hipLaunchKernelGGL((k_delta_join<64, true>), grid, blk, 0, st, a, j);
    else hipLaunchKernelGGL((k_delta_join<64, false>), grid, blk, 0, st, a, j);
  }
  return hipGetLastError();
}

}  // namespace zm
