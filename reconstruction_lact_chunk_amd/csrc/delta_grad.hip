// Gradient of the gated delta rule (delta_rule.h).  With dM' the gradient of M at a
// chunk's end and X = beta o R:
//   dU = P^T dO + dec o (K dM'),  dX = T^T dU,  dV = beta o dX,
//   dM = gam_C dM' + Q^T (scale gam o dO) - K^T (gam o beta o dX),
// which k_delta_reverse carries from chunk to chunk as the forward carries M (a
// wave 32 columns of d_v), and then for every chunk on its own (k_delta_grads)
//   dQ = scale gam o (dO M^T) + W K,             W_ij = scale G_ij (dO U^T)_ij, j <= i
//   dK = -gam o beta o (dX M^T) + dec o (U dM'^T) + W^T Q + (E + E^T) K,
//                                                E_ij = -beta_i G_ij (dX U^T)_ij, j < i
//   dbeta_i = dX_i.V_i - gam_i k_i.(M dX_i) - sum_j G_ij (dX U^T)_ij k_i.k_j
// and dg as the running sum from the end of the derivatives by c:
//   dc_i = scale gam_i q_i.(M dO_i) - gam_i beta_i k_i.(M dX_i) - dec_i k_i.(dM' U_i)
//          + (row sums - column sums)_i of W_ij q_i.k_j + E_ij k_i.k_j,
//   and for the chunk's last token gam_C <M, dM'> + sum_i dec_i k_i.(dM' U_i).
#include "delta_scan.h"

namespace zm {

namespace {

// TRANS: only the gradient that a segment adds to its start's from a zero one at its
// end (the rest of the transition is the transpose of the forward's).
template <int D, bool F32, bool TRANS>
__global__ __launch_bounds__(2 * D, 1) void k_delta_reverse(DeltaArgs a, DeltaGradArgs s) {
  using C = ScanCfg<D, F32>;
  using T = typename Tok<F32>::T;
  constexpr int NT = C::NT, KS = D / 32, MT = D / 16;
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * NT * C::TILE];
  uint16_t* const kl = lds;
  uint16_t* const ql = lds + NT * C::TILE;
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int h = blockIdx.x % a.heads, si = blockIdx.x / a.heads;
  const int4 sg = delta_seg(a.sq, si);
  if (sg.y < 0 || (TRANS && (sg.w & 1))) return;
  const int hk = h / (a.heads / a.heads_k);
  const int dv = 32 * (threadIdx.x >> 6) + 2 * c;
  const int64_t dd = (int64_t)D * D;

  f32x4 m[MT][2];
  const float* init = nullptr;
  if (!TRANS) {
    if (s.seg_end) init = s.seg_end + ((int64_t)si * a.heads + h) * dd;
    else if (s.dstate_out) init = s.dstate_out + ((int64_t)sg.z * a.heads + h) * dd;
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int ct = 0; ct < 2; ++ct)
      m[mt][ct] = init ? *(const f32x4*)(init + (int64_t)(dv + ct) * D + dim_row(mt, 4 * g))
                       : f32x4{0.f, 0.f, 0.f, 0.f};

  for (int j = sg.y - 1; j >= 0; --j) {
    const int ci = sg.x + j;
    const int4 ch = delta_chunk(a.sq, ci);
    const int count = ch.y;
    const int64_t slot = (int64_t)ci * a.heads + h;
    const uint16_t* const tf = a.tt_frags + slot * 3 * kTriFrags * kFragElems;
    const uint16_t* const pf = a.pt_frags + slot * 3 * kTriFrags * kFragElems;
    const float* const rows = a.rows + slot * 3 * kChunk;
    __syncthreads();
    stage<D, F32>(kl, (const T*)a.k.p + (int64_t)ch.x * a.k.ld + hk * D, a.k.ld, count);
    stage<D, F32>(ql, (const T*)a.q.p + (int64_t)ch.x * a.q.ld + hk * D, a.q.ld, count);
    __syncthreads();

    if (!TRANS) {
      float* const mo = s.d_m + slot * dd;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          *(f32x2*)(mo + (int64_t)dim_row(mt, 4 * g + r) * D + dv) = f32x2{m[mt][0][r], m[mt][1][r]};
    }
    // dU = dec o (K dM') + P^T dO
    f32x4 du[4][2], go[4][2];
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) du[it][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      Parts<3> b[2];
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) b[ct] = split_tiles<3>(m[2 * k][ct], m[2 * k + 1][ct]);
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const auto ka = lds_row<D, F32>(kl, token_row(it, c), 32 * k + 8 * g);
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) mma<2>(du[it][ct], ka, b[ct]);
      }
    }
    const T* const op = (const T*)s.d_o.p + (int64_t)ch.x * s.d_o.ld + h * D + dv;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int t0 = token_row(it, 4 * g);
      const f32x4 de = *(const f32x4*)(rows + kChunk + t0);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        f32x2 v = {0.f, 0.f};
        if (t0 + r < count) v = load_pair(op + (int64_t)(t0 + r) * s.d_o.ld);
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) {
          go[it][ct][r] = v[ct];
          du[it][ct][r] *= de[r];
        }
      }
    }
#pragma unroll
    for (int ts = 0; ts < 2; ++ts) {
      Parts<NT> b[2];
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) b[ct] = split_tiles<NT>(go[2 * ts][ct], go[2 * ts + 1][ct]);
#pragma unroll
      for (int it = 0; it < 2 * ts + 2; ++it) {
        const auto pa = frag<3>(pf, up_frag(it, ts), lane);
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) mma<2>(du[it][ct], pa, b[ct]);
      }
    }
    // dX = T^T dU
    f32x4 x[4][2];
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) x[it][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ts = 0; ts < 2; ++ts) {
      Parts<3> b[2];
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) b[ct] = split_tiles<3>(du[2 * ts][ct], du[2 * ts + 1][ct]);
#pragma unroll
      for (int it = 0; it < 2 * ts + 2; ++it) {
        const auto ta = frag<3>(tf, up_frag(it, ts), lane);
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) mma<2>(x[it][ct], ta, b[ct]);
      }
    }
    // dV, and the factors of the state's step: scale gam o dO and -gam o beta o dX
    T* const vp = (T*)s.dv + (int64_t)ch.x * s.ld_dv + h * D + dv;
    float* const xp = s.x + ((int64_t)ch.x * a.heads + h) * D + dv;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int t0 = token_row(it, 4 * g);
      const f32x4 gm = *(const f32x4*)(rows + t0), be = *(const f32x4*)(rows + 2 * kChunk + t0);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (!TRANS && t0 + r < count) {
          *(f32x2*)(xp + (int64_t)(t0 + r) * a.heads * D) = f32x2{x[it][0][r], x[it][1][r]};
          store_pair(vp + (int64_t)(t0 + r) * s.ld_dv, be[r] * x[it][0][r], be[r] * x[it][1][r]);
        }
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) {
          x[it][ct][r] *= -gm[r] * be[r];
          go[it][ct][r] *= a.scale * gm[r];
        }
      }
    }
    const float gl = rows[kChunk - 1];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int ct = 0; ct < 2; ++ct)
#pragma unroll
        for (int r = 0; r < 4; ++r) m[mt][ct][r] *= gl;
#pragma unroll
    for (int ts = 0; ts < 2; ++ts) {
      Parts<3> b[2], d[2];
#pragma unroll
      for (int ct = 0; ct < 2; ++ct) {
        b[ct] = split_tiles<3>(x[2 * ts][ct], x[2 * ts + 1][ct]);
        d[ct] = split_tiles<3>(go[2 * ts][ct], go[2 * ts + 1][ct]);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const auto ka = lds_col<D, F32>(kl, mt, ts, g, c);
        const auto qa = lds_col<D, F32>(ql, mt, ts, g, c);
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) {
          mma<2>(m[mt][ct], ka, b[ct]);
          mma<2>(m[mt][ct], qa, d[ct]);
        }
      }
    }
  }

  float* out = nullptr;
  if (TRANS) out = s.e_out + ((int64_t)si * a.heads + h) * dd;
  else if ((sg.w & 1) && s.dstate_in) out = s.dstate_in + ((int64_t)sg.z * a.heads + h) * dd;
  if (out) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int ct = 0; ct < 2; ++ct)
        *(f32x4*)(out + (int64_t)(dv + ct) * D + dim_row(mt, 4 * g)) = m[mt][ct];
  }
}

// Parts of 8 elements of a token's row, zero past the chunk.
template <int NP, typename T>
__device__ __forceinline__ Parts<NP> tok8(const T* p, int64_t ld, int t, int count, int col) {
  if (t < count) return load8(p + (int64_t)t * ld + col);
  return zero_parts<NP>();
}

__device__ __forceinline__ float sum_groups(float x) {
  x += __shfl_xor(x, 16, 64);
  return x + __shfl_xor(x, 32, 64);
}

__device__ __forceinline__ void load4(const uint16_t* p, float* v) {
  const u32x2 w = *(const u32x2*)p;
  v[0] = bf16lo(w[0]);
  v[1] = bf16hi(w[0]);
  v[2] = bf16lo(w[1]);
  v[3] = bf16hi(w[1]);
}
__device__ __forceinline__ void load4(const float* p, float* v) {
  const f32x4 w = *(const f32x4*)p;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = w[i];
}
__device__ __forceinline__ void store4(uint16_t* p, const f32x4& v) {
  *(u32x2*)p = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}
__device__ __forceinline__ void store4(float* p, const f32x4& v) { *(f32x4*)p = v; }

// Rows 16 mt + . of the transpose of a staged tile, slots = tokens 32 ts + 16 (e / 4) +
// 4 g + e % 4: those of two neighbouring result tiles.
template <int D, bool F32>
__device__ __forceinline__ Parts<Tok<F32>::NT> lds_col_plain(const uint16_t* lds, int mt, int ts,
                                                             int g, int c) {
  using C = ScanCfg<D, F32>;
  Parts<C::NT> p;
  const int row = 32 * ts + 4 * g + (c >> 2), col = 16 * mt + 4 * (c & 3);
#pragma unroll
  for (int k = 0; k < C::NT; ++k) {
    const uint16_t* at = lds + k * C::TILE + row * C::PITCH + col;
    p.p[k] = __builtin_shufflevector(delta_read_tr(at), delta_read_tr(at + 16 * C::PITCH), 0, 1, 2,
                                     3, 4, 5, 6, 7);
  }
  return p;
}

template <int D, bool F32>
__device__ __forceinline__ void stage256(uint16_t* lds, const typename Tok<F32>::T* src, int64_t ld,
                                         int count) {
  using C = ScanCfg<D, F32>;
  constexpr int CPR = D / 8;
  for (int i = threadIdx.x; i < kChunk * CPR; i += 256) {
    const int row = i / CPR, col = 8 * (i % CPR);
    const auto p = tok8<C::NT>(src, ld, row, count, col);
#pragma unroll
    for (int k = 0; k < C::NT; ++k) *(bf16x8*)(lds + k * C::TILE + row * C::PITCH + col) = p.p[k];
  }
}

// One workgroup per (chunk, head); wave w has the tokens 16 w + c as columns of every
// product, so that dQ^T and dK^T build up in registers (rows: dims) and the
// derivatives by c and beta are column sums.
template <int D, bool F32>
__global__ __launch_bounds__(256, 1) void k_delta_grads(DeltaArgs a, DeltaGradArgs s) {
  using C = ScanCfg<D, F32>;
  using T = typename Tok<F32>::T;
  constexpr int NT = C::NT, KS = D / 32, MT = D / 16, NW = NT == 1 ? 2 : 3;
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * NT * C::TILE];
  __shared__ double cs[kChunk];
  __shared__ float dcs[kChunk];
  __shared__ float ends[4], frob;
  uint16_t* const kl = lds;
  uint16_t* const ql = lds + NT * C::TILE;
  const int h = blockIdx.x % a.heads, ci = blockIdx.x / a.heads;
  const int4 ch = delta_chunk(a.sq, ci);
  const int count = ch.y;
  if (count == 0) return;
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int hk = h / (a.heads / a.heads_k);
  const int64_t slot = (int64_t)ci * a.heads + h, hd = (int64_t)a.heads * D;
  const float* const rows = a.rows + slot * 3 * kChunk;
  const T* const kp = (const T*)a.k.p + (int64_t)ch.x * a.k.ld + hk * D;
  const T* const qp = (const T*)a.q.p + (int64_t)ch.x * a.q.ld + hk * D;
  const T* const vp = (const T*)a.v.p + (int64_t)ch.x * a.v.ld + h * D;
  const T* const op = (const T*)s.d_o.p + (int64_t)ch.x * s.d_o.ld + h * D;
  const float* const up = s.u + ((int64_t)ch.x * a.heads + h) * D;
  const float* const xp = s.x + ((int64_t)ch.x * a.heads + h) * D;
  stage256<D, F32>(kl, kp, a.k.ld, count);
  stage256<D, F32>(ql, qp, a.q.ld, count);
  if (w == 0) {
    float gl = lane < count ? a.g[((int64_t)ch.x + lane) * a.heads + h] : 0.f;
    if (gl < kMinLogDecay) gl = kMinLogDecay;
    double sum = gl;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
      const double o = __shfl_up(sum, m, 64);
      if (lane >= m) sum += o;
    }
    cs[lane] = sum;
  }
  const int t = 16 * w + c;  // the lane's column
  const bool live = t < count;
  const float gam = rows[t], dec = rows[kChunk + t], beta = rows[2 * kChunk + t];
  Parts<NT> ob[KS];
  Parts<3> xb[KS], ub[KS];
  float xv = 0.f;
#pragma unroll
  for (int k = 0; k < KS; ++k) {
    const int col = 32 * k + 8 * g;
    ob[k] = tok8<NT>(op, s.d_o.ld, t, count, col);
    xb[k] = tok8<3>(xp, hd, t, count, col);
    ub[k] = tok8<3>(up, hd, t, count, col);
    if (live) {
      float v[8];
      load4(vp + (int64_t)t * a.v.ld + col, v);
      load4(vp + (int64_t)t * a.v.ld + col + 4, v + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) xv = fmaf(xp[(int64_t)t * hd + col + e], v[e], xv);
    }
  }
  __syncthreads();

  // the states' parts: dQ, dK by dims, and their products with q, k
  f32x4 dq[MT], dk[MT];
  float sq = 0.f, sx = 0.f, su = 0.f, fr = 0.f;
  const float* const m0 = s.m_in + slot * D * D;
  const float* const m1 = s.d_m + slot * D * D;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    f32x4 aq = {0.f, 0.f, 0.f, 0.f}, ax = aq, au = aq;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int64_t at = (int64_t)(16 * mt + c) * D + 32 * k + 8 * g;
      const Parts<3> p0 = load8(m0 + at), p1 = load8(m1 + at);
      mma<2>(aq, p0, ob[k]);
      mma<2>(ax, p0, xb[k]);
      mma<2>(au, p1, ub[k]);
      if (w == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) fr = fmaf(m0[at + e], m1[at + e], fr);
      }
    }
    float qv[4] = {0.f, 0.f, 0.f, 0.f}, kv[4] = {0.f, 0.f, 0.f, 0.f};
    if (live) {
      load4(qp + (int64_t)t * a.q.ld + 16 * mt + 4 * g, qv);
      load4(kp + (int64_t)t * a.k.ld + 16 * mt + 4 * g, kv);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float eq = a.scale * gam * aq[r], ex = gam * ax[r], eu = dec * au[r];
      sq = fmaf(eq, qv[r], sq);
      sx = fmaf(ex, kv[r], sx);
      su = fmaf(eu, kv[r], su);
      dq[mt][r] = eq;
      dk[mt][r] = fmaf(-beta, ex, eu);
    }
  }
  // the triangles, rows l = 16 it + 4 g + r against the column t
  f32x4 wl[4], wu[4], z[4];
  float rowp = 0.f, colp = 0.f, rowe = 0.f, cole = 0.f, xk = 0.f;
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    wl[it] = wu[it] = z[it] = f32x4{0.f, 0.f, 0.f, 0.f};
    f32x4 pl = wl[it], xl = wl[it], pu = wl[it], xu = wl[it], kk = wl[it], ql1 = wl[it], qu = wl[it];
    const int row = 16 * it + c;
    if (it <= w) {
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int col = 32 * k + 8 * g;
        const auto ua = tok8<3>(up, hd, row, count, col);
        mma<2>(pl, ua, ob[k]);
        mma<2>(xl, ua, xb[k]);
      }
    }
    if (it >= w) {
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int col = 32 * k + 8 * g;
        mma<2>(pu, tok8<NT>(op, s.d_o.ld, row, count, col), ub[k]);
        mma<2>(xu, tok8<3>(xp, hd, row, count, col), ub[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const int col = 32 * k + 8 * g;
      const auto ka = lds_row<D, F32>(kl, row, col), kb = lds_row<D, F32>(kl, t, col);
      mma<NT - 1>(kk, ka, kb);
      if (it <= w) mma<NT - 1>(ql1, ka, lds_row<D, F32>(ql, t, col));
      if (it >= w) mma<NT - 1>(qu, lds_row<D, F32>(ql, row, col), kb);
    }
    const f32x4 bl = *(const f32x4*)(rows + 2 * kChunk + 16 * it + 4 * g);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int l = 16 * it + 4 * g + r;
      if (l <= t) {
        const float gd = expf((float)(cs[t] - cs[l]));
        wl[it][r] = a.scale * gd * pl[r];
        if (l < t) {
          rowp = fmaf(wl[it][r], ql1[r], rowp);
          const float x = gd * xl[r];
          xk = fmaf(x, kk[r], xk);
          z[it][r] = -beta * x;
          rowe = fmaf(z[it][r], kk[r], rowe);
        }
      }
      if (l >= t) {
        const float gd = expf((float)(cs[l] - cs[t]));
        wu[it][r] = a.scale * gd * pu[r];
        if (l > t) {
          colp = fmaf(wu[it][r], qu[r], colp);
          z[it][r] = -bl[r] * gd * xu[r];
          cole = fmaf(z[it][r], kk[r], cole);
        }
      }
    }
  }
  // dQ += W K, dK += W^T Q + (E + E^T) K
#pragma unroll
  for (int ts = 0; ts < 2; ++ts) {
    const Parts<NW> bl = split_tiles<NW>(wl[2 * ts], wl[2 * ts + 1]);
    const Parts<NW> bu = split_tiles<NW>(wu[2 * ts], wu[2 * ts + 1]);
    const Parts<NW> bz = split_tiles<NW>(z[2 * ts], z[2 * ts + 1]);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const auto ka = lds_col_plain<D, F32>(kl, mt, ts, g, c);
      const auto qa = lds_col_plain<D, F32>(ql, mt, ts, g, c);
      mma<NW - 1>(dq[mt], ka, bl);
      mma<NW - 1>(dk[mt], ka, bz);
      mma<NW - 1>(dk[mt], qa, bu);
    }
  }
  if (live) {
    const int64_t tok = (int64_t)ch.x + t;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int col = 16 * mt + 4 * g;
      if (s.dq) {
        store4((T*)s.dq + tok * s.ld_dq + h * D + col, dq[mt]);
        store4((T*)s.dk + tok * s.ld_dk + h * D + col, dk[mt]);
      } else {
        store4(s.dq_part + (tok * a.heads + h) * D + col, dq[mt]);
        store4(s.dk_part + (tok * a.heads + h) * D + col, dk[mt]);
      }
    }
  }
  xv = sum_groups(xv);
  sq = sum_groups(sq);
  sx = sum_groups(sx);
  su = sum_groups(su);
  xk = sum_groups(xk);
  const float tri = sum_groups(rowp - colp) + sum_groups(rowe - cole);
  if (g == 0) {
    if (live) s.dbeta[((int64_t)ch.x + t) * a.heads + h] = xv - sx - xk;
    dcs[t] = sq - beta * sx - su + tri;
  }
  float all = su;
#pragma unroll
  for (int x = 1; x < 16; x *= 2) all += __shfl_xor(all, x, 64);
  if (lane == 0) ends[w] = all;
  if (w == 0) {
#pragma unroll
    for (int x = 1; x < 64; x *= 2) fr += __shfl_xor(fr, x, 64);
    if (lane == 0) frob = fr;
  }
  __syncthreads();
  if (w == 0) {
    double sum = dcs[lane];
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
      const double o = __shfl_down(sum, m, 64);
      if (lane + m < 64) sum += o;
    }
    sum += (double)(ends[0] + ends[1] + ends[2] + ends[3]) + (double)rows[kChunk - 1] * frob;
    if (lane < count) s.dg[((int64_t)ch.x + lane) * a.heads + h] = (float)sum;
  }
}

// dq and dk of key heads from their value heads' parts, in head order: a workgroup per
// (chunk, key head).
template <int D, bool F32>
__global__ __launch_bounds__(256) void k_delta_group_sum(DeltaArgs a, DeltaGradArgs s, void* dq,
                                                         void* dk) {
  using T = typename Tok<F32>::T;
  const int hk = blockIdx.x % a.heads_k;
  const int4 ch = delta_chunk(a.sq, blockIdx.x / a.heads_k);
  const int rep = a.heads / a.heads_k;
  for (int i = threadIdx.x; i < ch.y * (D / 4); i += 256) {
    const int64_t tok = (int64_t)ch.x + i / (D / 4);
    const int col = 4 * (i % (D / 4));
    f32x4 sq = {0.f, 0.f, 0.f, 0.f}, sk = sq;
    for (int r = 0; r < rep; ++r) {
      const int64_t at = (tok * a.heads + hk * rep + r) * D + col;
      sq += *(const f32x4*)(s.dq_part + at);
      sk += *(const f32x4*)(s.dk_part + at);
    }
    store4((T*)dq + tok * s.ld_dq + hk * D + col, sq);
    store4((T*)dk + tok * s.ld_dk + hk * D + col, sk);
  }
}

template <int D, bool F32>
hipError_t reverse_any(const DeltaArgs& a, const DeltaGradArgs& s, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.sq.n_segs * a.heads)), blk(2 * D);
  if (s.e_out) hipLaunchKernelGGL((k_delta_reverse<D, F32, true>), grid, blk, 0, st, a, s);
  else hipLaunchKernelGGL((k_delta_reverse<D, F32, false>), grid, blk, 0, st, a, s);
  return hipGetLastError();
}

template <int D, bool F32>
hipError_t grads_any(const DeltaArgs& a, const DeltaGradArgs& s, hipStream_t st) {
  DeltaGradArgs k = s;
  const bool grouped = a.heads != a.heads_k;
  if (grouped) k.dq = k.dk = nullptr;
  hipLaunchKernelGGL((k_delta_grads<D, F32>), dim3((unsigned)((int64_t)a.sq.n_chunks * a.heads)),
                     dim3(256), 0, st, a, k);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !grouped) return e;
  hipLaunchKernelGGL((k_delta_group_sum<D, F32>),
                     dim3((unsigned)((int64_t)a.sq.n_chunks * a.heads_k)), dim3(256), 0, st, a, s,
                     s.dq, s.dk);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_reverse(const DeltaArgs& a, const DeltaGradArgs& s, hipStream_t st) {
  if (a.d == 128) return a.f32 ? reverse_any<128, true>(a, s, st) : reverse_any<128, false>(a, s, st);
  return a.f32 ? reverse_any<64, true>(a, s, st) : reverse_any<64, false>(a, s, st);
}

hipError_t launch_delta_grads(const DeltaArgs& a, const DeltaGradArgs& s, hipStream_t st) {
  if (a.sq.n_chunks == 0) return hipSuccess;
  if (a.d == 128) return a.f32 ? grads_any<128, true>(a, s, st) : grads_any<128, false>(a, s, st);
  return a.f32 ? grads_any<64, true>(a, s, st) : grads_any<64, false>(a, s, st);
}

}  // namespace zm
