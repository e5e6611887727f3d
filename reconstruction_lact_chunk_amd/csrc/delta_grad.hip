// Gradient of the gated delta rule (delta_rule.h).  With dM' the gradient of M at a
// chunk's end and X = beta o R:
//   dU = P^T dO + dec o (K dM'),  dX = T^T dU,  dV = beta o dX,
//   dM = gam_C dM' + Q^T (scale gam o dO) - K^T (gam o beta o dX),
// which k_delta_reverse carries from chunk to chunk as the forward carries M (a
// wave 16 columns of d_v), and then for every chunk on its own (k_delta_grads)
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

// 8 consecutive elements of a token, as loaded.
template <bool F32>
struct Raw8 {
  u32x4 a;
  __device__ __forceinline__ void load(const uint16_t* p) { a = *(const u32x4*)p; }
  __device__ __forceinline__ Parts<1> parts() const { return Parts<1>{{as_bf16x8(a)}}; }
  __device__ __forceinline__ float at(int e) const { return e & 1 ? bf16hi(a[e >> 1]) : bf16lo(a[e >> 1]); }
};
template <>
struct Raw8<true> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *(const f32x4*)p;
    b = *(const f32x4*)(p + 4);
  }
  __device__ __forceinline__ Parts<3> parts() const { return split_tiles<3>(a, b); }
  __device__ __forceinline__ float at(int e) const { return e < 4 ? a[e & 3] : b[e & 3]; }
};

// Element `i` of uniform p: a chunk's offsets fit 32 bits (64 rows of at most 2^24).
template <typename T>
__device__ __forceinline__ T* elem(T* p, unsigned i) {
  return (T*)((char*)p + i * (unsigned)sizeof(T));
}
template <typename T>
__device__ __forceinline__ const T* elem(const T* p, unsigned i) {
  return (const T*)((const char*)p + i * (unsigned)sizeof(T));
}
// Keeps what follows from x inside the loop: hoisted addresses would not fit the registers.
__device__ __forceinline__ int pinned(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

__device__ __forceinline__ float to_float(uint16_t x) { return bf16lo(x); }
__device__ __forceinline__ float to_float(float x) { return x; }

__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = (uint16_t)pack_bf16x2(v, v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// TRANS: only the gradient that a segment adds to its start's from a zero one at its
// end (the rest of the transition is the transpose of the forward's).  What a chunk
// needs is loaded to registers while the chunk after it is computed; loaded when it is
// needed, by waves of 32 columns, a chunk took 32 us instead of 14.  Bound by the chain
// of a chunk's products: 8 sequences of 1374 bf16 tokens, 8 heads of 128, 87 us, TRANS
// 51 us.
template <int D, bool F32, bool TRANS>
__global__ __launch_bounds__(4 * D, 1) void k_delta_reverse(DeltaArgs a, DeltaGradArgs s) {
  using C = ScanCfg<D, F32>;
  using T = typename Tok<F32>::T;
  constexpr int NT = C::NT, KS = D / 32, MT = D / 16, THR = 4 * D, CPR = D / 8;
  constexpr int NI = kChunk * CPR / THR;                     // octets of K to a thread
  constexpr int FE = 3 * kTriFrags * kFragElems, NF = (2 * FE / 8 + THR - 1) / THR;
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * NT * C::TILE + 2 * FE];
  __shared__ __attribute__((aligned(16))) float rows[3 * kChunk];
  uint16_t* const kl = lds;
  uint16_t* const ql = lds + NT * C::TILE;
  uint16_t* const tf = lds + 2 * NT * C::TILE;  // T^T, P^T
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int h = blockIdx.x % a.heads, si = blockIdx.x / a.heads;
  const int4 sg = delta_seg(a.sq, si);
  if (sg.y < 0 || (TRANS && (sg.w & 1))) return;
  const int hk = h / (a.heads / a.heads_k);
  const int dv = 16 * (threadIdx.x >> 6) + c;
  const int64_t dd = (int64_t)D * D;

  f32x4 m[MT];
  const float* init = nullptr;
  if (!TRANS) {
    if (s.seg_end) init = s.seg_end + ((int64_t)si * a.heads + h) * dd;
    else if (s.dstate_out) init = s.dstate_out + ((int64_t)sg.z * a.heads + h) * dd;
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
    m[mt] = init ? *(const f32x4*)(init + (int64_t)dv * D + dim_row(mt, 4 * g))
                 : f32x4{0.f, 0.f, 0.f, 0.f};

  // all chunks of a segment but its last have kChunk tokens
  const int4 last = sg.y > 0 ? delta_chunk(a.sq, sg.x + sg.y - 1) : int4{0, 0, 0, 0};
  Raw8<F32> kr[NI], qr[NI];
  u32x4 fr[NF];
  float rr = 0.f;
  T orw[4][4];
  auto load = [&](int j) {
    const int count = j == sg.y - 1 ? last.y : kChunk;
    const int64_t first = (int64_t)last.x - (int64_t)kChunk * (sg.y - 1 - j);
    const int64_t slot = (int64_t)(sg.x + j) * a.heads + h;
    const T* const kp = (const T*)a.k.p + first * a.k.ld + hk * D;
    const T* const qp = (const T*)a.q.p + first * a.q.ld + hk * D;
    const T* const op = (const T*)s.d_o.p + first * s.d_o.ld + h * D;
    const int tid = pinned(threadIdx.x), tg = pinned(token_row(0, 4 * g));
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int at = tid + THR * i, row = at / CPR, col = 8 * (at % CPR);
      const int r = row < count ? row : count - 1;
      kr[i].load(elem(kp, r * (unsigned)a.k.ld + col));
      qr[i].load(elem(qp, r * (unsigned)a.q.ld + col));
    }
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      const int at = tid + THR * i;  // a wave's 64 lie in one of the two: FE is 18 of them
      if (at < 2 * FE / 8)
        fr[i] = *(const u32x4*)(at < FE / 8 ? elem(a.tt_frags + slot * FE, at * 8)
                                            : elem(a.pt_frags + slot * FE, at * 8 - FE));
    }
    if (threadIdx.x < 3 * kChunk) rr = a.rows[slot * 3 * kChunk + threadIdx.x];
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = token_row(it, 0) + tg + r;
        orw[it][r] = *elem(op, (t < count ? t : count - 1) * (unsigned)s.d_o.ld + dv);
      }
  };
  if (sg.y > 0) load(sg.y - 1);

  for (int j = sg.y - 1; j >= 0; --j) {
    const int count = j == sg.y - 1 ? last.y : kChunk;
    const int64_t first = (int64_t)last.x - (int64_t)kChunk * (sg.y - 1 - j);
    const int64_t slot = (int64_t)(sg.x + j) * a.heads + h;
    lds_barrier();  // the last chunk's reads are done
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int at = threadIdx.x + THR * i, row = at / CPR, col = 8 * (at % CPR);
      const auto kp = row < count ? kr[i].parts() : zero_parts<NT>();
      const auto qp = row < count ? qr[i].parts() : zero_parts<NT>();
#pragma unroll
      for (int p = 0; p < NT; ++p) {
        *(bf16x8*)(kl + p * C::TILE + row * C::PITCH + col) = kp.p[p];
        *(bf16x8*)(ql + p * C::TILE + row * C::PITCH + col) = qp.p[p];
      }
    }
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      const int at = threadIdx.x + THR * i;
      if (at < 2 * FE / 8) *(u32x4*)(tf + at * 8) = fr[i];
    }
    if (threadIdx.x < 3 * kChunk) rows[threadIdx.x] = rr;
    f32x4 go[4];
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        go[it][r] = token_row(it, 4 * g + r) < count ? to_float(orw[it][r]) : 0.f;
    if (j > 0) load(j - 1);
    lds_barrier();

    if (!TRANS) {
      float* const mo = s.d_m + slot * dd;
      const int at = pinned((dv >> 5) * D * 32 + dim_row(0, 4 * g) * 32 + (dv & 31));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 4; ++r) *elem(mo, at + (dim_row(mt, 0) + r) * 32) = m[mt][r];
    }
    // dU = dec o (K dM') + P^T dO
    f32x4 du[4];
#pragma unroll
    for (int it = 0; it < 4; ++it) du[it] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const Parts<3> b = split_tiles<3>(m[2 * k], m[2 * k + 1]);
#pragma unroll
      for (int it = 0; it < 4; ++it)
        mma<2>(du[it], lds_row<D, F32>(kl, token_row(it, c), 32 * k + 8 * g), b);
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) du[it] *= *(const f32x4*)(rows + kChunk + token_row(it, 4 * g));
#pragma unroll
    for (int ts = 0; ts < 2; ++ts) {
      const Parts<NT> b = split_tiles<NT>(go[2 * ts], go[2 * ts + 1]);
#pragma unroll
      for (int it = 0; it < 2 * ts + 2; ++it) mma<2>(du[it], frag<3>(tf + FE, up_frag(it, ts), lane), b);
    }
    // dX = T^T dU
    f32x4 x[4];
#pragma unroll
    for (int it = 0; it < 4; ++it) x[it] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ts = 0; ts < 2; ++ts) {
      const Parts<3> b = split_tiles<3>(du[2 * ts], du[2 * ts + 1]);
#pragma unroll
      for (int it = 0; it < 2 * ts + 2; ++it) mma<2>(x[it], frag<3>(tf, up_frag(it, ts), lane), b);
    }
    // dV, and the factors of the state's step: scale gam o dO and -gam o beta o dX
    T* const vp = (T*)s.dv + first * s.ld_dv + h * D;
    float* const xp = s.x + slot * kChunk * D + (dv >> 5) * kChunk * 32 + (dv & 31);
    const int tg = pinned(token_row(0, 4 * g));
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int t0 = token_row(it, 0) + tg;
      const f32x4 gm = *(const f32x4*)(rows + t0), be = *(const f32x4*)(rows + 2 * kChunk + t0);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (!TRANS && t0 + r < count) {
          xp[(t0 + r) * 32] = x[it][r];
          store1(elem(vp, (t0 + r) * (unsigned)s.ld_dv + dv), be[r] * x[it][r]);
        }
        x[it][r] *= -gm[r] * be[r];
        go[it][r] *= a.scale * gm[r];
      }
    }
    const float gl = rows[kChunk - 1];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) m[mt] *= gl;
#pragma unroll
    for (int ts = 0; ts < 2; ++ts) {
      const Parts<3> b = split_tiles<3>(x[2 * ts], x[2 * ts + 1]);
      const Parts<3> d = split_tiles<3>(go[2 * ts], go[2 * ts + 1]);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        mma<2>(m[mt], lds_col<D, F32>(kl, mt, ts, g, c), b);
        mma<2>(m[mt], lds_col<D, F32>(ql, mt, ts, g, c), d);
      }
    }
  }

  float* out = nullptr;
  if (TRANS) out = s.e_out + ((int64_t)si * a.heads + h) * dd;
  else if ((sg.w & 1) && s.dstate_in) out = s.dstate_in + ((int64_t)sg.z * a.heads + h) * dd;
  if (out) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
      *(f32x4*)(out + (TRANS ? join_b<D>(dv, mt, g) : dv * D + dim_row(mt, 4 * g))) = m[mt];
  }
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

// The chunk's operands in LDS as fragments: 16 tokens x 32 dims of one part are 512
// elements, octet g of token c those of lane 16 g + c.
constexpr int kSlice = 4 * kFragElems;  // 64 tokens x 32 dims

template <int NP>
__device__ __forceinline__ Parts<NP> slice_frag(const uint16_t* f, int tile, int lane) {
  Parts<NP> p;
#pragma unroll
  for (int k = 0; k < NP; ++k) p.p[k] = *(const bf16x8*)(f + k * kSlice + tile * kFragElems + lane * 8);
  return p;
}
template <int NP>
__device__ __forceinline__ void put_frag(uint16_t* f, int tile, int lane, const Parts<NP>& v) {
#pragma unroll
  for (int k = 0; k < NP; ++k) *(bf16x8*)(f + k * kSlice + tile * kFragElems + lane * 8) = v.p[k];
}
// Two transposing reads: elements 0..3 and 4..7, the latter's rows 4 further.
__device__ __forceinline__ bf16x8 read_tr8(const uint16_t* at) {
  return __builtin_shufflevector(delta_read_tr(at), delta_read_tr(at + 4 * 8), 0, 1, 2, 3, 4, 5, 6, 7);
}

// One workgroup per (chunk, head), a wave to 16 dims: M and dM' rows, loaded and
// taken apart by the one wave that needs them, times the chunk's dO, dX and U,
// which all waves share through LDS, 32 dims at a time and read ahead by one such
// slice.  W and E take three parts as all else: where a token replaced a large value W K takes
// it off M^T dO again.  The 16 x 16 tiles of the triangles go round the waves on the way; W and E
// are then shared through LDS for the products with K and Q.  8 sequences of 1374 bf16
// tokens, 8 heads of 128: 148 us, 3.1 TB/s; half of a workgroup's 25 us are the slices
// (M, dM', U and dX of fp32), half the start, the triangles and the sums, and its 99 KB
// of LDS let one run on a compute unit.  With every wave splitting all of M and dM' it
// took 505 us; workgroups that go on to the next chunk, or two slices read ahead, 152 of 146.
template <int D, bool F32>
__global__ __launch_bounds__(4 * D, 2) void k_delta_grads(DeltaArgs a, DeltaGradArgs s) {
  using T = typename Tok<F32>::T;
  constexpr int NT = Tok<F32>::NT, KS = D / 32, MT = D / 16, NW = 3, THR = 4 * D;
  constexpr int SETS = 512 / THR, TPW = (12 + MT - 1) / MT;
  // a buffer: dX and U of 3 parts, dO, and for fp32 K and Q; bf16 K and Q stay whole
  constexpr int BUF = (6 + NT + (F32 ? 2 * NT : 0)) * kSlice;
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * BUF + (F32 ? 0 : 2 * KS * kSlice)];
  __shared__ double cs[kChunk];
  __shared__ __attribute__((aligned(16))) float rows[3 * kChunk];
  __shared__ float red[3][MT][kChunk], tri_i[10][16], tri_j[10][16], tri_x[10][16], xvs[kChunk], frs[MT];
  uint16_t* const wl = lds;                              // W, E: after the slices
  uint16_t* const el = lds + NW * 2 * kSlice;
  const int h = blockIdx.x % a.heads, ci = blockIdx.x / a.heads;
  const int4 ch = delta_chunk(a.sq, ci);
  const int count = ch.y;
  if (count == 0) return;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int hk = h / (a.heads / a.heads_k);
  const int64_t slot = (int64_t)ci * a.heads + h;
  const T* const kp = (const T*)a.k.p + (int64_t)ch.x * a.k.ld + hk * D;
  const T* const qp = (const T*)a.q.p + (int64_t)ch.x * a.q.ld + hk * D;
  const T* const vp = (const T*)a.v.p + (int64_t)ch.x * a.v.ld + h * D;
  const T* const op = (const T*)s.d_o.p + (int64_t)ch.x * s.d_o.ld + h * D;
  const float* const up = s.u + slot * kChunk * D + 8 * g;
  const float* const xp = s.x + slot * kChunk * D + 8 * g;
  const float* const m0 = s.m_in + slot * D * D + (16 * w + c) * 32 + 8 * g;
  const float* const m1 = s.d_m + slot * D * D + (16 * w + c) * 32 + 8 * g;
  auto k_at = [&](int sl) { return F32 ? lds + (sl & 1) * BUF + 9 * kSlice : lds + 2 * BUF + sl * kSlice; };
  auto q_at = [&](int sl) {
    return F32 ? lds + (sl & 1) * BUF + 12 * kSlice : lds + 2 * BUF + (KS + sl) * kSlice;
  };

  // Set 0: dX, K, and V for dX.V; set 1: U, Q, dO.  Four waves take a set.
  const int st = 16 * (w & 3) + c, srow = st < count ? st : count - 1;
  f32x4 xr[SETS][2];
  Raw8<F32> br[SETS], cr[SETS];
  f32x4 mr[4];
  float xv = 0.f, fr = 0.f;
  auto load = [&](int sl) {
    const int col = 32 * sl + 8 * g;
#pragma unroll
    for (int i = 0; i < SETS; ++i) {
      const bool second = SETS == 1 ? w >= 4 : i == 1;
      const float* const f = (second ? up : xp) + sl * kChunk * 32 + srow * 32;
      xr[i][0] = *(const f32x4*)f;
      xr[i][1] = *(const f32x4*)(f + 4);
      br[i].load((second ? qp + srow * a.q.ld : kp + srow * a.k.ld) + col);
      cr[i].load((second ? op + srow * s.d_o.ld : vp + srow * a.v.ld) + col);
    }
    mr[0] = *(const f32x4*)(m0 + 32 * D * sl);
    mr[1] = *(const f32x4*)(m0 + 32 * D * sl + 4);
    mr[2] = *(const f32x4*)(m1 + 32 * D * sl);
    mr[3] = *(const f32x4*)(m1 + 32 * D * sl + 4);
  };
  auto put = [&](int sl) {
    uint16_t* const buf = lds + (sl & 1) * BUF;
    const bool live = st < count;
#pragma unroll
    for (int i = 0; i < SETS; ++i) {
      const bool second = SETS == 1 ? w >= 4 : i == 1;
      const auto x = split_tiles<3>(xr[i][0], xr[i][1]);
      put_frag(buf + (second ? 3 * kSlice : 0), w & 3, lane, live ? x : zero_parts<3>());
      put_frag(second ? q_at(sl) : k_at(sl), w & 3, lane, live ? br[i].parts() : zero_parts<NT>());
      if (second) {
        put_frag(buf + 6 * kSlice, w & 3, lane, live ? cr[i].parts() : zero_parts<NT>());
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) xv = fmaf(xr[i][e >> 2][e & 3], cr[i].at(e), xv);
      }
    }
  };
  Parts<3> p0, p1;
  auto take = [&]() {
    p0 = split_tiles<3>(mr[0], mr[1]);
    p1 = split_tiles<3>(mr[2], mr[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) fr = fmaf(mr[0][e], mr[2][e], fmaf(mr[1][e], mr[3][e], fr));
  };
  load(0);
  constexpr int SUMS = MT - 1;  // the wave of the sums over tokens: it has fewest tiles below
  float gl = 0.f, rv = 0.f;
  if (w == SUMS && lane < count) gl = a.g[((int64_t)ch.x + lane) * a.heads + h];
  if (threadIdx.x < 3 * kChunk) rv = a.rows[slot * 3 * kChunk + threadIdx.x];

  f32x4 dq[4], dk[4], au[4];             // dims 16 w + 4 g + r, tokens 16 tt + c
  f32x4 pt[TPW], xt[TPW], kk[TPW], qk[TPW];  // U dO^T, U dX^T, K K^T, K Q^T: tokens j, i
#pragma unroll
  for (int i = 0; i < 4; ++i) dq[i] = dk[i] = au[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < TPW; ++i) pt[i] = xt[i] = kk[i] = qk[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  put(0);
  take();
  load(1);
  // the next slice is split and written among this one's matrix instructions
#pragma unroll
  for (int sl = 0; sl < KS; ++sl) {
    uint16_t* const buf = lds + (sl & 1) * BUF;
    lds_barrier();
    if (sl == 0) {  // out of the way of the first slice
      if (threadIdx.x < 3 * kChunk) rows[threadIdx.x] = rv;
      if (w == SUMS) {
        double sum = (gl < kMinLogDecay ? kMinLogDecay : gl) * kLog2E;  // exponents of two
#pragma unroll
        for (int m = 1; m < 64; m *= 2) {
          const double o = __shfl_up(sum, m, 64);
          if (lane >= m) sum += o;
        }
        cs[lane] = sum;
      }
    }
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
      mma<2>(dq[tt], p0, slice_frag<NT>(buf + 6 * kSlice, tt, lane));
      mma<2>(dk[tt], p0, slice_frag<3>(buf, tt, lane));
      mma<2>(au[tt], p1, slice_frag<3>(buf + 3 * kSlice, tt, lane));
      if (tt == 1 && sl + 1 < KS) put(sl + 1);
    }
    if (sl + 1 < KS) take();
    if (sl + 2 < KS) load(sl + 2);
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      const int id = w + MT * i, it = id < 1 ? 0 : (id < 3 ? 1 : (id < 6 ? 2 : 3));
      const int jt = id - it * (it + 1) / 2;
      if (id >= 10) continue;
      const auto u = slice_frag<3>(buf + 3 * kSlice, jt, lane);
      mma<2>(pt[i], u, slice_frag<NT>(buf + 6 * kSlice, it, lane));
      mma<2>(xt[i], u, slice_frag<3>(buf, it, lane));
      const auto kj = slice_frag<NT>(k_at(sl), jt, lane);
      mma<NT - 1>(kk[i], kj, slice_frag<NT>(k_at(sl), it, lane));
      mma<NT - 1>(qk[i], kj, slice_frag<NT>(q_at(sl), it, lane));
    }
  }
  lds_barrier();  // the slices are read: their place takes W and E

  // the states' parts of dQ and dK, and their products with q and k
#pragma unroll
  for (int tt = 0; tt < 4; ++tt) {
    const int t = 16 * tt + c;
    const float gam = rows[t], dec = rows[kChunk + t], beta = rows[2 * kChunk + t];
    float qv[4] = {0.f, 0.f, 0.f, 0.f}, kv[4] = {0.f, 0.f, 0.f, 0.f};
    if constexpr (F32) {
      if (t < count) {
        load4(qp + t * a.q.ld + 16 * w + 4 * g, qv);
        load4(kp + t * a.k.ld + 16 * w + 4 * g, kv);
      }
    } else {
      const int at = tt * kFragElems + (16 * (2 * (w & 1) + (g >> 1)) + c) * 8 + 4 * (g & 1);
      load4(q_at(w >> 1) + at, qv);
      load4(k_at(w >> 1) + at, kv);
    }
    float sq = 0.f, sx = 0.f, su = 0.f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float eq = a.scale * gam * dq[tt][r], ex = gam * dk[tt][r], eu = dec * au[tt][r];
      sq = fmaf(eq, qv[r], sq);
      sx = fmaf(ex, kv[r], sx);
      su = fmaf(eu, kv[r], su);
      dq[tt][r] = eq;
      dk[tt][r] = fmaf(-beta, ex, eu);
    }
    sq = sum_groups(sq);
    sx = sum_groups(sx);
    su = sum_groups(su);
    if (g == 0) {
      red[0][w][t] = sq;
      red[1][w][t] = sx;
      red[2][w][t] = su;
    }
  }
  // the triangles, columns i = 16 it + c, rows j = 16 jt + 4 g + r; the last two ids are
  // the tiles above the diagonal that share an operand with one on it
#pragma unroll
  for (int n = 0; n < TPW; ++n) {
    const int id = w + MT * n;
    if (id >= 12) continue;
    const int it = id >= 10 ? 2 * (id - 10) : (id < 1 ? 0 : (id < 3 ? 1 : (id < 6 ? 2 : 3)));
    const int jt = id >= 10 ? it + 1 : id - it * (it + 1) / 2;
    const int i = 16 * it + c;
    const double sum_i = cs[i];
    const float beta = rows[2 * kChunk + i];
    float wv[4], ev[4], si = 0.f, sx = 0.f, sj[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int j = 16 * jt + 4 * g + r;
      const float gd = exp2_wide(j <= i ? sum_i - cs[j] : 0.0), x = j < i ? gd * xt[n][r] : 0.f;
      wv[r] = j <= i ? a.scale * gd * pt[n][r] : 0.f;
      ev[r] = -beta * x;
      sx += j < i ? x * kk[n][r] : 0.f;
      sj[r] = j < i ? fmaf(wv[r], qk[n][r], ev[r] * kk[n][r]) : 0.f;
      si += sj[r];
    }
    const int at = (2 * it + (jt >> 1)) * kFragElems + (16 * (2 * (jt & 1) + (g >> 1)) + c) * 8 + 4 * (g & 1);
#pragma unroll
    for (int p = 0; p < NW; ++p) {
      const u32x2 wp = {pack_bf16x2(wv[0], wv[1]), pack_bf16x2(wv[2], wv[3])};
      const u32x2 ep = {pack_bf16x2(ev[0], ev[1]), pack_bf16x2(ev[2], ev[3])};
      *(u32x2*)(wl + p * 2 * kSlice + at) = wp;
      *(u32x2*)(el + p * 2 * kSlice + at) = ep;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        wv[r] -= r & 1 ? bf16hi(wp[r >> 1]) : bf16lo(wp[r >> 1]);
        ev[r] -= r & 1 ? bf16hi(ep[r >> 1]) : bf16lo(ep[r >> 1]);
      }
    }
    if (id >= 10) continue;
    si = sum_groups(si);
    sx = sum_groups(sx);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int m = 1; m < 16; m *= 2) sj[r] += __shfl_xor(sj[r], m, 64);
    if (g == 0) {
      tri_i[id][c] = si;
      tri_x[id][c] = sx;
    }
    if (c == 0) {
#pragma unroll
      for (int r = 0; r < 4; ++r) tri_j[id][4 * g + r] = sj[r];
    }
  }
  xv = sum_groups(st < count ? xv : 0.f);
  if (w < 4 && g == 0) xvs[16 * w + c] = xv;
#pragma unroll
  for (int m = 1; m < 64; m *= 2) fr += __shfl_xor(fr, m, 64);
  if (lane == 0) frs[w] = fr;
  lds_barrier();

  // dQ += W K, dK += W^T Q + (E + E^T) K
#pragma unroll
  for (int ts = 0; ts < 2; ++ts) {
    Parts<NT> ka, qa;  // rows: dims 16 w + c, slots: tokens 32 ts + 8 g + e
    if constexpr (F32) {
      float kv[8], qv[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int t = 32 * ts + 8 * g + e, r = t < count ? t : count - 1;
        const float x = kp[r * a.k.ld + 16 * w + c], y = qp[r * a.q.ld + 16 * w + c];
        kv[e] = t < count ? x : 0.f;
        qv[e] = t < count ? y : 0.f;
      }
      ka = split8<NT>(kv);
      qa = split8<NT>(qv);
    } else {
      const int at = (2 * ts + (g >> 1)) * kFragElems +
                     (16 * (2 * (w & 1) + ((c & 3) >> 1)) + 8 * (g & 1) + (c >> 2)) * 8 + 4 * (c & 1);
      ka.p[0] = read_tr8(k_at(w >> 1) + at);
      qa.p[0] = read_tr8(q_at(w >> 1) + at);
    }
#pragma unroll
    for (int tt = 0; tt < 4; ++tt) {
      if (ts <= tt >> 1) {
        Parts<NW> wf, ef;
#pragma unroll
        for (int p = 0; p < NW; ++p) {
          const int at = p * 2 * kSlice + (2 * tt + ts) * kFragElems + lane * 8;
          wf.p[p] = *(const bf16x8*)(wl + at);
          ef.p[p] = *(const bf16x8*)(el + at);
        }
        mma<NW - 1>(dq[tt], ka, wf);
        mma<NW - 1>(dk[tt], ka, ef);
      }
      if (ts >= tt >> 1) {
        Parts<NW> wf, ef;
#pragma unroll
        for (int p = 0; p < NW; ++p) {
          const int at = p * 2 * kSlice + (2 * (2 * ts + (g >> 1)) + (tt >> 1)) * kFragElems +
                         (16 * (2 * (tt & 1) + ((c & 3) >> 1)) + 8 * (g & 1) + (c >> 2)) * 8 + 4 * (c & 1);
          wf.p[p] = read_tr8(wl + at);
          ef.p[p] = read_tr8(el + at);
        }
        mma<NW - 1>(dk[tt], qa, wf);
        mma<NW - 1>(dk[tt], ka, ef);
      }
    }
  }
#pragma unroll
  for (int tt = 0; tt < 4; ++tt) {
    if (16 * tt + c >= count) continue;
    const int64_t tok = (int64_t)ch.x + 16 * tt + c;
    const int col = 16 * w + 4 * g;
    if (s.dq) {
      store4((T*)s.dq + tok * s.ld_dq + h * D + col, dq[tt]);
      store4((T*)s.dk + tok * s.ld_dk + h * D + col, dk[tt]);
    } else {
      store4(s.dq_part + (tok * a.heads + h) * D + col, dq[tt]);
      store4(s.dk_part + (tok * a.heads + h) * D + col, dk[tt]);
    }
  }
  if (w == SUMS) {
    const int t = lane, it = t >> 4;
    float sq = 0.f, sx = 0.f, su = 0.f, sf = 0.f, xk = 0.f, tri = 0.f;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      sq += red[0][i][t];
      sx += red[1][i][t];
      su += red[2][i][t];
      sf += frs[i];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // its row of tiles, then its column
      const int low = it * (it + 1) / 2 + (j <= it ? j : it), up = j < it ? it : j;
      const float ti = tri_i[low][t & 15], tx = tri_x[low][t & 15], tj = tri_j[up * (up + 1) / 2 + it][t & 15];
      tri += j <= it ? ti : 0.f;
      xk += j <= it ? tx : 0.f;
      tri -= j >= it ? tj : 0.f;
    }
    if (t < count) s.dbeta[((int64_t)ch.x + t) * a.heads + h] = xvs[t] - sx - xk;
    double sum = sq - rows[2 * kChunk + t] * sx - su + tri;
    float all = su;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) all += __shfl_xor(all, m, 64);
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
      const double o = __shfl_down(sum, m, 64);
      if (lane + m < 64) sum += o;
    }
    sum += (double)all + (double)rows[kChunk - 1] * sf;
    if (t < count) s.dg[((int64_t)ch.x + t) * a.heads + h] = (float)sum;
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
  const dim3 grid((unsigned)((int64_t)a.sq.n_segs * a.heads)), blk(4 * D);
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
                     dim3(4 * D), 0, st, a, k);
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
