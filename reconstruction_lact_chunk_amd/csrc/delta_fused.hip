// The chunks of a segment in order for bf16 tokens (delta_rule.h), one workgroup per
// (segment, head) with two kinds of waves:
//   D / 16 state waves: 16 columns of M (d_v) each and all its rows.  M, R and U stay
//     in registers: each is the result of one product and the right operand of
//     the next.
//   4 triangle waves, one chunk ahead: T = (I + A)^-1 and P by blocks of 16, wave i the
//     block row i, left in LDS as operand tiles for the state waves.  They also
//     start the direct loads of K and Q two chunks ahead.
// Nothing of a chunk but q, k, v, o moves through memory.  The state waves are bound
// by their own issue (matrix instructions and the splitting of fp32 operands into
// bf16 parts); the triangle waves run in the gaps.  Measured, 137400 tokens, 8 heads of
// 128 in segments of 68 chunks: outputs 551 us, 8.1 us a chunk; transitions (two runs of
// a state) 623 us, 9.2 us a chunk.  A sixth of the outputs' matrix instructions are the
// third parts of M, P and U in O (507 us without them): O is a difference of large terms
// where a token replaces a large value.  State waves of 32 columns, or on 32 x 32
// instructions, came within 5% of it; triangles formed by a kernel of their own and read
// back took 4 times as long.
//
// Decays are taken out where they can be.  With a running exponent s (the state is
// 2^s M^) and U^ = U / 2^(s + c_i), c in powers of two,
//   U^ = T^ (V / 2^(s + c_i) - K M^),  T^ = (I + strictly_lower(b_i k_i.k_j))^-1 diag(b),
//   O = scale 2^(s + c_i) (Q M^ + lower(Q K^T) U^),  M^ <- M^ + K^T U^,  s <- s + c_C:
// the same numbers up to powers of two, whose factors come from 64-bit exponents
// (exp2_wide), so nothing is lost while |s + c_i| stays under kMaxShift.  A chunk that
// would leave that range takes 2^s into M^ first; one whose own decay is over it (a
// reset) is formed with the decays in place.
#include "delta_rule.h"

namespace zm {

namespace {

enum { kOutputs = 0, kKeep = 1, kTransition = 2 };

constexpr int kDPitch = 20;         // floats of a row of a 16 x 16 block in LDS
constexpr int kBlock = 16 * kDPitch;  // A^T's blocks (J, i), J <= i, and the diagonal ones' inverses
// K tiles in LDS: this chunk's, the next one's, the one in flight; Q's third takes the
// place of the first, whose last reader is done before its load starts.
constexpr int kRingK = 3, kRingQ = 2;
constexpr float kMaxShift = 60.f;  // products of 2^60 and what a model holds stay finite
// Row factors of a chunk in LDS: V's, O's, and those of a chunk formed with its decays,
// then scalars.
enum { kRowV = 0, kRowO = 64, kRowGam = 128, kRowDec = 192, kRowEnd = 256 };
enum { kFlags = kRowEnd, kPre, kLast, kScale0, kScale1, kRowFloats = kRowEnd + 8 };
enum { kGated = 1, kShift = 2 };

template <int V>
struct Const {
  static constexpr int value = V;
};

template <int D, int MODE>
struct FusedCfg {
  static constexpr int SW = D / 16;             // state waves
  static constexpr int TW = 4;                  // triangle waves
  static constexpr int THREADS = 64 * (SW + TW);
  static constexpr int GPR = D / 8;             // 16-byte granules of a row
  static constexpr int TILE = kChunk * D;       // elements of a K or Q tile
  static constexpr bool Q = MODE == kOutputs;
  static constexpr int TRI = kTriFrags * kFragElems;  // elements of one part of a triangle
  // byte offsets
  static constexpr int kOffK = 0;
  static constexpr int kOffQ = kRingK * TILE * 2;
  static constexpr int kOffT = kOffQ + (Q ? kRingQ * TILE * 2 : 0);
  static constexpr int kOffP = kOffT + 3 * TRI * 2;
  static constexpr int kOffV = kOffP + (Q ? 3 * TRI * 2 : 0);
  static constexpr int kOffRows = kOffV + TILE * 2;                    // two chunks' factors
  static constexpr int kOffAt = kOffRows + 2 * kRowFloats * 4;
  static constexpr int kOffD = kOffAt + 10 * kBlock * 4;
  static constexpr int kOffDt = kOffD + 4 * kBlock * 4;
  static constexpr int kOffCs = kOffDt + 4 * kBlock * 4;
  static constexpr int kOffBe = kOffCs + TW * kChunk * 8;
  static constexpr int BYTES = kOffBe + TW * kChunk * 4;
  static_assert(BYTES <= 160 * 1024, "LDS");
};

typedef __attribute__((address_space(3))) void lds_void;

// Row `row` of block (J, i) of A^T: columns J of A, rows i.
__device__ __forceinline__ constexpr int at_row(int J, int i, int row) {
  return (i * (i + 1) / 2 + J) * kBlock + row * kDPitch;
}

// Tiles hold row r's granule p at place p ^ swizzle(r): row reads (16 rows of tile
// order, two granules) and transposing reads spread over the banks.
template <int D>
__device__ __forceinline__ constexpr int swizzle(int r) {
  return D == 128 ? ((r & 3) << 2) | (((r >> 4) & 1) << 1) : (((r >> 1) & 1) << 2) | (((r >> 4) & 1) << 1);
}
template <int D>
__device__ __forceinline__ Parts<1> tile_row(const uint16_t* t, int row, int granule) {
  return Parts<1>{{*(const bf16x8*)(t + row * D + 8 * (granule ^ swizzle<D>(row)))}};
}
// What one wave issues is in order, and a matrix instruction leaves room for others
// while it runs: these place V vector operations after each of N matrix
// instructions, and LDS reads between such groups, ahead of their use.
template <int N, int V>
__device__ __forceinline__ void weave() {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // matrix
    __builtin_amdgcn_sched_group_barrier(0x002, V, 0);  // vector
  }
}
template <int N>
__device__ __forceinline__ void weave_reads() {
  __builtin_amdgcn_sched_group_barrier(0x100, N, 0);  // LDS reads
}

__device__ __forceinline__ void wait_direct_loads() { __builtin_amdgcn_s_waitcnt(0x0f70); }  // vmcnt(0)

template <int D, int MODE>
__global__ __launch_bounds__(64 * (D / 16 + 4)) void k_delta_fused(DeltaArgs a, DeltaScanArgs sa) {
  using C = FusedCfg<D, MODE>;
  constexpr int KS = D / 32, MT = D / 16;
  __shared__ __attribute__((aligned(16))) unsigned char smem[C::BYTES];
  const int h = blockIdx.x % a.heads, si = blockIdx.x / a.heads;
  const int4 sg = delta_seg(a.sq, si);
  if (sg.y < 0) return;
  // nothing follows the last segment; its N serves the way back
  if (MODE == kTransition && (sg.w & 2) && !sa.both) return;
  const int n = sg.y;
  const int hk = h / (a.heads / a.heads_k);
  int64_t tok0 = 0;
  int last = 0;  // tokens of the last chunk
  if (n > 0) {
    tok0 = delta_chunk(a.sq, sg.x).x;
    last = delta_chunk(a.sq, sg.x + n - 1).y;
  }
  auto k_tile = [&](int j) { return (uint16_t*)(smem + C::kOffK) + (j % kRingK) * C::TILE; };
  auto q_tile = [&](int j) { return (uint16_t*)(smem + C::kOffQ) + (j % kRingQ) * C::TILE; };
  uint16_t* const tf = (uint16_t*)(smem + C::kOffT);
  uint16_t* const pf = (uint16_t*)(smem + C::kOffP);
  uint16_t* const vt = (uint16_t*)(smem + C::kOffV);
  auto row_factors = [&](int j) { return (float*)(smem + C::kOffRows) + (j & 1) * kRowFloats; };
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;

  // the tiles' upper triangles stay zero
  for (int i = threadIdx.x; i < (C::kOffV - C::kOffT) / 16; i += C::THREADS)
    *(u32x4*)(smem + C::kOffT + 16 * i) = u32x4{0u, 0u, 0u, 0u};

  if (wave >= C::SW) {
    // ---- triangle waves: wave PW has block row PW of A and T and block row 3 - PW of P,
    // five tiles each ----
    const uint16_t* const kp = (const uint16_t*)a.k.p + tok0 * a.k.ld + hk * D;
    const uint16_t* const qp = (const uint16_t*)a.q.p + tok0 * a.q.ld + hk * D;
    const uint16_t* const vp = (const uint16_t*)a.v.p + tok0 * a.v.ld + h * D;
    float* const at = (float*)(smem + C::kOffAt);
    float* const dm = (float*)(smem + C::kOffD);
    float* const dt = (float*)(smem + C::kOffDt);
    auto triangle = [&](auto which) {
      constexpr int PW = decltype(which)::value, PI = 3 - PW;
      double* const cs = (double*)(smem + C::kOffCs) + PW * kChunk;  // the wave's own
      float* const bs = (float*)(smem + C::kOffBe) + PW * kChunk;
      double shift = 0.0;   // s, the same in every triangle wave
      bool gated = false;   // of the chunk at hand

      // Rows past the chunk's tokens take the last one's: finite where that is, and
      // their beta of zero leaves them out.
      // A lane's place in a load is a 32-bit offset from the load's first row, one of
      // two as the swizzle takes bit 4 of the row.
      constexpr int RPL = 64 / C::GPR, LOADS = kChunk / RPL / C::TW;  // rows of a load; loads of a wave
      const int lr = lane / C::GPR;
      struct Source {
        const char* base;
        int64_t ld;       // bytes
        unsigned off[2];
      };
      auto source = [&](const uint16_t* p, int64_t ld) {
        Source r{(const char*)p, ld * 2, {0u, 0u}};
#pragma unroll
        for (int i = 0; i < 2; ++i)
          r.off[i] = (unsigned)(lr * ld + 8 * ((lane % C::GPR) ^ swizzle<D>(lr + 16 * i))) * 2u;
        return r;
      };
      auto load_tile = [&](const Source& s, uint16_t* dst, int j) {
        if (j < n - 1 || last == kChunk) {
#pragma unroll
          for (int i = 0; i < LOADS; ++i) {
            const int r0 = (PW * LOADS + i) * RPL;
            const char* const from = s.base + ((int64_t)kChunk * j + r0) * s.ld;
            __builtin_amdgcn_global_load_lds((const void*)(from + s.off[(r0 >> 4) & 1]), (lds_void*)(dst + r0 * D), 16,
                                             0, 0);
          }
        } else {
          const int top = last - 1;
#pragma unroll 1
          for (int i = 0; i < LOADS; ++i) {
            const int r0 = (PW * LOADS + i) * RPL, r = r0 + lr;
            const char* const from = s.base + ((int64_t)kChunk * j + (r < top ? r : top)) * s.ld;
            const int col = 8 * ((lane % C::GPR) ^ swizzle<D>(r));
            __builtin_amdgcn_global_load_lds((const void*)(from + 2 * col), (lds_void*)(dst + r0 * D), 16, 0, 0);
          }
        }
      };
      const Source ks = source(kp, a.k.ld), qs = C::Q ? source(qp, a.q.ld) : ks, vs = source(vp, a.v.ld);
      auto load_k = [&](int j) { load_tile(ks, k_tile(j), j); };
      auto load_q = [&](int j) {
        if (C::Q) load_tile(qs, q_tile(j), j);
      };
      auto load_v = [&](int j) { load_tile(vs, vt, j); };
      float gn = 0.f, bn = 0.f;
      auto load_gates = [&](int j) {
        gn = bn = 0.f;
        if (lane < (j == n - 1 ? last : kChunk)) {
          const int64_t t = (tok0 + (int64_t)kChunk * j + lane) * a.heads + h;
          gn = a.g[t];
          bn = a.beta[t];
        }
      };
      f32x4 tt[4], pt[4];  // T^T and P^T: rows are columns of T and P
      auto tile = [&](const uint16_t* t, int block, Parts<1>* f) {
#pragma unroll
        for (int k = 0; k < KS; ++k) f[k] = tile_row<D>(t, 16 * block + c, 4 * k + g);
      };
      // K K^T, A^T and the diagonal block's inverse
      auto factor = [&](int j) {
        const uint16_t* const kt = k_tile(j);
        const float be = bn;
        double s = gn < kMinLogDecay ? kMinLogDecay : gn;
        s *= kLog2E;  // exponents of two from here
        if (j + 1 < n) load_gates(j + 1);
        Parts<1> ki[KS];
        tile(kt, PW, ki);
        // sums in 64 bits: a strong decay among weak ones must not blur their differences
#pragma unroll
        for (int m = 1; m < 64; m *= 2) {
          const double o = __shfl_up(s, m, 64);
          if (lane >= m) s += o;
        }
        bs[lane] = be;
        f32x4 kk[4];
#pragma unroll
        for (int J = 0; J <= PW; ++J) {
          kk[J] = f32x4{0.f, 0.f, 0.f, 0.f};
          Parts<1> kj[KS];
          if (J < PW) tile(kt, J, kj);
#pragma unroll
          for (int k = 0; k < KS; ++k) mma<0>(kk[J], ki[k], J < PW ? kj[k] : ki[k]);
        }
        // the chunk's form (a NaN decay keeps the decays in place)
        gated = __any(!(fabsf((float)s) <= kMaxShift));
        const bool move = gated ? shift != 0.0 : __any(!(fabsf((float)(shift + s)) <= kMaxShift));
        const double from = shift, end = __shfl(s, 63, 64);
        if (move) shift = 0.0;
        if (PW == 0) {
          float* const r = row_factors(j);
          const double at = shift + s;
          const float up = exp2_wide(at);
          r[kRowV + lane] = gated ? 1.f : exp2_wide(-at);
          r[kRowO + lane] = gated ? 1.f : C::Q ? a.scale * up : up;
          if (gated) {
            r[kRowGam + lane] = up;
            r[kRowDec + lane] = exp2_wide(end - s);
          }
          if (lane == 0) {
            ((unsigned*)r)[kFlags] = (gated ? kGated : 0) | (move ? kShift : 0);
            r[kPre] = exp2_wide(from);
            r[kLast] = exp2_wide(end);
            r[kScale0] = exp2_wide(shift);
            r[kScale1] = gated ? 1.f : exp2_wide(shift + end);
          }
        }
        if (gated) cs[lane] = s;
        else shift += end;
        const f32x4 bi = *(const f32x4*)(bs + 16 * PW + 4 * g);
#pragma unroll
        for (int J = PW; J >= 0; --J) {
          f32x4 av;
#pragma unroll
          for (int r = 0; r < 4; ++r) av[r] = J < PW || 4 * g + r > c ? bi[r] * kk[J][r] : 0.f;
          if (gated) {
            const double cj = cs[16 * J + c];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              // above the diagonal the exponent may be positive: not taken
              const float e = exp2_wide(cs[16 * PW + 4 * g + r] - cj);
              if (J < PW || 4 * g + r > c) av[r] *= e;
            }
          }
          *(f32x4*)(at + at_row(J, PW, c) + 4 * g) = av;
        }
        // row c of the inverse, from its end: a forward substitution, which (unlike a
        // product of powers of A) stays exact where keys repeat
        float x[16];
        const float* const blk = at + at_row(PW, PW, 0);
#pragma unroll
        for (int i = 15; i >= 0; --i) {
          f32x4 row[4];
#pragma unroll
          for (int q = 3; q >= 0; --q)
            if (4 * q + 3 > i) row[q] = *(const f32x4*)(blk + i * kDPitch + 4 * q);
          // two chains: the newest entry last
          float v = i == c ? 1.f : 0.f, y = 0.f;
#pragma unroll
          for (int q = 15; q > i; --q) {
            if (q & 1) v = fmaf(-row[q / 4][q % 4], x[q], v);
            else y = fmaf(-row[q / 4][q % 4], x[q], y);
          }
          x[i] = v + y;
        }
        if (g == 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *(f32x4*)(dm + (16 * PW + c) * kDPitch + 4 * i) =
                f32x4{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
#pragma unroll
          for (int i = 0; i < 16; ++i) dt[(16 * PW + i) * kDPitch + c] = x[i];
        }
      };
      // block row PW of T, transposed:  T_iw^T = -D_w^T sum_{w < j <= i} A_jw^T T_ij^T
      // on fp32 matrix instructions whose results are the next right operands
      auto solve = [&]() {
        f32x4 y[4], av[4][4], dv[4];
#pragma unroll
        for (int w = 0; w < PW; ++w) {
          y[w] = tt[w] = f32x4{0.f, 0.f, 0.f, 0.f};
          dv[w] = *(const f32x4*)(dt + (16 * w + c) * kDPitch + 4 * g);
#pragma unroll
          for (int j = w + 1; j <= PW; ++j) av[w][j] = *(const f32x4*)(at + at_row(w, j, c) + 4 * g);
        }
        tt[PW] = *(const f32x4*)(dm + (16 * PW + c) * kDPitch + 4 * g);
#pragma unroll
        for (int j = PW; j >= 0; --j) {
          if (j < PW) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              tt[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(-dv[j][r], y[j][r], tt[j], 0, 0, 0);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int w = j - 1; w >= 0; --w)
              y[w] = __builtin_amdgcn_mfma_f32_16x16x4f32(av[w][j][r], tt[j][r], y[w], 0, 0, 0);
        }
      };
      // four slots of an operand tile's lane at a time; `row` the block row of x
      auto store_tile = [&](uint16_t* to, int row, int J, const f32x4& x, int parts) {
        const int it = 2 * (row >> 1) + (c >> 3), m = 8 * (row & 1) + 4 * ((c >> 2) & 1) + (c & 3);
        uint16_t* const at2 =
            to + low_frag(it, J >> 1) * kFragElems + (16 * (2 * (J & 1) + (g & 1)) + m) * 8 + 4 * (g >> 1);
        float r[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int k = 0; k < 3; ++k) {
          if (k >= parts) continue;
          const u32x2 w = {pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3])};
          *(u32x2*)(at2 + k * C::TRI) = w;
          r[0] -= bf16lo(w[0]);
          r[1] -= bf16hi(w[0]);
          r[2] -= bf16lo(w[1]);
          r[3] -= bf16hi(w[1]);
        }
      };
      // T diag(b)
      auto store_t = [&]() {
#pragma unroll
        for (int J = 0; J <= PW; ++J) store_tile(tf, PW, J, tt[J] * *(const f32x4*)(bs + 16 * J + 4 * g), 3);
      };
      auto store_p = [&]() {
        if (!C::Q) return;
#pragma unroll
        for (int J = 0; J <= PI; ++J) store_tile(pf, PI, J, pt[J], 3);
      };
      // lower(Q K^T), or P with its decays
      auto scores = [&](int j) {
        if (!C::Q) return;
        const uint16_t* const kt = k_tile(j);
        Parts<1> qi[KS];
        tile(q_tile(j), PI, qi);
#pragma unroll
        for (int J = 0; J <= PI; ++J) {
          Parts<1> kj[KS];
          tile(kt, J, kj);
          f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < KS; ++k) mma<0>(p, kj[k], qi[k]);
#pragma unroll
          for (int r = 0; r < 4; ++r) pt[J][r] = J < PI || 4 * g + r <= c ? p[r] : 0.f;
          if (gated) {
            const double cp = cs[16 * PI + c];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float e = exp2_wide(cp - cs[16 * J + 4 * g + r]);
              if (J < PI || 4 * g + r <= c) pt[J][r] *= a.scale * e;
            }
          }
        }
      };

      __builtin_amdgcn_s_setprio(2);
      load_gates(0);
      load_k(0);
      load_q(0);
      load_v(0);
      if (n > 1) {
        load_k(1);
        load_q(1);
      }
      wait_direct_loads();
      lds_barrier();
      factor(0);
      lds_barrier();
      solve();
      store_t();
      scores(0);
      for (int j = 0; j < n; ++j) {
        wait_direct_loads();
        lds_barrier();  // everything of chunk j but P, K and Q of chunk j + 1
        store_p();      // chunk j's, first read after the next barriers
        if (j + 1 < n) factor(j + 1);
        if (j + 2 < n) load_k(j + 2);
        lds_barrier();  // A^T and the diagonal blocks; chunk j's Q and V have been read
        if (j + 1 < n) load_v(j + 1);
        if (j + 2 < n) load_q(j + 2);
        if (j + 1 < n) solve();
        lds_barrier();  // chunk j's T has been read
        if (j + 1 < n) {
          store_t();
          scores(j + 1);
        }
      }
    };
    if (n > 0) {
      switch (wave - C::SW) {
        case 0: triangle(Const<0>{}); break;
        case 1: triangle(Const<1>{}); break;
        case 2: triangle(Const<2>{}); break;
        default: triangle(Const<3>{}); break;
      }
    }
    return;
  }

  // ---- state waves ---------------------------------------------------------------
  const int dv = 16 * wave + c;  // the lane's column
  const int64_t dd = (int64_t)D * D;
  f32x4 m[MT], e[MODE == kTransition ? MT : 1];  // M; the second run of a transition's
  const float* init = nullptr;
  if (MODE != kTransition) {
    if (sa.seg_start) init = sa.seg_start + ((int64_t)si * a.heads + h) * dd;
    else if (sa.state_in) init = sa.state_in + ((int64_t)sg.z * a.heads + h) * dd;
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int dk = dim_row(mt, 4 * g);
    m[mt] = init ? *(const f32x4*)(init + (int64_t)dv * D + dk) : f32x4{0.f, 0.f, 0.f, 0.f};
    if (MODE == kTransition) {
#pragma unroll
      for (int r = 0; r < 4; ++r) e[mt][r] = dk + r == dv ? 1.f : 0.f;
    }
  }
  // Token token_row(it, 4 g + r) is the lane's first one and a uniform number of
  // rows on, so addresses are a scalar base and one 32-bit offset a lane.
  const int lt = token_row(0, 4 * g);
  const unsigned o_off = MODE == kOutputs ? (unsigned)(lt * sa.ld_o + dv) * 2u : 0u;
  char* const op = (char*)sa.o + (tok0 * sa.ld_o + h * D) * 2;
  // Byte offsets in LDS, formed anew for each chunk (pinned) rather than kept for
  // every use.  The swizzle's upper bits stand alone in a granule's address, so a
  // step along a row is an exclusive or and one down the rows an addition:
  // row token_row(0, c), granule g of a K or Q tile
  const unsigned row_off = (unsigned)(token_row(0, c) * D + 8 * (g ^ swizzle<D>(token_row(0, c)))) * 2u;
  // the transposing read of row dtau(g, c / 4), granule c % 4 of a K tile
  const int cr = dtau(g, c >> 2);
  const unsigned col_off = (unsigned)(cr * D + 8 * ((c & 3) ^ swizzle<D>(cr))) * 2u;
  // row token_row(0, 4 g), column dv of the V tile
  const unsigned v_off = (unsigned)(lt * D + 8 * ((dv / 8) ^ swizzle<D>(lt)) + dv % 8) * 2u + C::kOffV;

  if (n > 0) {
    lds_barrier();
    lds_barrier();
  }
  for (int j = 0; j < n; ++j) {
    lds_barrier();
    const int count = j == n - 1 ? last : kChunk;
    const float* const rows = row_factors(j);
    unsigned ko = row_off + (unsigned)((const unsigned char*)k_tile(j) - smem);
    unsigned qo = row_off + (unsigned)((const unsigned char*)q_tile(j) - smem);
    unsigned co = col_off + (unsigned)((const unsigned char*)k_tile(j) - smem), vo = v_off, lo = 16u * lane;
    pin(ko);
    pin(qo);
    pin(co);
    pin(vo);
    pin(lo);
    // rows of tile `it` at step s: the swizzle's high bits and s meet in bits of their own
    auto row_at = [&](unsigned off, int it, int s) {
      return *(const bf16x8*)(smem + ((off ^ (64u * s)) + (unsigned)token_row(it, 0) * D * 2));
    };
    const unsigned flags = __builtin_amdgcn_readfirstlane(((const unsigned*)rows)[kFlags]);
    // K M and Q M, the products of one order over all results in turn; operands are
    // read and M's next part is split during the step before theirs
    f32x4 km[4], qm[4];
    auto read_m = [&](const f32x4* mm, bool with_q) {
      bf16x8 kf[4], qf[4];
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        km[it] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (with_q) qm[it] = km[it];
        kf[it] = row_at(ko, it, 0);
      }
      Parts<3> b = split_tiles<3>(mm[0], mm[1]);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const bool more = s + 1 < KS;
        Parts<3> next = b;
        if (with_q) {
#pragma unroll
          for (int it = 0; it < 4; ++it) qf[it] = row_at(qo, it, s);
        }
#pragma unroll
        for (int p = 2; p >= 0; --p)
#pragma unroll
          for (int it = 0; it < 4; ++it) km[it] = mfma_bf16(kf[it], b.p[p], km[it]);
        if (more) {
#pragma unroll
          for (int it = 0; it < 4; ++it) kf[it] = row_at(ko, it, s + 1);
          next = split_tiles<3>(mm[2 * s + 2], mm[2 * s + 3]);
        }
        if (with_q) {
#pragma unroll
          for (int p = 2; p >= 0; --p)
#pragma unroll
            for (int it = 0; it < 4; ++it) qm[it] = mfma_bf16(qf[it], b.p[p], qm[it]);
        }
        if (with_q) weave_reads<4>();
        weave<12, 2>();
        if (more) weave_reads<4>();
        if (with_q) weave<12, 2>();
        __builtin_amdgcn_sched_barrier(0);
        b = next;
      }
    };
    // X = V o its factor - K M (with decays: gam o K M), in km
    auto form_x = [&](bool with_v) {
      if (flags & kGated) {
#pragma unroll
        for (int it = 0; it < 4; ++it) km[it] *= *(const f32x4*)(rows + kRowGam + token_row(it, 4 * g));
      }
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        if (!with_v) {
          km[it] = -km[it];
          continue;
        }
        const f32x4 fv = *(const f32x4*)(rows + kRowV + token_row(it, 4 * g));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float v =
              __uint_as_float((unsigned)*(const uint16_t*)(smem + ((vo ^ (64u * (D == 128 ? r : r >> 1))) +
                                                                  (token_row(it, r) * D * 2)))
                              << 16);
          km[it][r] = fmaf(v, fv[r], -km[it][r]);
        }
      }
    };
    // U = T X, part by part of T
    f32x4 u[4];
    auto t_part = [&](int ts, int k, bf16x8* f) {
#pragma unroll
      for (int it = 2 * ts; it < 4; ++it)
        f[it] = *(const bf16x8*)(smem + C::kOffT + lo + (k * C::TRI + low_frag(it, ts) * kFragElems) * 2);
    };
    auto apply_t = [&]() {
      bf16x8 fa[4], fb[4];
      auto products = [&](int ts, int k, const bf16x8* f, const Parts<3>& x) {
#pragma unroll
        for (int p = 2 - k; p >= 0; --p)
#pragma unroll
          for (int it = 2 * ts; it < 4; ++it) u[it] = mfma_bf16(f[it], x.p[p], u[it]);
      };
      t_part(0, 2, fa);
      t_part(0, 1, fb);
#pragma unroll
      for (int it = 0; it < 4; ++it) u[it] = f32x4{0.f, 0.f, 0.f, 0.f};
      const Parts<3> x0 = split_tiles<3>(km[0], km[1]);
      products(0, 2, fa, x0);
      t_part(0, 0, fa);
      const Parts<3> x1 = split_tiles<3>(km[2], km[3]);
      products(0, 1, fb, x0);
      t_part(1, 2, fb);
      products(0, 0, fa, x0);
      weave_reads<8>();
      weave<4, 2>();
      weave_reads<4>();
      weave<8, 2>();
      weave_reads<2>();
      weave<12, 2>();
      __builtin_amdgcn_sched_barrier(0);
      bf16x8 fc[4];
      t_part(1, 1, fa);
      t_part(1, 0, fc);
      products(1, 2, fb, x1);
      products(1, 1, fa, x1);
      products(1, 0, fc, x1);
      weave_reads<4>();
    };
    // a chunk formed with its decays: M and Q M take theirs
    auto decay = [&](f32x4* mm) {
      if (!(flags & kGated)) return;
      const float gl = rows[kLast];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) mm[mt] *= gl;
      if (C::Q) {
#pragma unroll
        for (int it = 0; it < 4; ++it) qm[it] *= *(const f32x4*)(rows + kRowGam + token_row(it, 4 * g)) * a.scale;
      }
    };
    // the parts of half ts of U that go into M, and those for O
    Parts<3> ub, ob;
    auto split_u = [&](int ts) {
      if (flags & kGated) {
        if (C::Q) ob = split_tiles<3>(u[2 * ts], u[2 * ts + 1]);
#pragma unroll
        for (int it = 2 * ts; it < 2 * ts + 2; ++it) u[it] *= *(const f32x4*)(rows + kRowDec + token_row(it, 4 * g));
      }
      ub = split_tiles<3>(u[2 * ts], u[2 * ts + 1]);
      if (C::Q && !(flags & kGated)) ob = ub;
    };
    // Q M + P U
    auto outputs = [&](int ts) {
      bf16x8 f[2][4];
      auto part = [&](int k) {
#pragma unroll
        for (int it = 2 * ts; it < 4; ++it)
          f[k & 1][it] = *(const bf16x8*)(smem + C::kOffP + lo + (k * C::TRI + low_frag(it, ts) * kFragElems) * 2);
      };
      part(2);
#pragma unroll
      for (int k = 2; k >= 0; --k) {
        if (k > 0) part(k - 1);
#pragma unroll
        for (int p = 2 - k; p >= 0; --p)
#pragma unroll
          for (int it = 2 * ts; it < 4; ++it) qm[it] = mfma_bf16(f[k & 1][it], ob.p[p], qm[it]);
      }
    };
    // M += K^T U, a half of the chunk's tokens at a time
    auto advance = [&](f32x4* mm, int ts) {
      bf16x8 f[2][4];
      auto fetch = [&](int m0, bf16x8* to) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const unsigned at = (co ^ (64u * ((m0 + i) >> 1))) + (32 * ts * D + 4 * (i & 1)) * 2;
          // 8 rows on: the same swizzle
          to[i] = __builtin_shufflevector(delta_read_tr((const uint16_t*)(smem + at)),
                                          delta_read_tr((const uint16_t*)(smem + at + 8 * D * 2)), 0, 1, 2, 3, 4, 5, 6,
                                          7);
        }
      };
      fetch(0, f[0]);
#pragma unroll
      for (int m0 = 0; m0 < MT; m0 += 4) {
        if (m0 + 4 < MT) fetch(m0 + 4, f[(m0 / 4 + 1) & 1]);
#pragma unroll
        for (int p = 2; p >= 0; --p)
#pragma unroll
          for (int i = 0; i < 4; ++i) mm[m0 + i] = mfma_bf16(f[(m0 / 4) & 1][i], ub.p[p], mm[m0 + i]);
      }
    };

    if (flags & kShift) {  // 2^s goes into the state
      const float f = rows[kPre];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        m[mt] *= f;
        if (MODE == kTransition) e[mt] *= f;
      }
    }
    if (MODE == kKeep) {
      const float f = rows[kScale0];
      char* const mo = (char*)(sa.m_out + ((int64_t)(sg.x + j) * a.heads + h) * dd);
      const unsigned m_off = (unsigned)((dv >> 5) * D * 32 + 8 * g * 32 + (dv & 31)) * 4u;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 4; ++r) *(float*)(mo + dim_row(mt, r) * 128 + m_off) = f * m[mt][r];
    }
    read_m(m, C::Q);
    form_x(true);
    apply_t();
    lds_barrier();
    if (MODE == kTransition) {
      decay(m);
      split_u(0);
      advance(m, 0);
      __builtin_amdgcn_sched_barrier(0);
      split_u(1);
      advance(m, 1);
      __builtin_amdgcn_sched_barrier(0);
      read_m(e, false);
      form_x(false);
      apply_t();
      lds_barrier();
    }
    if (MODE == kKeep) {
      char* const uo = (char*)(sa.u_out + ((int64_t)(sg.x + j) * a.heads + h) * kChunk * D);
      const unsigned u_off = (unsigned)((dv >> 5) * kChunk * 32 + lt * 32 + (dv & 31)) * 4u;
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const f32x4 fo = *(const f32x4*)(rows + kRowO + token_row(it, 4 * g));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int t = token_row(it, r);
          if (lt + t < count) *(float*)(uo + t * 128 + u_off) = fo[r] * u[it][r];
        }
      }
    }
    f32x4* const mm = MODE == kTransition ? e : m;
    decay(mm);
    split_u(0);
    if (C::Q) outputs(0);
    advance(mm, 0);
    if (MODE != kTransition) lds_barrier();
    split_u(1);
    if (C::Q) outputs(1);
    if (MODE == kOutputs) {
      char* const at = op + (int64_t)kChunk * j * sa.ld_o * 2;
      unsigned off = o_off, first = lt;
      pin(off);
      pin(first);
#pragma unroll
      for (int it = 0; it < 4; ++it) qm[it] *= *(const f32x4*)(rows + kRowO + token_row(it, 4 * g));
      if (count == kChunk) {
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            *(uint16_t*)(at + token_row(it, r) * sa.ld_o * 2 + off) = to_bf16(qm[it][r]);
      } else {
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if ((int)first + token_row(it, r) < count)
              *(uint16_t*)(at + token_row(it, r) * sa.ld_o * 2 + off) = to_bf16(qm[it][r]);
      }
    }
    advance(mm, 1);
    if (j == n - 1) {
      const float f = rows[kScale1];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        m[mt] *= f;
        if (MODE == kTransition) e[mt] *= f;
      }
    }
  }

  if (MODE == kTransition) {
    float* const to = sa.trans + ((int64_t)si * a.heads + h) * (sa.both ? 3 : 2) * dd;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int dk = dim_row(mt, 4 * g);
      // N and B for the join, and N's transpose for the one on the way back
#pragma unroll
      for (int r = 0; r < 4; ++r) to[join_n<D>(dk + r, dv)] = e[mt][r];
      *(f32x4*)(to + dd + join_b<D>(dv, mt, g)) = m[mt];
      if (sa.both) *(f32x4*)(to + 2 * dd + join_n<D>(dv, dk)) = e[mt];
    }
  } else if ((sg.w & 2) && sa.state_out) {
    float* const out = sa.state_out + ((int64_t)sg.z * a.heads + h) * dd + (int64_t)dv * D;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) *(f32x4*)(out + dim_row(mt, 4 * g)) = m[mt];
  }
}

template <int D>
hipError_t fused_any(const DeltaArgs& a, const DeltaScanArgs& s, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.sq.n_segs * a.heads)), blk(64 * (D / 16 + 4));
  if (s.trans)
    hipLaunchKernelGGL((k_delta_fused<D, kTransition>), grid, blk, 0, st, a, s);
  else if (s.m_out)
    hipLaunchKernelGGL((k_delta_fused<D, kKeep>), grid, blk, 0, st, a, s);
  else
    hipLaunchKernelGGL((k_delta_fused<D, kOutputs>), grid, blk, 0, st, a, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_fused(const DeltaArgs& a, const DeltaScanArgs& s, hipStream_t st) {
  return a.d == 128 ? fused_any<128>(a, s, st) : fused_any<64>(a, s, st);
}

}  // namespace zm
