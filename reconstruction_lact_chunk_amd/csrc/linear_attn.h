// Linear attention with decays: shared device code, argument blocks and launchers.
//
// Per sequence and value head, S in R^{d x d} (fp32), a_t = exp(g_t):
//   S_t = a_t S_{t-1} + v_t k_t^T,  o_t = scale S_t q_t.
// Tokens are taken C at a time.  With c_i the sum of g over the chunk's tokens up to i,
// G_ij = exp(c_i - c_j) for j <= i, and M = S^T at the chunk's start:
//   O = scale exp(c) o (Q M) + (scale G o Q K^T) V,   M' = exp(c_C) M + K^T (exp(c_C - c) o V).
// A pass over the chunks is the same for the outputs and for each gradient; only the
// tensors' parts and the direction change.  With D the gradient of M at the chunk's end:
//                 A    B    C    state          factor of A    of C in the state   order
//   o             Q    K    V    M              scale exp(c)   exp(c_C - c)        first to last
//   dq            dO   V    K    M^T            scale exp(c)   exp(c_C - c)        first to last
//   dv            K    Q    dO   D              exp(c_C - c)   scale exp(c)        last to first
//   dk            V    dO   Q    D^T            exp(c_C - c)   scale exp(c)        last to first
//   out = f o (A state) + T C,  T = scale G o (A B^T) (G^T, last to first),
//   state <- exp(c_C) state + B^T (w o C).
// So the gradients need no state of any chunk in memory.  Few long sequences are cut into
// segments: a first pass leaves what each adds to the state, a join makes the states at
// their starts (or ends) of these.
//
// The gradient by g_t is what flows past it, from tokens before t (or the first state) to
// t and later ones (or the last state):
//   dg_t = sum_{i >= t > j} X_ij + sum_{i >= t} q_i.dq'_i + sum_{j < t} v_j.dv'_j + exp(c_C) <M, D>
// with X_ij = T_ij (dO_i.v_j), and dq', dv' the parts that come from M and D.  Each term holds
// the factor a_t, so nothing large has to cancel where a decay is strong.
//
// Matrix products run on v_mfma_f32_16x16x32_bf16, operands in fp32 (states, T, w o C,
// fp32 tokens) as a sum of three bf16 parts (delta_rule.h): 24 bits, so the state and the
// outputs up to their own rounding are as exact as fp32 products would leave them.
//
// A wave holds CT * 16 columns of the state and all its rows; its accumulators are operands
// of the next product as they are, column mt = CT w + ct, c at dim_row(mt, c), and an
// output's rows (columns of the state) are consecutive in a lane.
#pragma once

#include "delta_rule.h"

namespace zm {

constexpr int kLinWaves = 4;  // waves to a state

template <int D, bool F32>
struct LinCfg {
  static constexpr int CH = F32 ? 32 : 64;       // tokens of a chunk
  static constexpr int NT = F32 ? 3 : 1;         // parts of a token element
  static constexpr int LIM = F32 ? 2 : 0;        // order of the parts' products of two tokens
  static constexpr int CT = D / (16 * kLinWaves);  // 16-column tiles of a wave
  static constexpr int KS = D / 32;              // steps over the head dims
  static constexpr int MT = D / 16;              // row tiles of the state
  static constexpr int IT = CH / 16;             // token tiles
  static constexpr int TS = CH / 32;             // steps over the tokens
  static constexpr int FRAGS = CH == 64 ? 6 : 2; // operand tiles of a triangle
  static constexpr int PITCH = D + 16;           // elements of a row in LDS
  static constexpr int PART = CH * PITCH;        // elements of one part of a tile
  static constexpr int TILE = NT * PART;
  static constexpr int TRI = 3 * FRAGS * kFragElems;
};

// What a chunk's tokens are multiplied with; computed by one wave.
struct LinFactors {
  float f[64];     // of A's rows
  float w[64];     // of C's rows in the state
  float ti[64];    // T = ti[out] tj[source], unless `gated`
  float tj[64];
  double cs[64];   // sums of decays, powers of two
  float last;      // of the state
  int gated;       // they span too much for ti tj: every element from its own difference
  float pad[2];
};
constexpr double kLinSpan = 60.0;  // ti and tj stay in 2^-60 .. 2^60

struct LinSeg {
  int tok, count;   // first token, tokens (-1: unused)
  int seq, flags;   // 1 first | 2 last of its sequence
  int chunk0;       // chunks before it (each segment but a sequence's last has seg_chunks)
  int slot;         // of its state, in a sequence of several segments
  int pad[2];
};

struct LinSeqs {
  const int* offsets;   // [n_seq + 1] or null: one sequence of all n tokens
  LinSeg* segs;         // null without a table (one sequence)
  int2* of_seq;         // [n_seq] {first slot, segments}, then {first token, end}, {chunks, -}
  int n, n_seq;
  int n_segs;           // upper bound over every content of offsets
  int seg_tokens;       // tokens of a segment, a multiple of the chunk
  int chunk;
};

struct LinTokens {
  const void* p;
  int64_t ld;
};

struct LinArgs {
  LinSeqs sq;
  LinTokens q, k, v, d_o;
  const float* g;      // decay of token t, head h: g[t ld_g + h]; null: none
  int64_t ld_g;
  int heads, heads_k;
  float scale;
  const float* state_in;    // [n_seq][heads][d][d] S or null (zeros)
  float* state_out;         // or null
  const float* dstate_out;  // gradients, or null
  float* dstate_in;
  // Sequences of several segments, [slots][heads][d][d]: the states at their starts, 1: the
  // gradients at their ends.  Before the join what the segment before (behind) adds is there.
  // So no pass reads state_in or dstate_out where another segment replaces it.
  float* part[2];
  float* decay[2];     // [slots][heads] factor of a segment
  void* o;             // o, or dq
  int64_t ld_o;
  void* dk;
  int64_t ld_dk;
  void* dv;
  int64_t ld_dv;
  float* o_part;       // dq and dk to each value head [n][heads][d], where these share key heads
  float* dk_part;
  float* flow;         // [n][heads]: the part of dg that the reverse pass forms, or null without g
  float* d_dump;       // D^T at every chunk's end
  float* dg;           // [n][heads], or, with ld_g = 0, the chunks' sums [chunks][heads]
};

// First token and end of all sequences together.
__device__ __forceinline__ int2 lin_range(const LinSeqs& s) {
  if (s.segs) return s.of_seq[s.n_seq];
  int a = 0, e = s.n;
  if (s.offsets) {
    a = clampi(s.offsets[0], 0, s.n);
    e = clampi(s.offsets[1], a, s.n);
  }
  return int2{a, e};
}
// Segments of a sequence of len tokens, and its chunks.
__device__ __forceinline__ int lin_segs(const LinSeqs& s, int len) {
  return len > 0 ? (int)(((int64_t)len + s.seg_tokens - 1) / s.seg_tokens) : 1;
}
__device__ __forceinline__ int lin_chunks(const LinSeqs& s, int len) {
  return (int)(((int64_t)len + s.chunk - 1) / s.chunk);
}

__device__ __forceinline__ LinSeg lin_seg(const LinSeqs& s, int si) {
  if (s.segs) return s.segs[si];
  const int2 r = lin_range(s);
  const int a = r.x, len = r.y - r.x, segs = lin_segs(s, len);
  LinSeg g;
  if (si >= segs) {
    g.count = -1;
    return g;
  }
  const int64_t at = (int64_t)si * s.seg_tokens;
  g.tok = a + (int)at;
  g.count = len - at < s.seg_tokens ? (int)(len - at) : s.seg_tokens;
  g.seq = 0;
  g.flags = (si == 0 ? 1 : 0) | (si == segs - 1 ? 2 : 0);
  g.chunk0 = (int)(at / s.chunk);
  g.slot = si;
  return g;
}

// Rows of a token tensor on their way from memory to LDS: THREADS threads, E-element
// granules.  Rows past `count` are zero in LDS.
template <int D, bool F32, int THREADS>
struct LinFetch {
  using C = LinCfg<D, F32>;
  using T = typename Tok<F32>::T;
  static constexpr int GPR = D / 8, N = C::CH * GPR / THREADS;
  static_assert(C::CH * GPR % THREADS == 0, "granules");
  u32x4 raw[N][F32 ? 2 : 1];

  __device__ __forceinline__ void load(const T* base, int64_t ld, int count) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int gr = threadIdx.x % THREADS + THREADS * i, row = gr / GPR, col = 8 * (gr % GPR);
      const T* const p = base + (int64_t)(row < count ? row : count - 1) * ld + col;
      raw[i][0] = *(const u32x4*)p;
      if constexpr (F32) raw[i][1] = *(const u32x4*)(p + 4);
    }
  }
  __device__ __forceinline__ void store(uint16_t* tile, int count) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int gr = threadIdx.x % THREADS + THREADS * i, row = gr / GPR, col = 8 * (gr % GPR);
      uint16_t* const at = tile + row * C::PITCH + col;
      const bool in = row < count;
      if constexpr (F32) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = in ? __uint_as_float(raw[i][e >> 2][e & 3]) : 0.f;
        const Parts<3> p = split8<3>(x);
#pragma unroll
        for (int k = 0; k < 3; ++k) *(bf16x8*)(at + k * C::PART) = p.p[k];
      } else {
        u32x4 x = raw[i][0];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = in ? x[e] : 0u;
        *(u32x4*)at = x;
      }
    }
  }
};

// Parts of 8 elements of a row, and of 8 tokens (order dtau) of column dim_row(mt, c).
template <int D, bool F32>
__device__ __forceinline__ Parts<LinCfg<D, F32>::NT> lin_row(const uint16_t* t, int row, int col) {
  using C = LinCfg<D, F32>;
  Parts<C::NT> p;
#pragma unroll
  for (int k = 0; k < C::NT; ++k) p.p[k] = *(const bf16x8*)(t + k * C::PART + row * C::PITCH + col);
  return p;
}
template <int D, bool F32>
__device__ __forceinline__ Parts<LinCfg<D, F32>::NT> lin_col(const uint16_t* t, int mt, int ts, int g, int c) {
  using C = LinCfg<D, F32>;
  Parts<C::NT> p;
  const int row = 32 * ts + dtau(g, c >> 2), col = 32 * (mt >> 1) + 8 * (c & 3) + 4 * (mt & 1);
#pragma unroll
  for (int k = 0; k < C::NT; ++k) {
    const uint16_t* const at = t + k * C::PART + row * C::PITCH + col;
    p.p[k] = __builtin_shufflevector(delta_read_tr(at), delta_read_tr(at + 8 * C::PITCH), 0, 1, 2, 3, 4, 5, 6, 7);
  }
  return p;
}

// The factors of a chunk from its lanes' log decays (zero past the tokens); one wave.
template <bool REV>
__device__ __forceinline__ void lin_factors(LinFactors* f, float gl, float scale) {
  const int lane = threadIdx.x & 63;
  if (gl < kMinLogDecay) gl = kMinLogDecay;
  // in 64 bits: a strong decay among weak ones must not blur their differences
  double s = gl * kLog2E;
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const double o = __shfl_up(s, m, 64);
    if (lane >= m) s += o;
  }
  const double last = __shfl(s, 63, 64), ref = 0.5 * (last + __shfl(s, 0, 64));
  const float in = scale * exp2_wide(s), out = exp2_wide(last - s);
  f->f[lane] = REV ? out : in;
  f->w[lane] = REV ? in : out;
  const float up = scale * exp2_wide(s - ref), down = exp2_wide(ref - s);
  f->ti[lane] = REV ? down : up;
  f->tj[lane] = REV ? up : down;
  f->cs[lane] = s;
  const bool wide = __any(!(fabs(s - ref) <= kLinSpan));
  if (lane == 0) {
    f->last = exp2_wide(last);
    f->gated = wide;
  }
}

// Operand tile f of a triangle (row tile, token step), and back.
template <int D, bool F32, bool REV>
__device__ __forceinline__ constexpr int lin_frag(int it, int ts) {
  return LinCfg<D, F32>::CH == 32 ? it : (REV ? up_frag(it, ts) : low_frag(it, ts));
}
template <int D, bool F32, bool REV>
__device__ __forceinline__ constexpr bool lin_in(int it, int ts) {
  return REV ? 32 * ts + 31 >= 16 * it : 32 * ts <= 16 * it + 15;
}

// Products of A's tokens 16 it + c (columns) with B's tokens token_row(jt, 4 g + r).
template <int D, bool F32>
__device__ __forceinline__ f32x4 lin_tri(const uint16_t* a, const uint16_t* b, int it, int jt, int g, int c) {
  using C = LinCfg<D, F32>;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < C::KS; ++s) {
    const auto bb = lin_row<D, F32>(b, token_row(jt, c), 32 * s + 8 * g);
    const auto aa = lin_row<D, F32>(a, 16 * it + c, 32 * s + 8 * g);
    mma<C::LIM>(acc, bb, aa);
  }
  return acc;
}

// The same with the decays and the mask.
template <bool REV>
__device__ __forceinline__ f32x4 lin_gate(const f32x4& x, const LinFactors* f, float scale, int it, int jt, int g,
                                          int c) {
  const int out = 16 * it + c, src = token_row(jt, 4 * g);
  f32x4 t;
  if (f->gated) {
    const double co = f->cs[out];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const double dif = REV ? f->cs[src + r] - co : co - f->cs[src + r];
      const bool in = REV ? src + r >= out : src + r <= out;
      t[r] = in ? x[r] * scale * exp2_wide(in ? dif : 0.0) : 0.f;
    }
  } else {
    const f32x4 w = *(const f32x4*)(f->tj + src);
    const float to = f->ti[out];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const bool in = REV ? src + r >= out : src + r <= out;
      t[r] = in ? x[r] * (to * w[r]) : 0.f;
    }
  }
  return t;
}

// Four sources of a triangle's tile into its operand tiles: element 4 (jt & 1) + r of lane.
__device__ __forceinline__ void lin_put(uint16_t* frags, int frags_each, int fi, int jt, int lane, const f32x4& t) {
  float r[4] = {t[0], t[1], t[2], t[3]};
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    u32x2 w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[i] = pack_bf16x2(r[2 * i], r[2 * i + 1]);
      r[2 * i] -= bf16lo(w[i]);
      r[2 * i + 1] -= bf16hi(w[i]);
    }
    *(u32x2*)(frags + (p * frags_each + fi) * kFragElems + lane * 8 + 4 * (jt & 1)) = w;
  }
}

template <int D, bool F32>
struct LinState {
  using C = LinCfg<D, F32>;
  f32x4 m[C::MT][C::CT];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
      for (int ct = 0; ct < C::CT; ++ct) m[mt][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // S [d (columns of the state)][d (rows)] in memory; TR: the other way round.
  template <bool TR>
  __device__ __forceinline__ void load(const float* s, int w, int g, int c) {
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
      for (int ct = 0; ct < C::CT; ++ct) {
        const int col = dim_row(C::CT * w + ct, c), row = dim_row(mt, 4 * g);
        if constexpr (TR) {
#pragma unroll
          for (int r = 0; r < 4; ++r) m[mt][ct][r] = s[(row + r) * D + col];
        } else {
          m[mt][ct] = *(const f32x4*)(s + col * D + row);
        }
      }
  }
  __device__ __forceinline__ void store(float* s, int w, int g, int c) const {
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
      for (int ct = 0; ct < C::CT; ++ct)
        *(f32x4*)(s + dim_row(C::CT * w + ct, c) * D + dim_row(mt, 4 * g)) = m[mt][ct];
  }
  __device__ __forceinline__ void scale(float x) {
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
      for (int ct = 0; ct < C::CT; ++ct)
#pragma unroll
        for (int r = 0; r < 4; ++r) m[mt][ct][r] *= x;
  }
};

// Output columns of a wave: rows 4 g + r of tile ct are CT * 4 consecutive dims from here.
template <int D>
__device__ __forceinline__ constexpr int lin_col0(int w, int g) {
  return D == 128 ? 32 * w + 8 * g : dim_row(w, 4 * g);
}

template <int D, bool F32>
struct LinOut {
  using C = LinCfg<D, F32>;
  f32x4 o[C::IT][C::CT];

  // f o (A state), transposed: columns are tokens
  __device__ __forceinline__ void read(const LinState<D, F32>& st, const uint16_t* a, const LinFactors* f, int g, int c) {
#pragma unroll
    for (int it = 0; it < C::IT; ++it)
#pragma unroll
      for (int ct = 0; ct < C::CT; ++ct) o[it][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < C::KS; ++s) {
      Parts<3> mp[C::CT];
#pragma unroll
      for (int ct = 0; ct < C::CT; ++ct) mp[ct] = split_tiles<3>(st.m[2 * s][ct], st.m[2 * s + 1][ct]);
#pragma unroll
      for (int it = 0; it < C::IT; ++it) {
        const auto aa = lin_row<D, F32>(a, 16 * it + c, 32 * s + 8 * g);
#pragma unroll
        for (int ct = 0; ct < C::CT; ++ct) mma<2>(o[it][ct], mp[ct], aa);
      }
    }
#pragma unroll
    for (int it = 0; it < C::IT; ++it) {
      const float x = f->f[16 * it + c];
#pragma unroll
      for (int ct = 0; ct < C::CT; ++ct)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[it][ct][r] *= x;
    }
  }
  // rows of the chunk's tokens, T elements (or fp32) of stride ld
  template <typename T>
  __device__ __forceinline__ void store(T* base, int64_t ld, int count, int w, int g, int c) const {
#pragma unroll
    for (int it = 0; it < C::IT; ++it) {
      const int tok = 16 * it + c;
      if (tok >= count) continue;
      T* const p = base + (int64_t)tok * ld + lin_col0<D>(w, g);
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int ct = 0; ct < C::CT; ++ct) *(f32x4*)((float*)p + 4 * ct) = o[it][ct];
      } else {
        unsigned x[2 * C::CT];
#pragma unroll
        for (int ct = 0; ct < C::CT; ++ct)
#pragma unroll
          for (int i = 0; i < 2; ++i) x[2 * ct + i] = pack_bf16x2(o[it][ct][2 * i], o[it][ct][2 * i + 1]);
        if constexpr (C::CT == 2) *(u32x4*)p = u32x4{x[0], x[1], x[2], x[3]};
        else *(u32x2*)p = u32x2{x[0], x[1]};
      }
    }
  }
};

// out += T C and state <- state + B^T (w o C) (the state has its factor already).
template <int D, bool F32, bool REV, bool OUT>
__device__ __forceinline__ void lin_tokens(LinOut<D, F32>* out, LinState<D, F32>& st, const uint16_t* frags,
                                           const uint16_t* b, const uint16_t* cc, const LinFactors* f, int w, int lane,
                                           int g, int c) {
  using C = LinCfg<D, F32>;
#pragma unroll
  for (int ts = 0; ts < C::TS; ++ts) {
    Parts<3> cw[C::CT];
#pragma unroll
    for (int ct = 0; ct < C::CT; ++ct) {
      const auto cf = lin_col<D, F32>(cc, C::CT * w + ct, ts, g, c);
      if constexpr (OUT) {
#pragma unroll
        for (int it = 0; it < C::IT; ++it) {
          if (!lin_in<D, F32, REV>(it, ts)) continue;
          Parts<3> t;
#pragma unroll
          for (int p = 0; p < 3; ++p)
            t.p[p] = *(const bf16x8*)(frags + (p * C::FRAGS + lin_frag<D, F32, REV>(it, ts)) * kFragElems + lane * 8);
          mma<2>(out->o[it][ct], cf, t);
        }
      }
      float x[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const u32x4 p0 = __builtin_bit_cast(u32x4, cf.p[0]);
        x[2 * i] = bf16lo(p0[i]);
        x[2 * i + 1] = bf16hi(p0[i]);
      }
      if constexpr (F32) {
        // the smaller parts first: their sum is exact, and so is the whole
        const u32x4 p1 = __builtin_bit_cast(u32x4, cf.p[1]), p2 = __builtin_bit_cast(u32x4, cf.p[2]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[2 * i] += bf16lo(p1[i]) + bf16lo(p2[i]);
          x[2 * i + 1] += bf16hi(p1[i]) + bf16hi(p2[i]);
        }
      }
      const f32x4 w0 = *(const f32x4*)(f->w + 32 * ts + dtau(g, 0)), w1 = *(const f32x4*)(f->w + 32 * ts + dtau(g, 4));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] *= w0[e];
        x[4 + e] *= w1[e];
      }
      cw[ct] = split8<3>(x);
    }
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt) {
      const auto bf = lin_col<D, F32>(b, mt, ts, g, c);
#pragma unroll
      for (int ct = 0; ct < C::CT; ++ct) mma<2>(st.m[mt][ct], bf, cw[ct]);
    }
  }
}

// ---- launchers ----------------------------------------------------------------
// The table of segments (n_seq > 1).
hipError_t launch_linear_table(const LinSeqs& s, hipStream_t st);
// What each segment adds to the state, all but the last of a sequence; with both, the
// gradients' too, all but the first.
hipError_t launch_linear_states(const LinArgs& a, int d, bool f32, bool both, hipStream_t st);
hipError_t launch_linear_join(const LinArgs& a, int d, bool both, hipStream_t st);
// The outputs and last states.
hipError_t launch_linear_out(const LinArgs& a, int d, bool f32, hipStream_t st);
// dk, dv, flow, d_dump and the first states' gradient; then dq and dg.
hipError_t launch_linear_dkdv(const LinArgs& a, int d, bool f32, hipStream_t st);
hipError_t launch_linear_dq(const LinArgs& a, int d, bool f32, hipStream_t st);
// y [n][heads_k][d] from x [n][heads][d] summed over the value heads of a key head.
hipError_t launch_linear_groups(const float* x, void* y, int64_t ld_y, const LinArgs& a, int d, bool f32,
                                hipStream_t st);
// dg [heads] from the chunks' sums.
hipError_t launch_linear_decay_sum(const float* sums, const LinSeqs& s, int heads, float* dg, hipStream_t st);

struct LinStepArgs {
  LinTokens q, k, v;
  const float* g;
  int64_t ld_g;
  float* state;
  void* o;
  int64_t ld_o;
  int n_seq, heads, heads_k;
  float scale;
};
hipError_t launch_linear_step(const LinStepArgs& a, int d, bool f32, hipStream_t st);

}  // namespace zm
