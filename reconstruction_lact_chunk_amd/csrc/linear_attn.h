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
// Decays are taken out where they can be.  With the state held as 2^s M^ and e_i = s plus the
// decay from the chunk's first (last) edge up to token i, all in powers of two,
//   out = 2^e_i (A M^ + lower(A B^T) (C_j / 2^e_j)),  M^ <- M^ + B^T (C / 2^e),  s <- s + c_C
// (scale with one of the two powers): the same numbers up to the powers, which come from 64-bit exponents
// (exp2_wide), while |e| stays under kLinSpan.  A chunk that would leave that range
// takes 2^s into M^ first; one whose own decays do (a reset) is formed with them in place.
// So only dg needs states of the chunks in memory (D^T, d_dump below).  Few long sequences are cut into
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
// fp32 tokens) as a sum of three bf16 parts (delta_rule.h): 24 bits, so states, gradients and
// outputs up to their own rounding are as exact as fp32 products would leave them, also where an
// output's terms cancel.
//
// A wave holds 16 columns of the state and all its rows; its accumulators are operands of
// the next product as they are.  Outputs are formed transposed, so that a lane has four
// consecutive dims of a token.
#pragma once

#include "delta_rule.h"

namespace zm {

template <int D, bool F32>
struct LinCfg {
  static constexpr int CH = F32 ? 32 : 64;       // tokens of a chunk
  static constexpr int NT = F32 ? 3 : 1;         // parts of a token element
  static constexpr int LIM = F32 ? 2 : 0;        // order of the parts' products of two tokens
  static constexpr int WAVES = D / 16;           // to a state
  static constexpr int THREADS = 64 * WAVES;
  static constexpr int KS = D / 32;              // steps over the head dims
  static constexpr int MT = D / 16;              // row tiles of the state
  static constexpr int IT = CH / 16;             // token tiles
  static constexpr int TS = CH / 32;             // steps over the tokens
  static constexpr int FRAGS = CH == 64 ? 6 : 2; // operand tiles of a triangle
  static constexpr int PITCH = F32 ? D + 16 : D; // elements of a row in LDS
  static constexpr int PART = CH * PITCH;        // elements of one part of a tile
  static constexpr int TILE = NT * PART;
  static constexpr int TRI = 3 * FRAGS * kFragElems;
};

// What a chunk's tokens are multiplied with; computed by one wave.
struct alignas(16) LinFactors {
  float up[64];    // of outputs; kLinGated: of A M^ alone
  float dn[64];    // of C in the state and, unless kLinGated, of T's columns
  double cs[64];   // sums of the chunk's decays, powers of two
  double s;        // exponent of the state
  double after;    // of the state behind the chunk
  double sum;      // of all decays up to the chunk's
  int count;       // tokens; dn is zero past them
  float pre;       // kLinScale: of the state before the chunk
  float last;      // kLinGated: of the state after the outputs' read
  float end;       // 2^exponent of the state behind the chunk
  int flags;
};
enum { kLinGated = 1, kLinScale = 2 };
template <bool B>
struct LinBool {
  static constexpr bool value = B;
};
constexpr double kLinSpan = 60.0;

struct LinSeg {
  int tok, count;   // first token, tokens (-1: unused)
  int seq, flags;   // 1 first | 2 last of its sequence
  int chunk0;       // chunks before it (each segment but a sequence's last has seg_chunks)
  int slot;         // of its state, in a sequence of several segments
  int segs;         // of its sequence
  int split;        // of its sequence, among those of several segments (in a table)
};
constexpr int kLinWaveSeqs = 64;  // sequences that need no table
constexpr int kLinSorted = 512;   // segments that the table puts in order

struct LinSeqs {
  const int* offsets;   // [n_seq + 1] or null: one sequence of all n tokens
  LinSeg* segs;         // null without a table (up to kLinWaveSeqs sequences)
  int* by_slot;         // [slots] the segment, -1: unused
  int* by_split;        // [n_split] the first segment of each sequence of several, -1: unused
  int4* all;            // {first token, end, chunks, -} of all sequences together
  int n, n_seq;
  int n_segs, n_slots;  // upper bounds over every content of offsets
  int n_split;          // the same of the sequences of several segments
  bool longest_first;   // the table's order, else that of the tokens
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
  float2* decay[2];    // [slots][heads] factor of a segment in two parts
  void* o;             // o, or dq
  int64_t ld_o;
  void* dk;
  int64_t ld_dk;
  void* dv;
  int64_t ld_dv;
  float* o_part;       // dq and dk to each value head [n][heads][d], where these share key heads
  float* dk_part;
  float* flow;         // [n][heads]: the parts of dg that the first two passes form, or null without dg
  float* d_dump;       // D^T at every chunk's end, less a power of two
  double* d_exp;       // [chunks][heads] that power
  float* dg;           // [n][heads], or, with ld_g = 0, the chunks' sums [chunks][heads]
};

// Segments of a sequence of len tokens, and its chunks (len and seg_tokens are under 2^31: 32
// bits without a sign hold their sum).
__device__ __forceinline__ int lin_segs(const LinSeqs& s, int len) {
  return len > 0 ? (int)(((unsigned)len + s.seg_tokens - 1) / (unsigned)s.seg_tokens) : 1;
}
__device__ __forceinline__ int lin_chunks(const LinSeqs& s, int len) {
  return (int)(((unsigned)len + s.chunk - 1) >> (s.chunk == 64 ? 6 : 5));
}

// Sums, and the largest, over the lanes up to each one: shifts within 16 lanes, then the
// rows' last lanes to the next row and to the upper half.  No addresses, as exchanges
// through LDS take them.
template <int CTRL, int ROWS>
__device__ __forceinline__ int lin_add_from(int x) {
  return x + __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ int lin_max_from(int x) {
  const int o = __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false);  // of nothing: 0
  return o > x ? o : x;
}
__device__ __forceinline__ int lin_prefix(int x) {
  x = lin_add_from<0x111, 0xf>(x);  // one lane on
  x = lin_add_from<0x112, 0xf>(x);
  x = lin_add_from<0x114, 0xf>(x);
  x = lin_add_from<0x118, 0xf>(x);
  x = lin_add_from<0x142, 0xa>(x);  // lane 15 to row 1, 47 to row 3
  return lin_add_from<0x143, 0xc>(x);  // lane 31 to rows 2 and 3
}
__device__ __forceinline__ int lin_prefix_max(int x) {  // x >= 0
  x = lin_max_from<0x111, 0xf>(x);
  x = lin_max_from<0x112, 0xf>(x);
  x = lin_max_from<0x114, 0xf>(x);
  x = lin_max_from<0x118, 0xf>(x);
  x = lin_max_from<0x142, 0xa>(x);
  return lin_max_from<0x143, 0xc>(x);
}

// Up to 64 sequences, a lane to each: what the table holds of more of them.  Every lane of a
// wave calls this.
struct LinWave {
  int begin, len, segs;    // of the lane's sequence; none past the last
  int chunk0, slot0;       // before it
  int first, end;          // of all sequences together
  int chunks;              // of all

  __device__ __forceinline__ explicit LinWave(const LinSeqs& s) {
    const int lane = threadIdx.x & 63;
    const bool in = lane < s.n_seq;
    int e = 0;
    first = 0;
    if (s.offsets) {
      first = clampi(s.offsets[0], 0, s.n);
      if (in) e = clampi(s.offsets[lane + 1], 0, s.n);
    } else if (in) {
      e = s.n;
    }
    if (e < first) e = first;
    e = lin_prefix_max(e);  // nondecreasing
    const int left = __shfl_up(e, 1, 64);
    begin = lane ? left : first;
    len = in ? e - begin : 0;
    segs = in ? lin_segs(s, len) : 0;
    const int c = lin_chunks(s, len), k = segs > 1 ? segs : 0;
    const int cs = lin_prefix(c);
    chunk0 = cs - c;
    slot0 = lin_prefix(k) - k;
    end = __builtin_amdgcn_readlane(e, 63);
    chunks = __builtin_amdgcn_readlane(cs, 63);
  }
  // Segment i of lane b's sequence, the same in every lane.
  __device__ __forceinline__ LinSeg get(const LinSeqs& s, int b, int i) const {
    LinSeg g;
    const int k = __builtin_amdgcn_readlane(segs, b), l = __builtin_amdgcn_readlane(len, b);
    const int from = i * s.seg_tokens;  // < l, or 0
    g.tok = __builtin_amdgcn_readlane(begin, b) + from;
    g.count = l - from < s.seg_tokens ? l - from : s.seg_tokens;
    g.seq = b;
    g.flags = (i == 0 ? 1 : 0) | (i == k - 1 ? 2 : 0);
    g.chunk0 = __builtin_amdgcn_readlane(chunk0, b) + lin_chunks(s, from);
    g.slot = __builtin_amdgcn_readlane(slot0, b) + i;
    g.segs = k;
    g.split = 0;
    return g;
  }
};

// First token and end of all sequences together, and their chunks.
__device__ __forceinline__ int4 lin_all(const LinSeqs& s) {
  if (s.segs) return *s.all;
  if (s.n_seq == 0) return int4{0, 0, 0, 0};
  const LinWave w(s);
  return int4{w.first, w.end, w.chunks, 0};
}

// Segment si: the full ones (which are a sequence's but its last) in the order of the tokens,
// then the others, longest first, so that long ones do not end last where there are more
// workgroups than run at once.
__device__ __forceinline__ LinSeg lin_seg(const LinSeqs& s, int si) {
  if (s.segs) return s.segs[si];
  const LinWave w(s);
  const int lane = threadIdx.x & 63;
  LinSeg none;
  none.count = -1;
  const int full = w.segs > 0 ? w.segs - 1 : 0, before = lin_prefix(full) - full;
  const int all = __builtin_amdgcn_readlane(before + full, 63);
  if (si < all) {
    const uint64_t at = __ballot(full > 0 && before <= si && si < before + full);
    const int b = __builtin_ctzll(at);
    return w.get(s, b, si - __builtin_amdgcn_readlane(before, b));
  }
  si -= all;
  if (si >= s.n_seq) return none;
  const int rest = w.segs > 0 ? w.len - full * s.seg_tokens : -1;  // len < 2^31
  int rank = 0;
  for (int i = 0; i < s.n_seq; ++i) {
    const int o = __builtin_amdgcn_readlane(rest, i);
    rank += o > rest || (o == rest && i < lane);
  }
  const uint64_t at = __ballot(lane < s.n_seq && rank == si);
  const int b = __builtin_ctzll(at);
  return w.get(s, b, __builtin_amdgcn_readlane(full, b));
}
// The segment whose state is in a slot: of sequences of several segments only.
__device__ __forceinline__ LinSeg lin_slot(const LinSeqs& s, int slot) {
  LinSeg g;
  g.count = -1;
  if (s.segs) {
    const int i = s.by_slot[slot];
    if (i >= 0) g = s.segs[i];
    return g;
  }
  const LinWave w(s);
  const uint64_t at = __ballot(w.segs > 1 && w.slot0 <= slot && slot < w.slot0 + w.segs);
  if (at == 0) return g;
  const int b = __builtin_ctzll(at);
  return w.get(s, b, slot - __builtin_amdgcn_readlane(w.slot0, b));
}

// The first segment of the r-th sequence of several.
__device__ __forceinline__ LinSeg lin_split(const LinSeqs& s, int r) {
  LinSeg g;
  g.count = -1;
  if (s.segs) {
    const int i = s.by_split[r];
    if (i >= 0) g = s.segs[i];
    return g;
  }
  const LinWave w(s);
  const int split = w.segs > 1 ? 1 : 0, upto = lin_prefix(split);
  const uint64_t at = __ballot(split && upto == r + 1);
  if (at == 0) return g;
  return w.get(s, __builtin_ctzll(at), 0);
}

// x as three bf16 parts, each what 8 bits hold of what the ones before leave, cut off: the sum
// is x to its last bit, and a part of two elements is one instruction.
__device__ __forceinline__ Parts<3> cut8(const float* x) {
  Parts<3> out;
  unsigned r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(x[i]);
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __builtin_amdgcn_perm(r[2 * i + 1], r[2 * i], 0x07060302u);
    out.p[p] = as_bf16x8(w);
    if (p < 2)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        r[i] = __float_as_uint(__uint_as_float(r[i]) - __uint_as_float(r[i] & 0xffff0000u));
  }
  return out;
}
__device__ __forceinline__ Parts<3> cut_tiles(const f32x4& a, const f32x4& b) {
  const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return cut8(x);
}

// Tiles of token rows in LDS.  bf16: the row's granules (8 elements) in the order p ^
// lin_swizzle(row), so that the 16 lanes that a read serves at once, of 4 + 4 rows and two
// granules, spread over the banks, and a wave's direct load can write 64 granules one after the other.
// fp32: three parts, rows of PITCH elements.
template <int D>
__device__ __forceinline__ constexpr int lin_swizzle(int r) {
  return D == 128 ? ((r & 3) << 2) | (((r >> 3) & 1) << 1) : (((r >> 1) & 1) << 2) | (((r >> 3) & 1) << 1);
}
template <int D, bool F32>
__device__ __forceinline__ int lin_at(int row, int granule) {
  return row * LinCfg<D, F32>::PITCH + 8 * (F32 ? granule : granule ^ lin_swizzle<D>(row));
}

// A lane's number that the compiler does not know to be the same every time: what follows from
// it (addresses) is formed again where it is used, and not kept in registers over the loop.
struct LinLane {
  int lane, g, c;
  __device__ __forceinline__ explicit LinLane(int l) {
    asm volatile("" : "+v"(l));
    lane = l;
    g = l >> 4;
    c = l & 15;
  }
};

__device__ __forceinline__ void lin_wait_loads() { __builtin_amdgcn_s_waitcnt(0x0f70); }  // vmcnt(0)

// A chunk's rows of a token tensor on their way from memory to a tile.  Rows past `count` are
// the last token's: finite where that is, and their dn of zero leaves them out.  A lane's
// place is a 32-bit offset from the chunk's first row (63 rows of 2^24 fp32 elements stay
// under 2^32).
//
// By way of registers (fp32 elements are cut into their parts there):
template <int D, bool F32>
struct LinFetch {
  using C = LinCfg<D, F32>;
  using T = typename Tok<F32>::T;
  static constexpr int GPR = D / 8, N = C::CH * GPR / C::THREADS, STEP = C::THREADS / GPR;
  static_assert(C::CH * GPR % C::THREADS == 0 && C::THREADS % GPR == 0, "granules");
  u32x4 raw[N][F32 ? 2 : 1];
  __device__ __forceinline__ void load(const T* base, unsigned ld, int count) {
    const int row = threadIdx.x % C::THREADS / GPR, col = 8 * (threadIdx.x % GPR);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const unsigned r = row + STEP * i, from = (int)r < count ? r : count - 1;
      const char* const p = (const char*)base + (from * ld + col) * (unsigned)sizeof(T);
      raw[i][0] = *(const u32x4*)p;
      if constexpr (F32) raw[i][1] = *(const u32x4*)(p + 16);
    }
  }
  __device__ __forceinline__ void store(uint16_t* tile) {
    const int row = threadIdx.x % C::THREADS / GPR, gr = threadIdx.x % GPR;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint16_t* const at = tile + lin_at<D, F32>(row + STEP * i, gr);
      if constexpr (F32) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(raw[i][e >> 2][e & 3]);
        const Parts<3> p = cut8(x);
#pragma unroll
        for (int k = 0; k < 3; ++k) *(bf16x8*)(at + k * C::PART) = p.p[k];
      } else {
        *(u32x4*)at = raw[i][0];
      }
    }
  }
};
// bf16 straight into LDS by the D / 16 waves of a state: the tile has to be free when the load
// starts, and is there after lin_wait_loads and a barrier.  LDS reads in between would
// wait for the load.
template <int D>
__device__ __forceinline__ void lin_load(uint16_t* tile, const uint16_t* base, unsigned ld, int count, int w, int lane) {
  using C = LinCfg<D, false>;
  constexpr int GPR = D / 8, RPL = 64 / GPR, N = C::CH / RPL / C::WAVES;  // rows of a load, loads of a wave
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r0 = (N * w + i) * RPL, r = r0 + lane / GPR;
    const unsigned from = r < count ? r : count - 1;
    const unsigned off = (from * ld + 8 * ((lane % GPR) ^ lin_swizzle<D>(r))) * 2u;
    __builtin_amdgcn_global_load_lds((const void*)((const char*)base + off),
                                     (__attribute__((address_space(3))) void*)(tile + r0 * D), 16, 0, 0);
  }
}

// Parts of granule `gr` of a row, and of 8 tokens (order dtau) of column dim_row(mt, c), or of
// column 16 w + c.
template <int D, bool F32>
__device__ __forceinline__ Parts<LinCfg<D, F32>::NT> lin_row(const uint16_t* t, int row, int gr) {
  using C = LinCfg<D, F32>;
  Parts<C::NT> p;
#pragma unroll
  for (int k = 0; k < C::NT; ++k) p.p[k] = *(const bf16x8*)(t + k * C::PART + lin_at<D, F32>(row, gr));
  return p;
}
template <int D, bool F32>
__device__ __forceinline__ Parts<LinCfg<D, F32>::NT> lin_read_tr(const uint16_t* t, int ts, int granule, int half, int g,
                                                                 int c) {
  using C = LinCfg<D, F32>;
  Parts<C::NT> p;
  const int row = 32 * ts + dtau(g, c >> 2);
#pragma unroll
  for (int k = 0; k < C::NT; ++k)
    p.p[k] = __builtin_shufflevector(delta_read_tr(t + k * C::PART + lin_at<D, F32>(row, granule) + half),
                                     delta_read_tr(t + k * C::PART + lin_at<D, F32>(row + 8, granule) + half), 0, 1, 2, 3,
                                     4, 5, 6, 7);
  return p;
}
template <int D, bool F32>
__device__ __forceinline__ Parts<LinCfg<D, F32>::NT> lin_row_dims(const uint16_t* t, int mt, int ts, int g, int c) {
  return lin_read_tr<D, F32>(t, ts, 4 * (mt >> 1) + (c & 3), 4 * (mt & 1), g, c);
}
template <int D, bool F32>
__device__ __forceinline__ Parts<LinCfg<D, F32>::NT> lin_columns(const uint16_t* t, int w, int ts, int g, int c) {
  return lin_read_tr<D, F32>(t, ts, 2 * w + ((c & 3) >> 1), 4 * (c & 1), g, c);
}

// 2^x in two parts, 48 bits.
__device__ __forceinline__ float2 lin_exp2_parts(double x) {
  const double f = exp2(x);
  const float hi = (float)f, rest = (float)(f - hi);
  return float2{hi, fabsf(rest) < INFINITY ? rest : 0.f};
}

template <int CTRL, int ROWS>
__device__ __forceinline__ double lin_add_from(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const unsigned lo = __builtin_amdgcn_update_dpp(0, (int)(unsigned)b, CTRL, ROWS, 0xf, false);
  const unsigned hi = __builtin_amdgcn_update_dpp(0, (int)(unsigned)(b >> 32), CTRL, ROWS, 0xf, false);
  return x + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lin_prefix(double x) {
  x = lin_add_from<0x111, 0xf>(x);  // one lane on
  x = lin_add_from<0x112, 0xf>(x);
  x = lin_add_from<0x114, 0xf>(x);
  x = lin_add_from<0x118, 0xf>(x);
  x = lin_add_from<0x142, 0xa>(x);  // lane 15 to row 1, 47 to row 3
  return lin_add_from<0x143, 0xc>(x);  // lane 31 to rows 2 and 3
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float lin_add_from(float x) {
  return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ float lin_prefix16(float x) {  // within 16 lanes
  x = lin_add_from<0x111, 0xf>(x);
  x = lin_add_from<0x112, 0xf>(x);
  x = lin_add_from<0x114, 0xf>(x);
  return lin_add_from<0x118, 0xf>(x);
}
__device__ __forceinline__ float lin_prefix(float x) {
  return lin_add_from<0x143, 0xc>(lin_add_from<0x142, 0xa>(lin_prefix16(x)));
}
__device__ __forceinline__ double lin_lane63(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const unsigned lo = __builtin_amdgcn_readlane((unsigned)b, 63), hi = __builtin_amdgcn_readlane((unsigned)(b >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// The factors of a chunk from its lanes' log decays; one wave.  before: those of the chunk
// before it in the pass, null for the first.
template <bool REV>
__device__ __forceinline__ void lin_factors(LinFactors* f, const LinFactors* before, float gl, int count, float scale) {
  const int lane = threadIdx.x & 63;
  if (lane >= count) gl = 0.f;
  if (gl < kMinLogDecay) gl = kMinLogDecay;
  double s = before ? before->after : 0.0;
  // in 64 bits: a strong decay among weak ones must not blur their differences
  const double c = lin_prefix(gl * kLog2E);
  const double last = lin_lane63(c), e0 = REV ? last - c : c;
  auto leaves = [&](double e) { return __any(!(fabs(e) <= kLinSpan)) || !(fabs(s + last) <= kLinSpan); };
  int flags = 0;
  float pre = 1.f;
  if (leaves(s + e0)) {
    flags = kLinScale;
    pre = exp2_wide(s);
    s = 0.0;
    if (leaves(e0)) flags |= kLinGated;
  }
  float up, dn;
  if (flags & kLinGated) {
    const float in = scale * exp2_wide(c), out = exp2_wide(last - c);
    up = REV ? out : in;
    dn = REV ? in : out;
  } else {
    up = exp2_wide(s + e0);
    dn = exp2_wide(-(s + e0));
    if (REV) dn *= scale;
    else up *= scale;
  }
  f->up[lane] = up;
  f->dn[lane] = lane < count ? dn : 0.f;
  f->cs[lane] = c;
  if (lane == 0) {
    const double after = flags & kLinGated ? 0.0 : s + last;
    f->s = s;
    f->after = after;
    f->sum = (before ? before->sum : 0.0) + last;
    f->count = count;
    f->pre = pre;
    f->last = exp2_wide(last);
    f->end = exp2_wide(after);
    f->flags = flags;
  }
}

// What a chunk's C is multiplied with where its part of the state is taken to the end of the
// chunks behind it, `after` them.
__device__ __forceinline__ void lin_reach(LinFactors* f, const LinFactors* after, float gl, int count) {
  const int lane = threadIdx.x & 63;
  if (lane >= count) gl = 0.f;
  if (gl < kMinLogDecay) gl = kMinLogDecay;
  const double c = lin_prefix(gl * kLog2E);
  const double last = lin_lane63(c), sum = after ? after->sum : 0.0;
  f->dn[lane] = lane < count ? exp2_wide(sum + last - c) : 0.f;
  if (lane == 0) f->sum = sum + last;
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
    const auto bb = lin_row<D, F32>(b, token_row(jt, c), 4 * s + g);
    const auto aa = lin_row<D, F32>(a, 16 * it + c, 4 * s + g);
    mma<C::LIM>(acc, bb, aa);
  }
  return acc;
}

// The same with the decays (GATED: all of them) and the mask.
template <bool REV, bool GATED>
__device__ __forceinline__ f32x4 lin_gate(const f32x4& x, const LinFactors* f, float scale, int it, int jt, int g,
                                          int c) {
  const int out = 16 * it + c, src = token_row(jt, 4 * g);
  f32x4 t;
  if constexpr (GATED) {
    const double co = f->cs[out];
    const int count = f->count;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const double dif = REV ? f->cs[src + r] - co : co - f->cs[src + r];
      const bool in = src + r < count && (REV ? src + r >= out : src + r <= out);
      t[r] = in ? x[r] * scale * exp2_wide(in ? dif : 0.0) : 0.f;
    }
  } else {
    const f32x4 w = *(const f32x4*)(f->dn + src);
#pragma unroll
    for (int r = 0; r < 4; ++r) t[r] = (REV ? src + r >= out : src + r <= out) ? x[r] * w[r] : 0.f;
  }
  return t;
}

// Four sources of a triangle's tile into its operand tiles: element 4 (jt & 1) + r of lane.
__device__ __forceinline__ void lin_put(uint16_t* frags, int frags_each, int fi, int jt, int lane, const f32x4& t) {
  unsigned r[4] = {__float_as_uint(t[0]), __float_as_uint(t[1]), __float_as_uint(t[2]), __float_as_uint(t[3])};
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    u32x2 w;
#pragma unroll
    for (int i = 0; i < 2; ++i) w[i] = __builtin_amdgcn_perm(r[2 * i + 1], r[2 * i], 0x07060302u);
    *(u32x2*)(frags + (p * frags_each + fi) * kFragElems + lane * 8 + 4 * (jt & 1)) = w;
    if (p < 2)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        r[i] = __float_as_uint(__uint_as_float(r[i]) - __uint_as_float(r[i] & 0xffff0000u));
  }
}

template <int D, bool F32>
struct LinState {
  using C = LinCfg<D, F32>;
  f32x4 m[C::MT];  // rows dim_row(mt, 4 g + r), column 16 w + c

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt) m[mt] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // S [d (columns of the state)][d (rows)] in memory; TR: the other way round.
  template <bool TR>
  __device__ __forceinline__ void load(const float* s, int w, int g, int c) {
    const int col = 16 * w + c;
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt) {
      const int row = dim_row(mt, 4 * g);
      if constexpr (TR) {
#pragma unroll
        for (int r = 0; r < 4; ++r) m[mt][r] = s[(row + r) * D + col];
      } else {
        m[mt] = *(const f32x4*)(s + col * D + row);
      }
    }
  }
  __device__ __forceinline__ void store(float* s, int w, int g, int c) const {
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt) *(f32x4*)(s + (16 * w + c) * D + dim_row(mt, 4 * g)) = m[mt];
  }
  __device__ __forceinline__ void scale(float x) {
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
      for (int r = 0; r < 4; ++r) m[mt][r] *= x;
  }
};

template <int D, bool F32>
struct LinOut {
  using C = LinCfg<D, F32>;
  f32x4 o[C::IT];  // dims 16 w + 4 g + r of token 16 it + c

  // A M^
  __device__ __forceinline__ void read(const LinState<D, F32>& st, const uint16_t* a, int g, int c) {
#pragma unroll
    for (int it = 0; it < C::IT; ++it) o[it] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < C::KS; ++s) {
      const Parts<3> mp = cut_tiles(st.m[2 * s], st.m[2 * s + 1]);
#pragma unroll
      for (int it = 0; it < C::IT; ++it) mma<2>(o[it], mp, lin_row<D, F32>(a, 16 * it + c, 4 * s + g));
    }
  }
  __device__ __forceinline__ void scale(const LinFactors* f, int c) {
#pragma unroll
    for (int it = 0; it < C::IT; ++it) {
      const float x = f->up[16 * it + c];
#pragma unroll
      for (int r = 0; r < 4; ++r) o[it][r] *= x;
    }
  }
  // rows of the chunk's tokens, T elements (or fp32) of stride ld
  template <typename T>
  __device__ __forceinline__ void store(T* base, unsigned ld, int count, int w, int g, int c) const {
    const unsigned at = (c * ld + 16 * w + 4 * g) * (unsigned)sizeof(T), step = 16 * ld * (unsigned)sizeof(T);
    auto put = [&](int it) {
      char* const p = (char*)base + (size_t)(it * step) + at;
      if constexpr (sizeof(T) == 4) *(f32x4*)p = o[it];
      else *(u32x2*)p = u32x2{pack_bf16x2(o[it][0], o[it][1]), pack_bf16x2(o[it][2], o[it][3])};
    };
    if (count == C::CH) {
#pragma unroll
      for (int it = 0; it < C::IT; ++it) put(it);
    } else {
#pragma unroll
      for (int it = 0; it < C::IT; ++it)
        if (16 * it + c < count) put(it);
    }
  }
};

// out += T C and M^ <- M^ + B^T (dn o C).
template <int D, bool F32, bool REV, bool OUT>
__device__ __forceinline__ void lin_tokens(LinOut<D, F32>* out, LinState<D, F32>& st, const uint16_t* frags,
                                           const uint16_t* b, const uint16_t* cc, const float* dn, int w, int lane,
                                           int g, int c) {
  using C = LinCfg<D, F32>;
#pragma unroll
  for (int ts = 0; ts < C::TS; ++ts) {
    const auto cf = lin_columns<D, F32>(cc, w, ts, g, c);
    if constexpr (OUT) {
#pragma unroll
      for (int it = 0; it < C::IT; ++it) {
        if (!lin_in<D, F32, REV>(it, ts)) continue;
        Parts<3> t;
#pragma unroll
        for (int p = 0; p < 3; ++p)
          t.p[p] = *(const bf16x8*)(frags + (p * C::FRAGS + lin_frag<D, F32, REV>(it, ts)) * kFragElems + lane * 8);
        mma<2>(out->o[it], cf, t);
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
    const f32x4 w0 = *(const f32x4*)(dn + 32 * ts + dtau(g, 0)), w1 = *(const f32x4*)(dn + 32 * ts + dtau(g, 4));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] *= w0[e];
      x[4 + e] *= w1[e];
    }
    const Parts<3> cw = cut8(x);
#pragma unroll
    for (int mt = 0; mt < C::MT; ++mt) mma<2>(st.m[mt], lin_row_dims<D, F32>(b, mt, ts, g, c), cw);
  }
}

// ---- launchers ----------------------------------------------------------------
// The table of segments (n_seq > kLinWaveSeqs).
hipError_t launch_linear_table(const LinSeqs& s, hipStream_t st);
// What each segment of a sequence adds to the state, all but its last.
hipError_t launch_linear_states(const LinArgs& a, int d, bool f32, hipStream_t st);
hipError_t launch_linear_join(const LinArgs& a, int d, bool both, hipStream_t st);
// The outputs and last states.
hipError_t launch_linear_out(const LinArgs& a, int d, bool f32, hipStream_t st);
// Gradients: what segments add to states and their gradients, and dg's part within the chunks;
// dk, dv, dg's part to the chunks' ends, d_dump and the first states' gradient; dq and dg.
hipError_t launch_linear_grad_states(const LinArgs& a, int d, bool f32, hipStream_t st);
hipError_t launch_linear_dkdv(const LinArgs& a, int d, bool f32, hipStream_t st);
hipError_t launch_linear_dq(const LinArgs& a, int d, bool f32, hipStream_t st);
// dq and dk from o_part and dk_part, summed over the value heads of a key head, and, unless dg is
// null, dg [heads] from the chunks' sums a.dg.
hipError_t launch_linear_groups(const LinArgs& a, int d, bool f32, float* dg, hipStream_t st);
// dg alone.
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
