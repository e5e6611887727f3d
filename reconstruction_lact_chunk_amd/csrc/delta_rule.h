// Gated delta rule: shared device code, argument blocks and launchers.
//
// Per sequence and value head, S in R^{d x d} (fp32), a_t = exp(g_t):
//   S_t = a_t S_{t-1} (I - b_t k_t k_t^T) + b_t v_t k_t^T,  o_t = scale S_t q_t.
// Tokens are taken kChunk at a time.  With c_i the sum of g over the chunk's
// tokens up to i, gam_i = exp(c_i), dec_i = exp(c_C - c_i), G_ij = exp(c_i - c_j)
// and M = S^T at the chunk's start:
//   A = strictly_lower(b_i G_ij k_i.k_j),  T = (I + A)^-1,  P = scale lower(G_ij q_i.k_j)
//   R = V - gam o (K M),  U = T (b o R),  O = scale gam o (Q M) + P U,
//   M' = gam_C M + K^T (dec o U).
// T and P do not depend on M.  fp32 tokens: delta_prep.hip forms them for all chunks
// at once, delta_scan.hip goes through the chunks of a sequence in order; bf16
// tokens: delta_fused.hip does both side by side.  A long sequence of few heads is cut
// into segments, whose transitions M -> N M + B are joined before the outputs.
//
// Matrix products run on v_mfma_f32_16x16x32_bf16.  An operand held in fp32
// (M, U, T, P, fp32 tokens) enters as a sum of bf16 parts: three parts carry 24
// bits, and of the products of parts those below 2^-24 are left out, so the
// state is as exact as fp32 products would leave it at 3 (bf16 tokens) or 6
// matrix instructions instead of the 16 that fp32 ones cost.  O takes as many parts
// where it ends as bf16: it can be what is left of terms much larger than itself.
//
// The matrix cores return rows 4 g + r (r < 4) of column c in lane 16 g + c, and
// take rows in slots 8 g + e (e < 8) of a 32-row step in the same lane.  With
// rows mapped to slots by tau (tokens) or 8 g + e (head dims) a product's result
// is the next product's right operand without leaving its registers.
#pragma once

#include "zm_internal.h"

namespace zm {

constexpr int kChunk = 64;             // tokens of a chunk
constexpr int kTriFrags = 6;           // 16 x 32 operand tiles of a 64 x 64 triangle
constexpr int kFragElems = 64 * 8;     // bf16 elements of one such tile
constexpr int kTableLds = 1024;        // sequences that the table's kernel keeps in LDS
constexpr float kMinLogDecay = -128.f; // exp of less is 0 in fp32
constexpr double kLog2E = 1.4426950408889634;

// Where the sequences lie.  Without a table (one sequence) a chunk follows from
// its index; offsets are clamped to 0 <= ... <= n and made nondecreasing, so that
// no content of them reaches outside the tokens.
struct DeltaSeqs {
  const int* offsets;    // [n_seq + 1] or null: one sequence of all n tokens
  int4* chunks;          // {first token, tokens, sequence, 0}, null without a table
  int4* segs;            // {first chunk, chunks (-1: unused), sequence,
                         //  1 first | 2 last | 4 * segments of the sequence}
  int* first_chunk;      // [n_seq + 1] scratch of the table's kernel
  int* begin;            // [n_seq + 1] scratch: clamped offsets
  int n, n_seq;
  int n_chunks, n_segs;  // upper bounds over every content of offsets
  int seg_chunks;        // chunks of a segment
  bool longest_first;    // segments (one to a sequence) in the order of their chunks
};

struct DeltaTokens {
  const void* p;
  int64_t ld;
};

struct DeltaArgs {
  DeltaSeqs sq;
  DeltaTokens q, k, v;
  const float* g;       // [n][heads]
  const float* beta;    // [n][heads]
  int heads, heads_k, d;
  float scale;
  bool f32;
  // per (chunk, head): operand tiles and row factors
  uint16_t* t_frags;    // [3][kTriFrags][kFragElems] parts of T
  uint16_t* p_frags;    // parts of P (these two: fp32 forward)
  uint16_t* tt_frags;   // parts of T^T, P^T (backward)
  uint16_t* pt_frags;
  float* rows;          // [3][kChunk] gam, dec, beta
};

struct DeltaScanArgs {
  const float* state_in;    // [n_seq][heads][d][d] or null (zeros)
  float* state_out;         // the same, or null
  const float* seg_start;   // [n_segs][heads][d][d]: states at the segments' starts, or null
  float* trans;             // pass of transitions: [n_segs][heads][2 or 3][d][d]: N, B and, with both,
                            // the transpose of N, as join_n and join_b place them
  bool both;
  void* o;
  int64_t ld_o;
  float* m_out;             // [n_chunks][heads][d][d]: M at each chunk's start (backward), as below
  float* u_out;             // U (backward), as below
};

// 2^x to 32 bits for an x of any size.  Of a sum of decays near 60 rounded to 32 bits as a
// whole up to 2^-19 is lost, 1.3e-6 of the factor, and between two tokens that does not
// cancel: so the whole part goes into the exponent and only the rest is rounded.
__device__ __forceinline__ float exp2_wide(double x) {
  const double whole = rint(x);
  return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f((float)(x - whole)),
                                 (int)fmin(fmax(whole, -4096.0), 4096.0));
}

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : (x > hi ? hi : x); }

// Chunk ci: {first token, tokens (0: unused), sequence, -}.
__device__ __forceinline__ int4 delta_chunk(const DeltaSeqs& s, int ci) {
  if (s.chunks) return s.chunks[ci];
  int a = 0, e = s.n;
  if (s.offsets) {
    a = clampi(s.offsets[0], 0, s.n);
    e = clampi(s.offsets[1], a, s.n);
  }
  const int64_t st = (int64_t)a + (int64_t)kChunk * ci;
  const int left = st < e ? (int)(e - st) : 0;
  return int4{left > 0 ? (int)st : 0, left < kChunk ? left : kChunk, 0, 0};
}

__device__ __forceinline__ int4 delta_seg(const DeltaSeqs& s, int si) {
  if (s.segs) return s.segs[si];
  int a = 0, e = s.n;
  if (s.offsets) {
    a = clampi(s.offsets[0], 0, s.n);
    e = clampi(s.offsets[1], a, s.n);
  }
  const int chunks = (int)(((int64_t)(e - a) + kChunk - 1) / kChunk);
  const int segs = chunks > 0 ? (chunks + s.seg_chunks - 1) / s.seg_chunks : 1;
  if (si >= segs) return int4{0, -1, 0, 0};
  const int f = si * s.seg_chunks;
  const int c = chunks - f < s.seg_chunks ? chunks - f : s.seg_chunks;
  return int4{f, c, 0, (si == 0 ? 1 : 0) | (si == segs - 1 ? 2 : 0) | segs << 2};
}

// Token of slot e of lane group g in a 32-token step (and, for row m = 4 g' + i of
// 16-row tile h of the step, token_row below): the order whose row and
// transposing LDS reads the update kernel already uses.
__device__ __forceinline__ constexpr int dtau(int g, int e) {
  return 16 * (g >> 1) + 4 * (g & 1) + 8 * (e >> 2) + (e & 3);
}
// Token of row m of tile `it` (16 rows; two tiles to a step).
__device__ __forceinline__ constexpr int token_row(int it, int m) {
  return 32 * (it >> 1) + dtau(m >> 2, 4 * (it & 1) + (m & 3));
}
// Head dim of row m of state tile mt.
__device__ __forceinline__ constexpr int dim_row(int mt, int m) {
  return 32 * (mt >> 1) + 8 * (m >> 2) + 4 * (mt & 1) + (m & 3);
}
// Where the join of segments finds element (row, col) of N, and the four of a state
// from (dim_row(mt, 4 g), column dv): as one load of a wave each.
template <int D>
__device__ __forceinline__ int join_n(int row, int col) {
  const int mt = 2 * (row >> 5) + ((row >> 2) & 1), m = 4 * ((row >> 3) & 3) + (row & 3);
  return ((mt * (D / 16) + (col >> 5) * 2 + ((col >> 2) & 1)) * 64 + 16 * ((col >> 3) & 3) + m) * 4 + (col & 3);
}
template <int D>
__device__ __forceinline__ int join_b(int dv, int mt, int g) {
  return (((dv >> 4) * (D / 16) + mt) * 64 + 16 * g + (dv & 15)) * 4;
}
// Operand tile (it, ts) of a lower (T, P) or upper (transposed) triangle.
__device__ __forceinline__ constexpr int low_frag(int it, int ts) { return it < 2 ? it : 2 * it - 2 + ts; }
__device__ __forceinline__ constexpr int up_frag(int it, int ts) { return it < 2 ? 2 * it + ts : it + 2; }

template <int NP>
struct Parts {
  bf16x8 p[NP];
};

// x as a sum of NP bf16 parts, each the rounding of what the ones before leave.
template <int NP>
__device__ __forceinline__ Parts<NP> split8(const float* x) {
  Parts<NP> out;
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = pack_bf16x2(r[2 * i], r[2 * i + 1]);
      if (p + 1 < NP) {
        r[2 * i] -= bf16lo(w[i]);
        r[2 * i + 1] -= bf16hi(w[i]);
      }
    }
    out.p[p] = as_bf16x8(w);
  }
  return out;
}
template <int NP>
__device__ __forceinline__ Parts<NP> split_tiles(const f32x4& a, const f32x4& b) {
  const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  return split8<NP>(x);
}

// acc += a b over the part products of order at most LIM, the smallest first.
template <int LIM, int NA, int NB>
__device__ __forceinline__ void mma(f32x4& acc, const Parts<NA>& a, const Parts<NB>& b) {
#pragma unroll
  for (int s = LIM; s >= 0; --s)
#pragma unroll
    for (int p = 0; p <= s; ++p)
      if (p < NA && s - p < NB) acc = mfma_bf16(a.p[p], b.p[s - p], acc);
}

typedef __attribute__((ext_vector_type(4))) __bf16 dbf16x4;
typedef __attribute__((address_space(3))) dbf16x4 lds_dbf16x4;

// Transposing LDS read: within 16 lanes, lane i gets element i % 4 of the 8-byte
// words at the addresses of lanes 4 e + i / 4, e = 0..3.
__device__ __forceinline__ dbf16x4 delta_read_tr(const uint16_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
      (lds_dbf16x4*)((__attribute__((address_space(3))) void*)(p)));
}

// LDS reads and writes of this wave are done, then the workgroup's barrier.  Loads
// and stores of global memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Token element type and the parts it takes.
template <bool F32>
struct Tok {
  using T = uint16_t;
  static constexpr int NT = 1;
};
template <>
struct Tok<true> {
  using T = float;
  static constexpr int NT = 3;
};

// Parts of 8 consecutive elements in memory.
__device__ __forceinline__ Parts<1> load8(const uint16_t* p) {
  return Parts<1>{{as_bf16x8(*(const u32x4*)p)}};
}
__device__ __forceinline__ Parts<3> load8(const float* p) {
  const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 4);
  return split_tiles<3>(a, b);
}
template <int NP>
__device__ __forceinline__ Parts<NP> zero_parts() {
  Parts<NP> z;
#pragma unroll
  for (int p = 0; p < NP; ++p) z.p[p] = as_bf16x8(u32x4{0u, 0u, 0u, 0u});
  return z;
}

struct DeltaJoinArgs {
  const float* init;     // [n_seq][heads][d][d] or null
  const float* trans;
  int stride;            // matrices to a segment of trans
  const float* e;        // the way back: what a segment adds (join_b), else null
  float* to;             // [n_segs][heads][d][d]
};

// Backward: buffers that the reverse pass and the chunks' gradients share, and outputs.
struct DeltaGradArgs {
  DeltaTokens d_o;           // gradient of o
  const float* dstate_out;   // gradient of the last states, or null
  float* dstate_in;          // receives the gradient of the first states, or null
  const float* seg_end;      // [n_segs][heads][d][d]: gradients of the states at the segments' ends, or null
  float* e_out;              // [n_segs][heads][d][d] (join_b): pass of transitions only
  // Of a chunk and head, 32 columns of d_v after the other, as k_delta_grads takes them
  // (rows of all of d_v would be read in pieces far apart):
  const float* m_in;         // [n_chunks][heads][d / 32][d_k][32] M at each chunk's start
  float* d_m;                // the same of the gradient of M at each chunk's end
  const float* u;            // [n_chunks][heads][d / 32][kChunk][32]
  float* x;                  // the same of the gradient of beta o R
  void* dv;
  int64_t ld_dv;
  void* dq;                  // with one value head to a key head, else null
  void* dk;
  int64_t ld_dq, ld_dk;
  float* dq_part;            // [n][heads][d] otherwise
  float* dk_part;
  float* dg;                 // [n][heads]
  float* dbeta;
};

// ---- launchers --------------------------------------------------------------------
// The tables of chunks and segments (n_seq > 1).
hipError_t launch_delta_table(const DeltaSeqs& s, hipStream_t st);
// T and P (backward: T of fp32 tokens, T^T, P^T) and the row factors of every chunk and head.
hipError_t launch_delta_prep(const DeltaArgs& a, bool backward, hipStream_t st);
// fp32 tokens: the chunks in order from the tiles of launch_delta_prep; bf16 tokens:
// the same with the triangles formed on the way (no tiles needed).
hipError_t launch_delta_scan(const DeltaArgs& a, const DeltaScanArgs& s, hipStream_t st);
hipError_t launch_delta_fused(const DeltaArgs& a, const DeltaScanArgs& s, hipStream_t st);
// The states at the segments' starts (gradients at their ends) from their transitions.
hipError_t launch_delta_join(const DeltaArgs& a, const DeltaJoinArgs& j, hipStream_t st);
// Backward through the chunks of each segment, last first: d_m, x, dv, dstate_in.
hipError_t launch_delta_reverse(const DeltaArgs& a, const DeltaGradArgs& s, hipStream_t st);
// dq, dk, dg, dbeta of every chunk and head from u, x, m_in, d_m.
hipError_t launch_delta_grads(const DeltaArgs& a, const DeltaGradArgs& s, hipStream_t st);
struct DeltaStepArgs {
  DeltaTokens q, k, v;
  const float* g;
  const float* beta;
  float* state;
  void* o;
  int64_t ld_o;
  int n_seq, heads, heads_k, d;
  float scale;
  bool f32;
};
hipError_t launch_delta_step(const DeltaStepArgs& a, hipStream_t st);

}  // namespace zm
