// What a chunk of the gated delta rule needs besides the state, for all chunks
// and heads at once: T = (I + A)^-1 and P as matrix-core operand tiles, and the
// row factors gam, dec, beta (delta_rule.h).
#include "delta_rule.h"

namespace zm {

namespace {

constexpr int kPitch = 68;     // floats of a row of the 64 x 64 matrices in LDS
constexpr int kBlk = 336;      // floats of a 16 x 16 diagonal block (rows of 20; blocks 16 banks apart)

// ---- tables -------------------------------------------------------------------
// One workgroup: the clamped, nondecreasing offsets, the prefix sums of chunks
// and segments, then every chunk's and segment's entry by a search in them.  A chain
// of dependent steps, so scans run within waves and the searches in LDS where the
// sequences fit it.
__global__ __launch_bounds__(1024) void k_delta_table(DeltaSeqs s) {
  __shared__ int part[3][16], first_l[kTableLds + 1], begin_l[kTableLds + 1], segs_l;
  __shared__ int len_l[kTableLds];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, per = (s.n_seq + 1023) / 1024;
  const bool in_lds = s.n_seq <= kTableLds;
  const int b0 = t * per, b1 = b0 + per < s.n_seq ? b0 + per : s.n_seq;
  // running maximum of the clamped ends
  const int start = clampi(s.offsets[0], 0, s.n);
  int top = start;
  for (int b = b0; b < b1; ++b) {
    const int e = clampi(s.offsets[b + 1], 0, s.n);
    if (e > top) top = e;
  }
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const int o = __shfl_up(top, m, 64);
    if (lane >= m && o > top) top = o;
  }
  if (lane == 63) part[0][w] = top;
  int run = __shfl_up(top, 1, 64);
  if (lane == 0) run = start;
  __syncthreads();
  for (int i = 0; i < w; ++i)
    if (part[0][i] > run) run = part[0][i];
  const int run0 = run;
  int nc = 0, ns = 0;
  for (int b = b0; b < b1; ++b) {
    int e = clampi(s.offsets[b + 1], 0, s.n);
    if (e < run) e = run;
    const int c = (int)(((int64_t)(e - run) + kChunk - 1) / kChunk);
    nc += c;
    ns += c > 0 ? (c + s.seg_chunks - 1) / s.seg_chunks : 1;
    run = e;
  }
  if (s.longest_first && t < s.n_seq) len_l[t] = nc;
  int c0 = nc, s0 = ns;
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const int oc = __shfl_up(c0, m, 64), os = __shfl_up(s0, m, 64);
    if (lane >= m) {
      c0 += oc;
      s0 += os;
    }
  }
  if (lane == 63) {
    part[1][w] = c0;
    part[2][w] = s0;
  }
  c0 -= nc;
  s0 -= ns;
  __syncthreads();
  for (int i = 0; i < w; ++i) {
    c0 += part[1][i];
    s0 += part[2][i];
  }
  // where a sequence is one segment: its place by length, then by number
  if (s.longest_first && t < s.n_seq) {
    s0 = 0;
    for (int b = 0; b < s.n_seq; ++b) s0 += len_l[b] > nc || (len_l[b] == nc && b < t);
  }
  // sequence by sequence: its first chunk, its begin and its segments
  int* const first = in_lds ? first_l : s.first_chunk;
  int* const begin = in_lds ? begin_l : s.begin;
  run = run0;
  for (int b = b0; b < b1; ++b) {
    int e = clampi(s.offsets[b + 1], 0, s.n);
    if (e < run) e = run;
    const int c = (int)(((int64_t)(e - run) + kChunk - 1) / kChunk);
    first[b] = c0;
    begin[b] = run;
    const int k = c > 0 ? (c + s.seg_chunks - 1) / s.seg_chunks : 1;
    for (int i = 0; i < k; ++i) {
      const int f = i * s.seg_chunks;
      s.segs[s0 + i] = int4{c0 + f, c - f < s.seg_chunks ? c - f : s.seg_chunks, b,
                            (i == 0 ? 1 : 0) | (i == k - 1 ? 2 : 0) | k << 2};
    }
    c0 += c;
    s0 += k;
    run = e;
    if (b == s.n_seq - 1) {
      first[s.n_seq] = c0;
      begin[s.n_seq] = e;
      segs_l = s.longest_first ? s.n_seq : s0;
    }
  }
  __syncthreads();
  __threadfence_block();
  const int all = first[s.n_seq];
  for (int i = segs_l + t; i < s.n_segs; i += 1024) s.segs[i] = int4{0, -1, 0, 0};
  for (int ci = t; ci < s.n_chunks; ci += 1024) {
    if (ci >= all) {
      s.chunks[ci] = int4{0, 0, 0, 0};
      continue;
    }
    int lo = 0, hi = s.n_seq;  // the last sequence whose first chunk is at most ci
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= ci) lo = mid; else hi = mid;
    }
    const int at = begin[lo] + kChunk * (ci - first[lo]);
    const int left = begin[lo + 1] - at;
    s.chunks[ci] = int4{at, left < kChunk ? left : kChunk, lo, 0};
  }
}

// ---- T and P --------------------------------------------------------------------
// Parts of tile `tile`'s row (lane c) at dims 32 s + 8 g; rows past the chunk's
// tokens are zero.
template <bool F32>
__device__ __forceinline__ Parts<Tok<F32>::NT> row_parts(const typename Tok<F32>::T* base, int64_t ld,
                                                         int tok, int count, int col) {
  const auto p = load8(base + (tok < count ? tok : count - 1) * ld + col);
  return tok < count ? p : zero_parts<Tok<F32>::NT>();
}

// Operand tiles of a 64 x 64 matrix in LDS: item i of 6 x 64 is tile i / 64, lane
// i % 64.  TR: of the transpose.
template <int NP, bool TR>
__device__ __forceinline__ void write_frags(const float* m, uint16_t* out) {
  for (int i = threadIdx.x; i < kTriFrags * 64; i += 256) {
    const int f = i >> 6, lane = i & 63, g = lane >> 4, c = lane & 15;
    int it, ts;
    if (!TR) {
      it = f < 2 ? f : 2 + (f - 2) / 2;
      ts = f < 2 ? 0 : (f - 2) & 1;
    } else {
      it = f < 4 ? f / 2 : f - 2;
      ts = f < 4 ? f & 1 : 1;
    }
    const int row = token_row(it, c);
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int col = 32 * ts + dtau(g, e);
      x[e] = TR ? m[col * kPitch + row] : m[row * kPitch + col];
    }
    const Parts<NP> p = split8<NP>(x);
#pragma unroll
    for (int k = 0; k < NP; ++k)
      *(bf16x8*)(out + (int64_t)(k * kTriFrags + f) * kFragElems + lane * 8) = p.p[k];
  }
}

// One workgroup per (chunk, head), wave w its 16-row block w of the products
// K K^T and Q K^T.  T by blocks of 16: the diagonal blocks' inverses by forward
// substitution (a column a lane; unlike a product of powers of A it stays exact
// where keys repeat), then block column w in wave w by
//   T_iw = -D_i sum_{w <= j < i} A_ij T_jw,
// on fp32 matrix instructions whose results are the next right operands.  Bound by that
// chain's latency; the many chunks run side by side: 1408 of 128 dims, bf16, 38 us.
template <int D, bool F32, bool BWD>
__global__ __launch_bounds__(256) void k_delta_prep(DeltaArgs a) {
  using T = typename Tok<F32>::T;
  constexpr int NT = Tok<F32>::NT, KS = D / 32, LIM = NT == 1 ? 0 : 2;
  __shared__ float ma[kChunk * kPitch], mp[kChunk * kPitch];
  __shared__ float diag[4 * kBlk];
  __shared__ double cs[kChunk];
  __shared__ float be[kChunk];
  const int h = blockIdx.x % a.heads, ci = blockIdx.x / a.heads;
  const int4 ch = delta_chunk(a.sq, ci);
  const int count = ch.y;
  if (count == 0) return;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15, hk = h / (a.heads / a.heads_k);
  const T* const kp = (const T*)a.k.p + (int64_t)ch.x * a.k.ld + hk * D;
  const T* const qp = (const T*)a.q.p + (int64_t)ch.x * a.q.ld + hk * D;
  const int64_t slot = (int64_t)ci * a.heads + h;

  float gl = 0.f, b = 0.f;
  if (w == 0 && lane < count) {
    gl = a.g[((int64_t)ch.x + lane) * a.heads + h];
    b = a.beta[((int64_t)ch.x + lane) * a.heads + h];
  }
  f32x4 kk[4], qk[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) kk[j] = qk[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const int col = 32 * s + 8 * g;
    const auto ka = row_parts<F32>(kp, a.k.ld, 16 * w + c, count, col);
    const auto qa = row_parts<F32>(qp, a.q.ld, 16 * w + c, count, col);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j > w) continue;
      const auto kb = row_parts<F32>(kp, a.k.ld, 16 * j + c, count, col);
      mma<LIM>(kk[j], ka, kb);
      mma<LIM>(qk[j], qa, kb);
    }
  }
  if (w == 0) {  // the wave with fewest products
    if (gl < kMinLogDecay) gl = kMinLogDecay;
    // sums in 64 bits: a strong decay among weak ones must not blur their differences
    double s = gl * kLog2E;  // exponents of two
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
      const double o = __shfl_up(s, m, 64);
      if (lane >= m) s += o;
    }
    cs[lane] = s;
    be[lane] = b;
    const double last = __shfl(s, 63, 64);
    float* const r = a.rows + slot * 3 * kChunk;
    r[lane] = exp2_wide(s);
    r[kChunk + lane] = exp2_wide(last - s);
    r[2 * kChunk + lane] = b;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int col = 16 * j + c;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * w + 4 * g + r;
      const float gd = row >= col ? exp2_wide(cs[row] - cs[col]) : 0.f;
      const float av = row > col ? be[row] * gd * kk[j][r] : 0.f;
      ma[row * kPitch + col] = av;
      mp[row * kPitch + col] = row >= col ? a.scale * gd * qk[j][r] : 0.f;
      if (j == w) diag[w * kBlk + (4 * g + r) * 20 + c] = av;
    }
  }
  __syncthreads();
  if (w == 0) {
    // column c of diagonal block g's inverse
    float x[16];
    const float* const blk = diag + g * kBlk;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == c ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < i; ++j) s = fmaf(-blk[i * 20 + j], x[j], s);
      x[i] = s;
    }
    // every lane has read the block: its 16 lanes run as one
#pragma unroll
    for (int i = 0; i < 16; ++i) diag[g * kBlk + i * 20 + c] = x[i];
  }
  if constexpr (BWD)
    write_frags<3, true>(mp, a.pt_frags + slot * 3 * kTriFrags * kFragElems);
  else
    write_frags<3, false>(mp, a.p_frags + slot * 3 * kTriFrags * kFragElems);
  __syncthreads();
  f32x4 tc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    tc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (i == w)
#pragma unroll
      for (int r = 0; r < 4; ++r) tc[i][r] = diag[i * kBlk + (4 * g + r) * 20 + c];
  }
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    if (i <= w) continue;
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < i; ++j) {
      if (j < w) continue;
      const f32x4 av = *(const f32x4*)(ma + (16 * i + c) * kPitch + 16 * j + 4 * g);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        y = __builtin_amdgcn_mfma_f32_16x16x4f32(av[r], tc[j][r], y, 0, 0, 0);
    }
    const f32x4 dv = *(const f32x4*)(diag + i * kBlk + c * 20 + 4 * g);
    f32x4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 4; ++r)
      t = __builtin_amdgcn_mfma_f32_16x16x4f32(-dv[r], y[r], t, 0, 0, 0);
    tc[i] = t;
  }
  // P's tiles are out: its place takes T
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) mp[(16 * i + 4 * g + r) * kPitch + 16 * w + c] = tc[i][r];
  __syncthreads();
  if constexpr (F32) write_frags<3, false>(mp, a.t_frags + slot * 3 * kTriFrags * kFragElems);
  if constexpr (BWD) write_frags<3, true>(mp, a.tt_frags + slot * 3 * kTriFrags * kFragElems);
}

template <int D>
hipError_t prep_any(const DeltaArgs& a, bool backward, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.sq.n_chunks * a.heads)), blk(256);
  if (!backward) hipLaunchKernelGGL((k_delta_prep<D, true, false>), grid, blk, 0, st, a);
  else if (a.f32) hipLaunchKernelGGL((k_delta_prep<D, true, true>), grid, blk, 0, st, a);
  else hipLaunchKernelGGL((k_delta_prep<D, false, true>), grid, blk, 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_table(const DeltaSeqs& s, hipStream_t st) {
  hipLaunchKernelGGL(k_delta_table, dim3(1), dim3(1024), 0, st, s);
  return hipGetLastError();
}

hipError_t launch_delta_prep(const DeltaArgs& a, bool backward, hipStream_t st) {
  if (a.sq.n_chunks == 0) return hipSuccess;
  return a.d == 128 ? prep_any<128>(a, backward, st) : prep_any<64>(a, backward, st);
}

}  // namespace zm
