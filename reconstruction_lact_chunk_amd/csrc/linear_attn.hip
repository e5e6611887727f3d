// Linear attention with decays (linear_attn.h): the table of segments, what segments add
// to the state, their join, and the outputs.
#include "linear_attn.h"

namespace zm {

namespace {

// ---- table --------------------------------------------------------------------
// One workgroup: the clamped, nondecreasing offsets, the prefix sums of chunks, segments,
// slots and sequences of several segments, and every segment's entry; longest first where there are more workgroups than
// run at once, so that long ones do not end last.  5 to 8 us.
__global__ __launch_bounds__(1024) void k_linear_table(LinSeqs s) {
  __shared__ int part[5][16], total, slots, splits;
  __shared__ LinSeg seg_l[kLinSorted];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6, per = (s.n_seq + 1023) / 1024;
  const int b0 = t * per < s.n_seq ? t * per : s.n_seq, b1 = b0 + per < s.n_seq ? b0 + per : s.n_seq;
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
  // chunks, segments, slots and sequences of several before this thread's sequences
  int v[4] = {0, 0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    int e = clampi(s.offsets[b + 1], 0, s.n);
    if (e < run) e = run;
    const int k = lin_segs(s, e - run);
    v[0] += lin_chunks(s, e - run);
    v[1] += k;
    v[2] += k > 1 ? k : 0;
    v[3] += k > 1;
    run = e;
  }
  int at[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    int x = v[j];
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
      const int o = __shfl_up(x, m, 64);
      if (lane >= m) x += o;
    }
    if (lane == 63) part[1 + j][w] = x;
    at[j] = x - v[j];
  }
  __syncthreads();
  for (int i = 0; i < w; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) at[j] += part[1 + j][i];
  run = run0;
  for (int b = b0; b < b1; ++b) {
    int e = clampi(s.offsets[b + 1], 0, s.n);
    if (e < run) e = run;
    const int len = e - run;
    const int k = lin_segs(s, len);
    for (int i = 0; i < k; ++i) {
      const int from = i * s.seg_tokens;  // < len, or 0
      LinSeg g;
      g.tok = run + from;
      g.count = len - from < s.seg_tokens ? len - from : s.seg_tokens;
      g.seq = b;
      g.flags = (i == 0 ? 1 : 0) | (i == k - 1 ? 2 : 0);
      g.chunk0 = at[0] + lin_chunks(s, from);
      g.slot = at[2] + i;
      g.segs = k;
      g.split = at[3];
      const int si = at[1] + i;
      if (s.longest_first) {
        seg_l[si] = g;
      } else {
        s.segs[si] = g;
        if (k > 1) {
          s.by_slot[g.slot] = si;
          if (i == 0) s.by_split[g.split] = si;
        }
      }
    }
    at[0] += lin_chunks(s, len);
    at[1] += k;
    at[2] += k > 1 ? k : 0;
    at[3] += k > 1;
    run = e;
  }
  if (t == 1023) {  // behind the last sequence, whosever that is
    total = at[1];
    slots = at[2];
    splits = at[3];
    *s.all = int4{start, run, at[0], 0};
  }
  __syncthreads();
  if (s.longest_first && t < total) {
    const int mine = seg_l[t].count;
    int rank = 0;
    for (int i = 0; i < total; ++i) {
      const int c = seg_l[i].count;
      rank += c > mine || (c == mine && i < t);
    }
    s.segs[rank] = seg_l[t];
    if (seg_l[t].segs > 1) {
      s.by_slot[seg_l[t].slot] = rank;
      if (seg_l[t].flags & 1) s.by_split[seg_l[t].split] = rank;
    }
  }
  for (int i = total + t; i < s.n_segs; i += 1024) s.segs[i].count = -1;
  for (int i = slots + t; i < s.n_slots; i += 1024) s.by_slot[i] = -1;
  for (int i = splits + t; i < s.n_split; i += 1024) s.by_split[i] = -1;
}

// ---- what a segment adds ----------------------------------------------------------
// One workgroup to a (segment, head).  Nothing is read from the state here, so the chunks go
// last to first: what this pass read last, and caches may still hold, is what the next
// one reads first (100 frames: 135 -> 119 us, their 563 MB of k and v at 4.7 TB/s).
template <int D, bool F32>
__global__ __launch_bounds__(4 * D, 4) void k_linear_states(LinArgs a) {
  using C = LinCfg<D, F32>;
  using T = typename Tok<F32>::T;
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * C::TILE];
  __shared__ LinFactors fac[2];
  const int h = blockIdx.x % a.heads;
  const LinSeg sg = lin_slot(a.sq, blockIdx.x / a.heads);
  if (sg.count <= 0 || (sg.flags & 2)) return;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int hk = h / (a.heads / a.heads_k);
  const T* const kp = (const T*)a.k.p + (int64_t)sg.tok * a.k.ld + hk * D;
  const T* const vp = (const T*)a.v.p + (int64_t)sg.tok * a.v.ld + h * D;
  const float* const gp = a.g ? a.g + (int64_t)sg.tok * a.ld_g + h : nullptr;
  const int n = (sg.count + C::CH - 1) / C::CH;
  LinState<D, F32> st;
  st.zero();
  LinFetch<D, F32> fk, fv;
  auto tokens = [&](int j) { return sg.count - j * C::CH < C::CH ? sg.count - j * C::CH : C::CH; };
  auto decay = [&](int j) {
    return gp && lane < tokens(j) ? gp[(int64_t)(j * C::CH + lane) * a.ld_g] : 0.f;
  };
  auto fetch = [&](int j) {
    fk.load(kp + (int64_t)j * C::CH * a.k.ld, (unsigned)a.k.ld, tokens(j));
    fv.load(vp + (int64_t)j * C::CH * a.v.ld, (unsigned)a.v.ld, tokens(j));
  };
  const bool mine = w == C::WAVES - 1;  // the factors are this wave's, a chunk ahead
  float gl = 0.f;
  fetch(n - 1);
  if (mine) {
    lin_reach(fac + ((n - 1) & 1), nullptr, decay(n - 1), tokens(n - 1));
    if (n > 1) gl = decay(n - 2);
  }
  for (int j = n - 1; j >= 0; --j) {
    fk.store(lds);
    fv.store(lds + C::TILE);
    __syncthreads();
    const LinFactors* const f = fac + (j & 1);
    if (j > 0) fetch(j - 1);
    if (mine && j > 0) {
      lin_reach(fac + (~j & 1), f, gl, tokens(j - 1));
      if (j > 1) gl = decay(j - 2);
    }
    lin_tokens<D, F32, false, false>(nullptr, st, nullptr, lds, lds + C::TILE, f->dn, w, lane, g, c);
    __syncthreads();
  }
  st.store(a.part[0] + ((int64_t)(sg.slot + 1) * a.heads + h) * D * D, w, g, c);
  if (mine && lane == 0) a.decay[0][(int64_t)sg.slot * a.heads + h] = lin_exp2_parts(fac[0].sum);
}

// ---- join ------------------------------------------------------------------------
// A wave to 256 elements of a state of a head of a sequence of several segments, a
// thread to four of them, the segments in order: each one's slot takes the state at its start
// (the gradients: the other way, at its end).  Loads of 8 segments are in flight
// (of 16, 256 threads a block: a frame's whole call 31.0 us against 29.4, of 24: 30.2).  The
// decays are taken in two parts: where they are all alike, a rounding to 24 bits would be too, and
// add up over the segments.  Bound by memory: 67 MB of 100 frames 17 us, both ways of 8 frames (125 MB)
// 27 us; a frame's 23 MB 8 us, the latency of three rounds of loads.
__global__ __launch_bounds__(64) void k_linear_join(LinArgs a, int dd, int ways) {
  const int blocks = dd / 256;  // of a state
  unsigned x = blockIdx.x;
  const int el = 4 * ((int)(x % blocks) * 64 + threadIdx.x);
  x /= blocks;
  const int h = x % a.heads;
  x /= a.heads;
  const int rev = x % ways;
  const LinSeg sg = lin_split(a.sq, x / ways);
  if (sg.count < 0) return;
  const int n = sg.segs;
  const float* const init = rev ? a.dstate_out : a.state_in;
  f32x4 m = {0.f, 0.f, 0.f, 0.f};
  if (init) m = *(const f32x4*)(init + ((int64_t)sg.seq * a.heads + h) * dd + el);
  const int64_t first = (int64_t)(rev ? sg.slot + n - 1 : sg.slot) * a.heads + h, step = rev ? -a.heads : a.heads;
  float* const part = a.part[rev] + el;
  const float2* const decay = a.decay[rev];
  *(f32x4*)(part + first * dd) = m;
  constexpr int U = 8;
  for (int i0 = 1; i0 < n; i0 += U) {
    f32x4 add[U];
    float2 f[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t at = first + (i0 + u < n ? i0 + u : n - 1) * step;
      add[u] = *(const f32x4*)(part + at * dd);
      f[u] = decay[at - step];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u >= n) break;
#pragma unroll
      for (int r = 0; r < 4; ++r) m[r] = fmaf(m[r], f[u].x, fmaf(m[r], f[u].y, add[u][r]));
      *(f32x4*)(part + (first + (i0 + u) * step) * dd) = m;
    }
  }
}

// ---- outputs -----------------------------------------------------------------------
// One workgroup to a (segment, head), two to a compute unit: while one waits for its tiles or at
// a barrier the other works.  Per chunk of 64 tokens and d = 128: 960 matrix instructions of 16
// cycles over 4 SIMDs (1.6 us), 5600 vector instructions (most of them the cutting of state and
// w o C into bf16 parts, 2.3 us) and 0.51 MB of LDS reads (1.7 us); 5.2 us a chunk and compute unit
// in all, since the phases between barriers bring the three one after the other.  137,400 tokens
// of 8 heads 346 us, 54,321 of 16 heads 302 us (2.2 TB/s) in a kernel trace, which clocks lower
// than calls alone (480 and 292 us with the passes before); of 342 without loads 262, without
// products 215.  Two parts of the state and of T save 0.3 us of matrix work and 0.3 of vector work (a
// tenth of the kernel) and lose what terms that cancel leave.  Four waves of 32 columns (half of the
// LDS reads, 256 registers) and tiles read ahead into registers gave nothing; stores past the
// caches, which help elsewhere, cost 11%, as q, k and v are all that the caches could keep.
template <int D, bool F32>
__global__ __launch_bounds__(4 * D, F32 ? 2 : D == 64 ? 3 : 4) void k_linear_out(LinArgs a) {
  using C = LinCfg<D, F32>;
  using T = typename Tok<F32>::T;
  __shared__ __attribute__((aligned(16))) uint16_t lds[3 * C::TILE + C::TRI];
  __shared__ LinFactors fac[2];
  __shared__ float next_decays[64];
  const int h = blockIdx.x % a.heads;
  const LinSeg sg = lin_seg(a.sq, blockIdx.x / a.heads);
  if (sg.count < 0) return;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int hk = h / (a.heads / a.heads_k);
  uint16_t* const q = lds;
  uint16_t* const k = q + C::TILE;
  uint16_t* const v = k + C::TILE;
  uint16_t* const tri = v + C::TILE;
  LinState<D, F32> st;
  const int64_t own = ((int64_t)sg.seq * a.heads + h) * D * D;
  if (sg.flags != 3) st.template load<false>(a.part[0] + ((int64_t)sg.slot * a.heads + h) * D * D, w, g, c);
  else if (a.state_in) st.template load<false>(a.state_in + own, w, g, c);
  else st.zero();
  const int n = (sg.count + C::CH - 1) / C::CH;
  if (n > 0) {
    const T* const qp = (const T*)a.q.p + (int64_t)sg.tok * a.q.ld + hk * D;
    const T* const kp = (const T*)a.k.p + (int64_t)sg.tok * a.k.ld + hk * D;
    const T* const vp = (const T*)a.v.p + (int64_t)sg.tok * a.v.ld + h * D;
    T* const op = (T*)a.o + (int64_t)sg.tok * a.ld_o + h * D;
    const float* const gp = a.g ? a.g + (int64_t)sg.tok * a.ld_g + h : nullptr;
    LinFetch<D, F32> fq, fk, fv;
    auto tokens = [&](int j) { return sg.count - j * C::CH < C::CH ? sg.count - j * C::CH : C::CH; };
    auto decay = [&](int j) {
      return gp && lane < tokens(j) ? gp[(int64_t)(j * C::CH + lane) * a.ld_g] : 0.f;
    };
    // bf16: straight into the tiles when all waves are done with a chunk; the other workgroup of
    // the compute unit works meanwhile
    auto fetch = [&](int j) {
      const int64_t t0 = (int64_t)j * C::CH;
      const LinLane l(lane);
      if constexpr (F32) {
        fq.load(qp + t0 * a.q.ld, (unsigned)a.q.ld, tokens(j));
        fk.load(kp + t0 * a.k.ld, (unsigned)a.k.ld, tokens(j));
        fv.load(vp + t0 * a.v.ld, (unsigned)a.v.ld, tokens(j));
      } else {
        lin_load<D>(q, qp + t0 * a.q.ld, (unsigned)a.q.ld, tokens(j), w, l.lane);
        lin_load<D>(k, kp + t0 * a.k.ld, (unsigned)a.k.ld, tokens(j), w, l.lane);
        lin_load<D>(v, vp + t0 * a.v.ld, (unsigned)a.v.ld, tokens(j), w, l.lane);
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
      if (mine) next_decays[lane] = gl;
      if constexpr (F32) {
        fq.store(q);
        fk.store(k);
        fv.store(v);
      } else {
        lin_wait_loads();
      }
      __syncthreads();
      const LinFactors* const f = fac + (j & 1);
      const int flags = f->flags;
      if (mine && j + 1 < n) {
        lin_factors<false>(fac + (~j & 1), f, next_decays[lane], tokens(j + 1), a.scale);
      }
      if (F32 && j + 1 < n) fetch(j + 1);
      if (flags & kLinScale) st.scale(f->pre);
      auto chunk = [&](auto gated) {
        constexpr bool GATED = decltype(gated)::value;
        for (int t = w; t < 2 * C::FRAGS; t += C::WAVES) {
          const LinLane l(lane);
          const int fr = t >> 1;
          const int it = C::CH == 32 || fr < 2 ? fr : 2 + (fr - 2) / 2, ts = C::CH == 32 || fr < 2 ? 0 : (fr - 2) & 1;
          const int jt = 2 * ts + (t & 1);
          const f32x4 x =
              lin_gate<false, GATED>(lin_tri<D, F32>(q, k, it, jt, l.g, l.c), f, a.scale, it, jt, l.g, l.c);
          lin_put(tri, C::FRAGS, fr, jt, l.lane, x);
        }
        LinOut<D, F32> out;
        const LinLane lr(lane);
        out.read(st, q, lr.g, lr.c);
        if (GATED) {
          out.scale(f, c);
          st.scale(f->last);
        }
        __syncthreads();
        const LinLane lt(lane);
        lin_tokens<D, F32, false, true>(&out, st, tri, k, v, f->dn, w, lt.lane, lt.g, lt.c);
        const LinLane lo(lane);
        if (!GATED) out.scale(f, lo.c);
        out.store(op + (int64_t)j * C::CH * a.ld_o, (unsigned)a.ld_o, tokens(j), w, lo.g, lo.c);
      };
      if (flags & kLinGated) chunk(LinBool<true>{});
      else chunk(LinBool<false>{});
      __syncthreads();
      if (!F32 && j + 1 < n) fetch(j + 1);
      gl = mine && j + 2 < n ? decay(j + 2) : 0.f;
    }
    st.scale(fac[(n - 1) & 1].end);
  }
  if ((sg.flags & 2) && a.state_out) st.store(a.state_out + own, w, g, c);
}

template <int D>
hipError_t states_any(const LinArgs& a, bool f32, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.sq.n_slots * a.heads)), blk(4 * D);
  if (f32) hipLaunchKernelGGL((k_linear_states<D, true>), grid, blk, 0, st, a);
  else hipLaunchKernelGGL((k_linear_states<D, false>), grid, blk, 0, st, a);
  return hipGetLastError();
}

template <int D>
hipError_t out_any(const LinArgs& a, bool f32, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.sq.n_segs * a.heads)), blk(4 * D);
  if (f32) hipLaunchKernelGGL((k_linear_out<D, true>), grid, blk, 0, st, a);
  else hipLaunchKernelGGL((k_linear_out<D, false>), grid, blk, 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_table(const LinSeqs& s, hipStream_t st) {
  hipLaunchKernelGGL(k_linear_table, dim3(1), dim3(1024), 0, st, s);
  return hipGetLastError();
}

hipError_t launch_linear_states(const LinArgs& a, int d, bool f32, hipStream_t st) {
  return d == 128 ? states_any<128>(a, f32, st) : states_any<64>(a, f32, st);
}

hipError_t launch_linear_join(const LinArgs& a, int d, bool both, hipStream_t st) {
  const int ways = both ? 2 : 1;
  const int64_t blocks = (int64_t)a.sq.n_split * ways * a.heads * (d * d / 256);
  hipLaunchKernelGGL(k_linear_join, dim3((unsigned)blocks), dim3(64), 0, st, a, d * d, ways);
  return hipGetLastError();
}

hipError_t launch_linear_out(const LinArgs& a, int d, bool f32, hipStream_t st) {
  return d == 128 ? out_any<128>(a, f32, st) : out_any<64>(a, f32, st);
}

}  // namespace zm
