// Rotary positions with several axes: pair p of a head, owned by axis a, turns
// by the angle pos[t][a] freqs[p]:
//   (x, y) -> (x cos - y sin, x sin + y cos),
// or by minus that angle (inverse), which is the rotation's transpose and so
// its gradient.  The dims of a pair, P pairs in all, axis a's pairs first[a]..:
//   layout 0  p, p + P
//   layout 1  2 p, 2 p + 1
//   layout 2  halves of the axis's own block of 2 s_a dims
// Dims from 2 P on pass unrotated.
// Bound by memory: q and k are read and written once, and a thread forms the
// angles of its V pairs once for all the heads it turns.  54960 fp32 tokens of 20 heads of
// 64 (563 MB): 132 us, 4.3 TB/s; 137400 bf16 tokens of 16 heads of 128 (1.13 GB) 220 us, 5.1 TB/s, and
// with sections of 5, 7 and 11 pairs, which take runs of one pair, 339; a frame of 1374 of them
// 7.9 us, loads and then angles of a few waves to a SIMD.
#include "rotary_dev.h"

namespace zm {

namespace {

constexpr int64_t kMaxRotaryBlocks = 1 << 20;  // more tokens than these take are looped over

struct RotaryPlan {
  int groups;       // V-pair groups of a token, at most 256: rotated ones, then the unrotated tail
  int turned;       // rotated ones among them
  int heads_each;   // heads of one thread
  int tokens;       // tokens of a block
};

// Thread i of a block: group i % groups of token i / groups of the block's
// `tokens`; blockIdx.y is the head split.
template <typename T, int V, bool ADJ>
__device__ __forceinline__ void turn_group(const RotaryArgs& a, const RotaryPlan& pl, int64_t t,
                                           int grp) {
  const bool turn = grp < pl.turned;
  const int p0 = grp * V;
  int c0, c1;  // first dims of the two runs of V elements
  rotary_runs<V, ADJ>(a, pl.turned, grp, c0, c1);
  const int all = a.q.heads + a.k.heads;
  const int h0 = blockIdx.y * pl.heads_each;
  const int h1 = h0 + pl.heads_each < all ? h0 + pl.heads_each : all;
  auto src = [&](int h) {
    return h < a.q.heads ? (const T*)a.q.x + t * a.q.ldx + (int64_t)h * a.d
                         : (const T*)a.k.x + t * a.k.ldx + (int64_t)(h - a.q.heads) * a.d;
  };
  // the first head's elements are on their way while the angles are formed
  Vec<T, V> nu = load_v<T, V>(src(h0) + c0), nv = load_v<T, V>(src(h0) + c1);
  float co[V], si[V];
  if (turn) {
    rotary_angles<V>(a, t, p0, co, si);
  }
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    const bool isq = h < a.q.heads;
    T* y = isq ? (T*)a.q.y + t * a.q.ldy + (int64_t)h * a.d
               : (T*)a.k.y + t * a.k.ldy + (int64_t)(h - a.q.heads) * a.d;
    Vec<T, V> u = nu, v = nv;
    if (h + 1 < h1) {
      nu = load_v<T, V>(src(h + 1) + c0);
      nv = load_v<T, V>(src(h + 1) + c1);
    }
    if (turn) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if constexpr (ADJ && V > 1) {
          // u then v hold pairs side by side
          Vec<T, V>& w = j < V / 2 ? u : v;
          const int e = 2 * (j < V / 2 ? j : j - V / 2);
          const float b = to_f(w.e[e]), c = to_f(w.e[e + 1]);
          w.e[e] = from_f<T>(b * co[j] - c * si[j]);
          w.e[e + 1] = from_f<T>(b * si[j] + c * co[j]);
        } else {
          const float b = to_f(u.e[j]), c = to_f(v.e[j]);
          u.e[j] = from_f<T>(b * co[j] - c * si[j]);
          v.e[j] = from_f<T>(b * si[j] + c * co[j]);
        }
      }
    }
    store_v<T, V>(y + c0, u);
    store_v<T, V>(y + c1, v);
  }
}

template <typename T, int V, bool ADJ>
__global__ __launch_bounds__(256) void k_rotary(RotaryArgs a, RotaryPlan pl) {
  const int tl = threadIdx.x / pl.groups, grp = threadIdx.x - tl * pl.groups;
  if (tl >= pl.tokens) return;
  for (int64_t t = (int64_t)blockIdx.x * pl.tokens + tl; t < a.n;
       t += (int64_t)gridDim.x * pl.tokens)
    turn_group<T, V, ADJ>(a, pl, t, grp);
}

template <typename T, int V, bool ADJ>
hipError_t rotary_launch(const RotaryArgs& a, hipStream_t st) {
  RotaryPlan pl;
  const int all = a.q.heads + a.k.heads;
  pl.turned = a.pairs / V;
  // the unrotated tail is copied only where the result goes elsewhere
  const bool tail = a.q.x != a.q.y || (a.k.heads && a.k.x != a.k.y);
  pl.groups = pl.turned + (tail ? (a.d - 2 * a.pairs) / (2 * V) : 0);
  // Threads for eight waves on each SIMD, as far as the heads can be split:
  // a thread with many heads forms its angles once, one with few starts sooner.
  const int64_t want = (int64_t)kTargetWgs * 4 * 8 * 64;
  int64_t splits = ceil_div(want, a.n * pl.groups);
  if (splits > all) splits = all;
  pl.heads_each = (int)ceil_div(all, splits);
  pl.tokens = 256 / pl.groups;
  int64_t blocks = ceil_div(a.n, pl.tokens);
  if (blocks > kMaxRotaryBlocks) blocks = kMaxRotaryBlocks;
  hipLaunchKernelGGL((k_rotary<T, V, ADJ>),
                     dim3((unsigned)blocks, (unsigned)ceil_div(all, pl.heads_each)), dim3(256), 0,
                     st, a, pl);
  return hipGetLastError();
}

template <typename T>
hipError_t rotary_any(const RotaryArgs& a, hipStream_t st) {
  const bool adj = a.layout == 1;
  if (rotary_fits(a, 8)) return adj ? rotary_launch<T, 8, true>(a, st) : rotary_launch<T, 8, false>(a, st);
  if (rotary_fits(a, 4)) return adj ? rotary_launch<T, 4, true>(a, st) : rotary_launch<T, 4, false>(a, st);
  return adj ? rotary_launch<T, 1, true>(a, st) : rotary_launch<T, 1, false>(a, st);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, hipStream_t st) {
  if (a.n == 0) return hipSuccess;
  return a.f32 ? rotary_any<float>(a, st) : rotary_any<uint16_t>(a, st);
}

}  // namespace zm
