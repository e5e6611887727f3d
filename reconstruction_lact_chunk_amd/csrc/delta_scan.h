// Operand fetches of the kernels that go through the chunks of the gated delta
// rule in order (delta_scan.hip, delta_grad.hip).
#pragma once

#include "delta_rule.h"

namespace zm {

template <int D, bool F32>
struct ScanCfg {
  static constexpr int NT = Tok<F32>::NT;
  static constexpr int PITCH = D + 16;
  static constexpr int TILE = kChunk * PITCH;   // one part of K or Q
};

// fp32 K (or Q) of the chunk into its LDS parts; rows past `count` are zero.
template <int D>
__device__ __forceinline__ void stage(uint16_t* lds, const float* src, int64_t ld, int count) {
  using C = ScanCfg<D, true>;
  constexpr int CPR = D / 8;
  for (int i = threadIdx.x; i < kChunk * CPR; i += 2 * D) {
    const int row = i / CPR, col = 8 * (i % CPR);
    Parts<C::NT> p = zero_parts<C::NT>();
    if (row < count) p = load8(src + (int64_t)row * ld + col);
#pragma unroll
    for (int k = 0; k < C::NT; ++k) *(bf16x8*)(lds + k * C::TILE + row * C::PITCH + col) = p.p[k];
  }
}

template <int D, bool F32>
__device__ __forceinline__ Parts<Tok<F32>::NT> lds_row(const uint16_t* lds, int row, int col) {
  using C = ScanCfg<D, F32>;
  Parts<C::NT> p;
#pragma unroll
  for (int k = 0; k < C::NT; ++k) p.p[k] = *(const bf16x8*)(lds + k * C::TILE + row * C::PITCH + col);
  return p;
}

// Rows dim_row(mt, .) of the transpose, slots = tokens of step ts.
template <int D, bool F32>
__device__ __forceinline__ Parts<Tok<F32>::NT> lds_col(const uint16_t* lds, int mt, int ts, int g,
                                                       int c) {
  using C = ScanCfg<D, F32>;
  Parts<C::NT> p;
  const int row = 32 * ts + dtau(g, c >> 2), col = 32 * (mt >> 1) + 8 * (c & 3) + 4 * (mt & 1);
#pragma unroll
  for (int k = 0; k < C::NT; ++k) {
    const uint16_t* at = lds + k * C::TILE + row * C::PITCH + col;
    p.p[k] = __builtin_shufflevector(delta_read_tr(at), delta_read_tr(at + 8 * C::PITCH), 0, 1, 2, 3,
                                     4, 5, 6, 7);
  }
  return p;
}

template <int NP>
__device__ __forceinline__ Parts<NP> frag(const uint16_t* f, int i, int lane) {
  Parts<NP> p;
#pragma unroll
  for (int k = 0; k < NP; ++k)
    p.p[k] = *(const bf16x8*)(f + (k * kTriFrags + i) * kFragElems + lane * 8);
  return p;
}

}  // namespace zm
