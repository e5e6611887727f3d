// What the kernels with rotary positions share (rotary.hip, norm_rotary.hip): vectors of
// elements, the dims of a group of pairs and the angles.
#pragma once

#include "seq_ops.h"

namespace zm {

template <typename T, int V>
struct Vec {
  T e[V];
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<uint16_t>(uint16_t x) { return __uint_as_float((unsigned)x << 16); }
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ uint16_t from_f<uint16_t>(float x) { return to_bf16(x); }
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }

// V elements at p, as wide as their alignment (V elements, 16 bytes at most).
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> load_v(const T* p) {
  Vec<T, V> r;
  constexpr int B = V * (int)sizeof(T);
  if constexpr (B % 16 == 0) {
#pragma unroll
    for (int i = 0; i < B / 16; ++i) ((u32x4*)&r)[i] = ((const u32x4*)p)[i];
  } else if constexpr (B == 8) {
    *(u32x2*)&r = *(const u32x2*)p;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) r.e[i] = p[i];
  }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const Vec<T, V>& r) {
  constexpr int B = V * (int)sizeof(T);
  if constexpr (B % 16 == 0) {
#pragma unroll
    for (int i = 0; i < B / 16; ++i) ((u32x4*)p)[i] = ((const u32x4*)&r)[i];
  } else if constexpr (B == 8) {
    *(u32x2*)p = *(const u32x2*)&r;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = r.e[i];
  }
}

// First dims c0, c1 of the two runs of V elements of group grp: a rotated one of V pairs, or
// of the unrotated tail.
template <int V, bool ADJ>
__device__ __forceinline__ void rotary_runs(const RotaryArgs& a, int turned, int grp, int& c0, int& c1) {
  const int p0 = grp * V;
  int ax = 0;  // of the first pair; a run of V > 1 pairs has one axis in layout 2 only
  if (grp < turned) {
    while (ax + 1 < a.axes && p0 >= a.first[ax + 1]) ++ax;
    if (ADJ) {
      c0 = 2 * p0;
      c1 = c0 + V;
    } else if (a.layout == 0) {
      c0 = p0;
      c1 = p0 + a.pairs;
    } else {
      c0 = p0 + a.first[ax];
      c1 = p0 + a.first[ax + 1];
    }
  } else {
    c0 = 2 * a.pairs + (grp - turned) * 2 * V;
    c1 = c0 + V;
  }
}

// Cosine and sine of the angles of pairs p0 .. p0 + V - 1 at token t, with the sign of the
// direction.  An angle is a 64-bit product taken in revolutions, whose nearest integer goes
// off before the rounding to 32 bits, and what that rounding leaves is put back: cosine and
// sine are those of the 64-bit angle.
template <int V>
__device__ __forceinline__ void rotary_angles(const RotaryArgs& a, int64_t t, int p0, float* co, float* si) {
  // all loads first: an axis picked pair by pair would wait for each on its own
  int raw[4];
  float fq[V];
#pragma unroll
  for (int i = 0; i < 4; ++i) raw[i] = ((const int*)a.pos)[t * a.axes + (i < a.axes ? i : 0)];
#pragma unroll
  for (int j = 0; j < V; ++j) fq[j] = a.freqs[p0 + j];
  double pos[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) pos[i] = a.pos_f32 ? (double)__int_as_float(raw[i]) : (double)raw[i];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    double p = pos[0];
#pragma unroll
    for (int i = 1; i < 4; ++i)
      if (i < a.axes && p0 + j >= a.first[i]) p = pos[i];
    const double rev = p * (double)fq[j] * 0.15915494309189533577;  // 1 / (2 pi)
    const double turn = rev - rint(rev);
    const float f = (float)turn;
    // what the rounding of up to half a turn leaves, 9e-8 of an angle at most, to first order
    const float rest = (float)(turn - (double)f) * 6.2831853f;
    float s, c;
    sincospif(2.f * f, &s, &c);
    si[j] = fmaf(rest, c, s);
    co[j] = fmaf(-rest, s, c);
    if (a.inverse) si[j] = -si[j];
  }
}

// Runs of V pairs fit: whole runs in the rotated and the unrotated part, and in
// layout 2 in every axis's block.
inline bool rotary_fits(const RotaryArgs& a, int v) {
  if (a.pairs % v || (a.d - 2 * a.pairs) % (2 * v)) return false;
  if (a.layout == 2)
    for (int i = 0; i < a.axes; ++i)
      if ((a.first[i + 1] - a.first[i]) % v) return false;
  return true;
}

// Applies the angles to a group's elements u (at c0) and v (at c1), in fp32.
template <int V, bool ADJ>
__device__ __forceinline__ void rotary_turn(float* u, float* v, const float* co, const float* si) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if constexpr (ADJ && V > 1) {
      // u then v hold pairs side by side
      float* const w = j < V / 2 ? u : v;
      const int e = 2 * (j < V / 2 ? j : j - V / 2);
      const float b = w[e], c = w[e + 1];
      w[e] = b * co[j] - c * si[j];
      w[e + 1] = b * si[j] + c * co[j];
    } else {
      const float b = u[j], c = v[j];
      u[j] = b * co[j] - c * si[j];
      v[j] = b * si[j] + c * co[j];
    }
  }
}

}  // namespace zm
