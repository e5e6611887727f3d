// The global norm N = sqrt(sum over all tensors of x^2) and the clipping
// y = x min(1, max / (N + 1e-6)).
// Bound by memory: every element is read for the norm and again for the scaling, and
// written once.  Squares are added in 64 bits (a square of an fp32 element and all sums of them are in
// range, and a conversion and a multiply-add an element hide behind the loads); the partial sums
// go to the workgroups' slots and every workgroup of the scaling adds all of them in the
// same order, so there is no third launch, no atomic, and the same bits every time.
// 277 MB of 24 layers' gradients (two launches of each kernel): 49 us for the squares, 100 for the
// scaling, which finds part of its input in the caches: 832 MB of reads and writes at 5.6 TB/s.  Next
// piece's loads ahead of this one's sums: 2% slower; pieces of 32 or 8 KB 153 and 164 us against 149 of
// 16 KB, of 2048 workgroups 161.  6 MB: 4 + 5 us.
#include "grad_clip.h"

namespace zm {

namespace {

constexpr int kThreads = 256;
constexpr int kWords = kClipPieceBytes / 16;     // 16-byte words of a piece
constexpr int kEach = kWords / kThreads;         // of a thread

// Piece p of the table: tensor i and the piece's number in it.
__device__ __forceinline__ int find_piece(const ClipTable& t, unsigned p, int& in) {
  int lo = 0, hi = t.count;  // the last tensor whose first piece is at most p (empty ones share theirs)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= p) lo = mid;
    else hi = mid;
  }
  in = (int)(p - t.first[lo]);
  return lo;
}

__device__ __forceinline__ float get(const uint16_t* p) { return __uint_as_float((unsigned)*p << 16); }
__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ void put(uint16_t* p, float x) { *p = to_bf16(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }

template <typename T>
__device__ __forceinline__ void unpack(const u32x4& w, float* v) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16lo(w[i]);
      v[2 * i + 1] = bf16hi(w[i]);
    }
  }
}
template <typename T>
__device__ __forceinline__ u32x4 pack(const float* v) {
  u32x4 w;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  }
  return w;
}

// Sum over the workgroup, the same bits in every thread.
__device__ __forceinline__ double block_sum(double s, double* red) {
#pragma unroll
  for (int m = 1; m < 64; m *= 2) s += __shfl_xor(s, m, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  return red[0] + red[1] + red[2] + red[3];
}

// Elements of a piece: words of 16 bytes from the one that holds the first element; word w holds
// the elements first + E w ..  of the tensor, of which those before 0 and from n on are not there.
template <typename T>
struct Piece {
  static constexpr int E = 16 / sizeof(T);
  const T* x;
  int64_t first, n;
  __device__ __forceinline__ Piece(const void* p, int64_t count, int piece) {
    const int skip = (int)(((uintptr_t)p & 15) / sizeof(T));
    x = (const T*)p;
    n = count;
    first = (int64_t)piece * kWords * E - skip;
  }
  __device__ __forceinline__ int64_t at(int w) const { return first + (int64_t)w * E; }
  __device__ __forceinline__ bool whole(int64_t e) const { return e >= 0 && e + E <= n; }
};

template <typename T>
__device__ __forceinline__ double piece_squares(const void* p, int64_t n, int piece) {
  const Piece<T> pc(p, n, piece);
  constexpr int E = Piece<T>::E;
  u32x4 raw[kEach];
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int64_t e = pc.at(threadIdx.x + kThreads * i);
    raw[i] = u32x4{0u, 0u, 0u, 0u};
    if (pc.whole(e)) raw[i] = *(const u32x4*)(pc.x + e);
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    float v[E];
    unpack<T>(raw[i], v);
#pragma unroll
    for (int j = 0; j < E; ++j) s = fma((double)v[j], (double)v[j], s);
    const int64_t e = pc.at(threadIdx.x + kThreads * i);
    if (!pc.whole(e) && e < n && e + E > 0) {  // a word at an end
      for (int j = 0; j < E; ++j)
        if (e + j >= 0 && e + j < n) {
          const double x = get(pc.x + e + j);
          s = fma(x, x, s);
        }
    }
  }
  return s;
}

__global__ __launch_bounds__(kThreads) void k_grad_squares(ClipTable t, double* part) {
  __shared__ double red[4];
  double s = 0.0;
  const unsigned pieces = t.first[t.count];
  for (unsigned p = blockIdx.x; p < pieces; p += gridDim.x) {
    int in;
    const int i = find_piece(t, p, in);
    if (t.f32[i >> 5] >> (i & 31) & 1) s += piece_squares<float>(t.x[i], t.n[i], in);
    else s += piece_squares<uint16_t>(t.x[i], t.n[i], in);
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The partial sums in a fixed order.
__device__ __forceinline__ double all_squares(const double* part, int count, double* red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < count; i += kThreads) s += part[i];
  return block_sum(s, red);
}

__global__ __launch_bounds__(kThreads) void k_grad_norm(const double* part, int count, float* norm) {
  __shared__ double red[4];
  const double s = all_squares(part, count, red);
  if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

template <typename T>
__device__ __forceinline__ void piece_scale(const void* p, void* q, int64_t n, int piece, double c) {
  const Piece<T> pc(p, n, piece);
  constexpr int E = Piece<T>::E;
  T* const y = (T*)q;
  // whole words where the output lies as its input does to 16 bytes
  const bool alike = (((uintptr_t)p ^ (uintptr_t)q) & 15) == 0;
  u32x4 raw[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int64_t e = pc.at(threadIdx.x + kThreads * i);
    if (alike && pc.whole(e)) raw[i] = *(const u32x4*)(pc.x + e);
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int64_t e = pc.at(threadIdx.x + kThreads * i);
    if (alike && pc.whole(e)) {
      float v[E];
      unpack<T>(raw[i], v);
#pragma unroll
      for (int j = 0; j < E; ++j) v[j] = (float)((double)v[j] * c);
      // past the caches, which then keep the elements still to be read: 24 layers' 277 MB 173 -> 148 us
      __builtin_nontemporal_store(pack<T>(v), (u32x4*)(y + e));
    } else if (alike && e < n && e + E > 0) {  // a word at an end
      for (int j = 0; j < E; ++j)
        if (e + j >= 0 && e + j < n) put(y + e + j, (float)((double)get(pc.x + e + j) * c));
    }
  }
  if (!alike) {
    const int64_t end = pc.first + (int64_t)kWords * E < n ? pc.first + (int64_t)kWords * E : n;
    for (int64_t e = (pc.first > 0 ? pc.first : 0) + threadIdx.x; e < end; e += kThreads)
      put(y + e, (float)((double)get(pc.x + e) * c));
  }
}

__global__ __launch_bounds__(kThreads) void k_grad_scale(ClipTable t, const double* part, int count, float max_norm,
                                                         float* norm) {
  __shared__ double red[4];
  const double s = sqrt(all_squares(part, count, red));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)s;
  const double ratio = (double)max_norm / (s + 1e-6), c = ratio < 1.0 || ratio != ratio ? ratio : 1.0;
  const unsigned pieces = t.first[t.count];
  // the last pieces first: they are what the caches still hold of the norm's pass
  for (unsigned behind = blockIdx.x; behind < pieces; behind += gridDim.x) {
    int in;
    const int i = find_piece(t, pieces - 1 - behind, in);
    if (c == 1.0 && t.x[i] == t.y[i]) continue;  // the same values
    if (t.f32[i >> 5] >> (i & 31) & 1) piece_scale<float>(t.x[i], t.y[i], t.n[i], in, c);
    else piece_scale<uint16_t>(t.x[i], t.y[i], t.n[i], in, c);
  }
}

}  // namespace

hipError_t launch_grad_squares(const ClipTable& t, double* part, hipStream_t st) {
  const int blocks = clip_blocks(t.first[t.count]);
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL(k_grad_squares, dim3(blocks), dim3(kThreads), 0, st, t, part);
  return hipGetLastError();
}

hipError_t launch_grad_norm(const double* part, int count, float* norm, hipStream_t st) {
  hipLaunchKernelGGL(k_grad_norm, dim3(1), dim3(kThreads), 0, st, part, count, norm);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const ClipTable& t, const double* part, int count, float max_norm, float* norm,
                             hipStream_t st) {
  const int blocks = clip_blocks(t.first[t.count]);
  if (blocks == 0 && !norm) return hipSuccess;
  hipLaunchKernelGGL(k_grad_scale, dim3(blocks > 0 ? blocks : 1), dim3(kThreads), 0, st, t, part, count, max_norm, norm);
  return hipGetLastError();
}

}  // namespace zm
