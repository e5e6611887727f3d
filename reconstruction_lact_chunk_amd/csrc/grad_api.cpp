// C-ABI layer of the gradients' norm and clipping: argument checks (host only, before any HIP
// call), the tables of tensors and the launches.
#include "zm_ttt.h"

#include <math.h>

#include <algorithm>
#include <memory>
#include <new>

#include "api_util.h"
#include "grad_clip.h"

using namespace zm;

namespace {

constexpr int kMaxTensors = 8192;
constexpr int64_t kMaxElements = (int64_t)1 << 36;  // of one tensor
static_assert(kClipTensors * clip_pieces(kMaxElements, true) + kClipBlocks < (int64_t)1 << 32,
              "pieces of a table and the kernels' steps over them are counted in 32 bits without a sign");

struct Span {
  uintptr_t at, end;
  bool operator<(const Span& o) const { return at < o.at; }
};

// No two of the arrays that are written may share memory: an element would be scaled twice, or
// by two workgroups at once.
bool overlapping(Span* s, int count) {
  bool sorted = true;
  for (int i = 1; i < count && sorted; ++i) sorted = s[i - 1].at <= s[i].at;
  if (!sorted) std::sort(s, s + count);
  for (int i = 1; i < count; ++i)
    if (s[i].at < s[i - 1].end) return true;
  return false;
}

int check_tensors(const zm_tensor* t, int32_t count, bool write) {
  if (count < 0 || (count > 0 && !t)) return ZM_ERR_INVALID_ARG;
  if (count > kMaxTensors) return ZM_ERR_UNSUPPORTED;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].n < 0 || t[i].n > kMaxElements || t[i].reserved != 0) return ZM_ERR_INVALID_ARG;
    if (t[i].dtype != ZM_BF16 && t[i].dtype != ZM_F32) return ZM_ERR_INVALID_ARG;
    if (t[i].n == 0) continue;
    const size_t size = t[i].dtype == ZM_F32 ? 4 : 2;
    if (!t[i].x || !aligned(t[i].x, size)) return ZM_ERR_INVALID_ARG;
    if (write && (!t[i].y || !aligned(t[i].y, size))) return ZM_ERR_INVALID_ARG;
  }
  return ZM_OK;
}

// What is written must not overlap another tensor, read or written, but its own input exactly.
// Up to kFewSpans lie on the stack (16 KB), more on the heap: the caller's stack may be small.
constexpr int kFewSpans = 1024;
int check_written(const zm_tensor* t, int32_t count, const float* norm, const void* ws, size_t bytes) {
  Span few[kFewSpans];
  std::unique_ptr<Span[]> many;
  Span* s = few;
  if (2 * (int64_t)count + 2 > kFewSpans) {
    many.reset(new (std::nothrow) Span[2 * (size_t)count + 2]);
    if (!many) {
      set_last_error("no host memory for the spans of %d tensors", (int)count);
      return ZM_ERR_HIP;
    }
    s = many.get();
  }
  int m = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].n == 0) continue;
    const size_t size = (size_t)t[i].n * (t[i].dtype == ZM_F32 ? 4 : 2);
    s[m++] = Span{(uintptr_t)t[i].y, (uintptr_t)t[i].y + size};
    if (t[i].x != t[i].y) s[m++] = Span{(uintptr_t)t[i].x, (uintptr_t)t[i].x + size};
  }
  s[m++] = Span{(uintptr_t)norm, (uintptr_t)norm + 4};
  s[m++] = Span{(uintptr_t)ws, (uintptr_t)ws + bytes};
  return overlapping(s, m) ? ZM_ERR_INVALID_ARG : ZM_OK;
}

// The partial sums must not be written into a tensor that is still read.
int check_read(const zm_tensor* t, int32_t count, const void* ws, size_t bytes) {
  const uintptr_t at = (uintptr_t)ws;
  for (int32_t i = 0; i < count; ++i) {
    const uintptr_t x = (uintptr_t)t[i].x;
    const size_t size = (size_t)t[i].n * (t[i].dtype == ZM_F32 ? 4 : 2);
    if (t[i].n > 0 && x < at + bytes && at < x + size) return ZM_ERR_INVALID_ARG;
  }
  return ZM_OK;
}

// Tables of up to kClipTensors tensors (empty ones left out), one after the other.
struct Tables {
  const zm_tensor* t;
  int32_t count;
  // the table that starts at tensor `from`; returns where the next one does
  int32_t fill(ClipTable& out, int32_t from) const {
    int m = 0;
    int64_t pieces = 0;
    for (uint32_t& w : out.f32) w = 0;
    for (; from < count && m < kClipTensors; ++from) {
      if (t[from].n == 0) continue;
      const bool f32 = t[from].dtype == ZM_F32;
      out.x[m] = t[from].x;
      out.y[m] = t[from].y;
      out.n[m] = t[from].n;
      out.first[m] = (uint32_t)pieces;
      if (f32) out.f32[m >> 5] |= 1u << (m & 31);
      pieces += clip_pieces(t[from].n, f32);
      ++m;
    }
    out.first[m] = (uint32_t)pieces;
    out.count = m;
    return from;
  }
};

size_t clip_bytes(int32_t count) {
  const size_t tables = (size_t)count / kClipTensors + 1;
  return round_up(tables * kClipBlocks * sizeof(double), 256);
}

int check_workspace(const void* ws, size_t have, size_t need) {
  if (!ws) return ZM_ERR_WORKSPACE;
  if (!aligned(ws, 256)) return ZM_ERR_INVALID_ARG;
  return have < need ? ZM_ERR_WORKSPACE : ZM_OK;
}

// The squares of all tables; returns the partial sums in `slots`.
hipError_t squares(const Tables& all, double* part, int& slots, hipStream_t st) {
  slots = 0;
  ClipTable t;
  for (int32_t from = 0; from < all.count;) {
    from = all.fill(t, from);
    const hipError_t e = launch_grad_squares(t, part + slots, st);
    if (e != hipSuccess) return e;
    slots += clip_blocks(t.first[t.count]);
  }
  return hipSuccess;
}

}  // namespace

extern "C" {

int zm_grad_norm_workspace_size(int32_t count, size_t* bytes) {
  if (!bytes || count < 0) return ZM_ERR_INVALID_ARG;
  if (count > kMaxTensors) return ZM_ERR_UNSUPPORTED;
  *bytes = clip_bytes(count);
  return ZM_OK;
}

int zm_grad_norm(const zm_tensor* tensors, int32_t count, float* norm, void* workspace, size_t workspace_bytes,
                 void* stream) {
  ZM_TRY(check_tensors(tensors, count, false));
  if (!norm || !aligned(norm, 4)) return ZM_ERR_INVALID_ARG;
  ZM_TRY(check_workspace(workspace, workspace_bytes, clip_bytes(count)));
  ZM_TRY(check_read(tensors, count, workspace, clip_bytes(count)));
  const hipStream_t st = (hipStream_t)stream;
  int slots;
  ZM_HIP(squares(Tables{tensors, count}, (double*)workspace, slots, st));
  ZM_HIP(launch_grad_norm((const double*)workspace, slots, norm, st));
  return ZM_OK;
}

int zm_clip_grads(const zm_tensor* tensors, int32_t count, float max_norm, float* norm, void* workspace,
                  size_t workspace_bytes, void* stream) {
  ZM_TRY(check_tensors(tensors, count, true));
  if (!(max_norm >= 0.f) || isinf(max_norm) || !norm || !aligned(norm, 4)) return ZM_ERR_INVALID_ARG;
  ZM_TRY(check_workspace(workspace, workspace_bytes, clip_bytes(count)));
  ZM_TRY(check_written(tensors, count, norm, workspace, clip_bytes(count)));
  const hipStream_t st = (hipStream_t)stream;
  const Tables all{tensors, count};
  double* const part = (double*)workspace;
  int slots;
  ZM_HIP(squares(all, part, slots, st));
  // the last table first, as its tensors are the last that were read
  int32_t starts[kMaxTensors / kClipTensors + 2], m = 0;
  ClipTable t;
  for (int32_t from = 0; from < count;) {
    starts[m++] = from;
    from = all.fill(t, from);
  }
  if (m == 0) {
    t.count = 0;
    t.first[0] = 0;
    ZM_HIP(launch_grad_scale(t, part, slots, max_norm, norm, st));
  }
  for (int i = m - 1; i >= 0; --i) {
    all.fill(t, starts[i]);
    ZM_HIP(launch_grad_scale(t, part, slots, max_norm, i == m - 1 ? norm : nullptr, st));
  }
  return ZM_OK;
}

}  // extern "C"
