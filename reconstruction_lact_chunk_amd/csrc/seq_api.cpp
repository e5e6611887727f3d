// C-ABI layer of the operators around a streamed token sequence: layer norm and
// rotary positions.  Arguments are checked on the host before any HIP call, as
// specified in include/zm_ttt.h.
#include "zm_ttt.h"

#include <math.h>

#include "api_util.h"
#include "seq_ops.h"

using namespace zm;

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 31;
constexpr int kMaxRotaryHeads = 64, kMaxRotaryHead = 256;

bool is_dtype(int32_t t) { return t == ZM_BF16 || t == ZM_F32; }

// Rows of token data: base alignment and stride.
int check_rows(const void* p, int64_t ld, int64_t width) {
  if (!p || !aligned(p, 16) || ld < width || ld % 8 != 0) return ZM_ERR_INVALID_ARG;
  return ZM_OK;
}

int check_norm(const zm_norm_desc* d, int64_t n) {
  if (!d || d->width < 1 || d->width % 8 != 0 || !is_dtype(d->io_dtype) || d->reserved != 0)
    return ZM_ERR_INVALID_ARG;
  if (!(d->eps > 0.f) || isinf(d->eps)) return ZM_ERR_INVALID_ARG;
  if (n < 0 || n > kMaxTokens) return ZM_ERR_INVALID_ARG;
  if (d->width > kMaxNormWidth) return ZM_ERR_UNSUPPORTED;
  return ZM_OK;
}

size_t norm_bytes(const zm_norm_desc* d, int64_t n) {
  return round_up((size_t)norm_slots(n) * 2 * d->width * sizeof(float), 256);
}

}  // namespace

extern "C" {

int zm_layer_norm(const zm_norm_desc* desc, int64_t n, const void* x, int64_t ld_x,
                  const float* gamma, const float* beta, void* y, int64_t ld_y, float* stats,
                  void* stream) {
  ZM_TRY(check_norm(desc, n));
  if (!aligned(gamma, 16) || !aligned(beta, 16) || !aligned(stats, 4)) return ZM_ERR_INVALID_ARG;
  if (n == 0) return ZM_OK;
  ZM_TRY(check_rows(x, ld_x, desc->width));
  ZM_TRY(check_rows(y, ld_y, desc->width));
  if (x == y && ld_x != ld_y) return ZM_ERR_INVALID_ARG;
  ZM_HIP(launch_layer_norm(x, ld_x, gamma, beta, desc->eps, y, ld_y, stats, desc->width, n,
                           desc->io_dtype == ZM_F32, (hipStream_t)stream));
  return ZM_OK;
}

int zm_layer_norm_backward_workspace_size(const zm_norm_desc* desc, int64_t n, size_t* bytes) {
  if (!bytes) return ZM_ERR_INVALID_ARG;
  ZM_TRY(check_norm(desc, n));
  *bytes = norm_bytes(desc, n);
  return ZM_OK;
}

int zm_layer_norm_backward(const zm_norm_desc* desc, int64_t n, const void* dy, int64_t ld_dy,
                           const void* x, int64_t ld_x, const float* gamma, const float* stats,
                           void* dx, int64_t ld_dx, float* dgamma, float* dbeta, void* workspace,
                           size_t workspace_bytes, void* stream) {
  ZM_TRY(check_norm(desc, n));
  if (!aligned(gamma, 16) || !aligned(dgamma, 4) || !aligned(dbeta, 4)) return ZM_ERR_INVALID_ARG;
  if (dgamma && dgamma == dbeta) return ZM_ERR_INVALID_ARG;  // one would be lost
  if (n > 0) {
    ZM_TRY(check_rows(dy, ld_dy, desc->width));
    ZM_TRY(check_rows(x, ld_x, desc->width));
    ZM_TRY(check_rows(dx, ld_dx, desc->width));
    if (!stats || !aligned(stats, 4)) return ZM_ERR_INVALID_ARG;
    if ((dx == dy && ld_dx != ld_dy) || (dx == x && ld_dx != ld_x)) return ZM_ERR_INVALID_ARG;
    if (dgamma || dbeta) {
      if (!workspace) return ZM_ERR_WORKSPACE;
      if (!aligned(workspace, 256)) return ZM_ERR_INVALID_ARG;
      if (workspace_bytes < norm_bytes(desc, n)) return ZM_ERR_WORKSPACE;
    }
  }
  ZM_HIP(launch_layer_norm_backward(dy, ld_dy, x, ld_x, gamma, stats, dx, ld_dx, dgamma, dbeta,
                                    (float*)workspace, desc->width, n, desc->io_dtype == ZM_F32,
                                    (hipStream_t)stream));
  return ZM_OK;
}

int zm_rotary(const zm_rotary_desc* desc, int64_t n, const void* pos, const float* freqs,
              const void* q, const void* k, void* q_out, void* k_out, void* stream) {
  const zm_rotary_desc* d = desc;
  if (!d || n < 0 || n > kMaxTokens || !is_dtype(d->io_dtype)) return ZM_ERR_INVALID_ARG;
  if (d->heads_q < 1 || d->heads_k < 0 || d->d_head < 8 || d->d_head % 8 != 0)
    return ZM_ERR_INVALID_ARG;
  if (d->layout < ZM_ROTARY_HALVES || d->layout > ZM_ROTARY_AXIS_HALVES ||
      (d->inverse & ~1) != 0 || (d->pos_f32 & ~1) != 0 || d->axes < 1 || d->axes > kMaxAxes)
    return ZM_ERR_INVALID_ARG;
  if (d->heads_q > kMaxRotaryHeads || d->heads_k > kMaxRotaryHeads || d->d_head > kMaxRotaryHead)
    return ZM_ERR_UNSUPPORTED;
  RotaryArgs a{};
  int64_t pairs = 0;
  for (int i = 0; i < kMaxAxes; ++i) {
    if (d->sections[i] < 0 || (i >= d->axes && d->sections[i] != 0)) return ZM_ERR_INVALID_ARG;
    pairs += d->sections[i];
    if (pairs > d->d_head / 2) return ZM_ERR_INVALID_ARG;
    a.first[i + 1] = (int)pairs;
  }
  if (pairs < 1) return ZM_ERR_INVALID_ARG;
  if (n == 0) return ZM_OK;
  if (!pos || !aligned(pos, 4) || !freqs || !aligned(freqs, 4)) return ZM_ERR_INVALID_ARG;
  ZM_TRY(check_rows(q, d->ld_q, (int64_t)d->heads_q * d->d_head));
  ZM_TRY(check_rows(q_out, d->ld_q_out, (int64_t)d->heads_q * d->d_head));
  if (q == q_out && d->ld_q != d->ld_q_out) return ZM_ERR_INVALID_ARG;
  if (d->heads_k) {
    ZM_TRY(check_rows(k, d->ld_k, (int64_t)d->heads_k * d->d_head));
    ZM_TRY(check_rows(k_out, d->ld_k_out, (int64_t)d->heads_k * d->d_head));
    if (k == k_out && d->ld_k != d->ld_k_out) return ZM_ERR_INVALID_ARG;
    if (q_out == k_out || q_out == k || k_out == q) return ZM_ERR_INVALID_ARG;
  }
  a.q = RotaryTensor{q, q_out, d->ld_q, d->ld_q_out, d->heads_q};
  a.k = RotaryTensor{k, k_out, d->ld_k, d->ld_k_out, d->heads_k};
  a.pos = pos;
  a.freqs = freqs;
  a.n = n;
  a.d = d->d_head;
  a.pairs = (int)pairs;
  a.axes = d->axes;
  a.layout = d->layout;
  a.f32 = d->io_dtype == ZM_F32;
  a.pos_f32 = d->pos_f32 != 0;
  a.inverse = d->inverse != 0;
  ZM_HIP(launch_rotary(a, (hipStream_t)stream));
  return ZM_OK;
}

}  // extern "C"
