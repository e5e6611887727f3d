// What the C-ABI translation units share: pointer checks and the early-return
// macros of their entry points.
#pragma once

#include "zm_internal.h"

namespace zm {

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

}  // namespace zm

#define ZM_TRY(expr)            \
  do {                          \
    const int _s = (expr);      \
    if (_s != ZM_OK) return _s; \
  } while (0)

#define ZM_HIP(expr)                                                                \
  do {                                                                              \
    const hipError_t _e = (expr);                                                   \
    if (_e != hipSuccess) {                                                         \
      zm::set_last_error("%s: %s (%d)", #expr, hipGetErrorString(_e), (int)_e);     \
      return ZM_ERR_HIP;                                                            \
    }                                                                               \
  } while (0)
