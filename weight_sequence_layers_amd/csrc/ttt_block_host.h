// Argument-check helpers shared by the host code of the block and the attention calls.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>

#include "ttt_internal.h"

namespace ttt {

inline ttt_status failf(ttt_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return report(st, buf);
}

#define BLK_HIP(expr)                                                                   \
  do {                                                                                  \
    hipError_t e_ = (expr);                                                             \
    if (e_ != hipSuccess)                                                               \
      return failf(TTT_E_HIP, "%s failed: %s (%s:%d)", #expr, hipGetErrorString(e_),    \
                   __FILE__, __LINE__);                                                 \
  } while (0)

#define BLK_TRY(expr)                  \
  do {                                 \
    ttt_status s_ = (expr);            \
    if (s_ != TTT_OK) return s_;       \
  } while (0)

inline ttt_status need(const void* p, const char* name) {
  if (!p) return failf(TTT_E_NULL, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % 16)
    return failf(TTT_E_ALIGN, "%s is not 16-byte aligned", name);
  return TTT_OK;
}

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const char *pa = static_cast<const char*>(a), *pb = static_cast<const char*>(b);
  return pa < pb + nb && pb < pa + na;
}

}  // namespace ttt
