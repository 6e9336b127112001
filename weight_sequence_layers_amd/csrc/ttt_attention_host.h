// Checks of strides and overlaps shared by the host code of the attention and the mixer calls.
#pragma once

#include <initializer_list>

#include "ttt_block_host.h"

namespace ttt {

constexpr int64_t LD_MAX = (int64_t)1 << 28;   // keeps every byte offset within int64

// A matrix of `rows` rows of `width` bytes, `ld` bytes apart.
struct Rows {
  const void* p;
  int64_t rows, width, ld;
};

// Whether two such matrices share a byte.  Matrices of one stride whose rows lie side by side
// (thirds of one projection's rows) do not.
inline bool share(const Rows& a, const Rows& b) {
  if (a.rows <= 0 || b.rows <= 0) return false;
  const size_t na = (size_t)((a.rows - 1) * a.ld + a.width), nb = (size_t)((b.rows - 1) * b.ld + b.width);
  if (!overlaps(a.p, na, b.p, nb)) return false;
  if (a.ld != b.ld) return true;
  const int64_t d = (int64_t)(reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p));
  const int64_t m = ((d % a.ld) + a.ld) % a.ld;   // b's column offset in a's rows
  return m < a.width || m + b.width > a.ld;
}

// `bytes` bytes in a row; NULL, or a call that does not touch them, is none.
inline Rows flat(const void* p, int64_t bytes) { return {p, p && bytes > 0 ? 1 : 0, bytes, bytes}; }

// Whether what a call writes shares a byte with the tables it reads or with its other outputs.
inline bool clash(std::initializer_list<Rows> outs, std::initializer_list<Rows> ins) {
  for (const Rows* o = outs.begin(); o != outs.end(); ++o) {
    for (const Rows& r : ins)
      if (share(*o, r)) return true;
    for (const Rows* x = outs.begin(); x != o; ++x)
      if (share(*o, *x)) return true;
  }
  return false;
}

inline ttt_status check_ld(int64_t ld, int64_t width, int size, const char* name) {
  if (ld < width || ld > LD_MAX || ld * size % 16)
    return failf(TTT_E_SHAPE, "%s %lld: at least %lld, rows 16-byte aligned", name, (long long)ld,
                 (long long)width);
  return TTT_OK;
}

inline ttt_status optional(const void* p, const char* name) { return p ? need(p, name) : TTT_OK; }

}  // namespace ttt
