// Internal interface between the mixer's host code (ttt_mixer.cpp) and its kernels
// (ttt_mixer_*.hip).  Not part of the public ABI.
#pragma once

#include "ttt_internal.h"
#include "ttt_mixer.h"

namespace ttt {

// A pointer as one to global memory: the compiler takes a pointer chosen at run time among several
// for a generic one, whose accesses also count as LDS accesses.
template <typename T>
__device__ __forceinline__ __attribute__((address_space(1))) T* as_global(T* p) {
  return (__attribute__((address_space(1))) T*)p;
}

// ------------------------------------------------------------------------ linear attention
constexpr int LIN_C = 64;          // tokens of a chunk
constexpr int LIN_MAX_ROLES = 3;

// One recurrence over the sequences, S <- decay S + k v^T read by q: the layer itself, or one of its
// gradients with other operands, forward or backward in time.  q and k have heads of DA, v and
// out heads of DB elements.
struct LinRole {
  const u16 *q, *k, *v;
  u16* out;
  int64_t ldq, ldk, ldv, ldo;
  const float* init;      // states before the first token [.][heads][...], or null
  float* fin;             // states behind the last one, or null
  float* ws;              // [batch * heads][nseg][...] states before each segment, or null (one segment)
  int32_t rev;            // 1: from a sequence's last token to its first
  int32_t trans;          // 1: the states lie as [DB][DA]
  float scale_p, scale_s, scale_w;   // of a token's own products, of the state's, of what the state takes
};

struct LinArgs {
  LinRole role[LIN_MAX_ROLES];
  const float* decay;
  const int32_t* starts;
  const int32_t* slot;
  int64_t tokens;
  int32_t roles, slots, batch, heads, T;   // T: the longest sequence
  int32_t DB;                               // elements of a head of v
  int32_t nseg, L;                          // segments of a sequence at most, tokens of one
  int32_t slices, total;
  int32_t nt;                               // 1: rows are read past the last-level cache
};

// A sequence's first row and its length.
__host__ __device__ inline void lin_span(const int32_t* starts, int32_t b, int64_t tokens, int32_t T,
                                         int64_t& row0, int32_t& len) {
  if (!starts) {
    row0 = (int64_t)b * T;
    len = T;
    return;
  }
  int64_t s = starts[b], e = starts[b + 1];
  s = s < 0 ? 0 : s > tokens ? tokens : s;
  e = e < s ? s : e > tokens ? tokens : e;
  row0 = s;
  len = e - s > T ? T : (int32_t)(e - s);
}

// A sequence's entry in the pools, or -1.
__host__ __device__ inline int64_t lin_slot(const int32_t* slot, int32_t b, int32_t slots) {
  const int32_t i = slot ? slot[b] : b;
  return i >= 0 && i < slots ? i : -1;
}

// dims: elements of a head of q and k (DA); NW: waves of a workgroup, 16 elements of v each.
// states: only each segment's own sum, into ws, of all but the last; scan: ws from those to the
// states before each segment.
hipError_t launch_linear_walk(const LinArgs& a, int DA, int NW, hipStream_t st);
hipError_t launch_linear_states(const LinArgs& a, int DA, int NW, hipStream_t st);
hipError_t launch_linear_scan(const LinArgs& a, int DA, hipStream_t st);

// ------------------------------------------------------------------------ one token
struct LinStepArgs {
  const u16 *q, *k, *v;
  u16* out;
  int64_t ldq, ldk, ldv, ldo;
  const float* decay;
  const float* in;
  float* fin;
  const int32_t* slot;
  int32_t slots, seqs, heads, K, V, slices, total;
  float scale;
};

hipError_t launch_linear_step(const LinStepArgs& a, int cols, hipStream_t st);

// ------------------------------------------------------------------------ residual norm
struct NormArgs {
  const void *h, *y, *gate, *wy, *rs, *wn, *dho, *dn;
  void *ho, *n;                  // forward
  void *dh, *dy, *dg;            // backward
  int64_t ldh, ldy, ldg, ldho, ldn, lddho, lddn, lddh, lddy, lddg;
  int64_t tokens;
  int32_t D, gw;                 // gw: elements of a group
  int32_t norm_y, gate_kind;
  float eps;
  float* part;                   // backward: [3][wgs][D] partial sums, or null
  double* sofar;                 // [3][D] their sums over the rows of earlier launches
  int32_t wgs, begun, more;      // begun, more: there are launches before, behind
  float *dwy, *drs, *dwn;
};

// Workgroups of a launch at most: a launch's threads, up to 1024 of each, are counted in 32 bits.
constexpr int64_t NORM_LAUNCH = (int64_t)1 << 20;

// A call's rows from `first` on, at most n, of elements of `size` bytes.
inline NormArgs norm_part(const NormArgs& a, int64_t first, int64_t n, int size) {
  NormArgs p = a;
  const auto from = [&](auto*& x, int64_t ld) {
    if (x) x = (char*)x + first * ld * size;
  };
  from(p.h, a.ldh);
  from(p.y, a.ldy);
  from(p.gate, a.ldg);
  from(p.ho, a.ldho);
  from(p.n, a.ldn);
  from(p.dho, a.lddho);
  from(p.dn, a.lddn);
  from(p.dh, a.lddh);
  from(p.dy, a.lddy);
  from(p.dg, a.lddg);
  p.tokens = a.tokens - first < n ? a.tokens - first : n;
  return p;
}

hipError_t launch_residual_norm(const NormArgs& a, int bf16, hipStream_t st);
hipError_t launch_residual_norm_backward(const NormArgs& a, int bf16, hipStream_t st);
int32_t residual_norm_wgs(int32_t D, int64_t tokens);   // workgroups of a backward launch of so many rows
int64_t residual_norm_chunk(int32_t D);                  // rows of a backward launch at most

}  // namespace ttt
