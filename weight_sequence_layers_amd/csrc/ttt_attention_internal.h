// Internal interface between the attention host code (ttt_attention.cpp) and its kernels
// (ttt_attention_*.hip).  Not part of the public ABI.
#pragma once

#include "ttt_attention.h"
#include "ttt_block_internal.h"

namespace ttt {

// A pointer as one to global memory.  The compiler takes a pointer chosen at run time among
// several for a generic one, whose accesses also count as LDS accesses: every wait for an LDS
// read would then wait for the global loads under way.
template <typename T>
__device__ __forceinline__ __attribute__((address_space(1))) T* as_global(T* p) {
  return (__attribute__((address_space(1))) T*)p;
}

// ------------------------------------------------------------------------ norm and rotation
constexpr int ROPE_NT = 256;           // threads of a workgroup
constexpr int ROPE_TURNS = 2048;       // cos / sin pairs a workgroup keeps in LDS
constexpr int ROPE_MAX_TB = 16;        // tokens of a workgroup's block, at most
constexpr int ROPE_BWD_WGS = 512;      // workgroups of a side of a backward launch, at most

// heads x head_dim values per token: rows of x, rows of y, the learned scale
struct RopeSide {
  const void* x;
  const void* dy;      // backward
  void* y;             // forward: the output; backward: dx
  const void* w;
  int64_t ldx, lddy, ldy;
  int32_t heads;
};

struct RopeArgs {
  RopeSide q, k;
  const void* v;       // append
  int64_t ldv;
  const float* freq;
  const int32_t* pos;
  int64_t tokens;
  int32_t D, rot, axes, pairs, norm, lph, tb;   // lph: lanes per head, a power of two
  float eps;
  // append
  u16* kc;
  u16* vc;             // e4m3 caches: byte pointers behind the same fields
  const float *ks, *vs;
  const int64_t* slot;
  int64_t page_stride;
  int32_t page_size;
  int64_t slots;       // pages * page_size
  int32_t e4m3;
  // backward
  float* part;         // [2][workgroups][D]: partial sums of the scales' gradients, or null
  int32_t wgs;
};

struct RopeDwArgs {
  const float* part;   // [2][n][D]
  float *dq, *dk;      // either may be null
  int32_t n, D;
};

hipError_t launch_rope(const RopeArgs& a, int bf16, hipStream_t st);
hipError_t launch_rope_append(const RopeArgs& a, hipStream_t st);
hipError_t launch_rope_backward(const RopeArgs& a, int bf16, hipStream_t st);
hipError_t launch_rope_dw(const RopeDwArgs& a, hipStream_t st);

// ------------------------------------------------------------------------ paged attention
constexpr int PG_NT = 256, PG_WAVES = 4;
constexpr int PG_BLOCK = 128;                    // tokens of a part: a multiple of this
constexpr int PG_HEADS = 16;                     // query heads of a workgroup

struct PagedArgs {
  const u16* q;
  int64_t ldq;
  const char *k, *v;
  const float *ks, *vs;
  int64_t page_bytes;   // bytes between pages
  int32_t pages, page_size, kv_heads;
  const int32_t* table;
  const int32_t* lens;
  u16* out;
  int64_t ldo;
  float* lse;
  int32_t seqs, heads, group, htiles, max_pages, window, splits;
  float scale;          // of the scores, natural
  float* po;            // [seqs][heads][splits][D] partial sums (splits > 1)
  float* pm;            // [seqs][heads][splits][2]: running maximum (base 2), normaliser
};

hipError_t launch_paged(const PagedArgs& a, int D, int e4m3, hipStream_t st);

// The tokens of a sequence that its new token sees, [lo, hi).
__host__ __device__ inline void paged_span(int32_t len, int32_t max_pages, int32_t page_size,
                                           int32_t window, int32_t& lo, int32_t& hi) {
  const int32_t cap = max_pages * page_size;   // at most 2^30: a host check
  hi = len < 0 ? 0 : len > cap ? cap : len;
  lo = window > 0 && hi > window ? hi - window : 0;
}

// Byte offset of a cached row from the cache's base, or -1 for a page outside the cache.
__host__ __device__ inline int64_t paged_row(int32_t page, int32_t pages, int64_t page_bytes,
                                             int32_t head, int32_t page_size, int32_t place,
                                             int32_t row_bytes) {
  if (page < 0 || page >= pages) return -1;
  return page * page_bytes + ((int64_t)head * page_size + place) * row_bytes;
}

// Tokens that each part of a sequence's span takes when n tokens are split into at most
// `splits` parts: whole steps of a workgroup.
__host__ __device__ inline int32_t paged_part(int32_t n, int32_t splits) {
  const int32_t steps = (n + PG_BLOCK - 1) / PG_BLOCK;
  return (steps + splits - 1) / splits * PG_BLOCK;
}

// ------------------------------------------------------------------------ window training
struct WindowArgs {
  const u16 *q, *k, *v;
  int64_t ld;
  u16* out;              // written by the forward, read by the backward
  int64_t ldo;
  float* lse;
  const u16* dout;       // backward
  u16 *dq, *dk, *dv;
  float* delta;
  int64_t lddo, ldd;
  int32_t T, heads, window, mode, blocks, total;
  float scale, scale2;   // 1 / sqrt(ATT_D), and times log2(e)
};

// problems: batch * heads; blocks and total are filled in here
hipError_t launch_window_fwd(WindowArgs a, int64_t problems, hipStream_t st);
hipError_t launch_window_bwd(WindowArgs a, int64_t problems, hipStream_t st);

}  // namespace ttt
