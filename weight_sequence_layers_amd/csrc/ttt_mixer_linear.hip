// Linear attention with a decay for each head over whole sequences, and its backward
// (include/ttt_mixer.h).
//
// Mathematics.  S_t = a S_{t-1} + k_t v_t^T, o_t = c S_t^T q_t.  Over a chunk of n tokens that starts
// with S:
//   o_i = c (a^(i+1) S^T q_i + sum_{j <= i} a^(i-j) (q_i . k_j) v_j),
//   S  <- a^n S + sum_j a^(n-1-j) k_j v_j^T.
// The gradients are the same recurrence with its operands in other places:
//   dq_i = c S_i do_i                       (q, k, v) <- (do, v, k), the state S^T;
//   dv_j = P_j^T k_j,  P_j = a P_{j+1} + c q_j do_j^T    <- (k, q, do), backward in time;
//   dk_j = P_j v_j                                        <- (v, do, q), backward in time, P^T,
// so that one kernel computes all four ("roles").
#include "ttt_device.hpp"
#include "ttt_mixer_internal.h"

namespace ttt {
namespace {

// A tile keeps the 16-byte chunk c of row r at chunk c ^ lin_swz(r) of the row (P bytes): 16
// consecutive rows at one chunk, and 32 elements of 4 consecutive rows, lie on distinct banks,
// whether it is read along its rows or along its columns.
template <int P>
__device__ __forceinline__ int lin_swz(int r) {
  return P == 128 ? (((r >> 1) & 1) << 2) | ((r >> 2) & 3) : ((r & 3) << 2) | ((r >> 2) & 3);
}

// Loads of a tile of LIN_C rows of P bytes, straight into LDS, by NW waves.
template <int P, int NW>
struct LinLoad {
  static constexpr int ROWS = 1024 / P;                     // rows of one wave's load
  static constexpr int N = LIN_C / ROWS / NW;               // loads of a wave
  static constexpr int VAR = NW * ROWS < 16 ? 16 / (NW * ROWS) : 1;   // the swizzle repeats after 16 rows
  int32_t off[VAR], step;
  uint32_t ld2;
  int slice;
  __device__ __forceinline__ void init(int64_t ld, int rev) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    ld2 = (uint32_t)(ld * 2);
    slice = wave * 1024;
    const int32_t row = rev ? -(int32_t)ld2 : (int32_t)ld2;
    step = NW * ROWS * VAR * row;
#pragma unroll
    for (int i = 0; i < VAR; ++i) {
      const int r = (wave + i * NW) * ROWS + lane / (P / 16);
      off[i] = r * row + ((lane % (P / 16)) ^ lin_swz<P>(r)) * 16;
    }
  }
  // The n rows at p, in their order or (rev) from the last to the first; the others read as 0:
  // their offsets lie behind the n rows, or wrap to 2^31 and more.
  __device__ __forceinline__ void issue(char* tile, const u16* p, int n, int rev) const {
    const uint32_t last = (uint32_t)(n - 1) * ld2;
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)(last + P), 0x00020000);
    const int32_t top = rev ? (int32_t)last : 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
      dma16(rs, (lds_void_t*)(tile + slice + i * NW * 1024), (uint32_t)(off[i % VAR] + (i / VAR) * step + top));
  }
};

// Offsets of a lane's fragments in a tile.  PERM: along the columns the second and third four of every
// 16 elements change places.  An accumulator's element v is row 8 (v / 4) + 4 (lane / 32) + v % 4 of its
// tile; rows taken in that order make a lane's eight of 16 neighbours, 8 (lane / 32) .. + 7, which is how
// an operand along the rows is read in one piece.
template <int P, bool PERM>
struct LinAt {
  int row;   // along the rows: elements 8 (lane / 32) .. + 7 of row lane % 32
  int col;   // along the columns: elements 16 (g & 1) + 4 (j & 3) .. + 3 of row 4 (g / 2) + j / 4
  __device__ __forceinline__ void init() {
    const int lane = threadIdx.x & 63, r = lane & 31, g = lane >> 4, j = lane & 15;
    row = r * P + ((lin_swz<P>(r) ^ (lane >> 5)) << 4);
    const int four = PERM ? ((j & 1) << 1) | ((j >> 1) & 1) : j & 3;
    const int m = 16 * (g & 1) + 4 * four, rc = 4 * (g >> 1) + (j >> 2);
    col = rc * P + (((m >> 3) ^ lin_swz<P>(rc)) << 4) + (m & 7) * 2;
  }
};

typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Row base_row + lane % 32, elements base + 8 (lane / 32) .. + 7.  base_row a multiple of 32, base of 16.
template <int P, bool PERM>
__device__ __forceinline__ bf16x8 lin_row(const char* tile, const LinAt<P, PERM>& at, int base_row, int base) {
  return *reinterpret_cast<const bf16x8*>(tile + base_row * P + (at.row ^ (base * 2)));
}
// Element base + lane % 32 (in the order of PERM) of rows row + 4 (lane / 32) + (0..3) and + 8.  base a
// multiple of 32, row of 16.
template <int P, bool PERM>
__device__ __forceinline__ bf16x8 lin_col(const char* tile, const LinAt<P, PERM>& at, int base, int row) {
  s16x4 x[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const char* p = tile + (row + 8 * i) * P + (at.col ^ (base << 1) ^ (i << 5));
    x[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p));
  }
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7));
}

__device__ __forceinline__ f32x16 lin_mma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Two numbers rounded to bf16, and their values.
__device__ __forceinline__ uint32_t lin_pack(float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
__device__ __forceinline__ float lin_first(uint32_t u) { return __builtin_bit_cast(float, u << 16); }
__device__ __forceinline__ float lin_second(uint32_t u) { return __builtin_bit_cast(float, u & 0xffff0000u); }

// x as N bf16 numbers whose sum it is, to 8 N bits, and what is left of it.
template <int N>
__device__ __forceinline__ void lin_split(float (&x)[8], bf16x8 (&p)[N]) {
  u32x4 u[N];
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      u[i][e] = lin_pack(x[2 * e], x[2 * e + 1]);
      x[2 * e] -= lin_first(u[i][e]);
      x[2 * e + 1] -= lin_second(u[i][e]);
    }
#pragma unroll
  for (int i = 0; i < N; ++i) p[i] = __builtin_bit_cast(bf16x8, u[i]);
}

// a^n, in 64 bits: a table made of rounded products would drift over long sequences
__device__ __forceinline__ float lin_power(float a, int n) {
  double p = 1.0, x = (double)a;
  for (; n; n >>= 1) {
    if (n & 1) p *= x;
    x *= x;
  }
  return (float)p;
}

// Waits until at most n of the wave's memory operations are under way (loads end in the order of
// their issue), then for the workgroup: what the waves had loaded is there, what they had read is free.
template <int N>
__device__ __forceinline__ void lin_wait() {
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
  lds_barrier();
}

// A workgroup's place in a launch: role, sequence, head, segment and columns.
struct LinPlace {
  int slice;       // (in the order in which they are taken from the workgroup's number)
  const LinRole& r;
  int h, seg, b, len, t0, cnt, chunks;
  int64_t row0;
  bool none;       // nothing to do
  static __device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
  static __device__ __forceinline__ int take(int& id, int n) {
    const int q = uniform(id / n), x = uniform(id - q * n);
    id = q;
    return x;
  }
  __device__ __forceinline__ LinPlace(const LinArgs& a, int nseg, int id, bool out)
      : slice(take(id, a.slices)), r(a.role[take(id, a.roles)]), h(take(id, a.heads)), seg(take(id, nseg)), b(id) {
    lin_span(a.starts, b, a.tokens, a.T, row0, len);
    t0 = seg * a.L;                                          // first token, in the role's time
    none = out ? seg > 0 && t0 >= len : t0 + a.L >= len;
    cnt = min(a.L, len - t0);
    chunks = (cnt + LIN_C - 1) / LIN_C;
  }
};

// Powers of the decay, and the weights of a chunk's tokens in the state behind it: of 64 tokens, and of
// the last chunk's.
struct LinTables {
  float pw[LIN_C + 4];
  float wt[2][LIN_C];
  __device__ __forceinline__ void init(float lam, const LinPlace& at) {
    const int i = threadIdx.x, last = at.cnt - (at.chunks - 1) * LIN_C;
    if (i <= LIN_C) pw[i] = lin_power(lam, i);
    if (i < LIN_C) {
      wt[0][i] = lin_power(lam, LIN_C - 1 - i) * at.r.scale_w;
      wt[1][i] = lin_power(lam, max(last - 1 - i, 0)) * at.r.scale_w;   // rows behind the last are 0
    }
  }
};

// The state of a wave: element v of tile rt is row 32 rt + 16 (v / 8) + 8 hl + v % 8, column li of its 32.
template <int RT>
struct LinState {
  f32x16 s[RT];
  // s <- f s + k^T (w v) over a chunk; vf: the wave's columns of v.  w v enters as two bf16 numbers, or
  // as three.
  template <int PA>
  __device__ __forceinline__ void add(const char* k, const LinAt<PA, true>& at, const bf16x8 (&vf)[LIN_C / 16],
                                      const float* wt, float f, int hl, bool three) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int v = 0; v < 16; ++v) s[rt][v] *= f;
#pragma unroll
    for (int x = 0; x < LIN_C / 16; ++x) {
      float w[8];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const f32x4 t = *reinterpret_cast<const f32x4*>(wt + 16 * x + 8 * g + 4 * hl);
        const u32x4 u = __builtin_bit_cast(u32x4, vf[x]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          w[4 * g + 2 * e] = lin_first(u[2 * g + e]) * t[2 * e];
          w[4 * g + 2 * e + 1] = lin_second(u[2 * g + e]) * t[2 * e + 1];
        }
      }
      bf16x8 wp[2], kf[RT];
      lin_split(w, wp);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) kf[rt] = lin_col(k, at, 32 * rt, 16 * x);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) s[rt] = lin_mma(kf[rt], wp[i], s[rt]);
      if (three) {   // what is left of w, w now
        bf16x8 rest[1];
        lin_split(w, rest);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) s[rt] = lin_mma(kf[rt], rest[0], s[rt]);
      }
    }
  }
  __device__ __forceinline__ void store(float* p, int ld, int hl, float f) const {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int v = 0; v < 16; ++v)
        *as_global(p + (int64_t)(32 * rt + 16 * (v >> 3) + 8 * hl + (v & 7)) * ld) = s[rt][v] * f;
  }
};

// A workgroup walks one segment of one sequence, head and role, 64 tokens at a time; its NW waves hold 32
// columns of the state each, all DA rows of it, as accumulators.  The output is computed transposed
// (a lane is a token), so that the accumulators of the state and of the scores are the operands of the
// products that follow as they lie.  The scores' three tiles of 32 x 32 (two of the diagonal, one below) are a wave's
// each, which leaves them, decayed and split, in LDS for the others: the barrier that they need is
// there for v.
//
// Four areas of LDS take turns: while q, k and v of a chunk lie in three, the next chunk's q comes into
// the fourth; once q has been read its k comes into q's, and once all has been read its v into k's: each
// load has half a chunk's work or more to arrive.
template <int DA, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(DA == 256 ? 1 : 2)))
void k_linear(LinArgs a) {
  constexpr int PA = DA * 2, PV = NW * 64;                    // bytes of a tile's row
  constexpr int AREA = LIN_C * (PA > PV ? PA : PV), RT = DA / 32;
  __shared__ __attribute__((aligned(1024))) char a0[AREA];
  __shared__ __attribute__((aligned(1024))) char a1[AREA];
  __shared__ __attribute__((aligned(1024))) char a2[AREA];
  __shared__ __attribute__((aligned(1024))) char a3[AREA];
  __shared__ __attribute__((aligned(1024))) bf16x8 scores[3][2][2][64];   // [tile][keys of 16][part][lane]
  __shared__ __attribute__((aligned(16))) LinTables tb;
  const LinPlace at(a, a.nseg, xcd_block(blockIdx.x, a.total), true);
  if (at.none) return;
  const LinRole& r = at.r;
  const int rev = r.rev, h = at.h, b = at.b, len = at.len, t0 = at.t0, cnt = at.cnt, chunks = at.chunks;
  const int lane = threadIdx.x & 63, hl = lane >> 5, li = lane & 31;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const float lam = a.decay[h];

  const int col0 = at.slice * 32 * NW;                       // the workgroup's first column
  const u16* qb = r.q + (int64_t)h * DA;
  const u16* kb = r.k + (int64_t)h * DA;
  const u16* vb = r.v + (int64_t)h * a.DB + col0;
  LinLoad<PA, NW> lq, lk;
  LinLoad<PV, NW> lv;
  lq.init(r.ldq, rev);
  lk.init(r.ldk, rev);
  lv.init(r.ldv, rev);
  auto size = [&](int c) __attribute__((always_inline)) { return min(LIN_C, cnt - c * LIN_C); };
  auto row = [&](int c) __attribute__((always_inline)) {     // of chunk c's lowest token
    const int t = t0 + c * LIN_C;
    return at.row0 + (rev ? len - t - size(c) : t);
  };
  if (chunks) {
    lq.issue(a0, qb + row(0) * r.ldq, size(0), rev);
    lk.issue(a1, kb + row(0) * r.ldk, size(0), rev);
    lv.issue(a2, vb + row(0) * r.ldv, size(0), rev);
  }
  tb.init(lam, at);

  const int64_t elems = (int64_t)DA * a.DB;
  const int colw = col0 + 32 * wave + li;
  const int64_t entry = lin_slot(a.slot, b, a.slots);
  LinState<RT> S;
  float* fin = nullptr;
  if (r.fin && entry >= 0 && t0 + a.L >= len) fin = r.fin + (entry * a.heads + h) * elems + colw;
  const float* init = nullptr;
  if (r.ws) init = r.ws + (((int64_t)b * a.heads + h) * a.nseg + at.seg) * elems;
  else if (r.init && entry >= 0) init = r.init + (entry * a.heads + h) * elems;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) S.s[rt] = f32x16{};
  if (init) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int i = 32 * rt + 16 * (g >> 1) + 8 * hl + 4 * (g & 1);
        if (r.trans) {
          const f32x4 x = *as_global(reinterpret_cast<const f32x4*>(init + (int64_t)colw * DA + i));
#pragma unroll
          for (int e = 0; e < 4; ++e) S.s[rt][4 * g + e] = x[e];
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) S.s[rt][4 * g + e] = *as_global(init + (int64_t)(i + e) * a.DB + colw);
        }
      }
  }
  LinAt<PA, true> ta;
  LinAt<PV, false> tv;
  ta.init();
  tv.init();
  lin_wait<0>();
  // element v of a tile of scores: key 8 (v / 4) + 4 hl + v % 4, query li
  float dm[16];
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    const int j = 8 * (v >> 2) + 4 * hl + (v & 3);
    dm[v] = li >= j ? tb.pw[li >= j ? li - j : 0] * r.scale_p : 0.f;
  }
  const float f21 = tb.pw[li + 1] * (r.scale_p / r.scale_w);   // with wt's second half: a^(32 + li - j)

  uint32_t ow[2][8];
  auto step = [&](char* qa, char* ka, char* va, char* spare, int c) __attribute__((always_inline)) {
    const int n = size(c);
    const bool more = c + 1 < chunks;
    if (more) lq.issue(spare, qb + row(c + 1) * r.ldq, size(c + 1), rev);
    // backward in time the state before the first token (the gradient of the last state) is that
    // of the first token itself: one power less
    const int e0 = rev && t0 + c == 0 ? 0 : 1;
    for (int tile = wave; tile < 3; tile += NW) {   // queries and keys: second and first half; both first; both second
      const int qi = tile == 1 ? 0 : 32, ki = tile == 2 ? 32 : 0;
      f32x16 p = f32x16{};
#pragma unroll
      for (int x = 0; x < 2 * RT; ++x) p = lin_mma(lin_row(ka, ta, ki, 16 * x), lin_row(qa, ta, qi, 16 * x), p);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float pv[8];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const f32x4 t = *reinterpret_cast<const f32x4*>(&tb.wt[0][32 + 16 * x + 8 * g + 4 * hl]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int v = 8 * x + 4 * g + e;
            pv[4 * g + e] = p[v] * (tile ? dm[v] : f21 * t[e]);
          }
        }
        bf16x8 pp[2];
        lin_split(pv, pp);
#pragma unroll
        for (int i = 0; i < 2; ++i) scores[tile][x][i][lane] = pp[i];
      }
    }
    f32x16 o1 = f32x16{}, o2 = f32x16{};
#pragma unroll
    for (int x = 0; x < 2 * RT; ++x) {
      const bf16x8 q1 = lin_row(qa, ta, 0, 16 * x), q2 = lin_row(qa, ta, 32, 16 * x);
      float sv[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) sv[e] = S.s[x >> 1][8 * (x & 1) + e];
      bf16x8 sp[2];
      lin_split(sv, sp);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        o1 = lin_mma(sp[i], q1, o1);
        o2 = lin_mma(sp[i], q2, o2);
      }
    }
    if (more) lin_wait<LinLoad<PA, NW>::N>();   // v and the scores are there, q is free
    else lin_wait<0>();
    if (more) lk.issue(qa, kb + row(c + 1) * r.ldk, size(c + 1), rev);
    bf16x8 vf[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) vf[x] = lin_col(va, tv, 32 * wave, 16 * x);
    const float f1 = tb.pw[li + e0] * r.scale_s, f2 = tb.pw[32 + li + e0] * r.scale_s;
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      o1[v] *= f1;
      o2[v] *= f2;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        o1 = lin_mma(vf[x], scores[1][x][i][lane], o1);
        o2 = lin_mma(vf[x], scores[0][x][i][lane], o2);
        o2 = lin_mma(vf[2 + x], scores[2][x][i][lane], o2);
      }
    // the halves of the wave swapped in pairs: 8 neighbouring elements of a row in a lane
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int g = 0; g < 4; g += 2)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const f32x16& o = i ? o2 : o1;
          const auto w = __builtin_amdgcn_permlane32_swap(lin_pack(o[4 * g + 2 * e], o[4 * g + 2 * e + 1]),
                                                          lin_pack(o[4 * g + 4 + 2 * e], o[4 * g + 5 + 2 * e]), false, false);
          ow[i][2 * g + e] = w[0];
          ow[i][2 * g + 2 + e] = w[1];
        }
    S.template add<PA>(ka, ta, vf, tb.wt[more ? 0 : 1], tb.pw[n - 1 + e0], hl, fin != nullptr);
    lin_wait<0>();   // the next chunk's q and k are there, k and v are free
    if (more) lv.issue(ka, vb + row(c + 1) * r.ldv, size(c + 1), rev);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (32 * i + li < n) {
        const int t = t0 + c * LIN_C + 32 * i + li;
        u16* y = r.out + (at.row0 + (rev ? len - 1 - t : t)) * r.ldo + (int64_t)h * a.DB + col0 + 32 * wave + 8 * hl;
#pragma unroll
        for (int g = 0; g < 2; ++g)
          *as_global(reinterpret_cast<u32x4*>(y + 16 * g)) =
              u32x4{ow[i][4 * g], ow[i][4 * g + 1], ow[i][4 * g + 2], ow[i][4 * g + 3]};
      }
  };
  int c = 0;
  while (c < chunks) {
    step(a0, a1, a2, a3, c++);
    if (c == chunks) break;
    step(a3, a0, a1, a2, c++);
    if (c == chunks) break;
    step(a2, a3, a0, a1, c++);
    if (c == chunks) break;
    step(a1, a2, a3, a0, c++);
  }

  if (fin)   // behind the last step back lies the state before the first token
    S.store(fin, a.DB, hl, rev && len > 0 ? lam : 1.f);
}

// Each segment's own sum, from zeros, of all but the last.
template <int DA, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(DA == 256 ? 1 : 2)))
void k_linear_states(LinArgs a) {
  constexpr int PA = DA * 2, PV = NW * 64, VO = LIN_C * PA, RT = DA / 32;
  __shared__ __attribute__((aligned(1024))) char st0[LIN_C * (PA + PV)];
  __shared__ __attribute__((aligned(1024))) char st1[LIN_C * (PA + PV)];
  __shared__ __attribute__((aligned(16))) LinTables tb;
  const LinPlace at(a, a.nseg - 1, xcd_block(blockIdx.x, a.total), false);
  if (at.none) return;
  const LinRole& r = at.r;
  const int rev = r.rev, lane = threadIdx.x & 63, hl = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int col0 = at.slice * 32 * NW;
  const u16* kb = r.k + (int64_t)at.h * DA;
  const u16* vb = r.v + (int64_t)at.h * a.DB + col0;
  LinLoad<PA, NW> lk;
  LinLoad<PV, NW> lv;
  lk.init(r.ldk, rev);
  lv.init(r.ldv, rev);
  auto issue = [&](char* st, int c) __attribute__((always_inline)) {   // every chunk is whole
    const int t = at.t0 + c * LIN_C;
    const int64_t row = at.row0 + (rev ? at.len - t - LIN_C : t);
    lk.issue(st, kb + row * r.ldk, LIN_C, rev);
    lv.issue(st + VO, vb + row * r.ldv, LIN_C, rev);
  };
  issue(st0, 0);
  tb.init(a.decay[at.h], at);
  LinState<RT> S;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) S.s[rt] = f32x16{};
  LinAt<PA, true> ta;
  LinAt<PV, false> tv;
  ta.init();
  tv.init();
  lin_wait<0>();
  auto step = [&](const char* cur, char* nxt, int c) __attribute__((always_inline)) {
    if (c + 1 < at.chunks) issue(nxt, c + 1);
    bf16x8 vf[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) vf[x] = lin_col(cur + VO, tv, 32 * wave, 16 * x);
    S.template add<PA>(cur, ta, vf, tb.wt[0], tb.pw[LIN_C], hl, r.fin != nullptr);
    lin_wait<0>();
  };
  int c = 0;
  for (; c + 1 < at.chunks; c += 2) {
    step(st0, st1, c);
    step(st1, st0, c + 1);
  }
  if (c < at.chunks) step(st0, st1, c);
  S.store(r.ws + (((int64_t)at.b * a.heads + at.h) * a.nseg + at.seg) * DA * a.DB + col0 + 32 * wave + (lane & 31), a.DB,
          hl, 1.f);
}

// From the segments' own sums to the states before each: a thread takes four elements of a state
// along the segments.
__global__ __launch_bounds__(256) void k_linear_scan(LinArgs a, int DA) {
  const int64_t elems = (int64_t)DA * a.DB;
  const int blocks = (int)(elems / 1024);
  const int pid = blockIdx.x / blocks, part = blockIdx.x - pid * blocks;
  const LinRole& r = a.role[blockIdx.y];
  const int b = pid / a.heads, h = pid - b * a.heads;
  int64_t row0;
  int len;
  lin_span(a.starts, b, a.tokens, a.T, row0, len);
  const int cnt = max(1, (len + a.L - 1) / a.L);
  const int64_t at = (int64_t)part * 1024 + 4 * threadIdx.x;
  float* w = r.ws + (int64_t)pid * a.nseg * elems + at;
  const int64_t entry = lin_slot(a.slot, b, a.slots);
  f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
  if (r.init && entry >= 0)
    s = *as_global(reinterpret_cast<const f32x4*>(r.init + (entry * a.heads + h) * elems + at));
  const float lam = a.decay[h], f = lin_power(lam, a.L);
  float f0 = r.rev ? lin_power(lam, a.L - 1) : f;
  for (int i = 0; i < cnt; i += 8) {
    f32x4 x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      x[j] = i + j < cnt - 1 ? *as_global(reinterpret_cast<const f32x4*>(w + (i + j) * elems)) : f32x4{};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < cnt) {
        *as_global(reinterpret_cast<f32x4*>(w + (i + j) * elems)) = s;
        s = s * f0 + x[j];
        f0 = f;
      }
  }
}

template <int DA>
hipError_t launch_nw(const LinArgs& a, int NW, bool out, hipStream_t st) {
  const dim3 grid(a.total), block(64 * NW);
  if (out && NW == 2) hipLaunchKernelGGL((k_linear<DA, 2>), grid, block, 0, st, a);
  else if (out) hipLaunchKernelGGL((k_linear<DA, 4>), grid, block, 0, st, a);
  else if (NW == 2) hipLaunchKernelGGL((k_linear_states<DA, 2>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_linear_states<DA, 4>), grid, block, 0, st, a);
  return hipGetLastError();
}

hipError_t launch_da(const LinArgs& a, int DA, int NW, bool out, hipStream_t st) {
  if (a.total == 0) return hipSuccess;
  return DA == 64 ? launch_nw<64>(a, NW, out, st)
         : DA == 128 ? launch_nw<128>(a, NW, out, st) : launch_nw<256>(a, NW, out, st);
}

}  // namespace

hipError_t launch_linear_walk(const LinArgs& a, int DA, int NW, hipStream_t st) {
  return launch_da(a, DA, NW, true, st);
}

hipError_t launch_linear_states(const LinArgs& a, int DA, int NW, hipStream_t st) {
  return launch_da(a, DA, NW, false, st);
}

hipError_t launch_linear_scan(const LinArgs& a, int DA, hipStream_t st) {
  const unsigned n = (unsigned)((int64_t)a.batch * a.heads * ((int64_t)DA * a.DB / 1024));
  hipLaunchKernelGGL(k_linear_scan, dim3(n, a.roles), dim3(256), 0, st, a, DA);
  return hipGetLastError();
}

}  // namespace ttt
