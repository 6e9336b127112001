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
// consecutive rows at one chunk lie on distinct banks (read along the rows), and so do 4 neighbouring
// chunks of 4 consecutive rows (along the columns, where a product reads the first or the second halves
// of chunks only: two fifths of the LDS's busy cycles are conflicts; halves in turn by lane, without
// conflicts, made k_linear_states no faster).
template <int P>
__device__ __forceinline__ int lin_swz(int r) {
  return P == 128 ? (((r >> 1) & 1) << 2) | ((r >> 2) & 3) : ((r & 3) << 2) | ((r >> 2) & 3);
}

// A value of every lane, held in scalar registers: the launch's arguments are read once, not at every use.
template <typename T>
__device__ __forceinline__ T lin_scalar(T x) {
  static_assert(sizeof(T) == 4 || sizeof(T) == 8, "one or two registers");
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x)));
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)u), hi = __builtin_amdgcn_readfirstlane((int)(u >> 32));
    return __builtin_bit_cast(T, (uint64_t)hi << 32 | lo);
  }
}

// Loads of the chunks of one operand in turn, tiles of LIN_C rows of P bytes, straight into LDS, by NW
// waves.
template <int P, int NW>
struct LinLoad {
  static constexpr int ROWS = 1024 / P;                     // rows of one wave's load
  static constexpr int N = LIN_C / ROWS / NW;               // loads of a wave
  static constexpr int VAR = NW * ROWS < 16 ? 16 / (NW * ROWS) : 1;   // the swizzle repeats after 16 rows
  const char* p;         // the next chunk's lowest token
  int32_t off[VAR], step;
  uint32_t ld2;
  int slice, rev, nt;
  // base: the head's columns of row 0; row: the lowest token of the first chunk
  __device__ __forceinline__ void init(const u16* base, int64_t ld, int64_t row, int rev_, int nt_) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    p = lin_scalar(reinterpret_cast<const char*>(base + row * ld));
    ld2 = lin_scalar((uint32_t)(ld * 2));
    rev = rev_;
    nt = nt_;
    slice = wave * 1024;
    const int32_t line = rev ? -(int32_t)ld2 : (int32_t)ld2;
    step = NW * ROWS * VAR * line;
#pragma unroll
    for (int i = 0; i < VAR; ++i) {
      const int r = (wave + i * NW) * ROWS + lane / (P / 16);
      off[i] = r * line + ((lane % (P / 16)) ^ lin_swz<P>(r)) * 16;
    }
  }
  // The chunk's n rows, in their order or (rev) from the last to the first; the others read as 0: their
  // offsets lie behind the n rows, or wrap to 2^31 and more.  next: rows of the chunk behind it.
  __device__ __forceinline__ void issue(char* tile, int n, int next) {
    const uint32_t last = (uint32_t)(n - 1) * ld2;
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)(last + P), 0x00020000);
    const int32_t top = rev ? (int32_t)last : 0;
    if (nt) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)(tile + slice + i * NW * 1024), 16,
                                                 (uint32_t)(off[i % VAR] + (i / VAR) * step + top), 0, 0, 2);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        dma16(rs, (lds_void_t*)(tile + slice + i * NW * 1024), (uint32_t)(off[i % VAR] + (i / VAR) * step + top));
    }
    p += rev ? -(int64_t)next * ld2 : (int64_t)LIN_C * ld2;
  }
};

typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// The lanes in a 16 x 16 x 32 product, lane = 16 g + j: an operand's row (column) j, of the 32 summed
// over the numbers 8 g .. 8 g + 7; the result's column j, rows 4 g .. 4 g + 3.  What is summed over may
// come in any order that both operands have.  Two results over one another are an operand as they lie:
// rows 4 g + e of the first and of the second are its 8 g + e and 8 g + 4 + e.
//
// Row j of 16, elements 8 g .. 8 g + 7 of 32 (at + 64 bytes times their number).
template <int P>
__device__ __forceinline__ int lin_row_at() {
  const int lane = threadIdx.x & 63, g = lane >> 4, j = lane & 15;
  return j * P + ((g ^ lin_swz<P>(j)) << 4);
}
__device__ __forceinline__ bf16x8 lin_row(const char* tile, int at, int y) {
  return *reinterpret_cast<const bf16x8*>(tile + (at ^ (y << 6)));
}
// Along the columns, 16 of them: rows 4 g + (0..3) and 16 + 4 g + (0..3).  Four columns that lie
// together go to lanes that do; `chunk` and `byte` say where lane j & 3's four are.
template <int P>
__device__ __forceinline__ int lin_col_at(int chunk, int byte) {
  const int lane = threadIdx.x & 63, r = 4 * (lane >> 4) + ((lane & 15) >> 2);
  return r * P + ((chunk ^ lin_swz<P>(r)) << 4) + byte;
}
template <int P>
__device__ __forceinline__ bf16x8 lin_col(const char* tile, int at) {
  s16x4 x[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    x[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(tile + 16 * i * P + at));
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7));
}

__device__ __forceinline__ f32x4 lin_mma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
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
__device__ __forceinline__ double lin_power64(float a, int n) {
  double p = 1.0, x = (double)a;
  for (; n; n >>= 1) {
    if (n & 1) p *= x;
    x *= x;
  }
  return p;
}
__device__ __forceinline__ float lin_power(float a, int n) { return (float)lin_power64(a, n); }

// The state's factor for each whole chunk, a^LIN_C: of the two fp32 numbers around it, each as often as keeps
// their product within one step of a's power.  The nearer one alone is off to the same side at every chunk (the
// state 1.6e-5 after 131072 tokens at a decay of 1 - 2^-16, 4e-6 after 32768 at 1 - 2^-12).
struct LinDecay {
  uint32_t lower, share, sum;   // the number nearer to 0; the other's share of the chunks, of 2^32; and its sum so far
  __device__ __forceinline__ void init(float a) {
    const double p = lin_power64(a, LIN_C);
    uint32_t u = __builtin_bit_cast(uint32_t, (float)p);
    if (fabs((double)(float)p) > fabs(p)) --u;
    const double x = (double)__builtin_bit_cast(float, u), step = fabs((double)__builtin_bit_cast(float, u + 1) - x);
    lower = lin_scalar(u);
    // the step is a power of 2, and what p is past x is less; no share where the decay is not finite
    share = lin_scalar(step < INFINITY ? (uint32_t)__builtin_ldexp(fabs(p - x), 33 - __builtin_amdgcn_frexp_exp(step)) : 0u);
    sum = 1u << 31;
  }
  __device__ __forceinline__ float next() {
    sum += share;
    return __builtin_bit_cast(float, lower + (sum < share));
  }
};

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

// The state of a wave, 16 columns: element e of tile 2 y + t is row 32 y + 8 g + 4 t + e, column j.  fp32 in
// accumulators over a whole segment.  As an operand it is two bf16 parts, 16 bits of what out, which has 8, is made
// of: 0.3 % of out's roundings go the other way than with fp32 products (1e-4 of its norm), its error against 64 bits
// is the same 1.66e-3.  Three parts would be half as many products again.
template <int DA>
struct LinState {
  static constexpr int P = DA * 2, N = DA / 16;
  f32x4 s[N];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  __device__ __forceinline__ void decay(float f) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] *= f;
  }
  // rows 32 y .. + 31 as an operand, in two bf16 parts
  __device__ __forceinline__ void parts(int y, bf16x8 (&p)[2]) const {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = s[2 * y + (e >> 2)][e & 3];
    lin_split(x, p);
  }
  // 32 tokens of the wave's columns of v by their weights
  static __device__ __forceinline__ void weigh(bf16x8 vf, const float* wt, int g, float (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4 t = *reinterpret_cast<const f32x4*>(wt + 16 * i + 4 * g);
      const u32x4 u = __builtin_bit_cast(u32x4, vf);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        w[4 * i + 2 * e] = lin_first(u[2 * i + e]) * t[2 * e];
        w[4 * i + 2 * e + 1] = lin_second(u[2 * i + e]) * t[2 * e + 1];
      }
    }
  }
  // s += k^T (w v) over a chunk; vf: the wave's columns of v.  w v enters as two bf16 numbers, or as
  // three.  at: lane j & 3's columns of k are 8 (j & 3) .. + 3, of every 32.
  __device__ __forceinline__ void add(const char* k, int at, const bf16x8 (&vf)[LIN_C / 32], const float* wt, int g,
                                      bool three) {
#pragma unroll
    for (int z = 0; z < LIN_C / 32; ++z) {
      float w[8];
      weigh(vf[z], wt + 32 * z, g, w);
      bf16x8 wp[2], rest[1];
      lin_split(w, wp);
      if (three) lin_split(w, rest);
      // four tiles in turn: a product that goes on with the last one's result waits for it
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        bf16x8 kf[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) kf[t] = lin_col<P>(k + 32 * z * P, (at ^ (((i + t) >> 1) << 6)) + 8 * (t & 1));
#pragma unroll
        for (int t = 0; t < 4; ++t) s[i + t] = lin_mma(kf[t], wp[0], s[i + t]);
#pragma unroll
        for (int t = 0; t < 4; ++t) s[i + t] = lin_mma(kf[t], wp[1], s[i + t]);
        if (three)
#pragma unroll
          for (int t = 0; t < 4; ++t) s[i + t] = lin_mma(kf[t], rest[0], s[i + t]);
      }
    }
  }
  __device__ __forceinline__ void store(float* p, int ld, int g, float f) const {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *as_global(p + (int64_t)(16 * (i & ~1) + 8 * g + 4 * (i & 1) + e) * ld) = s[i][e] * f;
  }
};

// A workgroup walks one segment of one sequence, head and role, 64 tokens at a time; its NW waves hold 16
// columns of the state each, all DA rows of it, as accumulators.  The output is computed transposed
// (a lane is a token), so that the accumulators of the state and of the scores are the operands of the
// products that follow as they lie.  The scores' ten tiles of 16 x 16 are spread over the waves, which
// leave them, decayed and split, in LDS for all: the barrier that they need is there for v.
//
// A wave's matrix and vector instructions do not run side by side, those of two waves do (4 products
// and 24 multiplications: 120 ns of one wave, 70 a wave of two): many narrow waves, at the price of
// reading q and k from LDS for each.  A SIMD holds four of them at key dimensions of 64 and 128 with eight
// waves to a workgroup, three at 64 x 64, two at 128 x 64 and at 256, one at 256 x 64: what LDS and
// registers leave.  Columns of 32 a wave, half as many to a SIMD, were as fast on long sequences (131072
// tokens of 8 heads of 128: 403 us, 417 so) and slower on the others (24 ragged prompts 198 -> 182, a training
// step of 3 x 777 tokens 79 -> 75).  What bounds the long ones: loads and
// stores alone take 223 us of this kernel there, its work without loads 238, both 310; the matrix cores
// are busy 31 % of the cycles, the vector units 42, the LDS 44, at 1.6 to 1.9 GHz: four waves of a SIMD
// that each wait for their own chain of products, and power; neither another order of the instructions
// nor a deeper ring of loads nor fewer LDS conflicts changed the time.
//
// Four areas of LDS take turns: while q, k and v of a chunk lie in three, the next chunk's q comes into
// the fourth; once q has been read its k comes into q's, and once all has been read its v into k's.  Three
// stages of whole chunks, two of them under way, gain nothing even where a workgroup has a CU to itself
// (one prompt of 512 tokens of 8 heads: 34.7 us, 36.0 so): a chunk's chain of products is what takes the time.
template <int DA, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(DA == 256 ? 2 : 4)))
void k_linear(LinArgs a) {
  constexpr int PA = DA * 2, PV = NW * 32;                    // bytes of a tile's row
  constexpr int AREA = LIN_C * (PA > PV ? PA : PV), Y = DA / 32;
  __shared__ __attribute__((aligned(1024))) char a0[AREA];
  __shared__ __attribute__((aligned(1024))) char a1[AREA];
  __shared__ __attribute__((aligned(1024))) char a2[AREA];
  __shared__ __attribute__((aligned(1024))) char a3[AREA];
  // [queries of 16 with keys of 32: 0 0, 1 0, 2 0, 2 1, 3 0, 3 1][part][lane][keys of 16]
  __shared__ __attribute__((aligned(1024))) u32x2 scores[6][2][64][2];
  __shared__ __attribute__((aligned(16))) LinTables tb;
  const LinPlace at(a, a.nseg, xcd_block(blockIdx.x, a.total), true);
  if (at.none) return;
  const LinRole& r = at.r;
  const int rev = lin_scalar(r.rev), h = at.h, b = at.b;
  const int len = lin_scalar(at.len), t0 = at.t0, cnt = lin_scalar(at.cnt), chunks = lin_scalar(at.chunks);
  const float scale_p = lin_scalar(r.scale_p), scale_s = lin_scalar(r.scale_s);
  const int lane = threadIdx.x & 63, g = lane >> 4, j = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const float lam = a.decay[h];

  const int col0 = at.slice * 16 * NW;                       // the workgroup's first column
  auto size = [&](int c) __attribute__((always_inline)) { return max(0, min(LIN_C, cnt - c * LIN_C)); };
  LinLoad<PA, NW> lq, lk;
  LinLoad<PV, NW> lv;
  {
    const int64_t first = at.row0 + (rev ? len - t0 - size(0) : t0);
    const int nt = lin_scalar(a.nt);
    lq.init(r.q + (int64_t)h * DA, r.ldq, first, rev, nt);
    lk.init(r.k + (int64_t)h * DA, r.ldk, first, rev, nt);
    lv.init(r.v + (int64_t)h * a.DB + col0, r.ldv, first, rev, nt);
  }
  auto load_q = [&](char* p, int c) __attribute__((always_inline)) { lq.issue(p, size(c), size(c + 1)); };
  auto load_k = [&](char* p, int c) __attribute__((always_inline)) { lk.issue(p, size(c), size(c + 1)); };
  auto load_v = [&](char* p, int c) __attribute__((always_inline)) { lv.issue(p, size(c), size(c + 1)); };
  if (chunks) {
    load_q(a0, 0);
    load_k(a1, 0);
    load_v(a2, 0);
  }
  tb.init(lam, at);
  LinDecay chunk_decay;
  chunk_decay.init(lam);
  if (wave < 2) scores[0][wave][lane][1] = scores[3][wave][lane][1] = u32x2{0, 0};   // keys behind all of the queries

  const int64_t elems = (int64_t)DA * a.DB;
  const int colw = col0 + 16 * wave + j;
  const int64_t entry = lin_slot(a.slot, b, a.slots);
  LinState<DA> S;
  float* fin = nullptr;
  if (r.fin && entry >= 0 && t0 + a.L >= len) fin = r.fin + (entry * a.heads + h) * elems + colw;
  const float* init = nullptr;
  if (r.ws) init = r.ws + (((int64_t)b * a.heads + h) * a.nseg + at.seg) * elems;
  else if (r.init && entry >= 0) init = r.init + (entry * a.heads + h) * elems;
  S.clear();
  if (init) {
#pragma unroll
    for (int i = 0; i < DA / 16; ++i) {
      const int x = 16 * (i & ~1) + 8 * g + 4 * (i & 1);
      if (r.trans) {
        S.s[i] = *as_global(reinterpret_cast<const f32x4*>(init + (int64_t)colw * DA + x));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) S.s[i][e] = *as_global(init + (int64_t)(x + e) * a.DB + colw);
      }
    }
  }
  const int ra = lin_row_at<PA>();
  const int ka_at = lin_col_at<PA>(j & 3, 0), va_at = lin_col_at<PV>(2 * wave + ((j & 3) >> 1), 8 * (j & 1));
  lin_wait<0>();

  u32x4 ow[2];   // a chunk's output: 8 elements from 8 (g / 2) of token 16 (2 i + g % 2) + j
  // the workgroup's columns of the next chunk's first token, and the lane's place from there
  char* op = lin_scalar(reinterpret_cast<char*>(r.out + (at.row0 + (rev ? len - 1 - t0 : t0)) * r.ldo + (int64_t)h * a.DB + col0));
  const int32_t ldo2 = lin_scalar((int32_t)(rev ? -r.ldo : r.ldo) * 2);
  const int32_t ox = 16 * (g & 1) + j, oc = 32 * wave + 16 * (g >> 1);
  auto store = [&](int c) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (32 * i + ox < size(c)) *as_global(reinterpret_cast<u32x4*>(op + (int64_t)((32 * i + ox) * ldo2 + oc))) = ow[i];
    op += (int64_t)LIN_C * ldo2;
  };
  auto step = [&](char* qa, char* ka, char* va, char* spare, int c) __attribute__((always_inline)) {
    const int n = size(c);
    const bool more = c + 1 < chunks;
    if (more) load_q(spare, c + 1);
    // backward in time the state before the first token (the gradient of the last state) is that
    // of the first token itself: one power less
    const int e0 = rev && t0 + c == 0 ? 0 : 1;
    for (int tile = wave; tile < 10; tile += NW) {
      const int qi = tile >= 6 ? 3 : tile >= 3 ? 2 : tile >= 1 ? 1 : 0, ki = tile - qi * (qi + 1) / 2;
      f32x4 p = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int y = 0; y < Y; ++y)
        p = lin_mma(lin_row(ka + 16 * ki * PA, ra, y), lin_row(qa + 16 * qi * PA, ra, y), p);
      float pv[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {   // query j of 16, key 4 g + e
        const int d = 16 * (qi - ki) + j - 4 * g - e;
        pv[e] = d >= 0 ? p[e] * (tb.pw[d >= 0 ? d : 0] * scale_p) : 0.f;
      }
      u32x2 hi = u32x2{lin_pack(pv[0], pv[1]), lin_pack(pv[2], pv[3])};
      const u32x2 lo = u32x2{lin_pack(pv[0] - lin_first(hi[0]), pv[1] - lin_second(hi[0])),
                             lin_pack(pv[2] - lin_first(hi[1]), pv[3] - lin_second(hi[1]))};
      const int at = qi < 2 ? qi : 2 * qi - 2 + (ki >> 1);
      scores[at][0][lane][ki & 1] = hi;
      scores[at][1][lane][ki & 1] = lo;
    }
    f32x4 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int y = 0; y < Y; ++y) {
      bf16x8 sp[2];
      S.parts(y, sp);
      bf16x8 qf[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) qf[i] = lin_row(qa + 16 * i * PA, ra, y);
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = lin_mma(sp[x], qf[i], o[i]);
    }
    if (more) lin_wait<LinLoad<PA, NW>::N>();   // v and the scores are there, q is free
    else lin_wait<0>();
    if (more) load_k(qa, c + 1);
    bf16x8 vf[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) vf[z] = lin_col<PV>(va + 32 * z * PV, va_at);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= tb.pw[16 * i + j + e0] * scale_s;
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 2 * z; i < 4; ++i)
          o[i] = lin_mma(vf[z], *reinterpret_cast<const bf16x8*>(scores[i < 2 ? i : 2 * i - 2 + z][x][lane]), o[i]);
    S.decay(n - 1 + e0 == LIN_C ? chunk_decay.next() : tb.pw[n - 1 + e0]);
    S.add(ka, ka_at, vf, tb.wt[more ? 0 : 1], g, fin != nullptr);
    // rows of 16 lanes swapped in pairs: 8 neighbouring elements of a token in a lane
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const auto w = __builtin_amdgcn_permlane16_swap(lin_pack(o[2 * i][2 * e], o[2 * i][2 * e + 1]),
                                                        lin_pack(o[2 * i + 1][2 * e], o[2 * i + 1][2 * e + 1]), false, false);
        ow[i][e] = w[0];
        ow[i][2 + e] = w[1];
      }
    lin_wait<0>();   // the next chunk's q and k are there, k and v are free
    if (more) load_v(ka, c + 1);
    store(c);
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
    S.store(fin, a.DB, g, rev && len > 0 ? lam : 1.f);
}

// Each segment's own sum, from zeros, of all but the last.
template <int DA, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(DA == 256 ? 2 : 4)))
void k_linear_states(LinArgs a) {
  constexpr int PA = DA * 2, PV = NW * 32, VO = LIN_C * PA;
  __shared__ __attribute__((aligned(1024))) char st0[LIN_C * (PA + PV)];
  __shared__ __attribute__((aligned(1024))) char st1[LIN_C * (PA + PV)];
  __shared__ __attribute__((aligned(16))) LinTables tb;
  const LinPlace at(a, a.nseg - 1, xcd_block(blockIdx.x, a.total), false);
  if (at.none) return;
  const LinRole& r = at.r;
  const int rev = lin_scalar(r.rev), lane = threadIdx.x & 63, g = lane >> 4, j = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int col0 = at.slice * 16 * NW;
  const int chunks = lin_scalar(at.chunks);
  const bool three = lin_scalar(r.fin) != nullptr;
  LinLoad<PA, NW> lk;
  LinLoad<PV, NW> lv;
  {
    const int64_t first = at.row0 + (rev ? at.len - at.t0 - LIN_C : at.t0);   // every chunk is whole
    const int nt = lin_scalar(a.nt);
    lk.init(r.k + (int64_t)at.h * DA, r.ldk, first, rev, nt);
    lv.init(r.v + (int64_t)at.h * a.DB + col0, r.ldv, first, rev, nt);
  }
  auto load = [&](char* st) __attribute__((always_inline)) {
    lk.issue(st, LIN_C, LIN_C);
    lv.issue(st + VO, LIN_C, LIN_C);
  };
  load(st0);
  const float lam = a.decay[at.h];
  tb.init(lam, at);
  LinDecay chunk_decay;
  chunk_decay.init(lam);
  LinState<DA> S;
  S.clear();
  const int ka_at = lin_col_at<PA>(j & 3, 0), va_at = lin_col_at<PV>(2 * wave + ((j & 3) >> 1), 8 * (j & 1));
  int c = 0;
  auto step = [&](const char* cur, char* free) __attribute__((always_inline)) {
    lin_wait<0>();
    if (c + 1 < chunks) load(free);
    bf16x8 vf[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) vf[z] = lin_col<PV>(cur + VO + 32 * z * PV, va_at);
    S.decay(chunk_decay.next());
    S.add(cur, ka_at, vf, tb.wt[0], g, three);
    ++c;
  };
  while (c < chunks) {
    step(st0, st1);
    if (c == chunks) break;
    step(st1, st0);
  }
  S.store(r.ws + (((int64_t)at.b * a.heads + at.h) * a.nseg + at.seg) * DA * a.DB + col0 + 16 * wave + j, a.DB, g, 1.f);
}

// From the segments' own sums to the states before each: a thread takes four elements of a state
// along the segments.  The decay over a segment is two fp32 numbers, so that it does not drift over many.
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
  const float lam = a.decay[h];
  const double p = lin_power64(lam, a.L), p0 = r.rev ? lin_power64(lam, a.L - 1) : p;
  const float f = (float)p, low = (float)(p - (double)f);
  float f0 = (float)p0, low0 = (float)(p0 - (double)f0);
  for (int i = 0; i < cnt; i += 8) {
    f32x4 x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      x[j] = i + j < cnt - 1 ? *as_global(reinterpret_cast<const f32x4*>(w + (i + j) * elems)) : f32x4{};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < cnt) {
        *as_global(reinterpret_cast<f32x4*>(w + (i + j) * elems)) = s;
        s = s * f0 + (s * low0 + x[j]);
        f0 = f;
        low0 = low;
      }
  }
}

template <int DA>
hipError_t launch_nw(const LinArgs& a, int NW, bool out, hipStream_t st) {
  const dim3 grid(a.total), block(64 * NW);
  if (out && NW == 4) hipLaunchKernelGGL((k_linear<DA, 4>), grid, block, 0, st, a);
  else if (out) hipLaunchKernelGGL((k_linear<DA, 8>), grid, block, 0, st, a);
  else if (NW == 4) hipLaunchKernelGGL((k_linear_states<DA, 4>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_linear_states<DA, 8>), grid, block, 0, st, a);
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
