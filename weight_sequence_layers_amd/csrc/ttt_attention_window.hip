// The window attention's training form (include/ttt_attention.h): the forward that also gives
// each row's log-sum-exp, and the backward.
//
// Mathematics, with c = 1 / sqrt(128), p = exp(c q k - lse), dp = dout . v, delta = dout . out:
//   out = sum_j p v_j,
//   ds = p (dp - delta),  dq = c sum_j ds k_j,  dk = c sum_t ds q_t,  dv = sum_t p dout_t.
//
// The backward is two launches, each recomputing p and dp, so that every sum is one workgroup's
// in one order and nothing is added by atomics: seven products of 2 * 128 operations per (query,
// key) pair for the five that the formulas need.  The first takes 128 queries per workgroup and
// runs over their keys (dq, and delta for the second), as the forward does; the second takes 128
// keys and runs over their queries (dk, dv).  Four waves hold 32 queries (keys) each: the operand
// that stays (q and dout; k) in registers as MFMA fragments, the one that passes by (k and v; q
// and dout) in LDS tiles, loaded one step ahead.  The scores are computed transposed, so that a
// lane's elements are the B operand of the product that follows; k (or q and dout) is read from
// the same tile both along its rows and, transposed, along its columns.
//
// p and ds enter their products as one bf16 number each, ds with the delta of the rounded out (but
// see SUM below); scores, exponentials, statistics and sums are fp32. That is a choice: against 64
// bits out is 2.3e-3 of its norm off and the gradients 2.4e-3, where rounding the exact values to
// bf16 gives 1.65e-3. Two bf16 numbers apiece reach that (1.65e-3, 1.68e-3) and take a training
// step at 32768 tokens from 1190 to 1600 us, the forward in it from 288 to 384: the matrix cores
// take no mixed operands, and fp16 does not hold the range of v, k, q and dout.
//
// Measured at 32768 tokens, 8 heads, a sliding window of 2048, in a run of 180 steps: forward
// 294 us, backward 385 and 513 us, the step 1192; 906, 1037 and 1038 TFLOP/s of the products made
// (the largest library product of this card, 8192 cubed, runs at 1160 to 1200). The first
// launches after a pause take up to a third longer. The matrix cores are busy 49, 59 and 55 % of
// the cycles, the LDS 25, 30 and 41 %, at a clock of 1.6 to 1.7 GHz (2.1 to 2.2 where the memory
// bounds): power is what bounds them, and filling more of the cycles gains little. The forward
// with the next step's scores computed beside this step's exponentials, in the same wave: 315 to
// 320 us against 317 in turn.
#include "ttt_attention_internal.h"

namespace ttt {
namespace {

constexpr int WB_ROWS = 64;                    // rows of a tile
constexpr int WB_TILE = WB_ROWS * ATT_D * 2;   // bytes
constexpr int64_t WB_FEW = 256;                // workgroups: one per CU

// A tile keeps chunk c (16 bytes) of row r at chunk c ^ wb_swz(r) of the row: any 16
// consecutive rows at one chunk, and the two chunks of 32 dims over 4 consecutive rows, lie on
// distinct banks, so that both ways of reading it are free of conflicts.
__device__ __forceinline__ int wb_swz(int r) { return ((r & 3) << 2) | ((r >> 2) & 3); }

// Loads of a tile, straight into LDS, 16 rows at a time: the lanes' places in them are the same
// each time (the swizzle depends on a row's number modulo 16).
struct WbLoad {
  uint32_t off, ld2;   // byte offset of the lane's place, bytes of a row
  int slice;
  __device__ __forceinline__ void init(int64_t ld) {
    const int tid = threadIdx.x, r = tid >> 4;
    ld2 = (uint32_t)(ld * 2);
    off = (uint32_t)r * ld2 + (uint32_t)(((tid & 15) ^ wb_swz(r)) << 4);
    slice = __builtin_amdgcn_readfirstlane(tid >> 6) * 1024;
  }
  // ROWS rows at p, of which the first `rows` (> 0) are there: the others read as 0
  template <int ROWS>
  __device__ __forceinline__ void issue(char* tile, const u16* p, int rows) const {
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void*)p, (short)0, (int)((uint32_t)min(rows, ROWS) * ld2), 0x00020000);
#pragma unroll
    for (int c = 0; c < ROWS / 16; ++c)
      dma16(rs, (lds_void_t*)(tile + c * 4096 + slice), off + c * 16 * ld2);
  }
};

// Offsets of a lane's fragments in a tile.  Every fragment's offset is one of two bases with a
// constant added (rows) and one xored in (chunks).
struct WbAt {
  int row;   // along the rows: row lane % 32, dims 8 (lane / 32) .. + 7
  int col;   // along the columns: dims 16 (g & 1) + 4 (j & 3) .. + 3 of row 4 (g / 2) + j / 4
  __device__ __forceinline__ void init() {
    const int lane = threadIdx.x & 63, r = lane & 31;
    const int g = lane >> 4, j = lane & 15;
    row = r * (ATT_D * 2) + (((lane >> 5) ^ wb_swz(r)) << 4);
    const int m = 16 * (g & 1) + 4 * (j & 3), rc = 4 * (g >> 1) + (j >> 2);
    col = rc * (ATT_D * 2) + (((m >> 3) ^ wb_swz(rc)) << 4) + (m & 7) * 2;
  }
};

// Fragment along the rows: row row_base + lane % 32, dims 16 s + 8 (lane / 32) .. + 7.
// row_base a multiple of 32.
__device__ __forceinline__ bf16x8 wb_row(const char* tile, const WbAt& at, int row_base, int s) {
  return *reinterpret_cast<const bf16x8*>(tile + row_base * (ATT_D * 2) + (at.row ^ (s << 5)));
}
// Fragment along the columns: dim dim_base + lane % 32, rows row_base + 4 (lane / 32) + (0..3)
// and + 8.  dim_base a multiple of 32, row_base of 16; 8 rows further the swizzle has bit 1 of
// the chunk turned.
__device__ __forceinline__ bf16x8 wb_col(const char* tile, const WbAt& at, int dim_base, int row_base) {
  s16x4 x[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const char* p = tile + (row_base + 8 * i) * (ATT_D * 2) + (at.col ^ (dim_base << 1) ^ (i << 5));
    x[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p));
  }
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  const s16x8 v = __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(bf16x8, v);
}

__device__ __forceinline__ f32x16 wb_mma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Orders the instructions of a stretch of straight-line code: n of a kind next.  Left alone the
// compiler loads each fragment right before its product and waits for LDS every time.
#define WB_ORDER(kind, n) __builtin_amdgcn_sched_group_barrier(kind, n, 0)
constexpr int WB_VALU = 0x2, WB_MFMA = 0x8, WB_DS = 0x100;

// a row's 64 values of this lane: dims 16 s + 8 hl .. + 7
__device__ __forceinline__ void wb_frags(bf16x8 (&f)[8], const u16* row, int hl, bool in) {
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    if (in) f[s] = *reinterpret_cast<const bf16x8*>(row + 16 * s + 8 * hl);
    else f[s] = bf16x8{};
  }
}

// dims 32 d + 8 (v / 4) + 4 hl + v % 4 of a row, times f
__device__ __forceinline__ void wb_store(u16* row, const f32x16 (&o)[4], float f, int hl) {
#pragma unroll
  for (int d = 0; d < 4; ++d)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint2 x;
      x.x = f2bf(o[d][4 * g] * f) | ((uint32_t)f2bf(o[d][4 * g + 1] * f) << 16);
      x.y = f2bf(o[d][4 * g + 2] * f) | ((uint32_t)f2bf(o[d][4 * g + 3] * f) << 16);
      *reinterpret_cast<uint2*>(row + 32 * d + 8 * g + 4 * hl) = x;
    }
}

// With TTT_WINDOW_BLOCK the rows of a workgroup start at multiples of their number, not of the
// window: one that straddles a boundary walks both windows, and the forward and dq compute steps
// that are masked for all of a wave (windows of 250: up to 8 steps of 64 keys for 4).
//
// The keys that a workgroup's queries q0 .. qlast visit, [lo, lo + nsteps tiles), those of its
// wave at w0 that every one of its queries sees, [in_lo, in_hi) (empty for a wave of padding
// rows: a step wholly inside needs no mask), and the lane's query t's own, lo_t and len_t of them
// (none for a padding row).
struct WbKeys {
  int lo, nsteps, in_lo, in_hi, lo_t, len_t;
  __device__ __forceinline__ WbKeys(const WindowArgs& a, int q0, int qlast, int w0, int t) {
    const int T = a.T, W = a.window, wl = min(w0 + 31, T - 1);
    int hi, hi_t;
    if (a.mode == TTT_WINDOW_SLIDING) {
      lo = max(0, q0 - W + 1);
      hi = qlast + 1;
      lo_t = t - W + 1;
      hi_t = t + 1;
      in_lo = wl - W + 1;
      in_hi = w0 + 1;
    } else {
      lo = (q0 / W) * W;
      hi = (int)min<int64_t>(T, ((int64_t)(qlast / W) + 1) * W);
      lo_t = (t / W) * W;
      hi_t = (int)min<int64_t>(T, (int64_t)lo_t + W);
      in_lo = (wl / W) * W;
      in_hi = (int)min<int64_t>(T, ((int64_t)(w0 / W) + 1) * W);
    }
    // uniform values that come out of vector arithmetic (the divisions), back in scalar
    // registers: a buffer resource made of vector registers takes a loop over the lanes for
    // every load
    lo = __builtin_amdgcn_readfirstlane(lo);
    hi = __builtin_amdgcn_readfirstlane(hi);
    in_lo = __builtin_amdgcn_readfirstlane(in_lo);
    in_hi = __builtin_amdgcn_readfirstlane(in_hi);
    if (t >= T) lo_t = hi_t = 0;
    if (w0 >= T) {
      in_lo = 1;
      in_hi = 0;
    }
    len_t = hi_t - lo_t;
    nsteps = (hi - lo + WB_ROWS - 1) / WB_ROWS;
  }
};

// The second halves' sums added to the first halves' (waves w and w + 2 hold the same rows),
// 32 KB through buf.  Call from every wave.
__device__ __forceinline__ void wb_join(f32x16 (&o)[4], int w, int half, char* buf) {
  const int lane = threadIdx.x & 63;
  __syncthreads();   // buf has been read
  auto at = [&](int d, int v) __attribute__((always_inline)) {
    return reinterpret_cast<float*>(buf) + ((w * 4 + d) * 16 + v) * 64 + lane;
  };
  if (half)
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int v = 0; v < 16; ++v) *at(d, v) = o[d][v];
  __syncthreads();
  if (!half)
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int v = 0; v < 16; ++v) o[d][v] += *at(d, v);
}

// NH 1: the four waves take 32 rows each, 128 to a workgroup.  NH 2, for launches of at most
// WB_FEW workgroups of 64 rows: 64 rows to a workgroup and two waves to each 32, which take half
// of every step's tile and are joined at the end: twice the workgroups, and half the products in
// each SIMD's chain of steps, which is what such a launch waits for (one head of 1024 tokens: dq
// 29 -> 20 us, dk and dv 42 -> 26; eight waves over 128 rows gain nothing).  WB_FEW is one
// workgroup to a CU. The rule leaves time where it ends: 8 heads, a window of 2048, take 110 us a
// training step at 2048 tokens (256 blocks of 64) and 173 at 2112, where NH 1 launches 136
// workgroups on 256 CUs.
//
// Forward with each row's log-sum-exp.  The running maximum that the exponentials refer to moves
// only when a score passes it by more than 2^8: the sums stay far inside fp32, the rounding of
// the probabilities to bf16 is relative, and the 64 sums of a lane are rescaled in the first
// steps only instead of in nearly every one (a maximum over 64 more scores moves for some row
// of 32 nearly always).  The normaliser sums the probabilities before they are rounded, as the
// log-sum-exp has to.
template <int NH>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2)))
void k_window_fwd(WindowArgs a) {
  constexpr int RG = 4 / NH, QB = 32 * RG;   // row groups, queries of a workgroup
  __shared__ __attribute__((aligned(1024))) char st0[2 * WB_TILE];
  __shared__ __attribute__((aligned(1024))) char st1[2 * WB_TILE];
  const int id = xcd_block(blockIdx.x, a.total);
  const int qb = __builtin_amdgcn_readfirstlane(id % a.blocks);
  const int bh = __builtin_amdgcn_readfirstlane(id / a.blocks);
  const int b = __builtin_amdgcn_readfirstlane(bh / a.heads), h = bh - b * a.heads;
  const int lane = threadIdx.x & 63, hl = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int w = wave % RG, half = wave / RG;
  const int T = a.T;
  const int q0 = qb * QB, w0 = q0 + 32 * w;
  const int t = w0 + (lane & 31);
  const WbKeys r(a, q0, min(q0 + QB, T) - 1, w0, t);

  const int64_t row0 = (int64_t)b * T;
  const u16* kb = a.k + row0 * a.ld + (int64_t)h * ATT_D;
  const u16* vb = a.v + row0 * a.ld + (int64_t)h * ATT_D;
  WbLoad lk;
  lk.init(a.ld);
  const u16 *kp = kb + (int64_t)r.lo * a.ld, *vp = vb + (int64_t)r.lo * a.ld;   // the next step's rows
  const int64_t adv = WB_ROWS * a.ld;
  auto issue = [&](char* st, int rows) __attribute__((always_inline)) {
    lk.issue<WB_ROWS>(st, kp, rows);
    lk.issue<WB_ROWS>(st + WB_TILE, vp, rows);
    kp += adv;
    vp += adv;
  };
  issue(st0, T - r.lo);

  bf16x8 qf[8];
  wb_frags(qf, a.q + (row0 + t) * a.ld + (int64_t)h * ATT_D, hl, t < T);
  WbAt at;
  at.init();
  f32x16 o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = f32x16{};
  float m = -INFINITY, l = 0.f;

  auto step = [&](const char* cur, char* nxt, int i) __attribute__((always_inline)) {
    const int kv0 = r.lo + i * WB_ROWS;
    if (i + 1 < r.nsteps) issue(nxt, T - kv0 - WB_ROWS);
    constexpr int N = 2 / NH;                    // halves of this wave
    const int r0 = NH == 1 ? 0 : 32 * half;      // its first row of the tile
    f32x16 s[N];
#pragma unroll
    for (int kt = 0; kt < N; ++kt) s[kt] = f32x16{};
    if (kv0 < r.in_lo || kv0 + WB_ROWS > r.in_hi) {   // the mask as the scores' first summand
#pragma unroll
      for (int kt = 0; kt < N; ++kt) {
        const int base = kv0 + r0 + 32 * kt + 4 * hl - r.lo_t;
#pragma unroll
        for (int v = 0; v < 16; ++v)
          s[kt][v] = (unsigned)(base + 8 * (v >> 2) + (v & 3)) < (unsigned)r.len_t ? 0.f : -INFINITY;
      }
    }
#pragma unroll
    for (int x = 0; x < 8; ++x)
#pragma unroll
      for (int kt = 0; kt < N; ++kt) s[kt] = wb_mma(wb_row(cur, at, r0 + 32 * kt, x), qf[x], s[kt]);
    if constexpr (NH == 1) {
      WB_ORDER(WB_DS, 4);
#pragma unroll
      for (int x = 0; x < 12; ++x) {
        WB_ORDER(WB_MFMA, 1);
        WB_ORDER(WB_DS, 1);
      }
      WB_ORDER(WB_MFMA, 4);
    }
    // a wave past its scores goes before the SIMD's other one (354 -> 340 us with the order above)
    __builtin_amdgcn_s_setprio(1);
    float mx = -INFINITY;
#pragma unroll
    for (int kt = 0; kt < N; ++kt)
#pragma unroll
      for (int v = 0; v < 16; ++v) mx = fmaxf(mx, s[kt][v]);
    mx = fmaxf(mx, __shfl_xor(mx, 32)) * a.scale2;
    if (__any(mx > m + 8.f)) {   // wave-uniform
      const float mnew = fmaxf(m, mx);
      const float alpha = __builtin_amdgcn_exp2f(m - (mnew == -INFINITY ? 0.f : mnew));
      l *= alpha;
#pragma unroll
      for (int d = 0; d < 4; ++d)
#pragma unroll
        for (int v = 0; v < 16; ++v) o[d][v] *= alpha;
      m = mnew;
    }
    const float mref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int kt = 0; kt < N; ++kt)
#pragma unroll
      for (int sp = 0; sp < 2; ++sp) {
        bf16x8 pf;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float p = __builtin_amdgcn_exp2f(fmaf(s[kt][8 * sp + e], a.scale2, -mref));
          l += p;
          pf[e] = static_cast<__bf16>(p);
        }
#pragma unroll
        for (int d = 0; d < 4; ++d)
          o[d] = wb_mma(wb_col(cur + WB_TILE, at, 32 * d, r0 + 32 * kt + 16 * sp), pf, o[d]);
      }
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
  };
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  int i = 0;
  for (; i + 1 < r.nsteps; i += 2) {
    step(st0, st1, i);
    step(st1, st0, i + 1);
  }
  if (i < r.nsteps) step(st0, st1, i);

  l += __shfl_xor(l, 32);
  if constexpr (NH == 2) {   // to one reference, then the halves' sums together
    float* ms = reinterpret_cast<float*>(st1);
    if (lane < 32) {
      ms[32 * wave + lane] = m;
      ms[128 + 32 * wave + lane] = l;
    }
    __syncthreads();
    const int other = 32 * (w + RG * (1 - half)) + (lane & 31);
    const float mo = ms[other], mt = fmaxf(m, mo), mtr = mt == -INFINITY ? 0.f : mt;
    const float f = __builtin_amdgcn_exp2f(m - mtr);
    l = l * f + ms[128 + other] * __builtin_amdgcn_exp2f(mo - mtr);
    m = mt;
#pragma unroll
    for (int d = 0; d < 4; ++d)
#pragma unroll
      for (int v = 0; v < 16; ++v) o[d][v] *= f;
    wb_join(o, w, half, st0);
    if (half) return;
  }
  if (t < T) {
    wb_store(a.out + (row0 + t) * a.ldo + (int64_t)h * ATT_D, o, 1.f / l, hl);
    if (hl == 0) a.lse[((int64_t)b * a.heads + h) * T + t] = (m + log2f(l)) * 0.69314718055994531f;
  }
}

// First kernel of the backward.
//
// SUM: delta summed from p and dp in a walk of its own over the keys instead of from dout and
// out.  The rounding of out to bf16 moves delta by 2^-9 of |dout| |out|, which counts where a
// window holds few tokens and out is as long as they are: with it the gradients of a window of
// 2 are 1.7 times as far off as their own rounding alone, with the sum 1.4 times, as those of
// long windows are.  For windows of at most one step's keys, where the walk is short.
template <bool SUM, int NH>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2)))
void k_window_dq(WindowArgs a) {
  constexpr int RG = 4 / NH, QB = 32 * RG;   // row groups, queries of a workgroup
  __shared__ __attribute__((aligned(1024))) char st0[2 * WB_TILE];
  __shared__ __attribute__((aligned(1024))) char st1[2 * WB_TILE];
  const int id = xcd_block(blockIdx.x, a.total);
  const int qb = __builtin_amdgcn_readfirstlane(id % a.blocks);
  const int bh = __builtin_amdgcn_readfirstlane(id / a.blocks);
  const int b = __builtin_amdgcn_readfirstlane(bh / a.heads), h = bh - b * a.heads;
  const int lane = threadIdx.x & 63, hl = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int w = wave % RG, half = wave / RG;
  const int T = a.T;
  const int q0 = qb * QB, w0 = q0 + 32 * w;
  const int t = w0 + (lane & 31);

  const WbKeys r(a, q0, min(q0 + QB, T) - 1, w0, t);
  const int lo = r.lo, lo_t = r.lo_t, len_t = r.len_t, in_lo = r.in_lo, in_hi = r.in_hi, nsteps = r.nsteps;

  const int64_t row0 = (int64_t)b * T;
  const u16* kb = a.k + row0 * a.ld + (int64_t)h * ATT_D;
  const u16* vb = a.v + row0 * a.ld + (int64_t)h * ATT_D;
  WbLoad lk;
  lk.init(a.ld);
  const u16 *kp = kb + (int64_t)lo * a.ld, *vp = vb + (int64_t)lo * a.ld;   // the next step's rows
  const int64_t adv = WB_ROWS * a.ld;
  auto issue = [&](char* st, int rows) __attribute__((always_inline)) {
    lk.issue<WB_ROWS>(st, kp, rows);
    lk.issue<WB_ROWS>(st + WB_TILE, vp, rows);
    kp += adv;
    vp += adv;
  };
  issue(st0, T - lo);

  bf16x8 qf[8], gf[8];
  wb_frags(qf, a.q + (row0 + t) * a.ld + (int64_t)h * ATT_D, hl, t < T);
  wb_frags(gf, a.dout + (row0 + t) * a.lddo + (int64_t)h * ATT_D, hl, t < T);
  float delta = 0.f, lse2 = 0.f;
  const int64_t stat = ((int64_t)b * a.heads + h) * T + t;   // the row's place in lse and delta
  if (t < T) lse2 = a.lse[stat] * 1.44269504088896341f;
  if constexpr (!SUM) {
    const u16* orow = a.out + (row0 + t) * a.ldo + (int64_t)h * ATT_D;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      bf16x8 x = bf16x8{};
      if (t < T) x = *reinterpret_cast<const bf16x8*>(orow + 16 * s + 8 * hl);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        delta = fmaf(static_cast<float>(x[e]), static_cast<float>(gf[s][e]), delta);
    }
    delta += __shfl_xor(delta, 32);
  }

  WbAt at;
  at.init();
  f32x16 dq[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dq[i] = f32x16{};
  // Walks over the steps, each one's tiles loaded during the one before (the first's before the
  // call).
  auto walk = [&](auto work) __attribute__((always_inline)) {
    auto step = [&](const char* cur, char* nxt, int i) __attribute__((always_inline)) {
      if (i + 1 < nsteps) issue(nxt, T - lo - (i + 1) * WB_ROWS);
      work(cur, lo + i * WB_ROWS);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
    };
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    int i = 0;
    for (; i + 1 < nsteps; i += 2) {
      step(st0, st1, i);
      step(st1, st0, i + 1);
    }
    if (i < nsteps) step(st0, st1, i);
  };
  if constexpr (SUM) {
    walk([&](const char* cur, int kv0) __attribute__((always_inline)) {
#pragma unroll
      for (int kh = 0; kh < 2 / NH; ++kh) {
        const int kt = NH == 1 ? kh : half;
        f32x16 s = f32x16{}, dp = f32x16{};
#pragma unroll
        for (int x = 0; x < 8; ++x) s = wb_mma(wb_row(cur, at, 32 * kt, x), qf[x], s);
#pragma unroll
        for (int x = 0; x < 8; ++x) dp = wb_mma(wb_row(cur + WB_TILE, at, 32 * kt, x), gf[x], dp);
        const int base = kv0 + 32 * kt + 4 * hl - lo_t;
#pragma unroll
        for (int v = 0; v < 16; ++v)
          if ((unsigned)(base + 8 * (v >> 2) + (v & 3)) < (unsigned)len_t)
            delta = fmaf(__builtin_amdgcn_exp2f(fmaf(s[v], a.scale2, -lse2)), dp[v], delta);
      }
    });
    delta += __shfl_xor(delta, 32);
    if constexpr (NH == 2) {   // the halves' sums
      float* sum = reinterpret_cast<float*>(st1);
      if (lane < 32) sum[32 * wave + lane] = delta;
      __syncthreads();
      delta = sum[32 * w + (lane & 31)] + sum[32 * (w + RG) + (lane & 31)];
      __syncthreads();
    }
    kp = kb + (int64_t)lo * a.ld;
    vp = vb + (int64_t)lo * a.ld;
    issue(st0, T - lo);
  }
  if (t < T && hl == 0 && half == 0) a.delta[stat] = delta;
  walk([&](const char* cur, int kv0) __attribute__((always_inline)) {
    // The step's two halves run one behind the other, a half's exponentials beside the other's
    // products, in one stretch of straight-line code: the mask enters as the scores' first
    // summand.
    const bool edge = kv0 < in_lo || kv0 + WB_ROWS > in_hi;
    constexpr int N = 2 / NH;                    // halves of this wave
    const int r0 = NH == 1 ? 0 : 32 * half;      // its first row of the tile
    f32x16 s[N], dp[N];
    bf16x8 ds[N][2];
#pragma unroll
    for (int kt = 0; kt < N; ++kt) s[kt] = f32x16{};
    if (edge) {
#pragma unroll
      for (int kt = 0; kt < N; ++kt) {
        const int base = kv0 + r0 + 32 * kt + 4 * hl - lo_t;
#pragma unroll
        for (int v = 0; v < 16; ++v)
          s[kt][v] = (unsigned)(base + 8 * (v >> 2) + (v & 3)) < (unsigned)len_t ? 0.f : -INFINITY;
      }
    }
    auto scores = [&](int kt) __attribute__((always_inline)) {
      dp[kt] = f32x16{};
      const int row = r0 + 32 * kt;
#pragma unroll
      for (int x = 0; x < 8; ++x) s[kt] = wb_mma(wb_row(cur, at, row, x), qf[x], s[kt]);
#pragma unroll
      for (int x = 0; x < 8; ++x) dp[kt] = wb_mma(wb_row(cur + WB_TILE, at, row, x), gf[x], dp[kt]);
    };
    auto probs = [&](int kt) __attribute__((always_inline)) {
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const float p = __builtin_amdgcn_exp2f(fmaf(s[kt][v], a.scale2, -lse2));
        ds[kt][v >> 3][v & 7] = static_cast<__bf16>(p * (dp[kt][v] - delta));
      }
    };
    auto add = [&](int kt) __attribute__((always_inline)) {
#pragma unroll
      for (int sp = 0; sp < 2; ++sp)
#pragma unroll
        for (int d = 0; d < 4; ++d)
          dq[d] = wb_mma(wb_col(cur, at, 32 * d, r0 + 32 * kt + 16 * sp), ds[kt][sp], dq[d]);
    };
    scores(0);
    WB_ORDER(WB_DS, 4);
#pragma unroll
    for (int x = 0; x < 12; ++x) {
      WB_ORDER(WB_MFMA, 1);
      WB_ORDER(WB_DS, 1);
    }
    WB_ORDER(WB_MFMA, 4);
    if constexpr (NH == 2) {
      probs(0);
      add(0);
    } else {
      scores(1);
      probs(0);
      WB_ORDER(WB_DS, 4);
#pragma unroll
      for (int x = 0; x < 12; ++x) {
        WB_ORDER(WB_MFMA, 1);
        WB_ORDER(WB_VALU, 7);
        WB_ORDER(WB_DS, 1);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        WB_ORDER(WB_MFMA, 1);
        WB_ORDER(WB_VALU, 7);
      }
      add(0);
      probs(1);
      add(1);
      WB_ORDER(WB_DS, 6);
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        WB_ORDER(WB_MFMA, 1);
        WB_ORDER(WB_VALU, 13);
        WB_ORDER(WB_DS, 2);
      }
#pragma unroll
      for (int x = 0; x < 5; ++x) {
        WB_ORDER(WB_MFMA, 1);
        WB_ORDER(WB_DS, 2);
      }
      WB_ORDER(WB_MFMA, 3);
    }
  });
  if constexpr (NH == 2) {
    wb_join(dq, w, half, st0);
    if (half) return;
  }
  if (t < T) wb_store(a.dq + (row0 + t) * a.ldd + (int64_t)h * ATT_D, dq, a.scale, hl);
}

// The second kernel's queries come 32 for each half at a time: a stage is the tiles of q and
// dout, then the rows' lse and delta (64 places each: a load of a wave).  The workgroup's rows of
// v stay in LDS: with k and v both in registers beside the two sums it spills.
template <int NH>
struct WbStage {
  static constexpr int ROWS = 32 * NH, TILE = ROWS * ATT_D * 2, BYTES = 2 * TILE + 2 * 64 * 4;
};

template <int NH>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2)))
void k_window_dkv(WindowArgs a) {
  constexpr int RG = 4 / NH, KB = 32 * RG;   // row groups, keys of a workgroup
  constexpr int QROWS = WbStage<NH>::ROWS, QTILE = WbStage<NH>::TILE;
  __shared__ __attribute__((aligned(1024))) char st0[WbStage<NH>::BYTES];
  __shared__ __attribute__((aligned(1024))) char st1[WbStage<NH>::BYTES];
  __shared__ __attribute__((aligned(1024))) char vt[KB * ATT_D * 2];
  const int id = xcd_block(blockIdx.x, a.total);
  const int kb = __builtin_amdgcn_readfirstlane(id % a.blocks);
  const int bh = __builtin_amdgcn_readfirstlane(id / a.blocks);
  const int b = __builtin_amdgcn_readfirstlane(bh / a.heads), h = bh - b * a.heads;
  const int lane = threadIdx.x & 63, hl = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int w = wave % RG, half = wave / RG;
  const int T = a.T, W = a.window;
  const int k0 = kb * KB, w0 = k0 + 32 * w;
  const int j = w0 + (lane & 31);

  // queries the workgroup visits, the lane's own [lo_j, hi_j), and for the wave the range that
  // sees all of its keys (no mask) and the one that sees any
  auto uniform = [](int x) __attribute__((always_inline)) { return __builtin_amdgcn_readfirstlane(x); };
  auto first = [&](int x) __attribute__((always_inline)) {
    return a.mode == TTT_WINDOW_SLIDING ? x : (x / W) * W;
  };
  auto end = [&](int x) __attribute__((always_inline)) {
    return (int)min<int64_t>(T, a.mode == TTT_WINDOW_SLIDING ? (int64_t)x + W
                                                             : ((int64_t)(x / W) + 1) * W);
  };
  const int klast = min(k0 + KB, T) - 1, wl = min(w0 + 31, T - 1);
  const int lo = uniform(first(k0)), hi = uniform(end(klast));
  int lo_j = 0, hi_j = 0, in_lo = 1, in_hi = 0, any_lo = 0, any_hi = 0;
  if (j < T) {
    lo_j = first(j);
    hi_j = end(j);
  }
  if (w0 < T) {
    in_lo = uniform(first(wl));
    in_hi = uniform(end(w0));
    any_lo = uniform(first(w0));
    any_hi = uniform(end(wl));
  }
  const int len_j = hi_j - lo_j;
  const int nsteps = (hi - lo + QROWS - 1) / QROWS;

  const int64_t row0 = (int64_t)b * T;
  const u16* qb = a.q + row0 * a.ld + (int64_t)h * ATT_D;
  const u16* gb = a.dout + row0 * a.lddo + (int64_t)h * ATT_D;
  const float* lb = a.lse + ((int64_t)b * a.heads + h) * T;
  const float* db = a.delta + ((int64_t)b * a.heads + h) * T;
  WbLoad lq, lg;
  lq.init(a.ld);
  lg.init(a.lddo);
  const u16 *qp = qb + (int64_t)lo * a.ld, *gp = gb + (int64_t)lo * a.lddo;   // the next step's rows
  const float* sp0 = (wave ? db : lb) + lo;
  const int64_t advq = QROWS * a.ld, advg = QROWS * a.lddo;
  auto issue = [&](char* st, int rows) __attribute__((always_inline)) {
    lq.issue<QROWS>(st, qp, rows);
    lg.issue<QROWS>(st + QTILE, gp, rows);
    if (wave < 2) {
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
          (void*)sp0, (short)0, min(rows, QROWS) * 4, 0x00020000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t*)(st + 2 * QTILE + wave * 64 * 4), 4,
                                               lane * 4, 0, 0, 0);
    }
    qp += advq;
    gp += advg;
    sp0 += QROWS;
  };
  lq.issue<KB>(vt, a.v + (row0 + k0) * a.ld + (int64_t)h * ATT_D, T - k0);
  issue(st0, T - lo);

  bf16x8 kf[8];
  wb_frags(kf, a.k + (row0 + j) * a.ld + (int64_t)h * ATT_D, hl, j < T);
  WbAt at;
  at.init();
  const char* vw = vt + 32 * w * (ATT_D * 2);   // the wave's rows of v
  f32x16 dk[4], dv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dk[i] = dv[i] = f32x16{};

  auto step = [&](const char* cur, char* nxt, int i) __attribute__((always_inline)) {
    if (i + 1 < nsteps) issue(nxt, T - lo - (i + 1) * QROWS);
    const int r0 = NH == 1 ? 0 : 32 * half, tq = lo + i * QROWS + r0;   // this wave's 32 queries
    const char* gt = cur + QTILE;
    const float* ls = reinterpret_cast<const float*>(cur + 2 * QTILE) + r0;
    if (tq + 32 > any_lo && tq < any_hi) {   // wave-uniform: some query here sees some key
      f32x16 s, dp = f32x16{};
      if (tq < in_lo || tq + 32 > in_hi) {   // the mask as the scores' first summand
        const int base = tq + 4 * hl - lo_j;
#pragma unroll
        for (int v = 0; v < 16; ++v)
          s[v] = (unsigned)(base + 8 * (v >> 2) + (v & 3)) < (unsigned)len_j ? 0.f : -INFINITY;
      } else {
        s = f32x16{};
      }
      // The exponentials run beside the second product, the differences beside the third; a wave
      // past its scores goes before the SIMD's other one, so that the two stay apart (631 -> 602 us).
#pragma unroll
      for (int x = 0; x < 8; ++x) s = wb_mma(wb_row(cur, at, r0, x), kf[x], s);
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int x = 0; x < 8; ++x) dp = wb_mma(wb_row(gt, at, r0, x), wb_row(vw, at, 0, x), dp);
      // element v: query tq + 8 (v / 4) + 4 hl + v % 4
      bf16x8 pf[2], df[2];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 l4 = *reinterpret_cast<const f32x4*>(ls + 8 * g + 4 * hl);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int v = 4 * g + e;
          s[v] = __builtin_amdgcn_exp2f(fmaf(s[v], a.scale2, -l4[e] * 1.44269504088896341f));
          pf[v >> 3][v & 7] = static_cast<__bf16>(s[v]);
        }
      }
#pragma unroll
      for (int sp = 0; sp < 2; ++sp)
#pragma unroll
        for (int d = 0; d < 4; ++d) dv[d] = wb_mma(wb_col(gt, at, 32 * d, r0 + 16 * sp), pf[sp], dv[d]);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 d4 = *reinterpret_cast<const f32x4*>(ls + 64 + 8 * g + 4 * hl);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int v = 4 * g + e;
          df[v >> 3][v & 7] = static_cast<__bf16>(s[v] * (dp[v] - d4[e]));
        }
      }
#pragma unroll
      for (int sp = 0; sp < 2; ++sp)
#pragma unroll
        for (int d = 0; d < 4; ++d) dk[d] = wb_mma(wb_col(cur, at, 32 * d, r0 + 16 * sp), df[sp], dk[d]);
      __builtin_amdgcn_s_setprio(0);
      WB_ORDER(WB_DS, 3);
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        WB_ORDER(WB_MFMA, 1);
        WB_ORDER(WB_DS, 1);
      }
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
  };
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  int i = 0;
  for (; i + 1 < nsteps; i += 2) {
    step(st0, st1, i);
    step(st1, st0, i + 1);
  }
  if (i < nsteps) step(st0, st1, i);
  if constexpr (NH == 2) {
    wb_join(dk, w, half, st0);
    wb_join(dv, w, half, st1);
    if (half) return;
  }
  if (j < T) {
    const int64_t i0 = (row0 + j) * a.ldd + (int64_t)h * ATT_D;
    wb_store(a.dk + i0, dk, a.scale, hl);
    wb_store(a.dv + i0, dv, 1.f, hl);
  }
}

template <int NH>
hipError_t launch_window_bwd_nh(const WindowArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)a.total), block(256);
  if (a.window <= WB_ROWS) hipLaunchKernelGGL((k_window_dq<true, NH>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_window_dq<false, NH>), grid, block, 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_window_dkv<NH>, grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace

// the form of a launch: a.blocks and a.total, and whether it leaves CUs idle
static bool wb_form(WindowArgs& a, int64_t problems) {
  const int64_t small = (a.T + 63) / 64 * problems;
  const bool few = small <= WB_FEW;
  a.blocks = few ? (a.T + 63) / 64 : (a.T + 127) / 128;
  a.total = (int32_t)(a.blocks * problems);
  return few;
}

hipError_t launch_window_fwd(WindowArgs a, int64_t problems, hipStream_t st) {
  const bool few = wb_form(a, problems);
  const dim3 grid((unsigned)a.total), block(256);
  if (few) hipLaunchKernelGGL(k_window_fwd<2>, grid, block, 0, st, a);
  else hipLaunchKernelGGL(k_window_fwd<1>, grid, block, 0, st, a);
  return hipGetLastError();
}

hipError_t launch_window_bwd(WindowArgs a, int64_t problems, hipStream_t st) {
  return wb_form(a, problems) ? launch_window_bwd_nh<2>(a, st) : launch_window_bwd_nh<1>(a, st);
}

}  // namespace ttt
