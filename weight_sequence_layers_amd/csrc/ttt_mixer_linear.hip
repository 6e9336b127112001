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
  static constexpr int N = LIN_C / ROWS;                    // loads of a tile
  static constexpr int PER = (N + NW - 1) / NW;
  int32_t off[PER];
  uint32_t ld2;
  int wave;
  __device__ __forceinline__ void init(int64_t ld, int rev) {
    const int lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    ld2 = (uint32_t)(ld * 2);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int r = (wave + i * NW) * ROWS + lane / (P / 16), c = (lane % (P / 16)) ^ lin_swz<P>(r);
      const int32_t at = r * (int32_t)ld2;
      off[i] = (rev ? -at : at) + c * 16;
    }
  }
  // The n rows at p, in their order or (rev) from the last to the first; the others read as 0:
  // their offsets lie behind the n rows, or wrap to 2^31 and more.
  __device__ __forceinline__ void issue(char* tile, const u16* p, int n, int rev) const {
    const uint32_t last = (uint32_t)(n - 1) * ld2;
    const __amdgpu_buffer_rsrc_t rs =
        __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)(last + P), 0x00020000);
    const uint32_t top = rev ? last : 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (N % NW == 0 || wave + i * NW < N)   // wave-uniform
        dma16(rs, (lds_void_t*)(tile + (wave + i * NW) * 1024), (uint32_t)off[i] + top);
  }
};

// Offsets of a lane's fragments in a tile.
template <int P>
struct LinAt {
  int row;   // along the rows: elements 4 (lane / 32) .. + 3 of row lane % 32
  int col;   // along the columns: elements 16 (g & 1) + 4 (j & 3) .. + 3 of row 4 (g / 2) + j / 4
  __device__ __forceinline__ void init() {
    const int lane = threadIdx.x & 63, r = lane & 31, g = lane >> 4, j = lane & 15;
    row = r * P + (lin_swz<P>(r) << 4) + 8 * (lane >> 5);
    const int m = 16 * (g & 1) + 4 * (j & 3), rc = 4 * (g >> 1) + (j >> 2);
    col = rc * P + (((m >> 3) ^ lin_swz<P>(rc)) << 4) + (m & 7) * 2;
  }
};

// Row lane % 32, elements base + 4 (lane / 32) + (0..3) and + 8: the order in which a lane holds the
// rows of an accumulator.  base a multiple of 16.
template <int P>
__device__ __forceinline__ bf16x8 lin_row(const char* tile, const LinAt<P>& at, int base) {
  s16x4 x[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) x[i] = *reinterpret_cast<const s16x4*>(tile + (at.row ^ (base * 2) ^ (i << 4)));
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  const s16x8 v = __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(bf16x8, v);
}
// Element base + lane % 32 of rows row + 4 (lane / 32) + (0..3) and + 8.  base a multiple of 32, row
// of 16.
template <int P>
__device__ __forceinline__ bf16x8 lin_col(const char* tile, const LinAt<P>& at, int base, int row) {
  s16x4 x[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const char* p = tile + (row + 8 * i) * P + (at.col ^ (base << 1) ^ (i << 5));
    x[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p));
  }
  typedef short s16x8 __attribute__((ext_vector_type(8)));
  const s16x8 v = __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(bf16x8, v);
}

__device__ __forceinline__ f32x16 lin_mma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// x as N bf16 numbers whose sum it is, to 8 N bits.
template <int N>
__device__ __forceinline__ void lin_split(const float (&x)[8], bf16x8 (&p)[N]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float r = x[e];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      p[i][e] = static_cast<__bf16>(r);
      r -= static_cast<float>(p[i][e]);
    }
  }
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

// A workgroup walks one segment of one sequence, head and role; its NW waves hold 32 columns of the
// state each, all DA rows of it, as accumulators.  The output is computed transposed (a lane is a
// token), so that the accumulators of the state and of the scores are the operands of the products
// that follow as they lie, in the order of an accumulator's rows; q and k are read from LDS in
// that order.  Every wave computes the chunk's 32 x 32 scores itself: an eighth more products, and no
// exchange between waves.
// OUT false: only the segment's own sum, from zeros.
template <int DA, int NW, bool OUT>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(DA == 256 ? 1 : 2)))
void k_linear(LinArgs a) {
  constexpr int PA = DA * 2, PV = NW * 64;                    // bytes of a tile's row
  constexpr int KO = OUT ? LIN_C * PA : 0, VO = KO + LIN_C * PA, STAGE = VO + LIN_C * PV;
  constexpr int RT = DA / 32;
  __shared__ __attribute__((aligned(1024))) char st0[STAGE];
  __shared__ __attribute__((aligned(1024))) char st1[STAGE];
  __shared__ float pw[LIN_C + 1];
  auto uniform = [](int x) __attribute__((always_inline)) { return __builtin_amdgcn_readfirstlane(x); };
  int id = xcd_block(blockIdx.x, a.total);
  const int slice = uniform(id % a.slices);
  id = uniform(id / a.slices);
  const int ri = uniform(id % a.roles);
  id = uniform(id / a.roles);
  const int h = uniform(id % a.heads);
  id = uniform(id / a.heads);
  const int nseg = OUT ? a.nseg : a.nseg - 1;
  const int seg = uniform(id % nseg), b = uniform(id / nseg);
  const LinRole& r = a.role[ri];
  const int rev = r.rev;
  int64_t row0;
  int len;
  lin_span(a.starts, b, a.tokens, a.T, row0, len);
  const int t0 = seg * a.L;                                  // first token, in the role's time
  if (OUT ? seg > 0 && t0 >= len : t0 + a.L >= len) return;
  const int cnt = min(a.L, len - t0), chunks = (cnt + LIN_C - 1) / LIN_C;

  const int lane = threadIdx.x & 63, hl = lane >> 5, li = lane & 31;
  const int wave = uniform((int)(threadIdx.x >> 6));
  const float lam = a.decay[h];
  if (threadIdx.x <= LIN_C) pw[threadIdx.x] = lin_power(lam, (int)threadIdx.x);

  const int col0 = slice * 32 * NW;                          // the workgroup's first column
  const u16* qb = r.q + (int64_t)h * DA;
  const u16* kb = r.k + (int64_t)h * DA;
  const u16* vb = r.v + (int64_t)h * a.DB + col0;
  LinLoad<PA, NW> lq, lk;
  LinLoad<PV, NW> lv;
  if (OUT) lq.init(r.ldq, rev);
  lk.init(r.ldk, rev);
  lv.init(r.ldv, rev);
  auto issue = [&](char* st, int c) __attribute__((always_inline)) {
    const int n = min(LIN_C, cnt - c * LIN_C), t = t0 + c * LIN_C;
    const int64_t row = row0 + (rev ? len - t - n : t);
    if (OUT) lq.issue(st, qb + row * r.ldq, n, rev);
    lk.issue(st + KO, kb + row * r.ldk, n, rev);
    lv.issue(st + VO, vb + row * r.ldv, n, rev);
  };
  if (chunks) issue(st0, 0);

  // the state: element v of tile rt is row 32 rt + 8 (v / 4) + 4 hl + v % 4, column li of the wave's
  const int64_t elems = (int64_t)DA * a.DB;
  const int colw = col0 + 32 * wave + li;
  const int64_t entry = lin_slot(a.slot, b, a.slots);
  f32x16 s[RT];
  const float* init = nullptr;
  if (OUT) {
    if (r.ws) init = r.ws + (((int64_t)b * a.heads + h) * a.nseg + seg) * elems;
    else if (r.init && entry >= 0) init = r.init + (entry * a.heads + h) * elems;
  }
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) s[rt] = f32x16{};
  if (init) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int row = 32 * rt + 8 * g + 4 * hl;
        if (r.trans) {
          const f32x4 x = *as_global(reinterpret_cast<const f32x4*>(init + (int64_t)colw * DA + row));
#pragma unroll
          for (int e = 0; e < 4; ++e) s[rt][4 * g + e] = x[e];
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[rt][4 * g + e] = *as_global(init + (int64_t)(row + e) * a.DB + colw);
        }
      }
  }
  LinAt<PA> at;
  LinAt<PV> av;
  at.init();
  av.init();
  __syncthreads();
  // element v of the scores: key 8 (v / 4) + 4 hl + v % 4 of the chunk, query li
  float dm[16];
  if (OUT)
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int j = 8 * (v >> 2) + 4 * hl + (v & 3);
      dm[v] = li >= j ? pw[li >= j ? li - j : 0] * r.scale_p : 0.f;
    }

  auto step = [&](const char* cur, char* nxt, int c) __attribute__((always_inline)) {
    const int n = min(LIN_C, cnt - c * LIN_C);
    if (c + 1 < chunks) issue(nxt, c + 1);
    // backward in time the state before the first token (the gradient of the last state) is that
    // of the first token itself: one power less
    const int e0 = rev && t0 + c == 0 ? 0 : 1;
    bf16x8 vf[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) vf[x] = lin_col<PV>(cur + VO, av, 32 * wave, 16 * x);
    if constexpr (OUT) {
      f32x16 p = f32x16{}, o = f32x16{}, o1 = f32x16{};
#pragma unroll
      for (int x = 0; x < 2 * RT; ++x) {
        const bf16x8 qf = lin_row<PA>(cur, at, 16 * x);
        p = lin_mma(lin_row<PA>(cur + KO, at, 16 * x), qf, p);
        float sv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) sv[e] = s[x >> 1][8 * (x & 1) + e];
        bf16x8 sp[2];
        lin_split(sv, sp);
        o = lin_mma(sp[0], qf, o);
        o1 = lin_mma(sp[1], qf, o1);
      }
      const float f = pw[li + e0] * r.scale_s;
#pragma unroll
      for (int v = 0; v < 16; ++v) o[v] = (o[v] + o1[v]) * f;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float pv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) pv[e] = p[8 * x + e] * dm[8 * x + e];
        bf16x8 pp[2];
        lin_split(pv, pp);
        o = lin_mma(vf[x], pp[0], o);
        o = lin_mma(vf[x], pp[1], o);
      }
      if (li < n) {
        const int t = t0 + c * LIN_C + li;
        u16* row = r.out + (row0 + (rev ? len - 1 - t : t)) * r.ldo + (int64_t)h * a.DB + col0 + 32 * wave + 4 * hl;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
          *as_global(reinterpret_cast<u32x2*>(row + 8 * g)) =
              u32x2{f2bf(o[4 * g]) | ((uint32_t)f2bf(o[4 * g + 1]) << 16),
                    f2bf(o[4 * g + 2]) | ((uint32_t)f2bf(o[4 * g + 3]) << 16)};
        }
      }
    }
    const float sd = pw[n - 1 + e0];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int v = 0; v < 16; ++v) s[rt][v] *= sd;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = 16 * x + 8 * (e >> 2) + 4 * hl + (e & 3);   // rows behind the last token are 0
        w[e] = static_cast<float>(vf[x][e]) * (pw[max(n - 1 - j, 0)] * r.scale_w);
      }
      bf16x8 wp[3];
      lin_split(w, wp);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const bf16x8 kf = lin_col<PA>(cur + KO, at, 32 * rt, 16 * x);
#pragma unroll
        for (int i = 0; i < 3; ++i) s[rt] = lin_mma(kf, wp[i], s[rt]);
      }
    }
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
  };
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  int c = 0;
  for (; c + 1 < chunks; c += 2) {
    step(st0, st1, c);
    step(st1, st0, c + 1);
  }
  if (c < chunks) step(st0, st1, c);

  float* fin = nullptr;
  float f = 1.f;
  if constexpr (OUT) {
    if (r.fin && entry >= 0 && t0 + a.L >= len) fin = r.fin + (entry * a.heads + h) * elems;
    if (rev && len > 0) f = lam;   // behind the last step back lies the state before the first token
  } else {
    fin = r.ws + (((int64_t)b * a.heads + h) * a.nseg + seg) * elems;
  }
  if (fin) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int row = 32 * rt + 8 * (v >> 2) + 4 * hl + (v & 3);
        *as_global(fin + (int64_t)row * a.DB + colw) = s[rt][v] * f;
      }
  }
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

template <int DA, bool OUT>
hipError_t launch_nw(const LinArgs& a, int NW, hipStream_t st) {
  if (NW == 2) hipLaunchKernelGGL((k_linear<DA, 2, OUT>), dim3(a.total), dim3(128), 0, st, a);
  else hipLaunchKernelGGL((k_linear<DA, 4, OUT>), dim3(a.total), dim3(256), 0, st, a);
  return hipGetLastError();
}

template <bool OUT>
hipError_t launch_da(const LinArgs& a, int DA, int NW, hipStream_t st) {
  if (a.total == 0) return hipSuccess;
  return DA == 64 ? launch_nw<64, OUT>(a, NW, st)
         : DA == 128 ? launch_nw<128, OUT>(a, NW, st) : launch_nw<256, OUT>(a, NW, st);
}

}  // namespace

hipError_t launch_linear_walk(const LinArgs& a, int DA, int NW, hipStream_t st) {
  return launch_da<true>(a, DA, NW, st);
}

hipError_t launch_linear_states(const LinArgs& a, int DA, int NW, hipStream_t st) {
  return launch_da<false>(a, DA, NW, st);
}

hipError_t launch_linear_scan(const LinArgs& a, int DA, hipStream_t st) {
  const unsigned n = (unsigned)((int64_t)a.batch * a.heads * ((int64_t)DA * a.DB / 1024));
  hipLaunchKernelGGL(k_linear_scan, dim3(n, a.roles), dim3(256), 0, st, a, DA);
  return hipGetLastError();
}

}  // namespace ttt
