// Per-head norm of queries and keys with the position rotation in one pass, its backward, and
// the same pass storing keys and values into a paged cache (include/ttt_attention.h).
//
// Mathematics.  r = 1 / sqrt(mean(x^2) + eps), n = x r w; pair j of n turned by
// angle_j = sum_a pos_a freq_a,j.  Backward: g = dy turned back, dw = sum g x r, u = g w,
// dx = r (u - x r mean(u x r)).
//
// Every value is read once and written once, a few operations each: the memory bounds it, once
// the angles are out of the way.  An angle needs 64-bit products (fp32 positions past 2^24
// would lose the angle) and a sine and a cosine, but every head of a token turns by the same
// ones: a workgroup takes a block of tokens, computes their angles once into LDS, and its
// lanes then run over the block's heads.  A lane holds 16 elements of a head, chosen so that
// both members of a pair are its own: the rotation needs no exchange, the norm a few shuffles
// among the head's lanes.
//
// Measured (a copy of 4 GB reads and writes 4.8 to 5.0 TB/s on the same card): forward, 64320 tokens of
// 12 heads of 128 in 32 bits, three axes: 181 us, 4.4 TB/s; backward, 32768 tokens of 16 heads
// in bf16: 84 to 87 us with the scales' sums (4.7 of it), 4.7 TB/s.  It moves its least bytes to within
// 1 %.  Non-temporal stores gain 2 to 15 % in bf16, whose runs fill whole lines, and lose 20 % in
// 32 bits with a rotation of 96 of 128, whose runs do not: ordinary ones stay.  The smallest
// calls take 3.6 us on the GPU, what any launch takes, and 10.8 us of the host.
#include "ttt_attention_internal.h"

namespace ttt {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// 16 bytes of T and back: 8 bf16 or 4 fp32
template <typename T>
constexpr int VW = 16 / (int)sizeof(T);
__device__ __forceinline__ void load16(const u16* p, float* x) {
  const u32x4 u = *as_global(reinterpret_cast<const u32x4*>(p));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf2f((u16)(u[i] & 0xffffu));
    x[2 * i + 1] = bf2f((u16)(u[i] >> 16));
  }
}
__device__ __forceinline__ void load16(const float* p, float* x) {
  const f32x4 w = *as_global(reinterpret_cast<const f32x4*>(p));
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = w[e];
}
__device__ __forceinline__ void store16(u16* p, const float* x) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = f2bf(x[2 * i]) | ((uint32_t)f2bf(x[2 * i + 1]) << 16);
  *as_global(reinterpret_cast<u32x4*>(p)) = w;
}
__device__ __forceinline__ void store16(float* p, const float* x) {
  *as_global(reinterpret_cast<f32x4*>(p)) = f32x4{x[0], x[1], x[2], x[3]};
}

// 8 values / scale as e4m3, held to +-448 (the conversion alone would turn larger ones to
// NaN), a NaN kept.
__device__ __forceinline__ void store8_e4m3(char* p, const float* x, float scale) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = x[i] / scale;
    y[i] = v > 448.f ? 448.f : v < -448.f ? -448.f : v;
  }
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], hi, true);
  *as_global(reinterpret_cast<u32x2*>(p)) = u32x2{(uint32_t)lo, (uint32_t)hi};
}

// Sum over the lph lanes (a power of two) that share a head.
__device__ __forceinline__ float head_sum(float v, int lph) {
  for (int off = lph >> 1; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// cos and sin of the block's angles: entry t * (rot / 2) + j.  A product of a position and a
// frequency has up to 55 bits, and 2^31 radians in 64 bits are 2^-22 off: the products, their sum
// over the axes and the turn's reduction keep what each rounds off (a fused product or a two-term
// sum gives it exactly).  Sine and cosine are taken of the reduced turn rounded to 32 bits and
// turned by the rest d: (c - d s, s + d c), d d / 2 being below 2^-50.  Measured: up to 1.3 half
// steps of fp32 off at positions anywhere in int32; in plain 64-bit steps 6 to 22 at far ones, by
// the axes; without the rest d 1.9 at any.  64320 tokens in 32 bits: outputs 6.4e-8 of their norm
// off, without d 6.7e-8, at the same time; sines and cosines in 64 bits 6.3e-8, and 3 to 5 % slower
// backward.
__device__ __forceinline__ void turns(const RopeArgs& a, int64_t t0, int nt, float* cs, float* sn) {
#pragma clang fp contract(off)   // the differences below are of rounded sums and products
  const int half = a.rot >> 1, n = nt * half;
  constexpr double C = 0.15915494309189535, CL = -9.839338337591243e-18;   // 1 / (2 pi) = C + CL
  for (int i = threadIdx.x; i < n; i += ROPE_NT) {
    const int t = i / half, j = i - t * half;
    const double p0 = (double)a.pos[t0 + t], f0 = (double)a.freq[j];
    double ang = p0 * f0, low = fma(p0, f0, -ang);
    for (int x = 1; x < a.axes; ++x) {
      const double p = (double)a.pos[(int64_t)x * a.tokens + t0 + t], f = (double)a.freq[x * half + j];
      const double y = p * f, sum = ang + y, part = sum - ang;
      low += fma(p, f, -y) + ((ang - (sum - part)) + (y - part));
      ang = sum;
    }
    const double u = ang * C;
    const double r = (u - rint(u)) + fma(low, C, fma(ang, CL, fma(ang, C, -u)));
    float s, c;
    const float turn = (float)r, d = 6.28318530717958648f * (float)(r - (double)turn);
    sincospif(2.f * turn, &s, &c);
    cs[i] = fmaf(-d, s, c);
    sn[i] = fmaf(d, c, s);
  }
}

// The lane's 16 elements of a head, as 16-byte runs: neighbouring lanes take neighbouring runs,
// so that each load of a wave is contiguous.  Lanes i < rot / 16 hold what turns: with HALVES
// half of their runs in each half of the rotated elements, at the same places.
template <typename T, bool PAIRS>
struct LanePlan {
  static constexpr int N = 16 / VW<T>;          // runs
  static constexpr int TN = PAIRS ? N : N / 2;  // runs of turns, 8 / TN each
  int off[N], toff[TN];
  bool has, rot;
  __device__ __forceinline__ LanePlan(const RopeArgs& a, int i) {
    const int rc = a.rot >> 4, all = a.D >> 4;
    has = i < all;
    rot = i < rc;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (!rot) off[n] = a.rot + VW<T> * (i - rc + n * (all - rc));
      else if (PAIRS) off[n] = VW<T> * (i + n * rc);
      else off[n] = VW<T> * (i + n % (N / 2) * rc) + (n / (N / 2)) * (a.rot >> 1);
    }
#pragma unroll
    for (int n = 0; n < TN; ++n) toff[n] = 8 / TN * (i + n * rc);
  }
  __device__ __forceinline__ void load(const T* p, float* x) const {
#pragma unroll
    for (int n = 0; n < N; ++n) load16(p + off[n], x + VW<T> * n);
  }
  __device__ __forceinline__ void store(T* p, const float* x) const {
#pragma unroll
    for (int n = 0; n < N; ++n) store16(p + off[n], x + VW<T> * n);
  }
  // cos and sin of the lane's 8 pairs from a token's table
  __device__ __forceinline__ void turns(const float* cs, const float* sn, float* c, float* s) const {
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int e = 0; e < 8 / TN; ++e) {
        c[8 / TN * n + e] = cs[toff[n] + e];
        s[8 / TN * n + e] = sn[toff[n] + e];
      }
  }
};

// The lane's 8 pairs turned by (c, s): pair e is (x[e], x[8 + e]) or (x[2 e], x[2 e + 1]).
template <bool PAIRS>
__device__ __forceinline__ void turn(float* x, const float* c, const float* s) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i0 = PAIRS ? 2 * e : e, i1 = PAIRS ? 2 * e + 1 : 8 + e;
    const float a = x[i0], b = x[i1];
    x[i0] = a * c[e] - b * s[e];
    x[i1] = a * s[e] + b * c[e];
  }
}
template <typename T, bool PAIRS, bool APPEND>
__global__ __launch_bounds__(ROPE_NT) void k_rope(RopeArgs a) {
  __shared__ __attribute__((aligned(16))) float cs[ROPE_TURNS];
  __shared__ __attribute__((aligned(16))) float sn[ROPE_TURNS];
  __shared__ int64_t row[ROPE_MAX_TB];   // append: the token's first cache element, or -1
  const int64_t t0 = (int64_t)blockIdx.x * a.tb;
  const int nt = (int)min<int64_t>(a.tb, a.tokens - t0);
  turns(a, t0, nt, cs, sn);
  if (APPEND && (int)threadIdx.x < nt) {
    const int64_t s = a.slot[t0 + threadIdx.x];
    int64_t at = -1;
    if (s >= 0 && s < a.slots) {
      const int64_t page = s / a.page_size;
      at = page * a.page_stride + (s - page * a.page_size) * a.D;
    }
    row[threadIdx.x] = at;
  }
  __syncthreads();
  const int groups = ROPE_NT / a.lph;
  const int g = (int)threadIdx.x / a.lph, li = (int)threadIdx.x % a.lph;
  const LanePlan<T, PAIRS> p(a, li);
  const int heads = a.q.heads + (APPEND ? 2 : 1) * a.k.heads;
  const int items = nt * heads;
  // every lane of a wave runs the same rounds: the shuffles need the head's lanes together
  for (int it0 = 0; it0 < items; it0 += groups) {
    const int it = it0 + g;
    const bool on = it < items && p.has;
    const int tt = it / heads;
    int h = it - tt * heads;
    const int64_t t = t0 + tt;
    const int which = h < a.q.heads ? 0 : h < a.q.heads + a.k.heads ? 1 : 2;
    if (which) h -= a.q.heads + (which - 1) * a.k.heads;
    float x[16];
    float ss = 0.f;
    if (on) {
      const T* src = which == 0   ? static_cast<const T*>(a.q.x) + t * a.q.ldx
                     : which == 1 ? static_cast<const T*>(a.k.x) + t * a.k.ldx
                                  : static_cast<const T*>(a.v) + t * a.ldv;
      src += (int64_t)h * a.D;
      p.load(src, x);
#pragma unroll
      for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
    }
    if (a.norm == TTT_HEAD_NORM_RMS) ss = head_sum(ss, a.lph);
    if (!on) continue;
    if (which < 2) {
      if (a.norm == TTT_HEAD_NORM_RMS) {
        const float r = 1.f / sqrtf(ss / (float)a.D + a.eps);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] *= r;
        const T* w = static_cast<const T*>(which ? a.k.w : a.q.w);
        if (w) {
          float wv[16];
          p.load(w, wv);
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] *= wv[e];
        }
      }
      if (p.rot) {
        float c[8], s[8];
        p.turns(cs + tt * (a.rot >> 1), sn + tt * (a.rot >> 1), c, s);
        turn<PAIRS>(x, c, s);
      }
    }
    if constexpr (APPEND) {
      if (which) {
        if (row[tt] < 0) continue;
        const int64_t at = row[tt] + (int64_t)h * a.page_size * a.D;
        if (a.e4m3) {
          const float* sc = which == 1 ? a.ks : a.vs;
          const float scale = sc ? sc[h] : 1.f;
          char* dst = reinterpret_cast<char*>(which == 1 ? a.kc : a.vc) + at;
#pragma unroll
          for (int n = 0; n < 2; ++n) store8_e4m3(dst + p.off[n], x + 8 * n, scale);
        } else {
          p.store((which == 1 ? a.kc : a.vc) + at, x);
        }
        continue;
      }
    }
    T* dst = which ? static_cast<T*>(a.k.y) + t * a.k.ldy : static_cast<T*>(a.q.y) + t * a.q.ldy;
    p.store(dst + (int64_t)h * a.D, x);
  }
}

// Backward: blockIdx.y is the side (queries, keys); a side's workgroups walk over the token
// blocks, so that the partial sums of the scales' gradients are few, and a second launch adds
// them up in order.  (Both sides in one workgroup hold two sets of running sums: 140 registers,
// three waves per SIMD instead of four.)
template <typename T, bool PAIRS>
__global__ __launch_bounds__(ROPE_NT) void k_rope_bwd(RopeArgs a) {
  __shared__ __attribute__((aligned(16))) float cs[ROPE_TURNS];
  __shared__ __attribute__((aligned(16))) float sn[ROPE_TURNS];
  const RopeSide& sd = blockIdx.y ? a.k : a.q;
  const int groups = ROPE_NT / a.lph;
  const int g = (int)threadIdx.x / a.lph, li = (int)threadIdx.x % a.lph;
  const LanePlan<T, PAIRS> p(a, li);
  const bool rms = a.norm == TTT_HEAD_NORM_RMS;
  const T* sdx = static_cast<const T*>(sd.x);
  const T* sdy = static_cast<const T*>(sd.dy);
  T* sy = static_cast<T*>(sd.y);
  const int64_t ldx = sd.ldx, lddy = sd.lddy, ldy = sd.ldy;
  const int heads = sd.heads;
  float w[16], dw[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    w[e] = 1.f;
    dw[e] = 0.f;
  }
  if (sd.w && p.has) p.load(static_cast<const T*>(sd.w), w);
  const int64_t nb = (a.tokens + a.tb - 1) / a.tb;
  for (int64_t b = blockIdx.x; b < nb; b += gridDim.x) {
    const int64_t t0 = b * a.tb;
    const int nt = (int)min<int64_t>(a.tb, a.tokens - t0);
    __syncthreads();   // the last block's turns have been read
    turns(a, t0, nt, cs, sn);
    __syncthreads();
    const int items = nt * heads;
    for (int it0 = 0; it0 < items; it0 += groups) {
      const int it = it0 + g;
      const bool on = it < items && p.has;
      const int tt = it / heads, h = it - tt * heads;
      const int64_t t = t0 + tt, col = (int64_t)h * a.D;
      float x[16], u[16];
      float ss = 0.f, dot = 0.f;
      if (on) {
        p.load(sdy + t * lddy + col, u);
        if (rms) {
          p.load(sdx + t * ldx + col, x);
#pragma unroll
          for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
        }
        if (p.rot) {
          float c[8], s[8];
          p.turns(cs + tt * (a.rot >> 1), sn + tt * (a.rot >> 1), c, s);
#pragma unroll
          for (int e = 0; e < 8; ++e) s[e] = -s[e];
          turn<PAIRS>(u, c, s);
        }
      }
      if (rms) {
        ss = head_sum(ss, a.lph);
        const float r = 1.f / sqrtf(ss / (float)a.D + a.eps);
        if (on) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            x[e] *= r;
            dw[e] = fmaf(u[e], x[e], dw[e]);
            u[e] *= w[e];
            dot = fmaf(u[e], x[e], dot);
          }
        }
        dot = head_sum(dot, a.lph) / (float)a.D;
        if (on)
#pragma unroll
          for (int e = 0; e < 16; ++e) u[e] = r * fmaf(-x[e], dot, u[e]);
      }
      if (on) p.store(sy + t * ldy + col, u);
    }
  }
  if (!a.part) return;
  // the groups' sums: 16 values per thread through LDS (cs and sn hold 16 * 256 floats
  // together), then one thread per column adds the groups' values in order, in 64 bits: up to 256
  // roundings of a growing sum in fp32 are most of the error (32768 tokens, 8 heads of 128: 1.6e-7
  // of the gradient's norm, 1.1e-7 with this sum in 64 bits, at the same time)
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    cs[e * ROPE_NT + threadIdx.x] = dw[e];
    sn[e * ROPE_NT + threadIdx.x] = dw[8 + e];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.D; c += ROPE_NT) {
    const int lane = c >> 4, e = c & 15;
    const float* src = (e < 8 ? cs + e * ROPE_NT : sn + (e - 8) * ROPE_NT) + lane;
    double s = 0.0;
#pragma unroll 8
    for (int i = 0; i < groups; ++i) s += (double)src[i * a.lph];
    const LanePlan<T, PAIRS> q(a, lane);
    int at = 0;   // a register array takes no run-time index
#pragma unroll
    for (int n = 0; n < LanePlan<T, PAIRS>::N; ++n)
      if (e / VW<T> == n) at = q.off[n] + e % VW<T>;
    a.part[((int64_t)blockIdx.y * a.wgs + blockIdx.x) * a.D + at] = (float)s;
  }
}

// Columns of the partial sums added up over the workgroups: 16 columns per workgroup, 64 rows
// at a time, in 64 bits and one order.
__global__ __launch_bounds__(1024) void k_rope_dw(RopeDwArgs a) {
  __shared__ double acc[1024];
  const int side = blockIdx.y;
  float* out = side ? a.dk : a.dq;
  if (!out) return;
  const int c = blockIdx.x * 16 + (threadIdx.x & 15), r0 = threadIdx.x >> 4;
  const float* p = a.part + (int64_t)side * a.n * a.D + c;
  double s = 0.0;
#pragma unroll 8
  for (int r = r0; r < a.n; r += 64) s += (double)p[(int64_t)r * a.D];
  acc[threadIdx.x] = s;
  for (int half = 512; half >= 16; half >>= 1) {
    __syncthreads();
    if ((int)threadIdx.x < half) acc[threadIdx.x] += acc[threadIdx.x + half];
  }
  if (threadIdx.x < 16) out[c] = (float)acc[threadIdx.x];
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, int bf16, hipStream_t st) {
  const dim3 grid((unsigned)((a.tokens + a.tb - 1) / a.tb)), block(ROPE_NT);
  if (bf16) {
    if (a.pairs) hipLaunchKernelGGL((k_rope<u16, true, false>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_rope<u16, false, false>), grid, block, 0, st, a);
  } else {
    if (a.pairs) hipLaunchKernelGGL((k_rope<float, true, false>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_rope<float, false, false>), grid, block, 0, st, a);
  }
  return hipGetLastError();
}

hipError_t launch_rope_append(const RopeArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)((a.tokens + a.tb - 1) / a.tb)), block(ROPE_NT);
  if (a.pairs) hipLaunchKernelGGL((k_rope<u16, true, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_rope<u16, false, true>), grid, block, 0, st, a);
  return hipGetLastError();
}

hipError_t launch_rope_backward(const RopeArgs& a, int bf16, hipStream_t st) {
  const dim3 grid((unsigned)a.wgs, 2), block(ROPE_NT);
  if (bf16) {
    if (a.pairs) hipLaunchKernelGGL((k_rope_bwd<u16, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_rope_bwd<u16, false>), grid, block, 0, st, a);
  } else {
    if (a.pairs) hipLaunchKernelGGL((k_rope_bwd<float, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_rope_bwd<float, false>), grid, block, 0, st, a);
  }
  return hipGetLastError();
}

hipError_t launch_rope_dw(const RopeDwArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(k_rope_dw, dim3(a.D / 16, 2), dim3(1024), 0, st, a);
  return hipGetLastError();
}

}  // namespace ttt
