// What stands between two sub-layers in one pass, and its backward (include/ttt_mixer.h).
//
// Mathematics, with mean_g over a group and mean over a row:
//   r = 1 / sqrt(mean_g y^2 + eps), u = y r w_y, z = u act(g), h' = h + s z,
//   p = 1 / sqrt(mean h'^2 + eps), n = h' p w_n.
// Backward: with x = h' p, a = dn w_n:  d = dh' + p (a - x mean(a x)), dw_n = sum dn x,  dh = d,
//   ds = sum d z,  e = d s,  dg = e u act'(g),  f = e act(g),  dw_y = sum f y r,
//   dy = r (f w_y - y r mean_g(f w_y y r)).
//
// Every tensor is read or written once: the memory bounds it.  A lane holds 8 neighbouring elements of
// a row, the row some lanes of a wave or up to 16 whole waves, so that a group (a power of two of at
// most 512 elements) lies in neighbouring lanes of one wave, and few registers keep many waves, and
// with them many bytes, under way (16 or 32 elements a lane: one wave to a SIMD).  Nothing is kept
// between the forward and the backward, which reads h and y again instead of saved statistics.
//
// Measured: 64320 rows of 768 in fp32 (two read, two written, 791 MB) 150 us, 5.3 TB/s; backward with a
// gate of 32768 rows of 1024 in bf16 (537 MB) 117 us, of 24197 rows of 768 in fp32 (594 MB) 124, 4.6 and 4.8
// TB/s, 5 us of each the weights' second launch; a copy of 4 GB reaches 5.0.  Without a gate bf16 rows
// run at 6.2 to 6.7; backwards of rows of 4096 and 8192 at 3.3 to 4.5 (of 2056, half of whose lanes idle, at 2.2 to
// 3.8): one workgroup of 8 or 16 waves to a row and mostly one to a CU, whose barriers nothing hides, and with 16
// waves and a gate 2 to 24 of a lane's registers in memory.
#include "ttt_device.hpp"
#include "ttt_mixer_internal.h"

namespace ttt {
namespace {

constexpr int NORM_NT = 256;
constexpr int NORM_CHAIN = 64;   // rows of a lane in a backward launch at most, whose scales' gradients it adds up in fp32

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 8 elements of T as loaded, and their values
template <typename T>
struct Raw8;
template <>
struct Raw8<u16> {
  u32x4 w;
  __device__ __forceinline__ void load(const u16* p) { w = *as_global(reinterpret_cast<const u32x4*>(p)); }
  __device__ __forceinline__ void fill(float x) {
    const uint32_t b = f2bf(x);
    w = u32x4{b, b, b, b} * 0x10001u;
  }
  // what was computed from the elements is computed again from here on, not kept
  __device__ __forceinline__ void again() { asm("" : "+v"(w)); }
  __device__ __forceinline__ float operator[](int i) const {
    return __builtin_bit_cast(float, i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
};
template <>
struct Raw8<float> {
  f32x4 w[2];
  __device__ __forceinline__ void load(const float* p) {
    w[0] = *as_global(reinterpret_cast<const f32x4*>(p));
    w[1] = *as_global(reinterpret_cast<const f32x4*>(p + 4));
  }
  __device__ __forceinline__ void fill(float x) { w[0] = w[1] = f32x4{x, x, x, x}; }
  __device__ __forceinline__ void again() { asm("" : "+v"(w[0]), "+v"(w[1])); }
  __device__ __forceinline__ float operator[](int i) const { return w[i >> 2][i & 3]; }
};
__device__ __forceinline__ void store8(u16* p, const float* x) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i)   // two at once, rounded to the nearest even one
    w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{x[2 * i], x[2 * i + 1]}), bf16x2));
  *as_global(reinterpret_cast<u32x4*>(p)) = w;
}
__device__ __forceinline__ void store8(float* p, const float* x) {
  *as_global(reinterpret_cast<f32x4*>(p)) = f32x4{x[0], x[1], x[2], x[3]};
  *as_global(reinterpret_cast<f32x4*>(p + 4)) = f32x4{x[4], x[5], x[6], x[7]};
}

// The smaller of 1 / (1 + exp(-g)) and what that leaves of 1, with g's sign, within about ten half steps of fp32,
// for every g.  With e = exp(-|g|), which is at most 1, it is e / (1 + e): nothing overflows, and neither it nor
// 1 less it cancels.  e is the square of exp(-|g| / 2), so that it may be below fp32's normal numbers, which the
// exponential itself cannot give; the exponent keeps what its product rounds off, |g| held to 110 (e is 0 from 104
// on), and the reciprocal takes a Newton step.  NaN stays NaN.
constexpr float GATE_FAR = 110.f;
__device__ __forceinline__ float sigmoid_tail(float g) {
  constexpr float L = -0.72134752044448170f, LL = -9.6298149556e-9f;   // -log2(e) / 2, and what its rounding leaves
  const float a = __builtin_elementwise_minimum(fabsf(g), GATE_FAR);
  const float t = a * L, low = fmaf(a, L, -t) + a * LL;
  float x = __builtin_amdgcn_exp2f(t);
  x = fmaf(x, low * 0.693147181f, x);
  const float e = x * x, d = 1.f + e;
  float r = __builtin_amdgcn_rcpf(d);
  r = fmaf(r, fmaf(-d, r, 1.f), r);
  return copysignf(e * r, g);
}
// The gate's value from the tail q: the sigmoid, or for silu g times it, g held where it is 0 so that their
// product is; and its slope, s (1 - s) or s + g s (1 - s), g held on both sides.
__device__ __forceinline__ float from_tail(float q) {   // by the sign's bit: q may be -0
  return __builtin_bit_cast(int32_t, q) < 0 ? -q : 1.f - q;
}
template <int GATE>
__device__ __forceinline__ float gate_value(float g, float q) {
  return GATE == TTT_GATE_SILU ? from_tail(q) * __builtin_amdgcn_fmed3f(g, -GATE_FAR, INFINITY) : from_tail(q);
}
template <int GATE>
__device__ __forceinline__ float gate_slope(float g, float q) {
  const float m = fabsf(q) * (1.f - fabsf(q));
  return GATE == TTT_GATE_SILU ? fmaf(__builtin_amdgcn_fmed3f(g, -GATE_FAR, GATE_FAR), m, from_tail(q)) : m;
}

// Lanes of a row: a power of two of a wave's, or the workgroup.
__host__ __device__ inline int norm_lanes(int D) {
  int n = 1;
  while (n < 64 && n * 8 < D) n *= 2;
  return n;
}

// Sum over the n neighbouring lanes (a power of two, the same in every lane) that hold a row or a group,
// in vector instructions: through the LDS a row's four sums are 24 round trips in a row, more
// than its loads.  Every lane adds the same two halves at each step, so all get the same sum.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float lanes_sum(float v, int n) {
  if (n > 1) v += dpp<0xB1>(v);     // of pairs: lane ^ 1
  if (n > 2) v += dpp<0x4E>(v);     // lane ^ 2
  if (n > 4) v += dpp<0x141>(v);    // the mirrored lane of 8
  if (n > 8) v += dpp<0x140>(v);    // of 16
  if (n > 16) {                     // rows of 16 lanes swapped in pairs
    const uint32_t x = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    v = __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
  }
  if (n > 32) {                     // halves of the wave
    const uint32_t x = __builtin_bit_cast(uint32_t, v);
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    v = __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
  }
  return v;
}

// Sums over a row.  Of a row of W waves each call takes the other half of `scratch` in turn, so that one
// barrier keeps its readers from the next call's writers.
template <int W>
struct RowSum {
  float (*scratch)[16];
  int lanes, turn = 0;
  __device__ __forceinline__ float operator()(float v) {
    if constexpr (W == 1) {
      return lanes_sum(v, lanes);
    } else {
      v = lanes_sum(v, 64);
      float* s = scratch[turn];
      turn ^= 1;
      const int wave = threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0) s[wave] = v;
      lds_barrier();
      return total(s + wave / W * W);
    }
  }
  // two at once
  __device__ __forceinline__ void operator()(float& u, float& v) {
    if constexpr (W == 1) {
      u = lanes_sum(u, lanes);
      v = lanes_sum(v, lanes);
    } else {
      u = lanes_sum(u, 64);
      v = lanes_sum(v, 64);
      float* s = scratch[turn];
      turn ^= 1;
      const int wave = threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0) {
        s[wave] = u;
        s[32 + wave] = v;   // of the pair of halves that lies 32 floats on
      }
      lds_barrier();
      u = total(s + wave / W * W);
      v = total(s + 32 + wave / W * W);
    }
  }
  static __device__ __forceinline__ float total(const float* s) {
    float x = s[0];
#pragma unroll
    for (int i = 1; i < W; ++i) x += s[i];
    return x;
  }
};

template <int W>
constexpr int norm_threads = W > 4 ? 64 * W : NORM_NT;

// 1 / root mean square of the lane's group (or of the row).
template <int W>
__device__ __forceinline__ float inv_rms(float ss, const NormArgs& a, RowSum<W>& sum) {
  return 1.f / sqrtf((a.gw == a.D ? sum(ss) : lanes_sum(ss, a.gw >> 3)) / (float)a.gw + a.eps);
}

// W: waves of a row; GATE: the gate's kind (as a select of each element: 120 us instead of 118.7 for that backward).
template <typename T, int W, int GATE>
__global__ __launch_bounds__(norm_threads<W>) void k_norm(NormArgs a) {
  __shared__ float scratch[4][16];
  const int lanes = W == 1 ? norm_lanes(a.D) : 64 * W;
  RowSum<W> sum{scratch, lanes};
  const int64_t t = (int64_t)blockIdx.x * (norm_threads<W> / lanes) + threadIdx.x / lanes;
  const int col = (int)threadIdx.x % lanes * 8;
  const bool on = t < a.tokens && col < a.D;       // the sums need all lanes
  Raw8<T> y, h, g, w, s;
  y.fill(0.f);
  h.fill(0.f);
  g.fill(0.f);
  w.fill(1.f);
  s.fill(1.f);
  if (on) {
    y.load(static_cast<const T*>(a.y) + t * a.ldy + col);
    if (a.h) h.load(static_cast<const T*>(a.h) + t * a.ldh + col);
    if (GATE) g.load(static_cast<const T*>(a.gate) + t * a.ldg + col);
    if (a.wy) w.load(static_cast<const T*>(a.wy) + col);
    if (a.rs) s.load(static_cast<const T*>(a.rs) + col);
  }
  float r = 1.f;
  if (a.norm_y) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
    r = inv_rms<W>(ss, a, sum);
  }
  float x[8], hh = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float z = y[e] * r * w[e];
    if (GATE) z *= gate_value<GATE>(g[e], sigmoid_tail(g[e]));
    x[e] = fmaf(s[e], z, h[e]);
    hh = fmaf(x[e], x[e], hh);
  }
  if (a.ho && on) store8(static_cast<T*>(a.ho) + t * a.ldho + col, x);
  if (a.n) {
    const float p = 1.f / sqrtf(sum(hh) / (float)a.D + a.eps);
    if (on) {
      w.fill(1.f);
      if (a.wn) w.load(static_cast<const T*>(a.wn) + col);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] * p * w[e];
      store8(static_cast<T*>(a.n) + t * a.ldn + col, x);
    }
  }
}

// Backward: the workgroups walk over the rows, so that the partial sums of the scales' gradients are
// few; a second launch adds them up in order.  Rows past NORM_CHAIN to a lane go into further pairs of launches,
// whose sums are joined in 64 bits (added up in one launch, 1024 equal rows to a lane gave sums 1.4e-5 off; a join
// inside the loop took 10 to 20 more registers and a wave of a SIMD from every size).
template <typename T, int W, int GATE>
__global__ __launch_bounds__(norm_threads<W>) void k_norm_bwd(NormArgs a) {
  constexpr int NT = norm_threads<W>;
  // 128 registers a lane, for which values computed again are cheaper than what would not fit (rows of 8192: bf16 silu
  // 233 -> 161 us, fp32 182 -> 135)
  constexpr bool FEW = W == 16;
  __shared__ float scratch[4][16];
  __shared__ __attribute__((aligned(16))) float red[W > 2 ? 1 : NT * 8];
  const int lanes = W == 1 ? norm_lanes(a.D) : 64 * W, rows = NT / lanes;
  RowSum<W> sum{scratch, lanes};
  const int col = (int)threadIdx.x % lanes * 8;
  const bool has = col < a.D;
  Raw8<T> wy, rs, wn;
  float dw[3][8];
  wy.fill(1.f);
  rs.fill(1.f);
  wn.fill(1.f);
  if (has) {
    if (a.wy) wy.load(static_cast<const T*>(a.wy) + col);
    if (a.rs) rs.load(static_cast<const T*>(a.rs) + col);
    if (a.wn) wn.load(static_cast<const T*>(a.wn) + col);
  }
#pragma unroll
  for (int i = 0; i < 3; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
  // every lane of a workgroup runs the same rounds: sums need them together
  for (int64_t t0 = (int64_t)blockIdx.x * rows; t0 < a.tokens; t0 += (int64_t)gridDim.x * rows) {
    const int64_t t = t0 + (int)threadIdx.x / lanes;
    const bool on = has && t < a.tokens;
    if (FEW && GATE && sizeof(T) == 2) {
      wy.again();
      rs.again();
      wn.again();
    }
    Raw8<T> y, h, g, dho, dn;
    y.fill(0.f);
    h.fill(0.f);
    g.fill(0.f);
    dho.fill(0.f);
    dn.fill(0.f);
    if (on) {
      y.load(static_cast<const T*>(a.y) + t * a.ldy + col);
      if (a.h) h.load(static_cast<const T*>(a.h) + t * a.ldh + col);
      if (GATE) g.load(static_cast<const T*>(a.gate) + t * a.ldg + col);
      if (a.dho) dho.load(static_cast<const T*>(a.dho) + t * a.lddho + col);
      if (a.dn) dn.load(static_cast<const T*>(a.dn) + t * a.lddn + col);
    }
    float r = 1.f;
    if (a.norm_y) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
      r = inv_rms<W>(ss, a, sum);
    }
    // the gate's tail, and d, the gradient of h'
    float q[8], d[8];
    if (GATE)
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = sigmoid_tail(g[e]);
    auto act = [&](int e) __attribute__((always_inline)) { return GATE ? gate_value<GATE>(g[e], q[e]) : 1.f; };
    if (a.dn) {
      float hh = 0.f, ax = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[e] = fmaf(rs[e], y[e] * r * wy[e] * act(e), h[e]);
        hh = fmaf(d[e], d[e], hh);
        ax = fmaf(dn[e] * wn[e], d[e], ax);
      }
      sum(hh, ax);
      const float p = 1.f / sqrtf(hh / (float)a.D + a.eps);
      const float m = p > 0.f ? ax * p / (float)a.D : 0.f;   // p is 0 past the squares' range, where ax may be infinite
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = d[e] * p;
        d[e] = fmaf(p, fmaf(-x, m, dn[e] * wn[e]), dho[e]);
        dw[2][e] = fmaf(dn[e], x, dw[2][e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = dho[e];
    }
    if (a.dh && on) store8(static_cast<T*>(a.dh) + t * a.lddh + col, d);
    float dg[8], dot = 0.f;
    if (GATE) g.again();
    if (FEW) y.again();
    if (FEW && GATE && sizeof(T) == 2) {
      wy.again();
      rs.again();
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (GATE) asm("" : "+v"(q[e]));   // the gate's values again from the tail: kept, they took 16 more registers
      const float yr = y[e] * r, u = yr * wy[e], ac = act(e);
      dw[1][e] = fmaf(d[e], u * ac, dw[1][e]);
      const float ez = d[e] * rs[e];
      if (GATE) dg[e] = ez * u * gate_slope<GATE>(g[e], q[e]);
      const float f = ez * ac;
      dw[0][e] = fmaf(f, yr, dw[0][e]);
      d[e] = f * wy[e];
      dot = fmaf(d[e], yr, dot);
    }
    if (GATE && a.dg && on) store8(static_cast<T*>(a.dg) + t * a.lddg + col, dg);
    if (a.norm_y) {
      dot = (a.gw == a.D ? sum(dot) : lanes_sum(dot, a.gw >> 3)) / (float)a.gw;
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = r * fmaf(-y[e] * r, dot, d[e]);
    }
    if (a.dy && on) store8(static_cast<T*>(a.dy) + t * a.lddy + col, d);
  }
  if (!a.part) return;
  // the workgroup's rows together, in 64 bits and one order
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (!(i == 0 ? a.dwy : i == 1 ? a.drs : a.dwn)) continue;
    float* part = a.part + ((int64_t)i * a.wgs + blockIdx.x) * a.D;
    if constexpr (W > 2) {
      if (has) store8(part + col, dw[i]);
    } else {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) red[e * NT + threadIdx.x] = dw[i][e];
      __syncthreads();
      for (int c = threadIdx.x; c < lanes * 8; c += NT) {
        const int l = c >> 3, e = c & 7;
        double s = 0.0;
        for (int k = 0; k < rows; ++k) s += (double)red[e * NT + k * lanes + l];
        if (c < a.D) part[c] = (float)s;
      }
    }
  }
}

// Columns of the partial sums added up over the workgroups: 16 columns per workgroup, 64 rows at a
// time, in 64 bits and one order, behind what earlier launches' rows gave.
__global__ __launch_bounds__(1024) void k_norm_dw(NormArgs a) {
  __shared__ double acc[1024];
  const int which = blockIdx.y;
  float* out = which == 0 ? a.dwy : which == 1 ? a.drs : a.dwn;
  if (!out) return;
  const int c = blockIdx.x * 16 + (threadIdx.x & 15), r0 = threadIdx.x >> 4;
  const float* p = a.part + (int64_t)which * a.wgs * a.D + c;
  double s = 0.0;
  if (c < a.D)
#pragma unroll 8
    for (int r = r0; r < a.wgs; r += 64) s += (double)p[(int64_t)r * a.D];
  acc[threadIdx.x] = s;
  for (int half = 512; half >= 16; half >>= 1) {
    __syncthreads();
    if ((int)threadIdx.x < half) acc[threadIdx.x] += acc[threadIdx.x + half];
  }
  if (threadIdx.x < 16 && c < a.D) {
    double* sofar = a.sofar + which * a.D + c;
    s = acc[threadIdx.x] + (a.begun ? *sofar : 0.0);
    if (a.more) *sofar = s;
    else out[c] = (float)s;
  }
}

// Waves of a row, rows of a workgroup.
int norm_waves(int D) {
  int w = 1;
  while (w * 512 < D) w *= 2;
  return w;
}
int64_t norm_rows(int D) {
  const int w = norm_waves(D);
  return w > 4 ? 1 : NORM_NT / (w > 1 ? 64 * w : norm_lanes(D));
}

void launch_dw(const NormArgs& a, hipStream_t st) {
  hipLaunchKernelGGL(k_norm_dw, dim3((a.D + 15) / 16, 3), dim3(1024), 0, st, a);
}

template <typename T, bool BWD, int GATE, int W>
hipError_t launch_w(const NormArgs& a, hipStream_t st) {
  const dim3 block(norm_threads<W>);
  if constexpr (BWD) {
    const int64_t most = residual_norm_chunk(a.D);
    for (int64_t first = 0; first < a.tokens; first += most) {
      NormArgs p = norm_part(a, first, most, sizeof(T));
      p.wgs = residual_norm_wgs(a.D, p.tokens);
      p.begun = first > 0;
      p.more = first + most < a.tokens;
      hipLaunchKernelGGL((k_norm_bwd<T, W, GATE>), dim3(p.wgs), block, 0, st, p);
      if (a.part) launch_dw(p, st);
    }
  } else {
    const int64_t rows = norm_rows(a.D), most = NORM_LAUNCH * rows;
    for (int64_t first = 0; first < a.tokens; first += most) {
      const NormArgs p = norm_part(a, first, most, sizeof(T));
      hipLaunchKernelGGL((k_norm<T, W, GATE>), dim3((unsigned)((p.tokens + rows - 1) / rows)), block, 0, st, p);
    }
  }
  return hipGetLastError();
}

template <typename T, bool BWD, int GATE>
hipError_t launch_rows(const NormArgs& a, hipStream_t st) {
  switch (norm_waves(a.D)) {
    case 1: return launch_w<T, BWD, GATE, 1>(a, st);
    case 2: return launch_w<T, BWD, GATE, 2>(a, st);
    case 4: return launch_w<T, BWD, GATE, 4>(a, st);
    case 8: return launch_w<T, BWD, GATE, 8>(a, st);
    default: return launch_w<T, BWD, GATE, 16>(a, st);
  }
}

template <typename T, bool BWD>
hipError_t launch_norm(const NormArgs& a, hipStream_t st) {
  return a.gate_kind == TTT_GATE_NONE      ? launch_rows<T, BWD, TTT_GATE_NONE>(a, st)
         : a.gate_kind == TTT_GATE_SIGMOID ? launch_rows<T, BWD, TTT_GATE_SIGMOID>(a, st)
                                           : launch_rows<T, BWD, TTT_GATE_SILU>(a, st);
}

}  // namespace

int32_t residual_norm_wgs(int32_t D, int64_t tokens) {
  const int64_t rows = norm_rows(D), n = (tokens + rows - 1) / rows;
  // whole rounds of the CUs, which hold one workgroup of 16 waves, one or two of 8 and three or four of 4 (gated bf16
  // rows of 4096: 180 us with 384, whose second round fills half of the CUs, 147 with 512, 143 with 256; without a
  // gate 97, 92 and 111)
  const int w = norm_waves(D), most = w > 8 ? 256 : w > 4 ? 512 : 768;
  return (int32_t)(n < most ? n : most);
}

int64_t residual_norm_chunk(int32_t D) {
  return NORM_CHAIN * norm_rows(D) * residual_norm_wgs(D, (int64_t)1 << 25);
}

hipError_t launch_residual_norm(const NormArgs& a, int bf16, hipStream_t st) {
  return bf16 ? launch_norm<u16, false>(a, st) : launch_norm<float, false>(a, st);
}

hipError_t launch_residual_norm_backward(const NormArgs& a, int bf16, hipStream_t st) {
  if (a.tokens) return bf16 ? launch_norm<u16, true>(a, st) : launch_norm<float, true>(a, st);
  if (a.dwy || a.drs || a.dwn) launch_dw(a, st);   // zeros
  return hipGetLastError();
}

}  // namespace ttt
