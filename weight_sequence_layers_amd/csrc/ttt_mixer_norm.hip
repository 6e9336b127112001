// What stands between two sub-layers in one pass, and its backward (include/ttt_mixer.h).
//
// Mathematics, with mean_g over a group and mean over a row:
//   r = 1 / sqrt(mean_g y^2 + eps), u = y r w_y, z = u act(g), h' = h + s z,
//   p = 1 / sqrt(mean h'^2 + eps), n = h' p w_n.
// Backward: with x = h' p, a = dn w_n:  d = dh' + p (a - x mean(a x)), dw_n = sum dn x,  dh = d,
//   ds = sum d z,  e = d s,  dg = e u act'(g),  f = e act(g),  dw_y = sum f y r,
//   dy = r (f w_y - y r mean_g(f w_y y r)).
//
// Every tensor is read or written once: the memory bounds it.  A row belongs to some lanes of a wave
// (up to 2048 elements) or to a workgroup, 8 elements of a lane side by side, so that a group (a
// power of two of at most 512 elements) lies in neighbouring lanes of one wave; nothing is kept
// between the forward and the backward, which reads its 16 or 32 bits of h and y again instead of
// saved statistics.
#include "ttt_device.hpp"
#include "ttt_mixer_internal.h"

namespace ttt {
namespace {

constexpr int NORM_NT = 256;
constexpr int NORM_WGS = 1024;         // workgroups of a backward launch, at most

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
  __device__ __forceinline__ float operator[](int i) const { return w[i >> 2][i & 3]; }
};
__device__ __forceinline__ void store8(u16* p, const float* x) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = f2bf(x[2 * i]) | ((uint32_t)f2bf(x[2 * i + 1]) << 16);
  *as_global(reinterpret_cast<u32x4*>(p)) = w;
}
__device__ __forceinline__ void store8(float* p, const float* x) {
  *as_global(reinterpret_cast<f32x4*>(p)) = f32x4{x[0], x[1], x[2], x[3]};
  *as_global(reinterpret_cast<f32x4*>(p + 4)) = f32x4{x[4], x[5], x[6], x[7]};
}

// 1 / (1 + exp(-g)) within about two half steps of fp32: the exponent keeps what its product rounds
// off, the reciprocal takes a Newton step; beyond 2^126 it stays there (the sigmoid below 2^-126).
__device__ __forceinline__ float sigmoid(float g) {
  constexpr float L = -1.44269504088896341f, LL = -1.925963033500e-8f;
  float t = g * L;
  const float low = fmaf(g, L, -t) + g * LL;
  t = t > 126.f ? 126.f : t;
  const float x = __builtin_amdgcn_exp2f(t);
  const float d = 1.f + fmaf(x, low * 0.693147181f, x);
  const float r = __builtin_amdgcn_rcpf(d);
  return fmaf(r, fmaf(-d, r, 1.f), r);
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

// Sums over a row.  Of a workgroup's row each call takes the other half of `scratch` in turn, so that one
// barrier keeps its readers from the next call's writers.
template <bool BLOCK>
struct RowSum {
  float (*scratch)[4];
  int lanes, turn = 0;
  __device__ __forceinline__ float operator()(float v) {
    v = lanes_sum(v, BLOCK ? 64 : lanes);
    if constexpr (BLOCK) {
      float* s = scratch[turn];
      turn ^= 1;
      if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
      lds_barrier();
      v = s[0] + s[1] + s[2] + s[3];
    }
    return v;
  }
};

// 1 / root mean square of each vector's group (or of the row).
template <bool BLOCK, int NV>
__device__ __forceinline__ void inv_rms(const float (&ss)[NV], float (&r)[NV], const NormArgs& a, RowSum<BLOCK>& sum) {
  if (a.gw == a.D) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) s += ss[v];
    s = 1.f / sqrtf(sum(s) / (float)a.D + a.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) r[v] = s;
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) r[v] = 1.f / sqrtf(lanes_sum(ss[v], a.gw >> 3) / (float)a.gw + a.eps);
  }
}

// GATE: whether there is a gate; its kind is one select an element.
template <typename T, bool BLOCK, int NV, bool GATE>
__global__ __launch_bounds__(NORM_NT) void k_norm(NormArgs a) {
  __shared__ float scratch[2][4];
  const int lanes = BLOCK ? NORM_NT : norm_lanes(a.D);
  RowSum<BLOCK> sum{scratch, lanes};
  const int lane = (int)threadIdx.x % lanes;
  const int64_t t = BLOCK ? blockIdx.x : (int64_t)blockIdx.x * (NORM_NT / lanes) + threadIdx.x / lanes;
  const bool in = t < a.tokens;       // the sums need a wave's lanes together
  const bool silu = a.gate_kind == TTT_GATE_SILU;
  Raw8<T> y[NV], h[NV], g[NV];
  int col[NV];
  bool on[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    col[v] = (v * lanes + lane) * 8;
    on[v] = in && col[v] < a.D;
    y[v].fill(0.f);
    h[v].fill(0.f);
    g[v].fill(0.f);
    if (on[v]) {
      y[v].load(static_cast<const T*>(a.y) + t * a.ldy + col[v]);
      if (a.h) h[v].load(static_cast<const T*>(a.h) + t * a.ldh + col[v]);
      if (GATE) g[v].load(static_cast<const T*>(a.gate) + t * a.ldg + col[v]);
    }
  }
  float r[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) r[v] = 1.f;
  if (a.norm_y) {
    float ss[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      ss[v] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss[v] = fmaf(y[v][e], y[v][e], ss[v]);
    }
    inv_rms<BLOCK, NV>(ss, r, a, sum);
  }
  float x[NV][8], hh = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    Raw8<T> w, s;
    w.fill(1.f);
    s.fill(1.f);
    if (a.wy && on[v]) w.load(static_cast<const T*>(a.wy) + col[v]);
    if (a.rs && on[v]) s.load(static_cast<const T*>(a.rs) + col[v]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float z = y[v][e] * r[v] * w[e];
      if (GATE) z *= sigmoid(g[v][e]) * (silu ? g[v][e] : 1.f);
      x[v][e] = fmaf(s[e], z, h[v][e]);
      hh = fmaf(x[v][e], x[v][e], hh);
    }
  }
  if (a.ho)
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (on[v]) store8(static_cast<T*>(a.ho) + t * a.ldho + col[v], x[v]);
  if (a.n) {
    const float p = 1.f / sqrtf(sum(hh) / (float)a.D + a.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (on[v]) {
        Raw8<T> w;
        w.fill(1.f);
        if (a.wn) w.load(static_cast<const T*>(a.wn) + col[v]);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[v][e] = x[v][e] * p * w[e];
        store8(static_cast<T*>(a.n) + t * a.ldn + col[v], x[v]);
      }
  }
}

// Backward: the workgroups walk over the rows, so that the partial sums of the scales' gradients are
// few; a second launch adds them up in order.
template <typename T, bool BLOCK, int NV, bool GATE>
__global__ __launch_bounds__(NORM_NT) void k_norm_bwd(NormArgs a) {
  __shared__ float scratch[2][4];
  __shared__ __attribute__((aligned(16))) float red[NORM_NT * 8];
  const int lanes = BLOCK ? NORM_NT : norm_lanes(a.D);
  RowSum<BLOCK> sum{scratch, lanes};
  const int lane = (int)threadIdx.x % lanes, rows = NORM_NT / lanes;
  const bool silu = a.gate_kind == TTT_GATE_SILU;
  int col[NV];
  bool has[NV];
  Raw8<T> wy[NV], rs[NV], wn[NV];
  float dw[3][NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    col[v] = (v * lanes + lane) * 8;
    has[v] = col[v] < a.D;
    wy[v].fill(1.f);
    rs[v].fill(1.f);
    wn[v].fill(1.f);
    if (has[v]) {
      if (a.wy) wy[v].load(static_cast<const T*>(a.wy) + col[v]);
      if (a.rs) rs[v].load(static_cast<const T*>(a.rs) + col[v]);
      if (a.wn) wn[v].load(static_cast<const T*>(a.wn) + col[v]);
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[i][v][e] = 0.f;
  }
  // every lane of a workgroup runs the same rounds: sums need them together
  for (int64_t t0 = (int64_t)blockIdx.x * rows; t0 < a.tokens; t0 += (int64_t)gridDim.x * rows) {
    const int64_t t = t0 + (int)threadIdx.x / lanes;
    const bool in = t < a.tokens;
    Raw8<T> y[NV], h[NV], g[NV], dho[NV], dn[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      y[v].fill(0.f);
      h[v].fill(0.f);
      g[v].fill(0.f);
      dho[v].fill(0.f);
      dn[v].fill(0.f);
      if (in && has[v]) {
        y[v].load(static_cast<const T*>(a.y) + t * a.ldy + col[v]);
        if (a.h) h[v].load(static_cast<const T*>(a.h) + t * a.ldh + col[v]);
        if (GATE) g[v].load(static_cast<const T*>(a.gate) + t * a.ldg + col[v]);
        if (a.dho) dho[v].load(static_cast<const T*>(a.dho) + t * a.lddho + col[v]);
        if (a.dn) dn[v].load(static_cast<const T*>(a.dn) + t * a.lddn + col[v]);
      }
    }
    float r[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) r[v] = 1.f;
    if (a.norm_y) {
      float ss[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        ss[v] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss[v] = fmaf(y[v][e], y[v][e], ss[v]);
      }
      inv_rms<BLOCK, NV>(ss, r, a, sum);
    }
    // the gate's sigmoid, and d, the gradient of h'
    float sg[NV][8], d[NV][8];
    if (GATE)
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) sg[v][e] = sigmoid(g[v][e]);
    auto act = [&](int v, int e) __attribute__((always_inline)) { return GATE ? sg[v][e] * (silu ? g[v][e] : 1.f) : 1.f; };
    auto z = [&](int v, int e) __attribute__((always_inline)) { return y[v][e] * r[v] * wy[v][e] * act(v, e); };
    if (a.dn) {
      float hh = 0.f, ax = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          d[v][e] = fmaf(rs[v][e], z(v, e), h[v][e]);
          hh = fmaf(d[v][e], d[v][e], hh);
          ax = fmaf(dn[v][e] * wn[v][e], d[v][e], ax);
        }
      hh = sum(hh);
      ax = sum(ax);
      const float p = 1.f / sqrtf(hh / (float)a.D + a.eps);
      const float m = ax * p / (float)a.D;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = d[v][e] * p;
          d[v][e] = fmaf(p, fmaf(-x, m, dn[v][e] * wn[v][e]), dho[v][e]);
          dw[2][v][e] = fmaf(dn[v][e], x, dw[2][v][e]);
        }
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) d[v][e] = dho[v][e];
    }
    if (a.dh)
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (in && has[v]) store8(static_cast<T*>(a.dh) + t * a.lddh + col[v], d[v]);
    float dot[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float dg[8];
      dot[v] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float yr = y[v][e] * r[v], u = yr * wy[v][e], ac = act(v, e);
        dw[1][v][e] = fmaf(d[v][e], u * ac, dw[1][v][e]);
        const float ez = d[v][e] * rs[v][e];
        if (GATE) {   // s (1 - s), and for silu s + g s (1 - s)
          const float s = sg[v][e];
          dg[e] = ez * u * (silu ? fmaf(ac, 1.f - s, s) : s * (1.f - s));
        }
        const float f = ez * ac;
        dw[0][v][e] = fmaf(f, yr, dw[0][v][e]);
        d[v][e] = f * wy[v][e];
        dot[v] = fmaf(d[v][e], yr, dot[v]);
      }
      if (GATE && a.dg && in && has[v]) store8(static_cast<T*>(a.dg) + t * a.lddg + col[v], dg);
    }
    if (a.norm_y) {
      if (a.gw == a.D) {
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) s += dot[v];
        s = sum(s) / (float)a.D;
#pragma unroll
        for (int v = 0; v < NV; ++v) dot[v] = s;
      } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) dot[v] = lanes_sum(dot[v], a.gw >> 3) / (float)a.gw;
      }
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) d[v][e] = r[v] * fmaf(-y[v][e] * r[v], dot[v], d[v][e]);
    }
    if (a.dy)
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (in && has[v]) store8(static_cast<T*>(a.dy) + t * a.lddy + col[v], d[v]);
  }
  if (!a.part) return;
  // the workgroup's rows together, in 64 bits and one order
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (!(i == 0 ? a.dwy : i == 1 ? a.drs : a.dwn)) continue;
    float* part = a.part + ((int64_t)i * a.wgs + blockIdx.x) * a.D;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if constexpr (BLOCK) {
        if (has[v]) store8(part + col[v], dw[i][v]);
      } else {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) red[e * NORM_NT + threadIdx.x] = dw[i][v][e];
        __syncthreads();
        for (int c = threadIdx.x; c < lanes * 8; c += NORM_NT) {
          const int e = c / lanes, l = c - e * lanes, at = (v * lanes + l) * 8 + e;
          double s = 0.0;
          for (int k = 0; k < rows; ++k) s += (double)red[e * NORM_NT + k * lanes + l];
          if (at < a.D) part[at] = (float)s;
        }
      }
    }
  }
}

// Columns of the partial sums added up over the workgroups: 16 columns per workgroup, 64 rows at a
// time, in 64 bits and one order.
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
  if (threadIdx.x < 16 && c < a.D) out[c] = (float)acc[threadIdx.x];
}

// Whether a row belongs to a workgroup, and 16- or 32-byte runs of a lane.
constexpr int NORM_WAVE_D = 2048;
int norm_vectors(int D) {
  const int n = D > NORM_WAVE_D ? NORM_NT : norm_lanes(D);
  return (D + 8 * n - 1) / (8 * n);
}
int64_t norm_rows(int D) { return D > NORM_WAVE_D ? 1 : NORM_NT / norm_lanes(D); }

template <typename T, bool BWD, bool GATE>
hipError_t launch_rows(const NormArgs& a, hipStream_t st) {
  const int64_t rows = norm_rows(a.D);
  const dim3 grid(BWD ? (unsigned)a.wgs : (unsigned)((a.tokens + rows - 1) / rows)), block(NORM_NT);
#define NORM_CASE(B, N)                                                                      \
  if constexpr (BWD) hipLaunchKernelGGL((k_norm_bwd<T, B, N, GATE>), grid, block, 0, st, a); \
  else hipLaunchKernelGGL((k_norm<T, B, N, GATE>), grid, block, 0, st, a);                   \
  break;
  switch (norm_vectors(a.D) + (a.D > NORM_WAVE_D ? 4 : 0)) {
    case 1: NORM_CASE(false, 1)
    case 2: NORM_CASE(false, 2)
    case 3: NORM_CASE(false, 3)
    case 4: NORM_CASE(false, 4)
    case 6: NORM_CASE(true, 2)
    case 7: NORM_CASE(true, 3)
    case 8: NORM_CASE(true, 4)
    default: return hipErrorInvalidValue;
  }
#undef NORM_CASE
  return hipGetLastError();
}

template <typename T, bool BWD>
hipError_t launch_norm(const NormArgs& a, hipStream_t st) {
  return a.gate_kind ? launch_rows<T, BWD, true>(a, st) : launch_rows<T, BWD, false>(a, st);
}

}  // namespace

int32_t residual_norm_wgs(int32_t D, int64_t tokens) {
  const int64_t rows = norm_rows(D), n = (tokens + rows - 1) / rows;
  return (int32_t)(n < NORM_WGS ? n : NORM_WGS);
}

hipError_t launch_residual_norm(const NormArgs& a, int bf16, hipStream_t st) {
  return bf16 ? launch_norm<u16, false>(a, st) : launch_norm<float, false>(a, st);
}

hipError_t launch_residual_norm_backward(const NormArgs& a, int bf16, hipStream_t st) {
  if (a.tokens) {
    const hipError_t e = bf16 ? launch_norm<u16, true>(a, st) : launch_norm<float, true>(a, st);
    if (e != hipSuccess) return e;
  }
  if (a.dwy || a.drs || a.dwn) hipLaunchKernelGGL(k_norm_dw, dim3((a.D + 15) / 16, 3), dim3(1024), 0, st, a);
  return hipGetLastError();
}

}  // namespace ttt
