// Linear attention of one new token per sequence (include/ttt_mixer.h): S <- a S + k v^T, then
// o = c S^T q.
//
// Every state is read once and written once, three operations to an element: the memory bounds
// it.  A workgroup takes some columns of one state (a run of whole rows where there are enough
// sequences), its lanes four of them in one row each; the loads of a lane's rows are under way
// together, before the token's own values come in.  256 sequences of 8 heads of 128 (271 MB): 45 us when
// the last-level cache has some of the states (5.9 TB/s), 56 when it has none (4.8, a copy's rate); 61 of
// 12 heads of 64 (24 MB) 5.5; one sequence 3.5, a launch's time and one memory read's.
#include "ttt_device.hpp"
#include "ttt_mixer_internal.h"

namespace ttt {
namespace {

constexpr int STEP_NT = 256;

template <int K, int COLS>
__global__ __launch_bounds__(STEP_NT) void k_linear_step(LinStepArgs a) {
  constexpr int CL = COLS / 4, G = STEP_NT / CL;   // lanes of a row, rows at a time
  constexpr int R = K / G, RL = R < 16 ? R : 16;   // rows of a lane, and of one round of loads
  __shared__ float qs[K], ks[K];
  __shared__ __attribute__((aligned(16))) float sum[G][COLS];
  const int id = xcd_block(blockIdx.x, a.total);
  const int slice = id % a.slices, sh = id / a.slices;
  const int h = sh % a.heads, seq = sh / a.heads;
  const int g = (int)threadIdx.x / CL, c = 4 * ((int)threadIdx.x % CL);
  const int64_t entry = lin_slot(a.slot, seq, a.slots);
  const int64_t at = ((entry * a.heads + h) * K + g) * a.V + slice * COLS + c;
  const float* in = a.in && entry >= 0 ? a.in + at : nullptr;
  float* fin = a.fin && entry >= 0 ? a.fin + at : nullptr;
  f32x4 s[RL];
  auto load = [&](int i0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < RL; ++i)
      s[i] = in ? *as_global(reinterpret_cast<const f32x4*>(in + (int64_t)(i0 + i) * G * a.V)) : f32x4{};
  };
  load(0);
  if ((int)threadIdx.x < K) {
    qs[threadIdx.x] = bf2f(a.q[seq * a.ldq + (int64_t)h * K + threadIdx.x]);
    ks[threadIdx.x] = bf2f(a.k[seq * a.ldk + (int64_t)h * K + threadIdx.x]);
  }
  const u16* vp = a.v + seq * a.ldv + (int64_t)h * a.V + slice * COLS + c;
  f32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = bf2f(vp[e]);
  const float lam = a.decay[h];
  __syncthreads();
  f32x4 o = f32x4{};
#pragma unroll
  for (int i0 = 0; i0 < R; i0 += RL) {
    if (i0) load(i0);
#pragma unroll
    for (int i = 0; i < RL; ++i) {
      const int row = (i0 + i) * G + g;
      const float kr = ks[row], qr = qs[row];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[i][e] = fmaf(kr, v[e], lam * s[i][e]);
        o[e] = fmaf(qr, s[i][e], o[e]);
      }
      if (fin) *as_global(reinterpret_cast<f32x4*>(fin + (int64_t)(i0 + i) * G * a.V)) = s[i];
    }
  }
  *reinterpret_cast<f32x4*>(&sum[g][c]) = o;
  __syncthreads();
  if ((int)threadIdx.x < COLS) {
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < G; ++i) x += sum[i][threadIdx.x];
    a.out[seq * a.ldo + (int64_t)h * a.V + slice * COLS + threadIdx.x] = f2bf(x * a.scale);
  }
}

template <int K>
hipError_t launch_k(const LinStepArgs& a, int cols, hipStream_t st) {
  const dim3 grid(a.total), block(STEP_NT);
  if (cols == 32) hipLaunchKernelGGL((k_linear_step<K, 32>), grid, block, 0, st, a);
  else if (cols == 64) hipLaunchKernelGGL((k_linear_step<K, 64>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_linear_step<K, 128>), grid, block, 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_step(const LinStepArgs& a, int cols, hipStream_t st) {
  return a.K == 64 ? launch_k<64>(a, cols, st) : a.K == 128 ? launch_k<128>(a, cols, st) : launch_k<256>(a, cols, st);
}

}  // namespace ttt
