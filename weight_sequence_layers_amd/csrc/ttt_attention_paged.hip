// Attention of one new token per sequence over a paged key-value cache
// (include/ttt_attention.h).
//
// Mathematics.  o = sum_j p_j v_j / sum_j p_j with p_j = 2^(s_j c - m), s_j = q . k_j, c =
// scale log2(e) and m the running maximum: parts of the tokens are summed apart, each with its
// own m, and joined as sum_i 2^(m_i - m) o_i.
//
// Every cached byte is read once: the memory bounds it.  A workgroup takes one key head of one
// sequence, the query heads that share it (up to 16, the columns of a 16 x 16 x 32 MFMA; with
// fewer the spare columns cost nothing that counts) and one part of the tokens; its four waves
// take 32 tokens in turn (16 of heads of 256).  A step's rows are loaded into registers in the order they lie in
// memory while the step before is computed, and put into the wave's own LDS tiles: K is read
// back along its rows as the A operand of S^T = K Q^T, so each lane holds 8 tokens of one query
// head and P^T is already laid out as the second product's B operand; V is read transposed.
//
// Measured, with the join: one context of 131072 tokens, 8 heads: 86 to 91 us, 6.0 TB/s of cached
// bytes (reading alone, 4 GB in 16-byte loads, reaches 6.5 to 6.8); 64 sequences up to 8192 tokens,
// 32 query heads on 8: 193 us, 5.7 TB/s; 96 windows of 2048 in e4m3: 37 to 39 us, 4.2 TB/s (4.7 us
// of it the join, a few the chain length - page - row of a workgroup's start).  e4m3 halves the
// bytes under way, not the latency: one context takes 53 us, heads of 256 93 (79 at the rate of
// reading), bf16 heads of 256 174 (158); 16 ragged sequences of e4m3 heads of 256, 4 key heads, 39
// us (20), whose registers leave two waves to a SIMD.  The kernels read 1.001 times the cached
// bytes.  K's fragments straight from memory (64 bytes of a row per load) read 2 to 6 % slower than
// through LDS.
#include "ttt_attention_internal.h"

namespace ttt {
namespace {

typedef short s16x8 __attribute__((ext_vector_type(8)));

// what rows outside the sequence or the cache read: lanes of a step that has fewer tokens
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ const u32x4 k_zero_row = {0u, 0u, 0u, 0u};

// 8 e4m3 numbers as bf16 (exact: e4m3's 4 significant bits and its range lie within bf16's)
__device__ __forceinline__ u32x4 bf16_of_e4m3(uint32_t lo, uint32_t hi) {
  return u32x4{
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true))};
}

// place of 16-byte chunk c of row r of a V tile (rows of D bf16): the rows that one transposing
// read touches land on distinct banks
template <int D>
__device__ __forceinline__ int vt_chunk(int r, int c) {
  if (D == 64) return c ^ (((r >> 1) & 3) << 1);
  return c ^ ((r & 7) << 1);
}

// The wave's LDS accesses before come before those after (a wave's own are in order in the
// hardware: this holds the compiler to it).
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// place of 16-byte chunk c of row r of a K tile (rows as cached, RB bytes): 16 consecutive
// rows at one chunk lie on distinct banks
template <int RB>
__device__ __forceinline__ int kt_chunk(int r, int c) {
  if (RB == 64) return c ^ ((r >> 2) & 3);
  if (RB == 128) return c ^ ((r >> 1) & 7);
  return c ^ (r & 15);
}

// Four of an output row: sums times inv, an infinite one (of an infinite value) as NaN.  The two
// parts of its probability alone would make it an infinity or a NaN by their low bits.
__device__ __forceinline__ uint2 out4(const f32x4& acc, float inv) {
  float x[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const float y = acc[v] * inv;
    x[v] = fmaf(y, 0.f, y);
  }
  return uint2{f2bf(x[0]) | ((uint32_t)f2bf(x[1]) << 16), f2bf(x[2]) | ((uint32_t)f2bf(x[3]) << 16)};
}

// the first four of a lane's eight probabilities
__device__ __forceinline__ s16x4 low4(bf16x8 p) {
  const s16x8 x = __builtin_bit_cast(s16x8, p);
  return __builtin_shufflevector(x, x, 0, 1, 2, 3);
}

template <int D, bool E4>
struct PagedShape {
  static constexpr int RB = D * (E4 ? 1 : 2);         // bytes of a cached row
  static constexpr int STEP = D == 256 ? 16 : 32;     // tokens of a wave's step
  static constexpr int BLOCK = STEP * PG_WAVES;       // and of the workgroup's
  static_assert(PG_BLOCK % BLOCK == 0, "a part is whole steps");
  static constexpr int KL = STEP * RB / 16 / 64;      // 16-byte loads per lane of a step's rows
  static constexpr int LR = RB / 16;                  // lanes of a row
  static constexpr int RPI = 64 / LR;                 // rows per load
  static constexpr int KS = D / 32;                   // MFMA steps along D
  static constexpr int KT = STEP * RB;                // bytes of a wave's K tile, as cached
  static constexpr int VT = STEP * D * 2;             // bytes of a wave's V tile, bf16
};

// Registers held to three waves per SIMD for e4m3 heads of 128 (the compiler takes two's worth
// by itself): half the bytes per step leave too few in flight with two (96 windows of 2048:
// 47.7 -> 42.2 us).  For heads of 256 to two, with steps of 16 tokens: steps of 32 fill the LDS
// and the registers with one (16 sequences up to 8192 tokens, 4 key heads: bf16 64.8 -> 59.7 us,
// e4m3 49.1 -> 39.7 us; one of 65536: bf16 53.6 -> 49.6 us).
template <int D, bool E4>
__global__ __launch_bounds__(PG_NT, D == 256 ? 2 : D == 128 && E4 ? 3 : 1) void k_paged(PagedArgs a) {
  using S = PagedShape<D, E4>;
  // the waves' K and V tiles, and after the loop their sums
  constexpr int JOIN = PG_WAVES * PG_HEADS * D * 4;
  constexpr int TILES = PG_WAVES * (S::KT + S::VT);
  constexpr int LDS = TILES > JOIN ? TILES : JOIN;
  __shared__ __attribute__((aligned(1024))) char lds[LDS];
  __shared__ float wm[PG_WAVES][PG_HEADS], wl[PG_WAVES][PG_HEADS];

  int id = blockIdx.x;
  const int sp = id % a.splits;
  id /= a.splits;
  const int ht = id % a.htiles;
  id /= a.htiles;
  const int kh = id % a.kv_heads, seq = id / a.kv_heads;
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int h0 = ht * PG_HEADS;                       // first query head of the group
  const int nh = min(PG_HEADS, a.group - h0);

  int lo, hi;
  paged_span(a.lens[seq], a.max_pages, a.page_size, a.window, lo, hi);
  const int part = paged_part(hi - lo, a.splits);
  const int b0 = lo + min(hi - lo, sp * part), b1 = min(hi, b0 + part);
  if (b0 >= b1 && sp > 0) return;   // part 0 stays: it writes an empty sequence's row
  const bool whole = part >= hi - lo;                 // this part is all of it

  // Q fragments: column n, k index 8 g + i of step s
  bf16x8 qf[S::KS];
  {
    const u16* qr = a.q + (int64_t)seq * a.ldq + ((int64_t)kh * a.group + h0 + n) * D;
#pragma unroll
    for (int s = 0; s < S::KS; ++s) {
      const int d = E4 ? 64 * (s >> 1) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g;
      if (n < nh) qf[s] = *reinterpret_cast<const bf16x8*>(qr + d);
      else qf[s] = bf16x8{};
    }
  }
  const float ksc = E4 && a.ks ? a.ks[kh] : 1.f, vsc = E4 && a.vs ? a.vs[kh] : 1.f;
  const float c2 = a.scale * ksc * 1.44269504088896341f;

  const int32_t* tab = a.table + (int64_t)seq * a.max_pages;
  const char* zero = reinterpret_cast<const char*>(&k_zero_row);
  // lane l < STEP of a step at token k0: the page of token k0 + l, and its row's byte offset (-1
  // for none)
  auto page_of = [&](int k0) __attribute__((always_inline)) {
    const int key = k0 + (lane & (S::STEP - 1));
    return key < b1 ? tab[key / a.page_size] : -1;
  };
  auto row_of = [&](int page, int k0) __attribute__((always_inline)) {
    return paged_row(page, a.pages, a.page_bytes, kh, a.page_size, (k0 + (lane & (S::STEP - 1))) % a.page_size, S::RB);
  };
  auto at_lane = [](int64_t x, int l) __attribute__((always_inline)) {
    const int lo32 = __shfl((int)(uint32_t)x, l, 64), hi32 = __shfl((int)(x >> 32), l, 64);
    return (int64_t)(((uint64_t)(uint32_t)hi32 << 32) | (uint32_t)lo32);
  };
  // every row is read once: loads that leave no line behind (one 131072-token context: 5.4 ->
  // 6.2 TB/s)
  u32x4 kr[S::KL], vr[S::KL];
  auto load = [&](int64_t row) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < S::KL; ++i) {
      const int64_t off = at_lane(row, S::RPI * i + lane / S::LR);
      const int64_t at = off + 16 * (lane % S::LR);
      kr[i] = __builtin_nontemporal_load(as_global(reinterpret_cast<const u32x4*>(off >= 0 ? a.k + at : zero)));
      vr[i] = __builtin_nontemporal_load(as_global(reinterpret_cast<const u32x4*>(off >= 0 ? a.v + at : zero)));
    }
  };

  f32x4 o[D / 16];
#pragma unroll
  for (int i = 0; i < D / 16; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;
  char* kt = lds + w * (S::KT + S::VT);
  char* vt = kt + S::KT;

  int k0 = b0 + w * S::STEP;
  // Page numbers are loaded before the rows of the step ahead of theirs: loads return in order,
  // so waiting for them does not wait for rows still on their way.
  const int page0 = page_of(k0);
  int npage = page_of(k0 + S::BLOCK);
  int64_t row = row_of(page0, k0);
  load(row);
  for (; k0 < b1; k0 += S::BLOCK) {
    // this step's rows into the wave's tiles, the next step's on their way
#pragma unroll
    for (int i = 0; i < S::KL; ++i) {
      const int r = S::RPI * i + lane / S::LR, c = lane % S::LR;
      *reinterpret_cast<u32x4*>(kt + r * S::RB + (kt_chunk<S::RB>(r, c) << 4)) = kr[i];
    }
#pragma unroll
    for (int i = 0; i < S::KL; ++i) {
      const int r = S::RPI * i + lane / S::LR, c = lane % S::LR;
      char* dst = vt + r * D * 2;
      if constexpr (E4) {
        *reinterpret_cast<u32x4*>(dst + (vt_chunk<D>(r, 2 * c) << 4)) = bf16_of_e4m3(vr[i].x, vr[i].y);
        *reinterpret_cast<u32x4*>(dst + (vt_chunk<D>(r, 2 * c + 1) << 4)) = bf16_of_e4m3(vr[i].z, vr[i].w);
      } else {
        *reinterpret_cast<u32x4*>(dst + (vt_chunk<D>(r, c) << 4)) = vr[i];
      }
    }
    // tokens without a row (past the end, a page outside the cache) are left out
    const uint32_t have = (uint32_t)__ballot(row >= 0);
    row = row_of(npage, k0 + S::BLOCK);
    npage = page_of(k0 + 2 * S::BLOCK);
    load(row);
    wave_order();
    // scores: element v of tile t is token k0 + 16 t + 4 g + v of query head n
    constexpr int NT = S::STEP / 16;
    f32x4 sc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = 16 * t + n;
      sc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < S::RB / 64; ++s) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(kt + r * S::RB + (kt_chunk<S::RB>(r, 4 * s + g) << 4));
        if constexpr (E4) {
          sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, bf16_of_e4m3(x.x, x.y)), qf[2 * s], sc[t], 0, 0, 0);
          sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, bf16_of_e4m3(x.z, x.w)), qf[2 * s + 1], sc[t], 0, 0, 0);
        } else {
          sc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), qf[s], sc[t], 0, 0, 0);
        }
      }
    }
    float mx = -INFINITY;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        // x - x: a score of -inf is a NaN, not a token left out
        sc[t][v] = (have >> (16 * t + 4 * g + v)) & 1 ? fmaf(sc[t][v], c2, sc[t][v] - sc[t][v]) : -INFINITY;
        mx = fmaxf(mx, sc[t][v]);
      }
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float mnew = fmaxf(m, mx), mref = mnew == -INFINITY ? 0.f : mnew;
    if (__any(mnew != m)) {
      const float al = __builtin_amdgcn_exp2f(m - mref);
      l *= al;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) o[i][v] *= al;
    }
    m = mnew;
    // two bf16 numbers per probability: what the first leaves, the second holds, 16 bits in all
    bf16x8 ph, pl;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float p = __builtin_amdgcn_exp2f(sc[t][v] - mref);
        const __bf16 hi16 = static_cast<__bf16>(p);
        l += p;
        ph[4 * t + v] = hi16;
        pl[4 * t + v] = static_cast<__bf16>(p - static_cast<float>(hi16));
      }
    // O^T += V^T P^T: k slot (g, i) is token 4 g + i (i < 4) or 16 + 4 g + i - 4
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
      s16x4 part2[2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int r = 16 * t + 4 * g + (n >> 2), d = 16 * mt + 4 * (n & 3);
        const char* p = vt + r * D * 2 + (vt_chunk<D>(r, d >> 3) << 4) + (d & 7) * 2;
        part2[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p));
      }
      if constexpr (NT == 2) {
        const s16x8 vv = __builtin_shufflevector(part2[0], part2[1], 0, 1, 2, 3, 4, 5, 6, 7);
        const bf16x8 vf = __builtin_bit_cast(bf16x8, vv);
        o[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, ph, o[mt], 0, 0, 0);
        o[mt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pl, o[mt], 0, 0, 0);
      } else {
        o[mt] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(part2[0], low4(ph), o[mt], 0, 0, 0);
        o[mt] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(part2[0], low4(pl), o[mt], 0, 0, 0);
      }
    }
    wave_order();
  }

  // join the waves: l over the lanes of a head, then the four waves' sums through LDS
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (g == 0) {
    wm[w][n] = m;
    wl[w][n] = l;
  }
  __syncthreads();   // every wave is done with its V tile
  float* os = reinterpret_cast<float*>(lds) + (w * PG_HEADS + n) * D;
  if (n < nh)
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt)
      *reinterpret_cast<f32x4*>(os + 16 * mt + 4 * g) = o[mt];
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(lds);
  for (int i = threadIdx.x; i < nh * (D / 4); i += PG_NT) {
    const int h = i / (D / 4), d = (i % (D / 4)) * 4;
    float mm = -INFINITY, ll = 0.f;
    for (int x = 0; x < PG_WAVES; ++x) mm = fmaxf(mm, wm[x][h]);
    const float mr = mm == -INFINITY ? 0.f : mm;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int x = 0; x < PG_WAVES; ++x) {
      const float f = __builtin_amdgcn_exp2f(wm[x][h] - mr);
      ll += f * wl[x][h];
      const f32x4 ox = *reinterpret_cast<const f32x4*>(all + (x * PG_HEADS + h) * D + d);
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[v] += f * ox[v];
    }
    const int64_t head = (int64_t)kh * a.group + h0 + h;
    if (whole) {
      const float inv = ll == 0.f ? 0.f : vsc / ll;   // no token: zeros; a NaN stays one
      *reinterpret_cast<uint2*>(a.out + (int64_t)seq * a.ldo + head * D + d) = out4(acc, inv);
      if (d == 0 && a.lse)
        a.lse[(int64_t)seq * a.heads + head] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.69314718055994531f;
    } else {
      const int64_t at = ((int64_t)seq * a.heads + head) * a.splits + sp;
      *reinterpret_cast<f32x4*>(a.po + at * D + d) = acc;
      if (d == 0) {
        a.pm[2 * at] = mm;
        a.pm[2 * at + 1] = ll;
      }
    }
  }
}

// Joins the parts of every sequence that took more than one: a workgroup per query head, whose
// groups of D / 4 threads each sum every G-th part before the groups are joined through LDS.
template <int D>
__global__ __launch_bounds__(256) void k_paged_join(PagedArgs a) {
  constexpr int TPH = D / 4, G = 256 / TPH;
  __shared__ __attribute__((aligned(16))) float acc_s[G][D];
  __shared__ float m_s[G], l_s[G];
  const int64_t id = blockIdx.x;
  const int seq = (int)(id / a.heads), head = (int)(id % a.heads);
  const int g = threadIdx.x / TPH, d = (threadIdx.x % TPH) * 4;
  int lo, hi;
  paged_span(a.lens[seq], a.max_pages, a.page_size, a.window, lo, hi);
  const int part = paged_part(hi - lo, a.splits);
  if (part >= hi - lo) return;
  const int np = (hi - lo + part - 1) / part;
  const float* pm = a.pm + id * a.splits * 2;
  const float* po = a.po + id * a.splits * D + d;
  float mm = -INFINITY;
#pragma unroll 4
  for (int i = g; i < np; i += G) mm = fmaxf(mm, pm[2 * i]);
  const float mr = mm == -INFINITY ? 0.f : mm;
  float ll = 0.f;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int i = g; i < np; i += G) {
    const float f = __builtin_amdgcn_exp2f(pm[2 * i] - mr);
    const f32x4 ox = *reinterpret_cast<const f32x4*>(po + (int64_t)i * D);
    ll += f * pm[2 * i + 1];
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] += f * ox[v];
  }
  *reinterpret_cast<f32x4*>(&acc_s[g][d]) = acc;
  if (d == 0) {
    m_s[g] = mm;
    l_s[g] = ll;
  }
  __syncthreads();
  if (g) return;
  float mt = -INFINITY, lt = 0.f;
  for (int i = 0; i < G; ++i) mt = fmaxf(mt, m_s[i]);
  const float mtr = mt == -INFINITY ? 0.f : mt;
  acc = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < G; ++i) {
    const float f = __builtin_amdgcn_exp2f(m_s[i] - mtr);
    const f32x4 ox = *reinterpret_cast<const f32x4*>(&acc_s[i][d]);
    lt += f * l_s[i];
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] += f * ox[v];
  }
  const float vsc = a.vs ? a.vs[head / a.group] : 1.f;
  const float inv = lt == 0.f ? 0.f : vsc / lt;
  *reinterpret_cast<uint2*>(a.out + (int64_t)seq * a.ldo + (int64_t)head * D + d) = out4(acc, inv);
  if (d == 0 && a.lse)
    a.lse[id] = lt == 0.f ? -INFINITY : (mt + log2f(lt)) * 0.69314718055994531f;
}

template <int D>
hipError_t launch_paged_d(const PagedArgs& a, int e4m3, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.seqs * a.kv_heads * a.htiles * a.splits));
  if (e4m3) hipLaunchKernelGGL((k_paged<D, true>), grid, dim3(PG_NT), 0, st, a);
  else hipLaunchKernelGGL((k_paged<D, false>), grid, dim3(PG_NT), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL(k_paged_join<D>, dim3((unsigned)((int64_t)a.seqs * a.heads)), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_paged(const PagedArgs& a, int D, int e4m3, hipStream_t st) {
  if (D == 64) return launch_paged_d<64>(a, e4m3, st);
  if (D == 128) return launch_paged_d<128>(a, e4m3, st);
  if (D == 256) return launch_paged_d<256>(a, e4m3, st);
  return hipErrorInvalidValue;
}

}  // namespace ttt
