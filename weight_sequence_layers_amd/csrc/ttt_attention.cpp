// Host side of the attention calls (include/ttt_attention.h): argument checks, launch sizes,
// workspace layout.
#include "ttt_attention.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "ttt_attention_internal.h"
#include "ttt_block_host.h"

using namespace ttt;

namespace {

constexpr int64_t LD_MAX = (int64_t)1 << 28;   // keeps every byte offset within int64

// A matrix of `rows` rows of `width` bytes, `ld` bytes apart.
struct Rows {
  const void* p;
  int64_t rows, width, ld;
};

// Whether two such matrices share a byte.  Matrices of one stride whose rows lie side by side
// (thirds of one projection's rows) do not.
bool share(const Rows& a, const Rows& b) {
  if (a.rows <= 0 || b.rows <= 0) return false;
  const size_t na = (size_t)((a.rows - 1) * a.ld + a.width), nb = (size_t)((b.rows - 1) * b.ld + b.width);
  if (!overlaps(a.p, na, b.p, nb)) return false;
  if (a.ld != b.ld) return true;
  const int64_t d = (int64_t)(reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p));
  const int64_t m = ((d % a.ld) + a.ld) % a.ld;   // b's column offset in a's rows
  return m < a.width || m + b.width > a.ld;
}

// `bytes` bytes in a row; NULL, or a call that does not touch them, is none.
Rows flat(const void* p, int64_t bytes) { return {p, p && bytes > 0 ? 1 : 0, bytes, bytes}; }

// Whether what a call writes shares a byte with the tables it reads or with its other outputs.
bool clash(std::initializer_list<Rows> outs, std::initializer_list<Rows> ins) {
  for (const Rows* o = outs.begin(); o != outs.end(); ++o) {
    for (const Rows& r : ins)
      if (share(*o, r)) return true;
    for (const Rows* x = outs.begin(); x != o; ++x)
      if (share(*o, *x)) return true;
  }
  return false;
}

ttt_status check_rope(const ttt_rope_config* c) {
  if (!c) return failf(TTT_E_NULL, "config is NULL");
  if (c->q_heads < 1 || c->q_heads > 4096 || c->k_heads < 1 || c->k_heads > 4096)
    return failf(TTT_E_SHAPE, "q_heads %d, k_heads %d: in [1, 4096]", c->q_heads, c->k_heads);
  if (c->head_dim < 16 || c->head_dim > 1024 || c->head_dim % 16)
    return failf(TTT_E_SHAPE, "head_dim %d: a multiple of 16 in [16, 1024]", c->head_dim);
  if (c->rot_dim < 0 || c->rot_dim > c->head_dim || c->rot_dim % 16)
    return failf(TTT_E_SHAPE, "rot_dim %d: a multiple of 16 in [0, head_dim %d]", c->rot_dim,
                 c->head_dim);
  if (c->axes < 1 || c->axes > 4) return failf(TTT_E_SHAPE, "axes %d: in [1, 4]", c->axes);
  if (c->pairing != TTT_ROPE_HALVES && c->pairing != TTT_ROPE_PAIRS)
    return failf(TTT_E_CONFIG, "unknown pairing %d", c->pairing);
  if (c->norm != TTT_HEAD_NORM_NONE && c->norm != TTT_HEAD_NORM_RMS)
    return failf(TTT_E_CONFIG, "unknown head norm %d", c->norm);
  if (c->act != TTT_F32 && c->act != TTT_BF16)
    return failf(TTT_E_DTYPE, "unknown activation dtype %d", c->act);
  if (c->norm == TTT_HEAD_NORM_RMS && !(std::isfinite(c->eps) && c->eps > 0.f))
    return failf(TTT_E_CONFIG, "eps %g: finite and > 0", (double)c->eps);
  return TTT_OK;
}

int act_size(const ttt_rope_config* c) { return c->act == TTT_BF16 ? 2 : 4; }

// at most 2^23 workgroups of 256 threads (a block is at least 4 tokens for so many): a launch's
// threads are counted in 32 bits
ttt_status check_tokens(int64_t tokens) {
  if (tokens < 0 || tokens > ((int64_t)1 << 25))
    return failf(TTT_E_SHAPE, "tokens %lld: in [0, 2^25]", (long long)tokens);
  return TTT_OK;
}

ttt_status check_ld(int64_t ld, int64_t width, int size, const char* name) {
  if (ld < width || ld > LD_MAX || ld * size % 16)
    return failf(TTT_E_SHAPE, "%s %lld: at least %lld, rows 16-byte aligned", name, (long long)ld,
                 (long long)width);
  return TTT_OK;
}

ttt_status optional(const void* p, const char* name) { return p ? need(p, name) : TTT_OK; }

// The arguments that every norm-and-rotation call shares, checked.
ttt_status rope_common(const ttt_rope_config* c, const void* qw, const void* kw, const float* freq,
                       const int32_t* pos) {
  if (c->norm == TTT_HEAD_NORM_NONE && (qw || kw))
    return failf(TTT_E_CONFIG, "learned scales without a norm");
  BLK_TRY(optional(qw, "q_weight"));
  BLK_TRY(optional(kw, "k_weight"));
  if (c->rot_dim) {
    BLK_TRY(need(freq, "freq"));
    BLK_TRY(need(pos, "pos"));
  }
  return TTT_OK;
}

// The tables that every norm-and-rotation call reads.
struct RopeTables {
  Rows qw, kw, freq, pos;
};

RopeTables rope_tables(const ttt_rope_config* c, const void* qw, const void* kw, const float* freq,
                       const int32_t* pos, int64_t tokens) {
  const int64_t w = (int64_t)c->head_dim * act_size(c), turns = c->rot_dim ? c->axes * (int64_t)4 : 0;
  return {flat(qw, w), flat(kw, w), flat(freq, turns * (c->rot_dim / 2)), flat(pos, turns * tokens)};
}

RopeArgs rope_args(const ttt_rope_config* c, const void* qw, const void* kw, const float* freq,
                   const int32_t* pos, int64_t tokens) {
  RopeArgs a = {};
  a.q.w = qw;
  a.k.w = kw;
  a.q.heads = c->q_heads;
  a.k.heads = c->k_heads;
  a.freq = freq;
  a.pos = pos;
  a.tokens = tokens;
  a.D = c->head_dim;
  a.rot = c->rot_dim;
  a.axes = c->axes;
  a.pairs = c->pairing == TTT_ROPE_PAIRS;
  a.norm = c->norm;
  a.eps = c->eps;
  a.lph = 1;
  while (a.lph * 16 < a.D) a.lph *= 2;
  // tokens per workgroup: enough workgroups for eight to a CU first, then up to 16 tokens that fit
  // the LDS table (the angles are shared by a token's heads only).  A side of few small heads then
  // has fewer heads in a block than the workgroup's groups: with one query and one key head of 64,
  // 131072 tokens take 24 us and the backward 64, against 14 and 20 at a copy's rate.
  const int fit = a.rot ? std::min(ROPE_MAX_TB, ROPE_TURNS / (a.rot / 2)) : ROPE_MAX_TB;
  a.tb = (int32_t)std::max<int64_t>(1, std::min<int64_t>(fit, tokens / 2048));
  return a;
}

ttt_status check_cache(const ttt_kv_cache* c) {
  if (!c) return failf(TTT_E_NULL, "cache is NULL");
  if (c->dtype != TTT_CACHE_BF16 && c->dtype != TTT_CACHE_E4M3)
    return failf(TTT_E_DTYPE, "unknown cache dtype %d", c->dtype);
  if (c->reserved) return failf(TTT_E_CONFIG, "reserved field must be 0");
  if (c->pages < 1) return failf(TTT_E_SHAPE, "pages %d < 1", c->pages);
  if (c->page_size < 1 || c->page_size > 65536)
    return failf(TTT_E_SHAPE, "page_size %d: in [1, 65536]", c->page_size);
  if (c->kv_heads < 1 || c->kv_heads > 4096)
    return failf(TTT_E_SHAPE, "kv_heads %d: in [1, 4096]", c->kv_heads);
  if (c->head_dim < 16 || c->head_dim > 1024 || c->head_dim % 16)
    return failf(TTT_E_SHAPE, "head_dim %d: a multiple of 16 in [16, 1024]", c->head_dim);
  const int64_t page = (int64_t)c->kv_heads * c->page_size * c->head_dim;
  const int size = c->dtype == TTT_CACHE_BF16 ? 2 : 1;
  if (c->page_stride < page || c->page_stride > ((int64_t)1 << 40) || c->page_stride * size % 16)
    return failf(TTT_E_SHAPE, "page_stride %lld: at least %lld, pages 16-byte aligned",
                 (long long)c->page_stride, (long long)page);
  if ((double)c->pages * (double)c->page_stride >= 4611686018427387904.0)
    return failf(TTT_E_SHAPE, "pages * page_stride too large");
  if (c->dtype == TTT_CACHE_BF16 && (c->k_scale || c->v_scale))
    return failf(TTT_E_CONFIG, "scales with a bf16 cache");
  return TTT_OK;
}

ttt_status check_cache_pointers(const ttt_kv_cache* c) {
  BLK_TRY(need(c->k, "cache k"));
  BLK_TRY(need(c->v, "cache v"));
  BLK_TRY(optional(c->k_scale, "k_scale"));
  return optional(c->v_scale, "v_scale");
}

// keys or values of a cache: pages as rows
Rows cache_rows(const ttt_kv_cache* c, const void* p) {
  const int64_t size = c->dtype == TTT_CACHE_BF16 ? 2 : 1;
  return {p, c->pages, (int64_t)c->kv_heads * c->page_size * c->head_dim * size, c->page_stride * size};
}

// workgroups of a backward launch: one per token block, at most ROPE_BWD_WGS, which walk over
// the blocks
int32_t bwd_wgs(const RopeArgs& a) {
  return (int32_t)std::min<int64_t>((a.tokens + a.tb - 1) / a.tb, ROPE_BWD_WGS);
}

int64_t bwd_work_bytes(const ttt_rope_config* c, int64_t tokens) {
  if (c->norm == TTT_HEAD_NORM_NONE || tokens == 0) return 0;
  const RopeArgs a = rope_args(c, nullptr, nullptr, nullptr, nullptr, tokens);
  return (int64_t)2 * bwd_wgs(a) * a.D * (int64_t)sizeof(float);
}

// Parts that each sequence's tokens are split into, at most.  The lengths are on the device, so
// the rule goes by the longest span a sequence may have.
//   - enough workgroups to fill the CUs once, as many to a CU as keep the memory busy
//     (paged_per_cu): more parts than that only make the join longer (one 131072-token sequence
//     of 8 heads: 90.5 us at 512 workgroups, 95.7 at 2048).  Room is for one more of heads of 64 and
//     of bf16 heads of 256 (8 heads, one sequence of 131072 tokens, heads of 64: 49.2 us, 50.9 with
//     three to a CU; of 65536, heads of 256: 91.0 us, 92.5 with two);
//   - no part above PG_MAX_PART tokens, so that one long sequence among short ones is not left
//     to a few workgroups (64 sequences up to 8192 tokens: 193.5 us, against 199.8 unsplit), while
//     the launch stays below PG_WGS_MOST workgroups, most of which a ragged batch leaves empty;
//   - no part below PG_MIN_PART tokens: two steps of every wave.
constexpr int64_t PG_MAX_PART = 2048, PG_MIN_PART = 256, PG_WGS_MOST = 16384, NUM_CU = 256;

int64_t paged_per_cu(int32_t D, bool e4m3) { return D == 128 ? (e4m3 ? 3 : 2) : D == 64 || e4m3 ? 2 : 1; }

int32_t paged_splits(int64_t wgs, int64_t span, int64_t per_cu) {
  if (wgs == 0) return 1;
  const int64_t fill = (NUM_CU * per_cu + wgs - 1) / wgs;
  const int64_t even = std::min((span + PG_MAX_PART - 1) / PG_MAX_PART, PG_WGS_MOST / wgs);
  return (int32_t)std::max<int64_t>(1, std::min(std::max(fill, even), span / PG_MIN_PART));
}

struct PagedPlan {
  int32_t group, htiles, splits;
  int64_t bytes, sums;   // workspace; of which the parts' sums come first
};

ttt_status paged_plan(const ttt_kv_cache* c, int32_t seqs, int32_t heads, int32_t max_pages,
                      int32_t window, PagedPlan* p) {
  BLK_TRY(check_cache(c));
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return failf(TTT_E_UNSUPPORTED, "head_dim %d: 64, 128 or 256", c->head_dim);
  if (seqs < 0 || seqs > (1 << 20)) return failf(TTT_E_SHAPE, "seqs %d: in [0, 2^20]", seqs);
  if (heads < 1 || heads > 65536 || heads % c->kv_heads)
    return failf(TTT_E_SHAPE, "heads %d: a multiple of kv_heads %d in [1, 65536]", heads, c->kv_heads);
  // the join's threads, 256 to a row, are counted in 32 bits
  if ((int64_t)seqs * heads >= ((int64_t)1 << 24))
    return failf(TTT_E_SHAPE, "seqs * heads %lld: below 2^24", (long long)seqs * heads);
  if (max_pages < 0 || (int64_t)max_pages * c->page_size > ((int64_t)1 << 30))
    return failf(TTT_E_SHAPE, "max_pages %d of %d tokens: at most 2^30 tokens", max_pages, c->page_size);
  if (window < 0) return failf(TTT_E_SHAPE, "window %d < 0", window);
  p->group = heads / c->kv_heads;
  p->htiles = (p->group + PG_HEADS - 1) / PG_HEADS;
  int64_t span = (int64_t)max_pages * c->page_size;
  if (window) span = std::min<int64_t>(span, window);
  p->splits = paged_splits((int64_t)seqs * c->kv_heads * p->htiles, span,
                           paged_per_cu(c->head_dim, c->dtype == TTT_CACHE_E4M3));
  const int64_t parts = p->splits > 1 ? (int64_t)seqs * heads * p->splits : 0;
  p->sums = parts * c->head_dim * (int64_t)sizeof(float);
  p->bytes = p->sums + parts * 2 * (int64_t)sizeof(float);
  return TTT_OK;
}

WindowArgs window_args(const void* q, const void* k, const void* v, int64_t ld, void* out,
                       int64_t ld_out, float* lse, int32_t heads, int64_t T, int32_t window,
                       int32_t mode) {
  WindowArgs a = {};
  a.q = static_cast<const u16*>(q);
  a.k = static_cast<const u16*>(k);
  a.v = static_cast<const u16*>(v);
  a.ld = ld;
  a.out = static_cast<u16*>(out);
  a.ldo = ld_out;
  a.lse = lse;
  a.T = (int32_t)T;
  a.heads = heads;
  a.window = (int32_t)std::min<int64_t>(window, T);   // no row sees more
  a.mode = mode;
  a.scale = (float)(1.0 / std::sqrt((double)ATT_D));
  a.scale2 = (float)(1.4426950408889634 / std::sqrt((double)ATT_D));
  return a;
}

}  // namespace

extern "C" {

ttt_status ttt_validate_rope_config(const ttt_rope_config* cfg) { return check_rope(cfg); }

ttt_status ttt_qk_norm_rope(const ttt_rope_config* cfg, const void* q, int64_t ld_q,
                            const void* k, int64_t ld_k, const void* q_weight,
                            const void* k_weight, const float* freq, const int32_t* pos,
                            void* q_out, int64_t ld_qo, void* k_out, int64_t ld_ko,
                            int64_t tokens, void* stream) {
  BLK_TRY(check_rope(cfg));
  BLK_TRY(check_tokens(tokens));
  const int sz = act_size(cfg);
  const int64_t qn = (int64_t)cfg->q_heads * cfg->head_dim, kn = (int64_t)cfg->k_heads * cfg->head_dim;
  BLK_TRY(check_ld(ld_q, qn, sz, "ld_q"));
  BLK_TRY(check_ld(ld_k, kn, sz, "ld_k"));
  BLK_TRY(check_ld(ld_qo, qn, sz, "ld_qo"));
  BLK_TRY(check_ld(ld_ko, kn, sz, "ld_ko"));
  if (tokens == 0) return TTT_OK;
  BLK_TRY(need(q, "q"));
  BLK_TRY(need(k, "k"));
  BLK_TRY(need(q_out, "q_out"));
  BLK_TRY(need(k_out, "k_out"));
  BLK_TRY(rope_common(cfg, q_weight, k_weight, freq, pos));
  const Rows rq = {q, tokens, qn * sz, ld_q * sz}, rk = {k, tokens, kn * sz, ld_k * sz};
  const Rows oq = {q_out, tokens, qn * sz, ld_qo * sz}, ok = {k_out, tokens, kn * sz, ld_ko * sz};
  if ((share(oq, rq) && !(q_out == q && ld_qo == ld_q)) || share(oq, rk) ||
      (share(ok, rk) && !(k_out == k && ld_ko == ld_k)) || share(ok, rq) || share(oq, ok))
    return failf(TTT_E_CONFIG, "an output overlaps an input or the other output");
  const RopeTables t = rope_tables(cfg, q_weight, k_weight, freq, pos, tokens);
  if (clash({oq, ok}, {t.qw, t.kw, t.freq, t.pos}))
    return failf(TTT_E_CONFIG, "an output overlaps a scale, freq or pos");
  RopeArgs a = rope_args(cfg, q_weight, k_weight, freq, pos, tokens);
  a.q.x = q;
  a.q.ldx = ld_q;
  a.q.y = q_out;
  a.q.ldy = ld_qo;
  a.k.x = k;
  a.k.ldx = ld_k;
  a.k.y = k_out;
  a.k.ldy = ld_ko;
  BLK_HIP(launch_rope(a, cfg->act == TTT_BF16, static_cast<hipStream_t>(stream)));
  return TTT_OK;
}

ttt_status ttt_qk_norm_rope_backward_work(const ttt_rope_config* cfg, int64_t tokens, int64_t* bytes) {
  BLK_TRY(check_rope(cfg));
  BLK_TRY(check_tokens(tokens));
  if (!bytes) return failf(TTT_E_NULL, "bytes is NULL");
  *bytes = bwd_work_bytes(cfg, tokens);
  return TTT_OK;
}

ttt_status ttt_qk_norm_rope_backward(const ttt_rope_config* cfg, const void* q, int64_t ld_q,
                                     const void* k, int64_t ld_k, const void* q_weight,
                                     const void* k_weight, const float* freq,
                                     const int32_t* pos, const void* dq_out, int64_t ld_dqo,
                                     const void* dk_out, int64_t ld_dko, void* dq,
                                     int64_t ld_dq, void* dk, int64_t ld_dk, float* dq_weight,
                                     float* dk_weight, void* work, int64_t work_bytes,
                                     int64_t tokens, void* stream) {
  BLK_TRY(check_rope(cfg));
  BLK_TRY(check_tokens(tokens));
  const int sz = act_size(cfg);
  const int64_t qn = (int64_t)cfg->q_heads * cfg->head_dim, kn = (int64_t)cfg->k_heads * cfg->head_dim;
  BLK_TRY(check_ld(ld_q, qn, sz, "ld_q"));
  BLK_TRY(check_ld(ld_k, kn, sz, "ld_k"));
  BLK_TRY(check_ld(ld_dqo, qn, sz, "ld_dqo"));
  BLK_TRY(check_ld(ld_dko, kn, sz, "ld_dko"));
  BLK_TRY(check_ld(ld_dq, qn, sz, "ld_dq"));
  BLK_TRY(check_ld(ld_dk, kn, sz, "ld_dk"));
  if ((dq_weight && !q_weight) || (dk_weight && !k_weight))
    return failf(TTT_E_CONFIG, "a scale's gradient without the scale");
  BLK_TRY(optional(dq_weight, "dq_weight"));
  BLK_TRY(optional(dk_weight, "dk_weight"));
  hipStream_t st = static_cast<hipStream_t>(stream);
  const bool want = dq_weight || dk_weight;
  RopeDwArgs dw = {};
  dw.dq = dq_weight;
  dw.dk = dk_weight;
  dw.D = cfg->head_dim;
  const int64_t scale_bytes = (int64_t)cfg->head_dim * (int64_t)sizeof(float);
  const Rows wq = flat(dq_weight, scale_bytes), wk = flat(dk_weight, scale_bytes);
  if (tokens == 0) {   // a sum over no rows
    if (cfg->norm == TTT_HEAD_NORM_NONE && (q_weight || k_weight))
      return failf(TTT_E_CONFIG, "learned scales without a norm");
    if (share(wq, wk)) return failf(TTT_E_CONFIG, "dq_weight overlaps dk_weight");
    if (want) BLK_HIP(launch_rope_dw(dw, st));
    return TTT_OK;
  }
  BLK_TRY(need(q, "q"));
  BLK_TRY(need(k, "k"));
  BLK_TRY(need(dq_out, "dq_out"));
  BLK_TRY(need(dk_out, "dk_out"));
  BLK_TRY(need(dq, "dq"));
  BLK_TRY(need(dk, "dk"));
  BLK_TRY(rope_common(cfg, q_weight, k_weight, freq, pos));
  const int64_t bytes = bwd_work_bytes(cfg, tokens);
  if (bytes) {
    BLK_TRY(need(work, "work"));
    if (work_bytes < bytes)
      return failf(TTT_E_SHAPE, "work of %lld bytes, %lld needed", (long long)work_bytes,
                   (long long)bytes);
  }
  const Rows rq = {q, tokens, qn * sz, ld_q * sz}, rk = {k, tokens, kn * sz, ld_k * sz};
  const Rows gq = {dq_out, tokens, qn * sz, ld_dqo * sz}, gk = {dk_out, tokens, kn * sz, ld_dko * sz};
  const Rows oq = {dq, tokens, qn * sz, ld_dq * sz}, ok = {dk, tokens, kn * sz, ld_dk * sz};
  if (share(oq, rq) || share(oq, rk) || share(ok, rq) || share(ok, rk) || share(oq, gk) ||
      share(ok, gq) || share(oq, ok) || (share(oq, gq) && !(dq == dq_out && ld_dq == ld_dqo)) ||
      (share(ok, gk) && !(dk == dk_out && ld_dk == ld_dko)))
    return failf(TTT_E_CONFIG, "a gradient overlaps an input or the other gradient");
  const RopeTables t = rope_tables(cfg, q_weight, k_weight, freq, pos, tokens);
  if (clash({oq, ok, wq, wk, flat(work, bytes)}, {t.qw, t.kw, t.freq, t.pos}) ||
      clash({wq, wk, flat(work, bytes)}, {rq, rk, gq, gk}))
    return failf(TTT_E_CONFIG, "a gradient or work overlaps an input, work or another gradient");
  RopeArgs a = rope_args(cfg, q_weight, k_weight, freq, pos, tokens);
  a.q.x = q;
  a.q.ldx = ld_q;
  a.q.dy = dq_out;
  a.q.lddy = ld_dqo;
  a.q.y = dq;
  a.q.ldy = ld_dq;
  a.k.x = k;
  a.k.ldx = ld_k;
  a.k.dy = dk_out;
  a.k.lddy = ld_dko;
  a.k.y = dk;
  a.k.ldy = ld_dk;
  a.wgs = bwd_wgs(a);
  a.part = want ? static_cast<float*>(work) : nullptr;
  BLK_HIP(launch_rope_backward(a, cfg->act == TTT_BF16, st));
  if (want) {
    dw.part = a.part;
    dw.n = a.wgs;
    BLK_HIP(launch_rope_dw(dw, st));
  }
  return TTT_OK;
}

ttt_status ttt_qk_norm_rope_append(const ttt_rope_config* cfg, const void* q, int64_t ld_q,
                                   const void* k, int64_t ld_k, const void* v, int64_t ld_v,
                                   const void* q_weight, const void* k_weight,
                                   const float* freq, const int32_t* pos,
                                   const ttt_kv_cache* cache, const int64_t* slot,
                                   void* q_out, int64_t ld_qo, int64_t tokens, void* stream) {
  BLK_TRY(check_rope(cfg));
  BLK_TRY(check_tokens(tokens));
  BLK_TRY(check_cache(cache));
  if (cfg->act != TTT_BF16) return failf(TTT_E_DTYPE, "the cache takes bf16 activations");
  if (cfg->k_heads != cache->kv_heads || cfg->head_dim != cache->head_dim)
    return failf(TTT_E_SHAPE, "%d key heads of %d against a cache of %d of %d", cfg->k_heads,
                 cfg->head_dim, cache->kv_heads, cache->head_dim);
  const int64_t qn = (int64_t)cfg->q_heads * cfg->head_dim, kn = (int64_t)cfg->k_heads * cfg->head_dim;
  BLK_TRY(check_ld(ld_q, qn, 2, "ld_q"));
  BLK_TRY(check_ld(ld_k, kn, 2, "ld_k"));
  BLK_TRY(check_ld(ld_v, kn, 2, "ld_v"));
  BLK_TRY(check_ld(ld_qo, qn, 2, "ld_qo"));
  if (tokens == 0) return TTT_OK;
  BLK_TRY(need(q, "q"));
  BLK_TRY(need(k, "k"));
  BLK_TRY(need(v, "v"));
  BLK_TRY(need(q_out, "q_out"));
  BLK_TRY(need(slot, "slot"));
  BLK_TRY(rope_common(cfg, q_weight, k_weight, freq, pos));
  BLK_TRY(check_cache_pointers(cache));
  const Rows rq = {q, tokens, qn * 2, ld_q * 2}, rk = {k, tokens, kn * 2, ld_k * 2},
             rv = {v, tokens, kn * 2, ld_v * 2}, oq = {q_out, tokens, qn * 2, ld_qo * 2};
  const Rows ck = cache_rows(cache, cache->k), cv = cache_rows(cache, cache->v);
  if ((share(oq, rq) && !(q_out == q && ld_qo == ld_q)) || share(oq, rk) || share(oq, rv))
    return failf(TTT_E_CONFIG, "q_out overlaps an input");
  if (share(ck, cv) || share(ck, rq) || share(ck, rk) || share(ck, rv) || share(ck, oq) ||
      share(cv, rq) || share(cv, rk) || share(cv, rv) || share(cv, oq))
    return failf(TTT_E_CONFIG, "the cache's keys and values overlap each other or a tensor");
  const RopeTables t = rope_tables(cfg, q_weight, k_weight, freq, pos, tokens);
  const int64_t scales = (int64_t)cache->kv_heads * (int64_t)sizeof(float);
  if (clash({oq, ck, cv}, {t.qw, t.kw, t.freq, t.pos, flat(slot, tokens * (int64_t)sizeof(int64_t)),
                           flat(cache->k_scale, scales), flat(cache->v_scale, scales)}))
    return failf(TTT_E_CONFIG, "q_out or the cache overlaps a scale, freq, pos or slot");
  RopeArgs a = rope_args(cfg, q_weight, k_weight, freq, pos, tokens);
  a.q.x = q;
  a.q.ldx = ld_q;
  a.q.y = q_out;
  a.q.ldy = ld_qo;
  a.k.x = k;
  a.k.ldx = ld_k;
  a.v = v;
  a.ldv = ld_v;
  a.kc = static_cast<u16*>(cache->k);
  a.vc = static_cast<u16*>(cache->v);
  a.ks = cache->k_scale;
  a.vs = cache->v_scale;
  a.slot = slot;
  a.page_stride = cache->page_stride;
  a.page_size = cache->page_size;
  a.slots = (int64_t)cache->pages * cache->page_size;
  a.e4m3 = cache->dtype == TTT_CACHE_E4M3;
  BLK_HIP(launch_rope_append(a, static_cast<hipStream_t>(stream)));
  return TTT_OK;
}

ttt_status ttt_paged_attention_work(const ttt_kv_cache* cache, int32_t seqs, int32_t heads,
                                    int32_t max_pages, int32_t window, int64_t* bytes) {
  PagedPlan p;
  BLK_TRY(paged_plan(cache, seqs, heads, max_pages, window, &p));
  if (!bytes) return failf(TTT_E_NULL, "bytes is NULL");
  *bytes = p.bytes;
  return TTT_OK;
}

ttt_status ttt_paged_attention(const void* q, int64_t ld_q, const ttt_kv_cache* cache,
                               const int32_t* table, const int32_t* lens, void* out,
                               int64_t ld_out, float* lse, int32_t seqs, int32_t heads,
                               int32_t max_pages, int32_t window, float scale, void* work,
                               int64_t work_bytes, void* stream) {
  PagedPlan p;
  BLK_TRY(paged_plan(cache, seqs, heads, max_pages, window, &p));
  if (scale != 0.f && !(std::isfinite(scale) && scale > 0.f))
    return failf(TTT_E_CONFIG, "scale %g: 0, or finite and > 0", (double)scale);
  const int64_t n = (int64_t)heads * cache->head_dim;
  BLK_TRY(check_ld(ld_q, n, 2, "ld_q"));
  BLK_TRY(check_ld(ld_out, n, 2, "ld_out"));
  if (seqs == 0) return TTT_OK;
  BLK_TRY(need(q, "q"));
  BLK_TRY(need(out, "out"));
  BLK_TRY(need(lens, "lens"));
  if (max_pages) BLK_TRY(need(table, "table"));
  BLK_TRY(optional(lse, "lse"));
  BLK_TRY(check_cache_pointers(cache));
  if (p.bytes) {
    BLK_TRY(need(work, "work"));
    if (work_bytes < p.bytes)
      return failf(TTT_E_SHAPE, "work of %lld bytes, %lld needed", (long long)work_bytes,
                   (long long)p.bytes);
  }
  const Rows rq = {q, seqs, n * 2, ld_q * 2}, ro = {out, seqs, n * 2, ld_out * 2};
  const int64_t scales = (int64_t)cache->kv_heads * (int64_t)sizeof(float);
  if (clash({ro, flat(lse, (int64_t)seqs * heads * (int64_t)sizeof(float)), flat(work, p.bytes)},
            {rq, cache_rows(cache, cache->k), cache_rows(cache, cache->v), flat(cache->k_scale, scales),
             flat(cache->v_scale, scales), flat(lens, (int64_t)seqs * (int64_t)sizeof(int32_t)),
             flat(table, (int64_t)seqs * max_pages * (int64_t)sizeof(int32_t))}))
    return failf(TTT_E_CONFIG, "out, lse or work overlaps an input or each other");
  PagedArgs a = {};
  a.q = static_cast<const u16*>(q);
  a.ldq = ld_q;
  a.k = static_cast<const char*>(cache->k);
  a.v = static_cast<const char*>(cache->v);
  a.ks = cache->k_scale;
  a.vs = cache->v_scale;
  a.page_bytes = cache->page_stride * (cache->dtype == TTT_CACHE_BF16 ? 2 : 1);
  a.pages = cache->pages;
  a.page_size = cache->page_size;
  a.kv_heads = cache->kv_heads;
  a.table = table;
  a.lens = lens;
  a.out = static_cast<u16*>(out);
  a.ldo = ld_out;
  a.lse = lse;
  a.seqs = seqs;
  a.heads = heads;
  a.group = p.group;
  a.htiles = p.htiles;
  a.max_pages = max_pages;
  a.window = window;
  a.splits = p.splits;
  a.scale = scale != 0.f ? scale : (float)(1.0 / std::sqrt((double)cache->head_dim));
  a.po = static_cast<float*>(work);
  a.pm = reinterpret_cast<float*>(static_cast<char*>(work) + p.sums);
  BLK_HIP(launch_paged(a, cache->head_dim, cache->dtype == TTT_CACHE_E4M3,
                       static_cast<hipStream_t>(stream)));
  return TTT_OK;
}

ttt_status ttt_window_attention_lse(const void* q, const void* k, const void* v, int64_t ld,
                                    void* out, int64_t ld_out, float* lse, int32_t batch,
                                    int32_t heads, int64_t seq_len, int32_t window,
                                    int32_t window_mode, void* stream) {
  BLK_TRY(check_attention(ld, ld_out, batch, heads, seq_len, window, window_mode));
  BLK_TRY(check_ld(ld_out, 0, 2, "ld_out"));
  if (seq_len == 0) return TTT_OK;
  BLK_TRY(need(q, "q"));
  BLK_TRY(need(k, "k"));
  BLK_TRY(need(v, "v"));
  BLK_TRY(need(out, "out"));
  BLK_TRY(need(lse, "lse"));
  const int64_t rows = (int64_t)batch * seq_len, n = (int64_t)heads * ATT_D;
  const Rows ro = {out, rows, n * 2, ld_out * 2}, rl = {lse, 1, rows * heads * 4, rows * heads * 4};
  for (const void* p : {q, k, v}) {
    const Rows r = {p, rows, n * 2, ld * 2};
    if (share(ro, r) || share(rl, r)) return failf(TTT_E_CONFIG, "out or lse overlaps q, k or v");
  }
  if (share(ro, rl)) return failf(TTT_E_CONFIG, "lse overlaps out");
  WindowArgs a = window_args(q, k, v, ld, out, ld_out, lse, heads, seq_len, window, window_mode);
  BLK_HIP(launch_window_fwd(a, (int64_t)batch * heads, static_cast<hipStream_t>(stream)));
  return TTT_OK;
}

ttt_status ttt_window_attention_backward(const void* q, const void* k, const void* v,
                                         int64_t ld, const void* out, int64_t ld_out,
                                         const float* lse, const void* dout, int64_t ld_dout,
                                         void* dq, void* dk, void* dv, int64_t ld_d,
                                         float* work, int32_t batch, int32_t heads,
                                         int64_t seq_len, int32_t window, int32_t window_mode,
                                         void* stream) {
  BLK_TRY(check_attention(ld, ld_out, batch, heads, seq_len, window, window_mode));
  // dout is read as q is, the gradients are written as out is: the same limits
  BLK_TRY(check_attention(ld_dout, ld_d, batch, heads, seq_len, window, window_mode));
  BLK_TRY(check_ld(ld_out, 0, 2, "ld_out"));
  BLK_TRY(check_ld(ld_d, 0, 2, "ld_d"));
  if (seq_len == 0) return TTT_OK;
  BLK_TRY(need(q, "q"));
  BLK_TRY(need(k, "k"));
  BLK_TRY(need(v, "v"));
  BLK_TRY(need(out, "out"));
  BLK_TRY(need(lse, "lse"));
  BLK_TRY(need(dout, "dout"));
  BLK_TRY(need(dq, "dq"));
  BLK_TRY(need(dk, "dk"));
  BLK_TRY(need(dv, "dv"));
  BLK_TRY(need(work, "work"));
  const int64_t rows = (int64_t)batch * seq_len, n = (int64_t)heads * ATT_D * 2, stats = rows * heads * 4;
  const Rows ins[] = {{q, rows, n, ld * 2}, {k, rows, n, ld * 2}, {v, rows, n, ld * 2},
                      {out, rows, n, ld_out * 2}, {dout, rows, n, ld_dout * 2}, {lse, 1, stats, stats}};
  const Rows outs[] = {{dq, rows, n, ld_d * 2}, {dk, rows, n, ld_d * 2}, {dv, rows, n, ld_d * 2},
                       {work, 1, stats, stats}};
  for (int i = 0; i < 4; ++i) {
    for (const Rows& r : ins)
      if (share(outs[i], r)) return failf(TTT_E_CONFIG, "a gradient or work overlaps an input");
    for (int j = 0; j < i; ++j)
      if (share(outs[i], outs[j])) return failf(TTT_E_CONFIG, "the gradients and work overlap");
  }
  WindowArgs a = window_args(q, k, v, ld, const_cast<void*>(out), ld_out, const_cast<float*>(lse),
                             heads, seq_len, window, window_mode);
  a.dout = static_cast<const u16*>(dout);
  a.lddo = ld_dout;
  a.dq = static_cast<u16*>(dq);
  a.dk = static_cast<u16*>(dk);
  a.dv = static_cast<u16*>(dv);
  a.ldd = ld_d;
  a.delta = work;
  BLK_HIP(launch_window_bwd(a, (int64_t)batch * heads, static_cast<hipStream_t>(stream)));
  return TTT_OK;
}

}  // extern "C"
