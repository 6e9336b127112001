// Host side of the mixer calls (include/ttt_mixer.h): argument checks, launch sizes, workspace
// layout.
#include "ttt_mixer.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "ttt_attention_host.h"
#include "ttt_mixer_internal.h"

using namespace ttt;

namespace {

bool dim_ok(int32_t d) { return d == 64 || d == 128 || d == 256; }

ttt_status check_linear(const ttt_linear_attention_config* c) {
  if (!c) return failf(TTT_E_NULL, "config is NULL");
  if (c->heads < 1 || c->heads > 4096) return failf(TTT_E_SHAPE, "heads %d: in [1, 4096]", c->heads);
  if (!dim_ok(c->dim_k) || !dim_ok(c->dim_v))
    return failf(TTT_E_UNSUPPORTED, "dim_k %d, dim_v %d: 64, 128 or 256 each", c->dim_k, c->dim_v);
  if (c->scale != 0.f && !(std::isfinite(c->scale) && c->scale > 0.f))
    return failf(TTT_E_CONFIG, "scale %g: 0, or finite and > 0", (double)c->scale);
  return TTT_OK;
}

float linear_scale(const ttt_linear_attention_config* c) {
  return c->scale != 0.f ? c->scale : (float)(1.0 / std::sqrt((double)c->dim_k));
}

// below 2^24: the bytes of a chunk's rows are offsets of 32 bits
ttt_status linear_ld(int64_t ld, int64_t width, const char* name) {
  if (ld < width || ld >= (1 << 24) || ld % 8)
    return failf(TTT_E_SHAPE, "%s %lld: a multiple of 8, at least %lld, below 2^24", name, (long long)ld,
                 (long long)width);
  return TTT_OK;
}

ttt_status check_sizes(const ttt_linear_attention_config* c, int32_t batch, int64_t seq_len) {
  if (batch < 0 || batch > 65535 || (int64_t)batch * c->heads > (1 << 20))
    return failf(TTT_E_SHAPE, "batch %d of %d heads: batch in [0, 65535], at most 2^20 together", batch, c->heads);
  if (seq_len < 0 || seq_len > ((int64_t)1 << 30))
    return failf(TTT_E_SHAPE, "seq_len %lld: in [0, 2^30]", (long long)seq_len);
  return TTT_OK;
}

ttt_status check_rows(const int32_t* starts, int64_t tokens, int32_t batch, int64_t seq_len) {
  if (tokens < 0 || tokens > INT32_MAX)
    return failf(TTT_E_SHAPE, "tokens %lld: in [0, 2^31)", (long long)tokens);
  if (!starts && tokens != batch * seq_len)
    return failf(TTT_E_SHAPE, "tokens %lld of %d sequences of %lld without starts", (long long)tokens, batch,
                 (long long)seq_len);
  return starts ? need(starts, "starts") : TTT_OK;
}

// Segments that a sequence is cut into, and tokens of one.  A segment's own sum is computed first and the
// states before the segments from those: two more launches and one more reading of k and v, so that a
// sequence is cut only where its workgroups would leave CUs idle.
//   - as many workgroups as run at once (`slots`): with 8 heads of 131072 tokens 64 segments take 472 us, 32
//     take 507, 96 take 500; the three gradients of 32768 tokens take 424 us in a training step at 32
//     segments (768 workgroups for 512 places), 437 at 21, 450 at 42.  The gradients of 16384 tokens at half as
//     many segments, as many and twice as many take 164, 126, 136 us (heads of 64 by 64), 148, 143, 164 (128 by
//     128), 162, 124, 125 (128 by 64), 167, 166, 216 (256 by 128), but 125, 136, 155 (64 by 256), 157, 178, 224
//     (128 by 256) and 248, 306, 404 (256 by 256), where fewer would do: the rule does not ask for the dimensions;
//   - half as many again for prompts with starts, whose segments go by the longest: 24 of up to 4096 tokens of 12
//     heads of 64 take 187 us in 2 segments, 151 in 3, 141 in 4, 150 in 6.  Gradients make no difference between
//     batches with starts and without (12 of up to 3815 tokens, 8 heads of 128: 273 us, 242 at twice the segments);
//   - down to one chunk each (3 x 777 tokens of 2 heads, a training step: 104 us whole, 58 in segments of
//     129, 51 in segments of 65), but none for sequences of LIN_WHOLE tokens or fewer, for which the
//     launches cost more (a prompt of 8 heads: 192 tokens 17 us whole, 21 cut; 256 21 and 21; 384 28 and 22).
struct LinPlan {
  int32_t nseg, L;
};

constexpr int64_t NUM_CU = 256, LIN_WHOLE = 256;

LinPlan linear_plan(int64_t wgs, int64_t seq_len, int64_t slots) {
  const int64_t n = wgs && seq_len > LIN_WHOLE ? std::max<int64_t>(1, std::min(slots / wgs, seq_len / LIN_C)) : 1;
  LinPlan p;
  p.L = (int32_t)std::max<int64_t>(LIN_C, ((seq_len + n - 1) / n + LIN_C - 1) / LIN_C * LIN_C);
  p.nseg = (int32_t)std::max<int64_t>(1, (seq_len + p.L - 1) / p.L);
  return p;
}

// waves of a workgroup, 16 columns each
int32_t linear_waves(int32_t DB) { return DB == 64 ? 4 : 8; }

int64_t state_bytes(const ttt_linear_attention_config* c, int64_t n) {
  return n * c->heads * c->dim_k * c->dim_v * (int64_t)sizeof(float);
}

LinPlan forward_plan(const ttt_linear_attention_config* c, int32_t batch, int64_t seq_len, bool ragged) {
  // workgroups of a CU: what LDS and registers hold
  const int32_t NW = linear_waves(c->dim_v), per_cu = c->dim_k == 256 ? 1 : c->dim_k == 64 && NW == 4 ? 3 : 2;
  const int64_t slots = per_cu * NUM_CU;
  return linear_plan((int64_t)batch * c->heads * (c->dim_v / (16 * NW)), seq_len, ragged ? slots * 3 / 2 : slots);
}
LinPlan backward_plan(const ttt_linear_attention_config* c, int32_t batch, int64_t seq_len) {
  return linear_plan((int64_t)batch * c->heads * 3, seq_len, 3 * NUM_CU);
}

int64_t forward_bytes(const ttt_linear_attention_config* c, int32_t batch, const LinPlan& p) {
  return p.nseg > 1 ? state_bytes(c, (int64_t)batch * p.nseg) : 0;
}
int64_t backward_bytes(const ttt_linear_attention_config* c, int32_t batch, int64_t seq_len) {
  const LinPlan p = backward_plan(c, batch, seq_len);
  return p.nseg > 1 ? 2 * state_bytes(c, (int64_t)batch * p.nseg) : 0;
}

LinArgs linear_args(const ttt_linear_attention_config* c, const float* decay, const int32_t* starts,
                    const int32_t* slot, int32_t slots, int64_t tokens, int32_t batch, int64_t seq_len,
                    const LinPlan& p) {
  LinArgs a = {};
  a.decay = decay;
  a.starts = starts;
  a.slot = slot;
  a.slots = slots;
  a.tokens = tokens;
  a.batch = batch;
  a.heads = c->heads;
  a.T = (int32_t)seq_len;
  a.nseg = p.nseg;
  a.L = p.L;
  // rows that the last-level cache cannot keep for the walk after the segments' sums are read past it: a
  // prompt of 131072 tokens of 8 heads of 128 (805 MB) 3 % faster, 32768 tokens (201 MB) 10 % slower
  a.nt = 2 * tokens * c->heads * (2 * (int64_t)c->dim_k + c->dim_v) > ((int64_t)256 << 20);
  return a;
}

LinRole role(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv, void* out,
             int64_t ldo) {
  LinRole r = {};
  r.q = static_cast<const u16*>(q);
  r.k = static_cast<const u16*>(k);
  r.v = static_cast<const u16*>(v);
  r.out = static_cast<u16*>(out);
  r.ldq = ldq;
  r.ldk = ldk;
  r.ldv = ldv;
  r.ldo = ldo;
  return r;
}

// Sizes of a launch over heads of DB elements and nseg segments.
int32_t linear_grid(LinArgs& a, int32_t DB, int32_t nseg) {
  const int32_t NW = linear_waves(DB);
  a.DB = DB;
  a.slices = DB / (16 * NW);
  a.total = (int32_t)((int64_t)a.batch * a.heads * nseg * a.roles * a.slices);
  return NW;
}

ttt_status check_norm(const ttt_residual_norm_config* c) {
  if (!c) return failf(TTT_E_NULL, "config is NULL");
  if (c->dim < 8 || c->dim > 8192 || c->dim % 8)
    return failf(TTT_E_SHAPE, "dim %d: a multiple of 8 in [8, 8192]", c->dim);
  if (c->groups < 1 || c->dim % c->groups) return failf(TTT_E_SHAPE, "groups %d of dim %d", c->groups, c->dim);
  const int32_t w = c->dim / c->groups;
  if (c->groups > 1 && (w < 8 || w > 512 || (w & (w - 1))))
    return failf(TTT_E_SHAPE, "groups of %d elements: a power of two in [8, 512]", w);
  if (c->norm_y != 0 && c->norm_y != 1) return failf(TTT_E_CONFIG, "norm_y %d: 0 or 1", c->norm_y);
  if (c->gate < TTT_GATE_NONE || c->gate > TTT_GATE_SILU) return failf(TTT_E_CONFIG, "unknown gate %d", c->gate);
  if (c->act != TTT_F32 && c->act != TTT_BF16) return failf(TTT_E_DTYPE, "unknown activation dtype %d", c->act);
  if (!(std::isfinite(c->eps) && c->eps > 0.f)) return failf(TTT_E_CONFIG, "eps %g: finite and > 0", (double)c->eps);
  return TTT_OK;
}

ttt_status check_norm_tokens(int64_t tokens) {
  if (tokens < 0 || tokens > ((int64_t)1 << 25))
    return failf(TTT_E_SHAPE, "tokens %lld: in [0, 2^25]", (long long)tokens);
  return TTT_OK;
}

// A row tensor: its stride and pointer checked, where there is one.
ttt_status norm_rows(const ttt_residual_norm_config* c, const void* p, int64_t ld, int64_t tokens, bool must,
                     const char* name, Rows* r) {
  const int size = c->act == TTT_BF16 ? 2 : 4;
  *r = {p, 0, (int64_t)c->dim * size, ld * size};
  if (!p) return must && tokens ? failf(TTT_E_NULL, "%s is NULL", name) : TTT_OK;
  BLK_TRY(check_ld(ld, c->dim, size, name));
  BLK_TRY(need(p, name));
  r->rows = tokens;
  return TTT_OK;
}

// Whether o overlaps an input other than as that input itself.
bool partly(const Rows& o, std::initializer_list<Rows> ins) {
  for (const Rows& r : ins)
    if (share(o, r) && !(o.p == r.p && o.ld == r.ld)) return true;
  return false;
}

// The workgroups' partial sums, and behind them, where there are several launches, their sums so far.
int64_t norm_part_bytes(const ttt_residual_norm_config* c, int64_t tokens) {
  return (int64_t)3 * residual_norm_wgs(c->dim, tokens) * c->dim * (int64_t)sizeof(float);
}
int64_t norm_work_bytes(const ttt_residual_norm_config* c, int64_t tokens) {
  return norm_part_bytes(c, tokens) +
         (tokens > residual_norm_chunk(c->dim) ? (int64_t)3 * c->dim * (int64_t)sizeof(double) : 0);
}

struct NormInputs {
  Rows h, y, g, wy, rs, wn;
};

ttt_status norm_inputs(const ttt_residual_norm_config* c, const void* h, int64_t ld_h, const void* y, int64_t ld_y,
                       const void* gate, int64_t ld_gate, const void* wy, const void* rs, const void* wn, bool n,
                       int64_t tokens, NormInputs* in, NormArgs* a) {
  const int64_t w = (int64_t)c->dim * (c->act == TTT_BF16 ? 2 : 4);
  BLK_TRY(norm_rows(c, h, ld_h, tokens, false, "h", &in->h));
  BLK_TRY(norm_rows(c, y, ld_y, tokens, true, "y", &in->y));
  if (c->gate == TTT_GATE_NONE && gate) return failf(TTT_E_CONFIG, "a gate where the configuration has none");
  BLK_TRY(norm_rows(c, gate, ld_gate, tokens, c->gate != TTT_GATE_NONE, "gate", &in->g));
  if (wy && !c->norm_y) return failf(TTT_E_CONFIG, "y_weight without norm_y");
  if (wn && !n) return failf(TTT_E_CONFIG, "n_weight without its norm");
  BLK_TRY(optional(wy, "y_weight"));
  BLK_TRY(optional(rs, "res_scale"));
  BLK_TRY(optional(wn, "n_weight"));
  in->wy = flat(wy, w);
  in->rs = flat(rs, w);
  in->wn = flat(wn, w);
  *a = {};
  a->h = h;
  a->y = y;
  a->gate = gate;
  a->wy = wy;
  a->rs = rs;
  a->wn = wn;
  a->ldh = ld_h;
  a->ldy = ld_y;
  a->ldg = ld_gate;
  a->tokens = tokens;
  a->D = c->dim;
  a->gw = c->dim / c->groups;
  a->norm_y = c->norm_y;
  a->gate_kind = c->gate;
  a->eps = c->eps;
  return TTT_OK;
}

}  // namespace

extern "C" {

ttt_status ttt_validate_linear_attention_config(const ttt_linear_attention_config* cfg) {
  return check_linear(cfg);
}

ttt_status ttt_linear_attention_work(const ttt_linear_attention_config* cfg, int32_t batch, int64_t seq_len,
                                     int64_t* bytes) {
  BLK_TRY(check_linear(cfg));
  BLK_TRY(check_sizes(cfg, batch, seq_len));
  if (!bytes) return failf(TTT_E_NULL, "bytes is NULL");
  // for sequences with starts and without: the former take at least as many segments
  *bytes = std::max(forward_bytes(cfg, batch, forward_plan(cfg, batch, seq_len, true)),
                    forward_bytes(cfg, batch, forward_plan(cfg, batch, seq_len, false)));
  return TTT_OK;
}

ttt_status ttt_linear_attention(const ttt_linear_attention_config* cfg, const void* q, int64_t ld_q, const void* k,
                                int64_t ld_k, const void* v, int64_t ld_v, const float* decay,
                                const int32_t* starts, const float* state_in, float* state_out,
                                const int32_t* slot, int32_t slots, void* out, int64_t ld_out, int64_t tokens,
                                int32_t batch, int64_t seq_len, void* work, int64_t work_bytes, void* stream) {
  BLK_TRY(check_linear(cfg));
  BLK_TRY(check_sizes(cfg, batch, seq_len));
  const int64_t kn = (int64_t)cfg->heads * cfg->dim_k, vn = (int64_t)cfg->heads * cfg->dim_v;
  BLK_TRY(linear_ld(ld_q, kn, "ld_q"));
  BLK_TRY(linear_ld(ld_k, kn, "ld_k"));
  BLK_TRY(linear_ld(ld_v, vn, "ld_v"));
  BLK_TRY(linear_ld(ld_out, vn, "ld_out"));
  BLK_TRY(check_rows(starts, tokens, batch, seq_len));
  if (slots < 0 || (!slot && (state_in || state_out) && slots < batch))
    return failf(TTT_E_SHAPE, "%d slots for %d sequences", slots, batch);
  if (batch == 0) return TTT_OK;
  if (tokens) {
    BLK_TRY(need(q, "q"));
    BLK_TRY(need(k, "k"));
    BLK_TRY(need(v, "v"));
    BLK_TRY(need(out, "out"));
  }
  BLK_TRY(need(decay, "decay"));
  BLK_TRY(optional(slot, "slot"));
  BLK_TRY(optional(state_in, "state_in"));
  BLK_TRY(optional(state_out, "state_out"));
  const LinPlan p = forward_plan(cfg, batch, seq_len, starts != nullptr);
  const int64_t bytes = forward_bytes(cfg, batch, p);
  if (bytes) {
    BLK_TRY(need(work, "work"));
    if (work_bytes < bytes)
      return failf(TTT_E_SHAPE, "work of %lld bytes, %lld needed", (long long)work_bytes, (long long)bytes);
  }
  const Rows rq = {q, tokens, kn * 2, ld_q * 2}, rk = {k, tokens, kn * 2, ld_k * 2}, rv = {v, tokens, vn * 2, ld_v * 2};
  const Rows ro = {out, tokens, vn * 2, ld_out * 2};
  const Rows rd = flat(decay, cfg->heads * (int64_t)4), rs = flat(starts, (batch + (int64_t)1) * 4);
  const Rows rl = flat(slot, batch * (int64_t)4);
  const Rows si = flat(state_in, state_bytes(cfg, slots)), so = flat(state_out, state_bytes(cfg, slots));
  if (clash({ro, so, flat(work, bytes)}, {rq, rk, rv, rd, rs, rl}) || share(ro, si) ||
      share(flat(work, bytes), si) || (share(so, si) && state_out != state_in))
    return failf(TTT_E_CONFIG, "out, state_out or work overlaps an input or each other");
  LinArgs a = linear_args(cfg, decay, starts, slot, slots, tokens, batch, seq_len, p);
  a.roles = 1;
  LinRole& r = a.role[0];
  r = role(q, ld_q, k, ld_k, v, ld_v, out, ld_out);
  r.init = state_in;
  r.fin = state_out;
  r.scale_p = r.scale_s = linear_scale(cfg);
  r.scale_w = 1.f;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (p.nseg > 1) {
    r.ws = static_cast<float*>(work);
    const int32_t NW = linear_grid(a, cfg->dim_v, p.nseg - 1);
    BLK_HIP(launch_linear_states(a, cfg->dim_k, NW, st));
    BLK_HIP(launch_linear_scan(a, cfg->dim_k, st));
  }
  const int32_t NW = linear_grid(a, cfg->dim_v, p.nseg);
  BLK_HIP(launch_linear_walk(a, cfg->dim_k, NW, st));
  return TTT_OK;
}

ttt_status ttt_linear_attention_backward_work(const ttt_linear_attention_config* cfg, int32_t batch,
                                              int64_t seq_len, int64_t* bytes) {
  BLK_TRY(check_linear(cfg));
  BLK_TRY(check_sizes(cfg, batch, seq_len));
  if (!bytes) return failf(TTT_E_NULL, "bytes is NULL");
  *bytes = backward_bytes(cfg, batch, seq_len);
  return TTT_OK;
}

ttt_status ttt_linear_attention_backward(const ttt_linear_attention_config* cfg, const void* q, int64_t ld_q,
                                         const void* k, int64_t ld_k, const void* v, int64_t ld_v,
                                         const float* decay, const int32_t* starts, const float* state_in,
                                         const void* dout, int64_t ld_dout, const float* dstate_out, void* dq,
                                         int64_t ld_dq, void* dk, int64_t ld_dk, void* dv, int64_t ld_dv,
                                         float* dstate_in, int64_t tokens, int32_t batch, int64_t seq_len,
                                         void* work, int64_t work_bytes, void* stream) {
  BLK_TRY(check_linear(cfg));
  BLK_TRY(check_sizes(cfg, batch, seq_len));
  const int64_t kn = (int64_t)cfg->heads * cfg->dim_k, vn = (int64_t)cfg->heads * cfg->dim_v;
  BLK_TRY(linear_ld(ld_q, kn, "ld_q"));
  BLK_TRY(linear_ld(ld_k, kn, "ld_k"));
  BLK_TRY(linear_ld(ld_v, vn, "ld_v"));
  BLK_TRY(linear_ld(ld_dout, vn, "ld_dout"));
  BLK_TRY(linear_ld(ld_dq, kn, "ld_dq"));
  BLK_TRY(linear_ld(ld_dk, kn, "ld_dk"));
  BLK_TRY(linear_ld(ld_dv, vn, "ld_dv"));
  BLK_TRY(check_rows(starts, tokens, batch, seq_len));
  if (batch == 0) return TTT_OK;
  if (tokens) {
    BLK_TRY(need(q, "q"));
    BLK_TRY(need(k, "k"));
    BLK_TRY(need(v, "v"));
    BLK_TRY(need(dout, "dout"));
    BLK_TRY(need(dq, "dq"));
    BLK_TRY(need(dk, "dk"));
    BLK_TRY(need(dv, "dv"));
  }
  BLK_TRY(need(decay, "decay"));
  BLK_TRY(optional(state_in, "state_in"));
  BLK_TRY(optional(dstate_out, "dstate_out"));
  BLK_TRY(optional(dstate_in, "dstate_in"));
  const LinPlan p = backward_plan(cfg, batch, seq_len);
  const int64_t bytes = backward_bytes(cfg, batch, seq_len);
  if (bytes) {
    BLK_TRY(need(work, "work"));
    if (work_bytes < bytes)
      return failf(TTT_E_SHAPE, "work of %lld bytes, %lld needed", (long long)work_bytes, (long long)bytes);
  }
  const int64_t states = state_bytes(cfg, batch);
  const auto kr = [&](const void* x, int64_t ld) { return Rows{x, tokens, kn * 2, ld * 2}; };
  const auto vr = [&](const void* x, int64_t ld) { return Rows{x, tokens, vn * 2, ld * 2}; };
  if (clash({kr(dq, ld_dq), kr(dk, ld_dk), vr(dv, ld_dv), flat(dstate_in, states), flat(work, bytes)},
            {kr(q, ld_q), kr(k, ld_k), vr(v, ld_v), vr(dout, ld_dout), flat(decay, cfg->heads * (int64_t)4),
             flat(starts, (batch + (int64_t)1) * 4), flat(state_in, states), flat(dstate_out, states)}))
    return failf(TTT_E_CONFIG, "a gradient or work overlaps an input or each other");

  LinArgs a = linear_args(cfg, decay, starts, nullptr, batch, tokens, batch, seq_len, p);
  const float c = linear_scale(cfg);
  const int32_t K = cfg->dim_k, V = cfg->dim_v;
  hipStream_t st = static_cast<hipStream_t>(stream);
  // the states S before each segment, and backward in time the P behind each
  float *ws = nullptr, *wp = nullptr;
  if (p.nseg > 1) {
    ws = static_cast<float*>(work);
    wp = ws + bytes / 2 / (int64_t)sizeof(float);
    a.roles = 2;
    a.role[0] = role(nullptr, 0, k, ld_k, v, ld_v, nullptr, 0);
    a.role[0].init = state_in;
    a.role[0].ws = ws;
    a.role[0].scale_w = 1.f;
    a.role[1] = role(nullptr, 0, q, ld_q, dout, ld_dout, nullptr, 0);
    a.role[1].init = dstate_out;
    a.role[1].fin = dstate_in;
    a.role[1].ws = wp;
    a.role[1].rev = 1;
    a.role[1].scale_w = c;
    const int32_t NW = linear_grid(a, V, p.nseg - 1);
    BLK_HIP(launch_linear_states(a, K, NW, st));
    BLK_HIP(launch_linear_scan(a, K, st));
  }
  LinRole rq = role(dout, ld_dout, v, ld_v, k, ld_k, dq, ld_dq);
  rq.init = state_in;
  rq.ws = ws;
  rq.trans = 1;
  rq.scale_p = rq.scale_s = c;
  rq.scale_w = 1.f;
  LinRole rv = role(k, ld_k, q, ld_q, dout, ld_dout, dv, ld_dv);
  rv.init = dstate_out;
  rv.fin = dstate_in;
  rv.ws = wp;
  rv.rev = 1;
  rv.scale_p = rv.scale_w = c;
  rv.scale_s = 1.f;
  LinRole rk = role(v, ld_v, dout, ld_dout, q, ld_q, dk, ld_dk);
  rk.init = dstate_out;
  rk.ws = wp;
  rk.rev = rk.trans = 1;
  rk.scale_p = rk.scale_w = c;
  rk.scale_s = 1.f;
  if (K == V) {
    a.roles = 3;
    a.role[0] = rq;
    a.role[1] = rv;
    a.role[2] = rk;
    const int32_t NW = linear_grid(a, V, p.nseg);
    BLK_HIP(launch_linear_walk(a, K, NW, st));
    return TTT_OK;
  }
  a.roles = 1;
  a.role[0] = rv;
  const int32_t NV = linear_grid(a, V, p.nseg);
  BLK_HIP(launch_linear_walk(a, K, NV, st));
  a.roles = 2;
  a.role[0] = rq;
  a.role[1] = rk;
  const int32_t NK = linear_grid(a, K, p.nseg);
  BLK_HIP(launch_linear_walk(a, V, NK, st));
  return TTT_OK;
}

ttt_status ttt_linear_attention_step(const ttt_linear_attention_config* cfg, const void* q, int64_t ld_q,
                                     const void* k, int64_t ld_k, const void* v, int64_t ld_v, const float* decay,
                                     const float* state_in, float* state_out, const int32_t* slot, int32_t slots,
                                     void* out, int64_t ld_out, int32_t seqs, void* stream) {
  BLK_TRY(check_linear(cfg));
  if (seqs < 0 || seqs > (1 << 20) || (int64_t)seqs * cfg->heads > (1 << 22))
    return failf(TTT_E_SHAPE, "%d sequences of %d heads: at most 2^20, 2^22 together", seqs, cfg->heads);
  const int64_t kn = (int64_t)cfg->heads * cfg->dim_k, vn = (int64_t)cfg->heads * cfg->dim_v;
  BLK_TRY(linear_ld(ld_q, kn, "ld_q"));
  BLK_TRY(linear_ld(ld_k, kn, "ld_k"));
  BLK_TRY(linear_ld(ld_v, vn, "ld_v"));
  BLK_TRY(linear_ld(ld_out, vn, "ld_out"));
  if (slots < 0 || (!slot && (state_in || state_out) && slots < seqs))
    return failf(TTT_E_SHAPE, "%d slots for %d sequences", slots, seqs);
  if (seqs == 0) return TTT_OK;
  BLK_TRY(need(q, "q"));
  BLK_TRY(need(k, "k"));
  BLK_TRY(need(v, "v"));
  BLK_TRY(need(out, "out"));
  BLK_TRY(need(decay, "decay"));
  BLK_TRY(optional(slot, "slot"));
  BLK_TRY(optional(state_in, "state_in"));
  BLK_TRY(optional(state_out, "state_out"));
  const Rows ro = {out, seqs, vn * 2, ld_out * 2};
  const Rows si = flat(state_in, state_bytes(cfg, slots)), so = flat(state_out, state_bytes(cfg, slots));
  if (clash({ro, so}, {{q, seqs, kn * 2, ld_q * 2}, {k, seqs, kn * 2, ld_k * 2}, {v, seqs, vn * 2, ld_v * 2},
                       flat(decay, cfg->heads * (int64_t)4), flat(slot, seqs * (int64_t)4)}) ||
      share(ro, si) || (share(so, si) && state_out != state_in))
    return failf(TTT_E_CONFIG, "out or state_out overlaps an input or each other");
  LinStepArgs a = {};
  a.q = static_cast<const u16*>(q);
  a.k = static_cast<const u16*>(k);
  a.v = static_cast<const u16*>(v);
  a.out = static_cast<u16*>(out);
  a.ldq = ld_q;
  a.ldk = ld_k;
  a.ldv = ld_v;
  a.ldo = ld_out;
  a.decay = decay;
  a.in = state_in;
  a.fin = state_out;
  a.slot = slot;
  a.slots = slots;
  a.seqs = seqs;
  a.heads = cfg->heads;
  a.K = cfg->dim_k;
  a.V = cfg->dim_v;
  a.scale = linear_scale(cfg);
  // columns of a workgroup: as few as give two workgroups to a CU
  const int64_t states = (int64_t)seqs * cfg->heads;
  int32_t cols = std::min(cfg->dim_v, 128);
  while (cols > 32 && states * (cfg->dim_v / cols) < 2 * NUM_CU) cols /= 2;
  a.slices = cfg->dim_v / cols;
  a.total = (int32_t)(states * a.slices);   // at most 2^23: more than 128 columns only where few
  BLK_HIP(launch_linear_step(a, cols, static_cast<hipStream_t>(stream)));
  return TTT_OK;
}

ttt_status ttt_validate_residual_norm_config(const ttt_residual_norm_config* cfg) { return check_norm(cfg); }

ttt_status ttt_residual_norm(const ttt_residual_norm_config* cfg, const void* h, int64_t ld_h, const void* y,
                             int64_t ld_y, const void* gate, int64_t ld_gate, const void* y_weight,
                             const void* res_scale, const void* n_weight, void* h_out, int64_t ld_ho, void* n_out,
                             int64_t ld_n, int64_t tokens, void* stream) {
  BLK_TRY(check_norm(cfg));
  BLK_TRY(check_norm_tokens(tokens));
  NormInputs in;
  NormArgs a;
  BLK_TRY(norm_inputs(cfg, h, ld_h, y, ld_y, gate, ld_gate, y_weight, res_scale, n_weight, n_out != nullptr, tokens,
                      &in, &a));
  Rows ho, no;
  BLK_TRY(norm_rows(cfg, h_out, ld_ho, tokens, false, "h_out", &ho));
  BLK_TRY(norm_rows(cfg, n_out, ld_n, tokens, false, "n_out", &no));
  if (tokens == 0) return TTT_OK;
  if (!h_out && !n_out) return failf(TTT_E_NULL, "h_out and n_out are NULL");
  if (partly(ho, {in.h, in.y, in.g}) || partly(no, {in.h, in.y, in.g}) || clash({ho, no}, {in.wy, in.rs, in.wn}))
    return failf(TTT_E_CONFIG, "an output overlaps an input or the other output");
  a.ho = h_out;
  a.ldho = ld_ho;
  a.n = n_out;
  a.ldn = ld_n;
  BLK_HIP(launch_residual_norm(a, cfg->act == TTT_BF16, static_cast<hipStream_t>(stream)));
  return TTT_OK;
}

ttt_status ttt_residual_norm_backward_work(const ttt_residual_norm_config* cfg, int64_t tokens, int64_t* bytes) {
  BLK_TRY(check_norm(cfg));
  BLK_TRY(check_norm_tokens(tokens));
  if (!bytes) return failf(TTT_E_NULL, "bytes is NULL");
  *bytes = norm_work_bytes(cfg, tokens);
  return TTT_OK;
}

ttt_status ttt_residual_norm_backward(const ttt_residual_norm_config* cfg, const void* h, int64_t ld_h,
                                      const void* y, int64_t ld_y, const void* gate, int64_t ld_gate,
                                      const void* y_weight, const void* res_scale, const void* n_weight,
                                      const void* dh_out, int64_t ld_dho, const void* dn, int64_t ld_dn, void* dh,
                                      int64_t ld_dh, void* dy, int64_t ld_dy, void* dgate, int64_t ld_dgate,
                                      float* dy_weight, float* dres_scale, float* dn_weight, void* work,
                                      int64_t work_bytes, int64_t tokens, void* stream) {
  BLK_TRY(check_norm(cfg));
  BLK_TRY(check_norm_tokens(tokens));
  NormInputs in;
  NormArgs a;
  BLK_TRY(norm_inputs(cfg, h, ld_h, y, ld_y, gate, ld_gate, y_weight, res_scale, n_weight, dn != nullptr || !tokens,
                      tokens, &in, &a));
  Rows gh, gn, oh, oy, og;
  BLK_TRY(norm_rows(cfg, dh_out, ld_dho, tokens, false, "dh_out", &gh));
  BLK_TRY(norm_rows(cfg, dn, ld_dn, tokens, false, "dn", &gn));
  BLK_TRY(norm_rows(cfg, dh, ld_dh, tokens, false, "dh", &oh));
  BLK_TRY(norm_rows(cfg, dy, ld_dy, tokens, false, "dy", &oy));
  BLK_TRY(norm_rows(cfg, dgate, ld_dgate, tokens, false, "dgate", &og));
  if (dgate && cfg->gate == TTT_GATE_NONE) return failf(TTT_E_CONFIG, "dgate without a gate");
  if (dh && !h && tokens) return failf(TTT_E_CONFIG, "dh without h");
  if ((dy_weight && !y_weight) || (dres_scale && !res_scale) || (dn_weight && !n_weight))
    return failf(TTT_E_CONFIG, "a scale's gradient without the scale");
  BLK_TRY(optional(dy_weight, "dy_weight"));
  BLK_TRY(optional(dres_scale, "dres_scale"));
  BLK_TRY(optional(dn_weight, "dn_weight"));
  const bool want = dy_weight || dres_scale || dn_weight;
  const int64_t bytes = want ? norm_work_bytes(cfg, tokens) : 0;
  if (bytes) {
    BLK_TRY(need(work, "work"));
    if (work_bytes < bytes)
      return failf(TTT_E_SHAPE, "work of %lld bytes, %lld needed", (long long)work_bytes, (long long)bytes);
  }
  if (tokens && !dh_out && !dn) return failf(TTT_E_NULL, "dh_out and dn are NULL");
  const int64_t w = (int64_t)cfg->dim * (int64_t)sizeof(float);
  const Rows sums[] = {flat(dy_weight, w), flat(dres_scale, w), flat(dn_weight, w)}, wk = flat(work, bytes);
  if (clash({oh, oy, og, sums[0], sums[1], sums[2], wk}, {in.h, in.y, in.g, in.wy, in.rs, in.wn}) ||
      clash({sums[0], sums[1], sums[2], wk}, {gh, gn}) || partly(oh, {gh, gn}) || partly(oy, {gh, gn}) ||
      partly(og, {gh, gn}))
    return failf(TTT_E_CONFIG, "a gradient or work overlaps an input, work or another gradient");
  a.dho = dh_out;
  a.lddho = ld_dho;
  a.dn = dn;
  a.lddn = ld_dn;
  a.dh = dh;
  a.lddh = ld_dh;
  a.dy = dy;
  a.lddy = ld_dy;
  a.dg = dgate;
  a.lddg = ld_dgate;
  a.dwy = dy_weight;
  a.drs = dres_scale;
  a.dwn = dn_weight;
  a.part = want ? static_cast<float*>(work) : nullptr;
  if (want && tokens) a.sofar = reinterpret_cast<double*>(static_cast<char*>(work) + norm_part_bytes(cfg, tokens));
  BLK_HIP(launch_residual_norm_backward(a, cfg->act == TTT_BF16, static_cast<hipStream_t>(stream)));
  return TTT_OK;
}

}  // extern "C"
