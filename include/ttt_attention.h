/*
 * libttt attention API: what stands around the window attention of ttt_block.h, for training
 * and for serving one token at a time, on gfx950.
 *
 * The TTT-E2E page (jsqmd.com) trains its hybrid of sliding-window attention and TTT with
 * normalised queries and keys and rotary positions; the
 * LaCT page (peacm.com) uses the same layer on text (§3.2), on image sets (§3.1) and on video
 * (§3.3), where a token has several position axes.  This header adds
 *   - the per-head norm of queries and keys with the position rotation in the same pass, and
 *     its backward;
 *   - the same pass for new tokens with their keys and values stored into a paged cache;
 *   - the attention of one new token per sequence over that cache, whole or windowed;
 *   - the window attention's training form: the forward that also gives each row's
 *     log-sum-exp, and the backward.
 *
 * Conventions as in ttt_block.h: all tensors are device memory of the current HIP device,
 * caller-owned, 16-byte aligned; every call is enqueued on `stream` (a hipStream_t, NULL the
 * null stream) without host synchronisation and without allocation; argument checks run on
 * the host before anything is enqueued; status codes and ttt_last_error as in libttt.h.  All
 * calls can be captured into a HIP graph.  Workspaces are the caller's: two calls that may
 * overlap in time (two streams, two graphs in flight) need a workspace each.  Reads never
 * leave the tensors described, whatever positions, slots, page numbers and lengths hold.
 */
#ifndef TTT_ATTENTION_H
#define TTT_ATTENTION_H

#include "libttt.h"
#include "ttt_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Norm of each query and key head: NONE leaves them, RMS divides by sqrt(mean(x^2) + eps) and
 * multiplies by the learned scale, if one is given.                                        */
typedef enum { TTT_HEAD_NORM_NONE = 0, TTT_HEAD_NORM_RMS = 1 } ttt_head_norm;

/* Which elements turn together, j < rot_dim / 2: HALVES element j with j + rot_dim / 2, PAIRS
 * element 2 j with 2 j + 1.                                                               */
typedef enum { TTT_ROPE_HALVES = 0, TTT_ROPE_PAIRS = 1 } ttt_rope_pairing;

/*
 * Limits: q_heads, k_heads in [1, 4096]; head_dim a multiple of 16 in [16, 1024]; rot_dim a
 * multiple of 16 in [0, head_dim]; axes in [1, 4]; act bf16 or fp32; with RMS eps finite and
 * > 0 (with NONE it is ignored).
 */
typedef struct {
  int32_t q_heads, k_heads, head_dim;
  int32_t rot_dim;   /* the first rot_dim elements of every head are rotated             */
  int32_t axes;      /* position axes: 1 text, 2 an image, 3 time or view, row, column   */
  int32_t pairing;   /* ttt_rope_pairing */
  int32_t norm;      /* ttt_head_norm    */
  int32_t act;       /* ttt_dtype of queries, keys, values and learned scales            */
  float eps;
} ttt_rope_config;

/* Host-only check of a configuration (no HIP call). */
ttt_status ttt_validate_rope_config(const ttt_rope_config* cfg);

/*
 * For every token t and head h of the queries (and of the keys, with their own scale)
 *   n = x / sqrt(mean(x^2) + eps) * weight        (n = x without norm)
 *   angle_j = sum_a pos[a][t] freq[a][j],          j < rot_dim / 2
 *   y = n with every pair (n0, n1) of index j turned by its angle:
 *       (n0 cos - n1 sin, n0 sin + n1 cos)
 * rounded once to the activation dtype; everything before is fp32, but the angles are summed and
 * reduced in 64 bits with what those round off: sines and cosines are within two half steps of
 * fp32 at positions anywhere in int32.  The sum of squares is fp32 too: a head whose
 * squares add up past its range (values of about 1e18 and more) comes out as zeros.
 *   q, k     element e of head h of token t at  t * ld + h * head_dim + e
 *   q_out, k_out  the same with ld_qo, ld_ko.  q_out may be q itself (ld_qo == ld_q) and k_out
 *            k; other overlaps of an output with an input (weights, freq and pos
 *            among them) or the other output are TTT_E_CONFIG.  q and k may be parts of one
 *            projection's rows.
 *   q_weight, k_weight  [head_dim] learned scales, or NULL for ones (must be NULL without norm)
 *   freq     fp32 [axes][rot_dim / 2], radians per position: a pair that turns with one axis
 *            holds zeros for the others (may be NULL with rot_dim 0)
 *   pos      int32 [axes][tokens] (may be NULL with rot_dim 0)
 * Limits: 0 <= tokens <= 2^25; every ld at least heads * head_dim, at most 2^28 and such
 * that rows stay 16-byte aligned.  tokens 0 does nothing.
 */
ttt_status ttt_qk_norm_rope(const ttt_rope_config* cfg, const void* q, int64_t ld_q,
                            const void* k, int64_t ld_k, const void* q_weight,
                            const void* k_weight, const float* freq, const int32_t* pos,
                            void* q_out, int64_t ld_qo, void* k_out, int64_t ld_ko,
                            int64_t tokens, void* stream);

/*
 * Backward of ttt_qk_norm_rope: with dq_out, dk_out the gradients of its outputs (activation
 * dtype, their own row strides), writes the gradients of q and k (dq, dk, activation dtype)
 * and, where a weight and its gradient pointer are given, those of the learned scales
 * (dq_weight, dk_weight, fp32 [head_dim], overwritten: the sum over all tokens and heads, in
 * an order that depends only on the sizes).  q, k, weights, freq, pos as given to the forward.
 * dq may be dq_out itself (same stride) and dk dk_out; other overlaps of what is written (work
 * among it) with an input or each other are TTT_E_CONFIG.
 * work: workspace of the size that ttt_qk_norm_rope_backward_work gives (0 without norm; work
 * may then be NULL).  tokens 0 writes zero weight gradients.
 */
ttt_status ttt_qk_norm_rope_backward_work(const ttt_rope_config* cfg, int64_t tokens,
                                          int64_t* bytes);
ttt_status ttt_qk_norm_rope_backward(const ttt_rope_config* cfg, const void* q, int64_t ld_q,
                                     const void* k, int64_t ld_k, const void* q_weight,
                                     const void* k_weight, const float* freq,
                                     const int32_t* pos, const void* dq_out, int64_t ld_dqo,
                                     const void* dk_out, int64_t ld_dko, void* dq,
                                     int64_t ld_dq, void* dk, int64_t ld_dk, float* dq_weight,
                                     float* dk_weight, void* work, int64_t work_bytes,
                                     int64_t tokens, void* stream);

/* Element type of a key-value cache: bf16, or e4m3 (8 bits, largest value 448, no infinity). */
typedef enum { TTT_CACHE_BF16 = 0, TTT_CACHE_E4M3 = 1 } ttt_cache_dtype;

/*
 * A paged key-value cache.  Element e of key head h in place s of page p is at
 *   k[p * page_stride + (h * page_size + s) * head_dim + e]   (v the same),
 * so the pages of keys and values may be separate arrays or lie in turn in one.  With e4m3
 * the stored number times the head's scale is the value (k_scale, v_scale: device fp32
 * [kv_heads], finite and > 0; NULL: 1; must be NULL with bf16).
 * Limits: pages >= 1; page_size in [1, 65536]; kv_heads in [1, 4096]; head_dim as the call
 * allows; page_stride >= kv_heads * page_size * head_dim and such that rows stay 16-byte
 * aligned.
 */
typedef struct {
  void* k;
  void* v;
  const float* k_scale;
  const float* v_scale;
  int64_t page_stride;
  int32_t pages, page_size, kv_heads, head_dim;
  int32_t dtype;      /* ttt_cache_dtype */
  int32_t reserved;   /* 0 */
} ttt_kv_cache;

/*
 * ttt_qk_norm_rope for new tokens (bf16), the keys going to the cache instead of k_out, and
 * the values v (rows as k's, unchanged) with them.  slot: int64 [tokens], the place of each
 * token as page * page_size + place in the page.  A token whose slot lies outside
 * [0, pages * page_size) (a padding token: -1) stores nothing; its q_out row is written.  The
 * slots inside must differ from each other: which of two tokens in one slot stays is not
 * said.  Stored e4m3 values are x / scale held to +-448 and rounded to nearest (ties to
 * even); a NaN stays one.  The other places of the cache are left as they are.  cfg's k_heads
 * and head_dim must equal the cache's.  The cache may not overlap the other tensors.
 */
ttt_status ttt_qk_norm_rope_append(const ttt_rope_config* cfg, const void* q, int64_t ld_q,
                                   const void* k, int64_t ld_k, const void* v, int64_t ld_v,
                                   const void* q_weight, const void* k_weight,
                                   const float* freq, const int32_t* pos,
                                   const ttt_kv_cache* cache, const int64_t* slot,
                                   void* q_out, int64_t ld_qo, int64_t tokens, void* stream);

/*
 * Attention of one new token per sequence over its cached keys and values.  For sequence s,
 * query head h (key head h / (heads / kv_heads)) and n = lens[s] cached tokens (the new token
 * among them, if it is to see itself):
 *   out[s, h] = sum_j softmax_j(scale q[s, h] . k_j) v_j,   max(0, n - window) <= j < n
 * (all j < n with window 0: with window w the new token sees what the block's sliding window
 * of w shows it).  Token j of sequence s is in place j % page_size of page
 * table[s][j / page_size].
 *   q, out   bf16, element e of head h of sequence s at s * ld + h * head_dim + e
 *   table    int32 [seqs][max_pages];  lens int32 [seqs]
 *   lse      fp32 [seqs][heads] or NULL: the log of the sum of the exponentials
 * A length below 0 counts as 0, one above max_pages * page_size as that.  Tokens whose page
 * number lies outside [0, pages) are left out.  A sequence with no token left gets out 0 and
 * lse -inf.  Cached tokens that the new token does not see may hold anything, NaN and infinities
 * too.  Of those it sees, a key that is infinite or NaN in some element gives its query heads
 * NaN for out and lse, a value its own element of their out; so does a sum of p v past fp32's
 * range (p at most 1).
 * heads a multiple of kv_heads, at most 65536; head_dim 64, 128 or 256; 0 <= seqs <= 2^20,
 * seqs * heads below 2^24; max_pages >= 0, max_pages * page_size <= 2^30; window >= 0; scale 0
 * selects 1 / sqrt(head_dim), otherwise finite and > 0.  out, lse and work may not overlap the
 * inputs, the cache or each other.
 * Scores, softmax and sums are fp32; the probabilities enter the product with v as two bf16
 * numbers each (16 significant bits), so out is rounded once.
 * work: workspace of the size ttt_paged_attention_work gives for the same cache sizes, seqs,
 * heads, max_pages and window; its contents need not be kept or cleared between calls.
 */
ttt_status ttt_paged_attention_work(const ttt_kv_cache* cache, int32_t seqs, int32_t heads,
                                    int32_t max_pages, int32_t window, int64_t* bytes);
ttt_status ttt_paged_attention(const void* q, int64_t ld_q, const ttt_kv_cache* cache,
                               const int32_t* table, const int32_t* lens, void* out,
                               int64_t ld_out, float* lse, int32_t seqs, int32_t heads,
                               int32_t max_pages, int32_t window, float scale, void* work,
                               int64_t work_bytes, void* stream);

/*
 * The window attention of ttt_window_attention for training: also stores lse
 * [batch][heads][seq_len] (fp32), the log of each row's sum of exponentials of the scaled scores,
 * for the backward.  Scores, softmax and sums are fp32, the probabilities are rounded to bf16 for
 * the product with v and summed before that.  Limits as there, and ld_out at most 2^28; out and
 * lse may not overlap the inputs or each other.  All values, and the scores they give, must be
 * finite.
 */
ttt_status ttt_window_attention_lse(const void* q, const void* k, const void* v, int64_t ld,
                                    void* out, int64_t ld_out, float* lse, int32_t batch,
                                    int32_t heads, int64_t seq_len, int32_t window,
                                    int32_t window_mode, void* stream);

/*
 * Backward of ttt_window_attention: from its inputs, out and lse, and the gradient dout
 * (bf16, rows as out's with stride ld_dout), the gradients
 *   p = exp(scale q k - lse),  dp = dout . v,  ds = p (dp - dout . out)
 *   dq = scale sum ds k,   dk = scale sum ds q,   dv = sum p dout
 * bf16, rows of dq, dk and dv as q's with stride ld_d (they may be thirds of one buffer).
 * (dout . out, where no row sees more than 64 tokens, is summed as p dp: there the rounding of
 * out would weigh).  Scores, exponentials and sums are fp32; p and ds are rounded to bf16 for
 * their products.
 * Every sum has one order: the results are the same from run to run.  work: fp32
 * [batch][heads][seq_len] workspace.  The gradients and work may not overlap the inputs or
 * each other.  All values, and the scores they give, must be finite.  Limits as for
 * ttt_window_attention, ld_dout as ld; ld_out and ld_d at most 2^28.
 */
ttt_status ttt_window_attention_backward(const void* q, const void* k, const void* v,
                                         int64_t ld, const void* out, int64_t ld_out,
                                         const float* lse, const void* dout, int64_t ld_dout,
                                         void* dq, void* dk, void* dv, int64_t ld_d,
                                         float* work, int32_t batch, int32_t heads,
                                         int64_t seq_len, int32_t window, int32_t window_mode,
                                         void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TTT_ATTENTION_H */
