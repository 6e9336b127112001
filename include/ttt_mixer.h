/*
 * libttt mixer API: a second sequence layer to stand beside the TTT layer of libttt.h, linear
 * attention with a decay for each head, for training, for prompts and for single tokens; and
 * what stands between two sub-layers: norms, gate and residual in one pass, with their
 * backward.  On gfx950.
 *
 * The pages measure TTT layers against recurrent layers of linear cost whose state decays
 * (PAPER.md:199-214, 309, 472).  The TTT layer's linear fast weight learns its map from chunks of
 * tokens; the layer here adds each token's key and value to its state as it comes, which serves
 * one token at a time.
 * The pre-norm residual sub-layers are those of ttt_block.h, with the learned scales, gates and
 * post-norms that trained models of this kind put around them.
 *
 * Conventions as in ttt_attention.h: all tensors are device memory of the current HIP device,
 * caller-owned, 16-byte aligned; every call is enqueued on `stream` (a hipStream_t, NULL the
 * null stream) without host synchronisation and without allocation; argument checks run on
 * the host before anything is enqueued; status codes and ttt_last_error as in libttt.h.  All
 * calls can be captured into a HIP graph.  Workspaces are the caller's: two calls that may
 * overlap in time (two streams, two graphs in flight) need a workspace each; what a workspace
 * holds need not be kept or cleared between calls.  Reads and writes never leave the tensors
 * described, whatever starts and slots hold.
 */
#ifndef TTT_MIXER_H
#define TTT_MIXER_H

#include "libttt.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Linear attention.  For every sequence and head h a state S, fp32 [dim_k][dim_v]:
 *   S_t = decay[h] S_{t-1} + k_t v_t^T,      out_t = scale S_t^T q_t
 * that is out_t = scale (decay^(t+1) S_in^T q_t + sum_{j <= t} decay^(t-j) (q_t . k_j) v_j).
 * decay is a constant of the head (no gradient): fp32 [heads] on the device, in [0, 1]; 1 is
 * linear attention without decay, 0 leaves each token its own value only.  Another value is
 * taken by the formula where its powers up to seq_len are finite in fp32.
 * Limits: heads in [1, 4096]; dim_k and dim_v 64, 128 or 256, each; scale finite and > 0, or 0,
 * which selects 1 / sqrt(dim_k).
 */
typedef struct {
  int32_t heads, dim_k, dim_v;
  float scale;
} ttt_linear_attention_config;

/* Host-only check of a configuration (no HIP call). */
ttt_status ttt_validate_linear_attention_config(const ttt_linear_attention_config* cfg);

/*
 * A prompt, or a training forward: the layer over whole sequences.
 *   q, k, v, out  bf16, element e of head h of row r at r * ld + h * dim + e (dim_k for q and k,
 *            dim_v for v and out); they may be parts of one projection's rows.  out may not
 *            overlap the others.
 *   starts   int32 [batch + 1] or NULL.  NULL: sequence b has the rows b * seq_len ..
 *            (b + 1) * seq_len - 1, and tokens is batch * seq_len.  Otherwise it has the rows
 *            starts[b] .. starts[b + 1] - 1, seq_len is the longest length: numbers outside
 *            [0, tokens] count as the nearer end, an end before its start as an empty sequence,
 *            and what a sequence has beyond seq_len rows is not read.  Sequences must not
 *            overlap.  out's rows that belong to no sequence are left as they are.
 *   state_in, state_out  fp32 [slots][heads][dim_k][dim_v], each NULL (zeros; not wanted) or a
 *            pool of states; state_out may be state_in, other overlaps are TTT_E_CONFIG.
 *   slot     int32 [batch], sequence b's entry in both pools, or NULL: entry b, and slots is at
 *            least batch.  A sequence whose slot lies outside [0, slots) starts from zeros and
 *            its state is not kept.  The slots inside must differ from each other.  Other
 *            entries of state_out are left as they are.  An empty sequence's state is kept
 *            as it is.
 * All values must be finite: one that is not makes the rows of its sequence and head NaN from up
 * to 63 tokens before it on.
 * q k, sums, states and powers are fp32 or more.  What out is made of (states, a token's weights and
 * decayed values) enters its products as two bf16 numbers each (16 significant bits), so that out is
 * rounded once; for a state that is given back the decayed values enter as three (24 bits, as
 * fp32), so that out's last bit may differ with whether one is wanted.  A state's decay over many tokens stays
 * within one step of fp32, its product with the state is rounded once in 64 tokens.  Every sum has one
 * order: the results are the same from run to run.
 * Limits: batch in [0, 65535], batch * heads at most 2^20, 0 <= seq_len <= 2^30, 0 <= tokens < 2^31, every ld at
 * least heads * dim, below 2^24 and a multiple of 8.  tokens, seq_len and batch may be 0.
 * work: workspace of the size that ttt_linear_attention_work gives for the same configuration,
 * batch and seq_len.
 */
ttt_status ttt_linear_attention_work(const ttt_linear_attention_config* cfg, int32_t batch,
                                     int64_t seq_len, int64_t* bytes);
ttt_status ttt_linear_attention(const ttt_linear_attention_config* cfg, const void* q,
                                int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                                int64_t ld_v, const float* decay, const int32_t* starts,
                                const float* state_in, float* state_out, const int32_t* slot,
                                int32_t slots, void* out, int64_t ld_out, int64_t tokens,
                                int32_t batch, int64_t seq_len, void* work, int64_t work_bytes,
                                void* stream);

/*
 * Backward of ttt_linear_attention with states of the sequences themselves (slot NULL, slots
 * batch): from its inputs, dout (rows as out's, stride ld_dout) and dstate_out (fp32 [batch][heads]
 * [dim_k][dim_v], the gradient of the final states, or NULL for zeros), the gradients dq, dk
 * and dv (bf16, rows as those of q, k and v with their own strides; they may be parts of one
 * buffer's rows) and, where given, dstate_in, that of the initial states (fp32, as dstate_out).
 * With P_t = decay P_{t+1} + scale q_t dout_t^T (P_T the gradient of the final state over decay):
 *   dq_t = scale S_t dout_t,  dk_t = P_t v_t,  dv_t = P_t^T k_t,  dstate_in = decay P_0.
 * Precision, order, starts and limits as above; all values must be finite, one that is not reaches up
 * to 63 tokens back, and backward in time (dk, dv) as many on.  The gradients and work may not overlap the
 * inputs or each other.  Rows that belong to no sequence are left as they are.
 */
ttt_status ttt_linear_attention_backward_work(const ttt_linear_attention_config* cfg,
                                              int32_t batch, int64_t seq_len, int64_t* bytes);
ttt_status ttt_linear_attention_backward(
    const ttt_linear_attention_config* cfg, const void* q, int64_t ld_q, const void* k,
    int64_t ld_k, const void* v, int64_t ld_v, const float* decay, const int32_t* starts,
    const float* state_in, const void* dout, int64_t ld_dout, const float* dstate_out, void* dq,
    int64_t ld_dq, void* dk, int64_t ld_dk, void* dv, int64_t ld_dv, float* dstate_in,
    int64_t tokens, int32_t batch, int64_t seq_len, void* work, int64_t work_bytes, void* stream);

/*
 * One token of each sequence: row s of q, k, v and out, the state of sequence s in entry slot[s]
 * (or s) of the pools, as for a prompt of one token each.  state_in NULL: zeros; state_out NULL:
 * not wanted; state_out may be state_in.  Everything is fp32 until out is rounded; a value that
 * is not finite stays with its sequence and head.
 * Limits: 0 <= seqs <= 2^20, seqs * heads at most 2^22; the others as above.
 */
ttt_status ttt_linear_attention_step(const ttt_linear_attention_config* cfg, const void* q,
                                     int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                                     int64_t ld_v, const float* decay, const float* state_in,
                                     float* state_out, const int32_t* slot, int32_t slots,
                                     void* out, int64_t ld_out, int32_t seqs, void* stream);

/*
 * The gate of a sub-layer's output: none, sigmoid(g), or silu(g) = g sigmoid(g).  Any g may be given, the
 * lowest number of the type as a mask among them; at infinity they are their limits: sigmoid 0 and 1, silu
 * 0 at minus infinity.
 */
typedef enum { TTT_GATE_NONE = 0, TTT_GATE_SIGMOID = 1, TTT_GATE_SILU = 2 } ttt_gate;

/*
 * What stands between two sub-layers, in one pass over the rows.  For every row
 *   u = y / sqrt(mean over its group (y^2) + eps) * y_weight     (norm_y; without it u = y)
 *   z = u act(gate)                                              (without a gate z = u)
 *   h_out = h + res_scale z                                      (without h: res_scale z)
 *   n_out = h_out / sqrt(mean(h_out^2) + eps) * n_weight
 * groups splits a row into equal groups, such as the heads of a sequence layer, each with its
 * own mean.  Everything is fp32 (n_out is taken of the unrounded h_out) and rounded once.
 * Limits: dim a multiple of 8 in [8, 8192]; groups 1, or such that dim / groups is a power of
 * two in [8, 512]; act bf16 or fp32; eps finite and > 0.
 */
typedef struct {
  int32_t dim, groups;
  int32_t norm_y;   /* 0 or 1   */
  int32_t gate;     /* ttt_gate */
  int32_t act;      /* ttt_dtype of the rows and the learned scales */
  float eps;
} ttt_residual_norm_config;

/* Host-only check of a configuration (no HIP call). */
ttt_status ttt_validate_residual_norm_config(const ttt_residual_norm_config* cfg);

/*
 *   h, y, gate, h_out, n_out  rows of dim elements, row t at t * ld.  h may be NULL (no residual);
 *            gate is NULL exactly where the configuration has none; h_out or n_out may be NULL (not
 *            wanted), not both.  An output may be one of the inputs h, y and gate (the same
 *            stride); other overlaps of outputs with inputs or each other are TTT_E_CONFIG.
 *   y_weight, res_scale, n_weight  [dim] learned scales, each NULL for ones (y_weight must be
 *            NULL without norm_y, n_weight without n_out)
 * Limits: 0 <= tokens <= 2^25; every ld at least dim, at most 2^28 and such that rows stay
 * 16-byte aligned.  A row's sums of squares are fp32: squares that add up past its range give
 * zeros.  A value that is not finite stays with its row.
 */
ttt_status ttt_residual_norm(const ttt_residual_norm_config* cfg, const void* h, int64_t ld_h,
                             const void* y, int64_t ld_y, const void* gate, int64_t ld_gate,
                             const void* y_weight, const void* res_scale, const void* n_weight,
                             void* h_out, int64_t ld_ho, void* n_out, int64_t ld_n,
                             int64_t tokens, void* stream);

/*
 * Backward of ttt_residual_norm: from its inputs and the gradients dh_out and dn of h_out and n_out
 * (activation dtype; either NULL for zeros, not both; n_weight only with dn), the gradients dh (of
 * h; only with h), dy and dgate (of the gate before its activation; only with a gate), rows as
 * theirs, each NULL where not wanted, and those of the learned scales that are given (fp32 [dim],
 * overwritten, each NULL where not wanted: the sum over all rows, in an order that depends only
 * on the sizes).  A row gradient may be dh_out or dn (the same stride); other overlaps of what is
 * written (work among it) with an input or each other are TTT_E_CONFIG.  A row whose squares pass fp32's range
 * has a norm of zeros and no gradient through it.
 * work: workspace of the size that ttt_residual_norm_backward_work gives (needed where a scale's
 * gradient is wanted).  tokens 0 writes zero scale gradients.
 */
ttt_status ttt_residual_norm_backward_work(const ttt_residual_norm_config* cfg, int64_t tokens,
                                           int64_t* bytes);
ttt_status ttt_residual_norm_backward(
    const ttt_residual_norm_config* cfg, const void* h, int64_t ld_h, const void* y, int64_t ld_y,
    const void* gate, int64_t ld_gate, const void* y_weight, const void* res_scale,
    const void* n_weight, const void* dh_out, int64_t ld_dho, const void* dn, int64_t ld_dn,
    void* dh, int64_t ld_dh, void* dy, int64_t ld_dy, void* dgate, int64_t ld_dgate,
    float* dy_weight, float* dres_scale, float* dn_weight, void* work, int64_t work_bytes,
    int64_t tokens, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TTT_MIXER_H */
