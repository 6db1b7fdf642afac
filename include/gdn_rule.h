/*
 * gdn_rule.h -- C ABI of the gated delta rule over whole sequences on MI355X
 * (gfx950): the pass over prompts and training sequences, its gradients, and the
 * step by one token.
 *
 * gdn_tree.h verifies a draft tree from a prefix state S0; these calls make that
 * state from the prompt's tokens, train the layer, and decode without a draft.
 * The rule is gdn_tree.h's, along one sequence instead of a tree's paths:
 *
 *     P_t = g_t S_(t-1),  w_t = v_t - P_t k_t,  S_t = P_t + beta_t w_t k_t^T,  o_t = S_t q_t
 *
 * with S [d_v][d_k] per value head, and value head h reading key head h / (h_v / h_k).
 *
 * Conventions are those of gdn_tree.h (device pointers, 16-byte aligned; a negative
 * gdn_status for what the host can see; nothing allocated, nothing synchronised, kernels
 * on `stream`; no normalisation and no scale of q and k), and:
 *
 *  - q, k, v, o and their gradients are gdn_attn_rows: [rows][heads][d] with the last
 *    axis contiguous and any row and head stride >= 0, in elements, so that q, k and v
 *    can be slices of one projection's output.  They need their elements' alignment alone
 *    (rows and heads at multiples of 16 bytes are read fastest); output rows must not
 *    overlap each other.
 *  - beta and g are [rows][h_v] fp32, contiguous; g in [0, 1].
 *  - Sequences are packed: sequence b owns rows offsets[b] .. offsets[b+1] - 1 (device
 *    int32 [B + 1], non-decreasing from 0, 4-byte aligned), 0 rows allowed, n_rows rows in
 *    all tensors.  A sequence whose offsets are unusable (offsets[b] < 0, fewer than 0
 *    rows, rows past n_rows) has none of its rows read or written, and its state is
 *    passed through.  The others keep their results if each usable one begins at or after the
 *    end of the usable ones before it; where one begins earlier, as the third of offsets 0, 1000,
 *    50, 200 does, it and those that it goes back over have undefined results (still, nothing
 *    but their rows and states is written).  Rows that belong to no sequence are neither read
 *    nor written.
 *  - Elements have to be finite.  NaN or an infinity in a row can reach all results of its sequence,
 *    those of up to 63 rows before it in the forward pass included; other sequences keep theirs.
 *  - Outputs must not overlap inputs, except that S_out may be S0 and dS0 may be dS_out.
 *
 * Sizes: 1 <= d_k, d_v <= 256; h_k >= 1; h_v a multiple of h_k, <= 32768; batch <= 2^20;
 * n_rows / 64 + batch < 2^21; batch h_v d_v / 16 < 2^22 (d_v rounded up to 32).
 * gdn_rule_step: batch <= 65535.  batch = 0 launches nothing; row tensors of n_rows = 0 may
 * be NULL.  Every chunk of 64 rows looks for its sequence among all offsets, 64 at a time, and every
 * sequence of a step with slots among those before it: beyond some thousand sequences a call
 * takes time with the square of their number.
 *
 * Rounding.  States, sums, gates and their gradients are fp32.  The products run on
 * bf16 matrix instructions with fp32 sums; fp32 factors enter them as sums of bf16
 * terms, three wherever the result is fp32.  bf16 results are rounded once at the end,
 * from products whose fp32 factors have two terms.
 */
#ifndef GDN_RULE_H
#define GDN_RULE_H

#include "gdn_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int32_t batch, h_k, h_v, d_k, d_v, io_dtype;
} gdn_rule_dims;

/* Bytes of the workspace of gdn_rule_forward (backward = 0) or gdn_rule_backward
 * (backward = 1) for up to n_rows rows.  Its contents need no preparation and are of no
 * use after the call; calls that follow each other on a stream can share one. */
int gdn_rule_workspace_bytes(const gdn_rule_dims* dims, int64_t n_rows, int32_t backward, size_t* bytes);

/*
 * The rule along every sequence.
 *
 *   S0     [B][h_v][d_v][d_k] fp32  state before each sequence; NULL: zeros
 *   o      [rows][h_v][d_v]   io    out: o_t = S_t q_t
 *   S_out  [B][h_v][d_v][d_k] fp32  out: state after each sequence (NULL: not wanted)
 */
int gdn_rule_forward(const gdn_rule_dims* dims, const int32_t* offsets, int64_t n_rows, const float* S0,
                     const gdn_attn_rows* q, const gdn_attn_rows* k, const gdn_attn_rows* v, const float* beta,
                     const float* g, const gdn_attn_rows* o, float* S_out, void* workspace, hipStream_t stream);

/*
 * Gradients of gdn_rule_forward.  They are formed from the same inputs; nothing is kept
 * from the forward call.
 *
 *   d_o     [rows][h_v][d_v]   io    gradient of o
 *   dS_out  [B][h_v][d_v][d_k] fp32  gradient of S_out; NULL: zeros
 *   dq, dk  [rows][h_k][d_k]   io    out, summed over the value heads of a key head
 *   dv      [rows][h_v][d_v]   io    out
 *   dbeta   [rows][h_v]        fp32  out
 *   dlog_g  [rows][h_v]        fp32  out: gradient with regard to ln g (that with regard to g
 *                                    is dlog_g / g; ln g is what models compute, and dividing
 *                                    by a gate near 0 would only enlarge its error)
 *   dS0     [B][h_v][d_v][d_k] fp32  out: gradient of S0 (NULL: not wanted)
 */
int gdn_rule_backward(const gdn_rule_dims* dims, const int32_t* offsets, int64_t n_rows, const float* S0,
                      const gdn_attn_rows* q, const gdn_attn_rows* k, const gdn_attn_rows* v, const float* beta,
                      const float* g, const gdn_attn_rows* d_o, const float* dS_out, const gdn_attn_rows* dq,
                      const gdn_attn_rows* dk, const gdn_attn_rows* dv, float* dbeta, float* dlog_g, float* dS0,
                      void* workspace, hipStream_t stream);

/*
 * One token of every sequence, on a pool of states, in place.
 *
 *   q, k, v, o   [B] rows (row b: sequence b's token); beta, g [B][h_v]
 *   state        [n_slots][h_v][d_v][d_k] fp32  read and written at the sequences' slots
 *   slot         [B] int32  each sequence's slot; -1: no token, its row of o is left as it
 *                           is.  NULL: sequence b's is b.
 *
 * A slot outside [-1, n_slots), or one that an earlier sequence of the call has, gives a
 * NaN row of o and changes no state.
 */
int gdn_rule_step(const gdn_rule_dims* dims, const int32_t* slot, int32_t n_slots, const gdn_attn_rows* q,
                  const gdn_attn_rows* k, const gdn_attn_rows* v, const float* beta, const float* g, float* state,
                  const gdn_attn_rows* o, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_RULE_H */
