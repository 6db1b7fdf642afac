/*
 * gdn_score.h -- C ABI of token scores on MI355X (gfx950): log-probabilities of given
 * tokens, entropy and best alternatives of rows of logits, and their gradient.
 *
 * The other calls of a decode step take what these give: gdn_tree_build a drafter's
 * best continuations (top_logp, top_tok), gdn_tree_accept the verifier's token after each
 * node (top_tok with topk = 1).  Training a drafter needs logp of given tokens, the
 * alternatives' log-probabilities, and gradients.
 *
 * For a row x of `vocab` logits, with m = max x and s = sum_j e^(x_j - m):
 *
 *     lse = m + ln s        ln p_j = x_j - lse        entropy = -sum_j p_j ln p_j
 *
 * Logits of -inf are entries of probability 0 (their part of the entropy is 0).  A row
 * without a finite logit, with +inf or with NaN has NaN or infinite results, as the
 * formulas give them; no other row is touched by it.
 *
 * Conventions are those of gdn_tree.h: every pointer is 16-byte aligned (GDN_ERR_ALIGN), so that
 * labels from a tensor's second element on have to be copied; the rows of logits may lie at any
 * distance.  Sums and results are fp32.
 */
#ifndef GDN_SCORE_H
#define GDN_SCORE_H

#include "gdn_tree.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 0 <= rows <= 2^22 (0 launches nothing), 1 <= vocab <= 2^24, rows ceil(vocab / 16384) < 2^24,
 * 0 <= topk <= min(64, vocab), vocab <= row_stride <= 2^40: elements between rows of logits and of their
 * gradient.  Others: GDN_ERR_DIMS. */
typedef struct {
    int64_t rows, row_stride;
    int32_t vocab, topk, io_dtype;
} gdn_score_dims;

/* Bytes of the workspace of gdn_token_scores; its contents need no preparation.  Calls
 * that follow each other on a stream can share one. */
int gdn_score_workspace_bytes(const gdn_score_dims* dims, size_t* bytes);

/*
 *   logits   [rows][vocab]  io    row_stride elements apart
 *   tokens   [rows]         int32 (NULL: no logp); a token outside [0, vocab) gives NaN
 *   logp     [rows]         fp32  out: ln p of the token (NULL where tokens is NULL)
 *   entropy  [rows]         fp32  out (NULL: not wanted)
 *   lse      [rows]         fp32  out (NULL: not wanted)
 *   top_logp [rows][topk]   fp32  out: ln p of the best alternatives, best first
 *   top_tok  [rows][topk]   int32 out: their tokens; equal logits in order of the token.
 *                                 NaN orders before every number.  Both NULL where topk = 0
 */
int gdn_token_scores(const gdn_score_dims* dims, const void* logits, const int32_t* tokens, float* logp,
                     float* entropy, float* lse, float* top_logp, int32_t* top_tok, void* workspace,
                     hipStream_t stream);

/*
 * Gradient of the logits, from lse and entropy as gdn_token_scores wrote them for these logits:
 *
 *     d_x_j = -p_j (d_logp + sum_c d_top_logp_c + d_entropy (ln p_j + entropy))
 *             + [j = token] d_logp + sum_c [j = top_tok_c] d_top_logp_c
 *
 *   d_logp     [rows]       fp32 (NULL, as tokens: no such term)
 *   d_entropy  [rows]       fp32 (NULL: no such term; entropy may then be NULL)
 *   top_tok    [rows][topk] int32 any tokens, repeated ones too; one outside [0, vocab) has no
 *   d_top_logp [rows][topk] fp32  part in the gradient.  Both NULL: no such term
 *   d_logits   [rows][vocab] io  out, row_stride elements apart; may be logits
 *
 * A token outside [0, vocab) has no part in the gradient.  ln p_j is x_j - lse, with what lse's rounding
 * leaves of it (2^-24 |lse|); where |lse| >= 4096, as in rows that hold a mask's value alone, it
 * comes of the row's logits again.
 */
int gdn_token_scores_backward(const gdn_score_dims* dims, const void* logits, const int32_t* tokens, const float* lse,
                              const float* entropy, const float* d_logp, const float* d_entropy,
                              const int32_t* top_tok, const float* d_top_logp, void* d_logits, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_SCORE_H */
