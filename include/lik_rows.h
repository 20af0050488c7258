/*
 * lik_rows.h -- C ABI of the losses over rows of logits (gfx950), beside the
 * row cross-entropy of lik.h (lik_ce_rows).
 *
 * A row is R x C logits z: the scores of one query against C documents (a
 * MaxSim forward's [Nq, Nd] or [B, N] output), or a language model's logits
 * of one token over its vocabulary.  With y = scale * z and
 *
 *     q_c = softmax_c(y),   lse = log sum_c exp(y_c),   logp = y_t - lse,
 *
 * the operators are
 *
 *   lik_logprob_rows_fwd/bwd   logp of one target column per row, and the
 *                              gradient of any loss on it
 *   lik_distill_rows           KL divergence from a teacher that is known by
 *                              its top K logits, with its gradient
 *   lik_policy_rows            clipped policy loss with a KL term, with its
 *                              gradient
 *   lik_preference_rows        loss on paired log ratios of whole sequences
 *                              of rows, with its gradient
 *
 * The conventions of lik.h hold (memory, stream, workspace, errors,
 * determinism, reentrancy), and for every operator here:
 *
 * Rows.  A call without rows (R == 0) is a successful no-op that writes no
 *   output, a preference loss over empty sequences among them.
 * Logits.  float16, bfloat16 or float32 (LIK_F16, LIK_BF16, LIK_F32), row r
 *   at logits + r * ld elements (ld >= C), columns dense, aligned to the
 *   element.  Every exponential, sum and statistic is float32 or wider.
 * Gradient.  [R, C] in the logits' type with a row stride of its own
 *   (grad_ld >= C), each entry rounded once from float32; the logits' own
 *   type because it is what the backward of whatever made the logits takes,
 *   and half the traffic for 16-bit logits.  Columns from C to the stride are
 *   left as they were.  From its first to its last element it must lie outside
 *   the memory from the logits' first to their last (other columns of one matrix
 *   are refused too).  NULL skips it (the losses alone then read the logits once).
 * scale.  The logit multiplier (1 / temperature), within [2^-64, 2^64].
 * Targets.  int32 columns.  A negative target leaves the row out: its logits
 *   are not read, its outputs and its gradient row are 0.  A target >= C makes
 *   the row's outputs and its gradient row NaN.
 * Row weights.  float32 [R], or NULL for 1 / R each: loss = sum_r w_r l_r, and
 *   the gradient is that of this sum.  A row of weight 0 is left out like one
 *   with a negative target.  (A mean over the rows that count is the weight
 *   1 / count on them and 0 elsewhere; a loss scale multiplies the weights.)
 * Masked logits.  Columns of -inf, or of the type's lowest value beside larger
 *   ones, have probability 0.  A row whose columns are all -inf has no
 *   softmax: its outputs and gradient are NaN unless it is left out.
 * Sums over rows, tokens and pairs are taken in float64 in a fixed order, so
 * losses are bitwise reproducible.
 */
#ifndef LIK_ROWS_H_
#define LIK_ROWS_H_

#include "lik.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Operation codes for lik_rows_workspace_bytes. */
typedef enum {
  LIK_ROWS_LOGPROB_FWD = 0,
  LIK_ROWS_LOGPROB_BWD = 1,
  LIK_ROWS_DISTILL = 2,
  LIK_ROWS_POLICY = 3,
  LIK_ROWS_PREFERENCE = 4
} lik_rows_op;

/* The loss on a pair's log ratio (lik_preference_rows). */
typedef enum {
  LIK_PREF_SIGMOID = 0,   /* -(1-e) log sigmoid(h) - e log sigmoid(-h) */
  LIK_PREF_HINGE = 1,     /* max(0, 1 - h) */
  LIK_PREF_SQUARE = 2     /* (d - 1 / (2 beta))^2 */
} lik_pref_kind;

/*
 * Workspace bytes of one call: the same R, C and dtype; n_seqs the number of
 * sequences S (lik_preference_rows; ignored otherwise); flags bit 0: a
 * gradient will be asked for (a call that differs may need more and then
 * returns LIK_ERR_INVALID_ARG).  Returns 0 for calls that need none and for
 * zero-sized ones; SIZE_MAX for sizes that overflow or an unknown op or dtype.
 */
size_t lik_rows_workspace_bytes(lik_rows_op op, int64_t R, int64_t C,
                                int64_t n_seqs, lik_dtype dtype, int flags);

/*
 * logp[r] = y[r, t_r] - lse[r] and lse[r], float32.  Both 0 for rows left out;
 * for a target >= C logp is NaN and lse is the row's.  (lse is a float32: the
 * backward's probabilities are off by its rounding, 2^-24 |lse| relative, and
 * undefined where it overflows.)
 */
lik_status lik_logprob_rows_fwd(const void* logits, lik_dtype dtype, int64_t R,
                                int64_t C, int64_t ld, const int32_t* targets,
                                float scale, float* logp, float* lse,
                                void* workspace, size_t workspace_bytes,
                                void* stream);

/*
 * Gradient of sum_r grad_logp[r] * logp[r]:
 *   grad[r, c] = grad_logp[r] * scale * ([c == t_r] - exp(y[r, c] - lse[r])),
 * lse from the forward for the same logits and scale.  A row whose grad_logp
 * is 0 is left out.  No workspace.
 */
lik_status lik_logprob_rows_bwd(const void* logits, lik_dtype dtype, int64_t R,
                                int64_t C, int64_t ld, const int32_t* targets,
                                float scale, const float* lse,
                                const float* grad_logp, void* grad,
                                int64_t grad_ld, void* stream);

/*
 * Distillation from a teacher's top logits.  Row r lists K entries (column
 * teacher_idx[r, k], teacher logit teacher_val[r, k]); a negative column is an
 * absent entry, so lists may be ragged.
 *   teacher_lse NULL: the teacher's probabilities are renormalised over the
 *     listed entries, p_k = softmax_k(scale * val), and
 *     l_r = sum_k p_k (log p_k - log q[idx_k]).
 *   teacher_lse [R]: the teacher's log-sum-exp of scale * logit over all its
 *     columns; p_k = exp(scale * val_k - teacher_lse), and what is left,
 *     p_rest = max(0, 1 - sum_k p_k), is set against the student's mass on the
 *     columns not listed, q_rest:
 *     l_r += p_rest (log p_rest - log q_rest)
 *     (nothing is added where every column is listed).
 * With M the teacher's mass in the row's terms (1 up to rounding), the
 * gradient of w_r l_r is w_r scale (M q_j - sum of the p_k listed for j), and
 * w_r scale q_j (M - p_rest / q_rest) on columns not listed.  A column listed
 * twice counts once in q and with both entries in p.  A teacher logit of -inf
 * has p = 0.  A row without a present entry, or whose entries all have -inf
 * logits, has loss 0 and gradient 0 (without teacher_lse), or only the rest's
 * term (with it).  An entry with column >= C makes the row's loss and gradient
 * NaN.  K <= 1024 and C <= 2^20 (LIK_ERR_UNSUPPORTED beyond).  The usual
 * factor of the squared temperature is the caller's, in row_weight.
 * teacher_lse is a float32, so p_rest is off by up to 2^-22 (1 + |teacher_lse|):
 * where the student leaves no finite column outside the list, pass NULL, for
 * what rounding leaves of p_rest is set against a q_rest of 0 (infinite loss).
 * row_loss [R] float32, loss [1] float32.
 */
lik_status lik_distill_rows(const void* logits, lik_dtype dtype, int64_t R,
                            int64_t C, int64_t ld, const int32_t* teacher_idx,
                            const float* teacher_val, int64_t K,
                            const float* teacher_lse, float scale,
                            const float* row_weight, float* row_loss,
                            float* loss, void* grad, int64_t grad_ld,
                            void* workspace, size_t workspace_bytes,
                            void* stream);

/*
 * Clipped policy loss.  With rho = exp(logp - old_logp) and A = advantage,
 *   l_r = -min(rho A, clamp(rho, 1 - clip_low, 1 + clip_high) A)
 *         + kl_coef (exp(ref_logp - logp) - (ref_logp - logp) - 1),
 * the second term only with ref_logp (NULL: none) and a kl_coef other than 0;
 * it is infinite where either of the two rules the target out.
 * old_logp, advantage and ref_logp are float32 [R], constants of the gradient;
 * a row at the border of its clip still has the gradient of rho A.  0 <= clip_low <= 1,
 * clip_high >= 0 (infinity: no clip on that side), kl_coef finite.
 * row_loss, logp [R] float32, loss [1] float32.
 */
lik_status lik_policy_rows(const void* logits, lik_dtype dtype, int64_t R,
                           int64_t C, int64_t ld, const int32_t* targets,
                           const float* old_logp, const float* advantage,
                           const float* ref_logp, float scale, float clip_low,
                           float clip_high, float kl_coef,
                           const float* row_weight, float* row_loss,
                           float* logp, float* loss, void* grad,
                           int64_t grad_ld, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * Preference loss on paired log ratios.  The rows are the tokens of S
 * sequences: sequence s is rows seq_offsets[s] .. seq_offsets[s+1] - 1
 * (int32 [S + 1], on the device, not decreasing, within [0, R]); its
 * log-probability L_s is the sum of its rows' logp, or with mean_logp != 0
 * their mean over the rows that carry a target; 0 for a sequence without any.
 * Pair p sets sequence chosen[p] against rejected[p] (int32; a sequence may be
 * in any number of pairs):
 *   d_p = (L_chosen - ref_chosen) - (L_rejected - ref_rejected),
 *   h_p = beta d_p - margin
 * with ref_logp [S] float32 (NULL: 0), and its loss l_p is that of `kind`:
 * smoothing e (0 <= e <= 0.5) belongs to LIK_PREF_SIGMOID, margin to it and
 * to LIK_PREF_HINGE; both must be 0 elsewhere.  beta > 0.
 *   loss = sum_p w_p l_p, pair_weight float32 [P] or NULL for 1 / P; a pair of
 * weight 0 is left out (its pair_loss is written all the same).  A sequence
 * number outside [0, S) makes the pair's loss NaN and takes the pair out of
 * the gradient.  Rows outside every sequence are not read; their gradient is
 * 0.  Rows of a sequence in no pair have gradient 0 too.  A NaN in a sequence
 * (a target >= C, a NaN logit) makes it, its pairs' losses and the gradient of
 * every sequence in those pairs NaN.
 * pair_loss [P], seq_logp [S], loss [1]: float32.  S x P <= 2^40
 * (LIK_ERR_UNSUPPORTED beyond).
 */
lik_status lik_preference_rows(const void* logits, lik_dtype dtype, int64_t R,
                               int64_t C, int64_t ld, const int32_t* targets,
                               const int32_t* seq_offsets, int64_t S,
                               const int32_t* chosen, const int32_t* rejected,
                               int64_t P, const float* ref_logp,
                               lik_pref_kind kind, float beta, float margin,
                               float smoothing, int mean_logp, float scale,
                               const float* pair_weight, float* pair_loss,
                               float* seq_logp, float* loss, void* grad,
                               int64_t grad_ld, void* workspace,
                               size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LIK_ROWS_H_ */
