/*
 * The policy's loss on generated responses, from the logits, with its gradient: what follows the rollout
 * (pg_rollout.h) and the packed forward in a GRPO step.  Prefix Grouper changes how the forward of a
 * group is computed and leaves the objective as it is (skill page "prefix-grouper-grpo"); the logits of
 * the prefix's last token, computed once for all responses of a group, are where each of them has its
 * first token.
 * Same conventions as pg_grouped_attn.h: caller-owned device buffers, asynchronous on `stream`,
 * host-side argument checks, no allocation.
 */
#ifndef PG_POLICY_H
#define PG_POLICY_H

#include "pg_grouped_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct pg_policy_opts {
  float temperature;  /* T, at least 2^-126 and finite: the distribution is softmax(logits / T) */
  float clip_low;     /* the ratio is clipped to [1 - clip_low, 1 + clip_high]; both >= 0 */
  float clip_high;
  float kl_coef;      /* weight of the KL term, >= 0 */
} pg_policy_opts;

/*
 * Log-probabilities of the tokens, their loss and, if asked for, its gradient.  With z = logits / T,
 * lse_r = ln sum_i exp(z_ri), and for a token n of row r:
 *   lp_n = z_r,token(n) - lse_r,   ratio = exp(lp_n - old_n),   gap = ref_n - lp_n
 *   token_loss[n] = w_n (-min(ratio A_n, clip(ratio) A_n) + kl_coef (exp(gap) - gap - 1))
 *   token_grad[n] = d token_loss[n] / d lp_n
 *                 = w_n (-(ratio A_n if ratio A_n <= clip(ratio) A_n else 0) + kl_coef (1 - exp(gap)))
 *   loss = sum_n token_loss[n]
 *   dlogits[r, i] = 1/T sum_{n of r} token_grad[n] ([i = token(n)] - exp(z_ri - lse_r))
 *   logits [rows, vocab] of dtype `dtype`, rows ld elements apart; dlogits like it, rows ldd apart, NULL:
 *   no gradient; it may be logits itself (ldd = ld)
 *   row_starts int32 [rows + 1] (device): tokens [row_starts[r], row_starts[r + 1]) belong to row r, which
 *   may have any number of them, row_starts[0] = 0, row_starts[rows] = n_tokens; NULL: token n is row
 *   n's, n_tokens = rows
 *   tokens int32 [n_tokens]; old_logprobs, ref_logprobs, advantages, weights fp32 [n_tokens] (device)
 *   lse fp32 [rows], logprobs, token_loss, token_grad fp32 [n_tokens], loss fp32 [1]
 * A row's targets beyond 256 (where rows are longer and many up to 1024) cost a look-up each at every 16 bytes of the row.
 * advantages NULL: log-probabilities only (old_logprobs, ref_logprobs, weights, token_loss, token_grad,
 * loss and dlogits must be NULL too).  old_logprobs NULL: the ratio is 1 (its gradient is not: this is
 * the first step on a rollout, old = lp); ref_logprobs NULL: no KL term; weights NULL: 1.
 * A row without a token is not read: its lse is 0 and its gradient 0.  A token below 0 is padding: its
 * log-probability, loss and gradient are 0.  One of vocab or above is taken as such and recorded
 * as PG_ERR_DEVICE in the status word, like a row_starts that decreases, leaves [0, n_tokens] or leaves a token to
 * no row (whose results are then not written).  A token
 * of weight 0 has loss 0 and gradient 0 whatever the rest is, and a row whose tokens all have gradient 0
 * has gradient 0.  Logits of -inf have probability 0; a row of them throughout has lse and
 * log-probabilities -inf, its tokens loss 0 and gradient 0.  A NaN or +inf logit makes its row's
 * lse, log-probabilities, losses and gradients NaN (weight 0 apart).
 * Arithmetic in fp32, sums in a fixed order, the loss in fp64; one rounding to the type of dlogits.  A log-probability's
 * error goes by the row's differences, not by its logits' size; that of lse is 2^-22 of it besides.
 * rows >= 1, 1 <= vocab < 2^30, n_tokens >= 0, pointers aligned to their element type.
 * Errors: PG_ERR_INVALID_ARG (host check, nothing launched); PG_ERR_CUDA on a launch failure.
 */
pg_status pg_policy_loss(pg_dtype dtype, int64_t rows, int32_t vocab, const void* logits, int64_t ld,
                         int64_t n_tokens, const int32_t* row_starts, const int32_t* tokens,
                         const float* old_logprobs, const float* ref_logprobs,
                         const float* advantages, const float* weights, const pg_policy_opts* opts,
                         float* lse, float* logprobs, float* token_loss, float* token_grad,
                         float* loss, void* dlogits, int64_t ldd, pg_stream_t stream);

/*
 * The gradient alone, from the lse that pg_policy_loss wrote and any gradient of the log-probabilities:
 *   dlogits[r, i] = grad_output / T sum_{n of r} token_grad[n] ([i = token(n)] - exp(logits[r, i] / T - lse[r]))
 * (so the rounding of lse[r] to fp32, 2^-24 of it, is in every probability, where pg_policy_loss takes x - max first).
 * grad_output fp32 [1] (device; NULL: 1).  Rows, tokens and padding as above; a row whose tokens all have
 * gradient 0 is not read.  With lse = -inf the probabilities are 0.
 */
pg_status pg_policy_loss_bwd(pg_dtype dtype, int64_t rows, int32_t vocab, const void* logits,
                             int64_t ld, int64_t n_tokens, const int32_t* row_starts,
                             const int32_t* tokens, float temperature, const float* lse,
                             const float* token_grad, const float* grad_output, void* dlogits,
                             int64_t ldd, pg_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* PG_POLICY_H */
