/*
 * libpalu — verification of drafted tokens (speculative decoding; page "add
 * TurboQuant KV cache compression", the pull request's review: speculative
 * rollback), from given random numbers.
 *
 * A draft model proposes up to k tokens for a sequence, the target model
 * scores all of them in one step, and a prefix of the drafts is kept so that
 * the kept tokens and the one sampled behind them are distributed as the
 * target's own samples.  The lengths that remain go straight to
 * palu_cache_truncate_ragged, or into the lengths of a paged cache.
 *
 * Conventions are those of palu.h.
 */
#ifndef PALU_DRAFT_H
#define PALU_DRAFT_H

#include "palu.h"

#ifdef __cplusplus
extern "C" {
#endif

/* For sequence b with drafts x_0 .. x_{n-1} (n = n_drafts[b]), target rows
 * p_0 .. p_n and draft rows q_0 .. q_{n-1}:
 *   draft i is kept while accept_u[b, i] * q_i(x_i) < p_i(x_i) has held for
 *   it and every draft before it; a = the number kept;
 *   one more token is drawn from the weights w(t) = max(p_a(t) - q_a(t), 0)
 *   if a < n (from p_a where these are all zero), and from p_n if a = n:
 *   the lowest t with w(0) + .. + w(t) > sample_u[b] * (w(0) + .. + w(V-1)).
 * The test of a draft is exact.  A running sum and u times the total are
 * together right to (278 + 12 ceil(V / 16384)) 2^-48 of the total (2^-39 for a
 * vocabulary of 152,065): a draw nearer than that to a border between two
 * tokens may give either, and the other one in a batch of another size (a call
 * that is repeated repeats its answer).  Weights that are NaN
 * count as 0; probabilities must be finite and need not be normalised.  A
 * draft outside 0 .. V-1 is never kept.
 *   target   device fp32, row (b, i) at target + b * target_strides[0] +
 *            i * target_strides[1] (elements), V contiguous values, i in 0 .. k.
 *   draft    device fp32, the same for i in 0 .. k-1; NULL where the drafts
 *            come from no distribution (copied from the prompt): then q_i is 1
 *            at x_i and 0 elsewhere.
 *   drafts   device int64 [batch, k]; n_drafts device int32 [batch] (NULL: k
 *            each; values are clamped to 0 .. k).
 *   accept_u device fp32 [batch, k] and sample_u device fp32 [batch], in [0, 1).
 *   lengths  device int64 [batch] (may be NULL): each sequence's length with
 *            all its n drafts; new_lengths device int64 [batch] =
 *            lengths - (n - a) (may be the same array).
 *   tokens   device int64 [batch, k+1]: the kept drafts, the drawn token,
 *            then -1.  The drawn token is -1 where no weight is positive.
 *   n_kept   device int32 [batch]: a (may be the array n_drafts).
 * Outputs must overlap neither an input nor each other, but for the two that
 * may be the same array.
 * k in 1 .. 256.  One kernel launch, no workspace. */
palu_status palu_draft_verify(int64_t batch, int32_t k, int64_t vocab, const float* target,
                              const int64_t target_strides[2], const float* draft, const int64_t draft_strides[2],
                              const int64_t* drafts, const int32_t* n_drafts, const float* accept_u,
                              const float* sample_u, const int64_t* lengths, int64_t* tokens, int32_t* n_kept,
                              int64_t* new_lengths, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PALU_DRAFT_H */
