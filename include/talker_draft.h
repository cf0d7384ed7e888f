/*
 * talker_draft.h — C-ABI of the verification of drafted tokens (speculative
 * decoding): drafted tokens of each sequence are taken or refused by the target's
 * logits and given random numbers, and the token after them is drawn.
 *
 * No handle: the caller owns every buffer; the call enqueues its kernels on
 * cuda_stream (NULL = legacy stream) of the current device and returns. Nothing is
 * allocated and the call may be captured into a CUDA graph. All pointers are
 * device pointers, aligned to their elements.
 */
#ifndef TALKER_DRAFT_H
#define TALKER_DRAFT_H

#include "talker.h"

#ifdef __cplusplus
extern "C" {
#endif

/* For each sequence s, with drafted tokens x_i, i < count (counts[s], or n_draft
 * without counts), uniform numbers u_0 .. u_n_draft and temperature T:
 *   p_i = softmax(target[s][i] / T), i <= count;  q_i = softmax(draft[s][i] / T),
 *   or, without draft logits, all of q_i on x_i;
 *   x_i is taken while u_i q_i(x_i) < p_i(x_i);  n: how many are taken;
 *   the next token t is the first with sum_{v <= t} w(v) > u_n_draft sum_v w(v),
 *   w = max(p_n - q_n, 0) where x_n was refused (p_n if that is 0 everywhere, which
 *   only rounding can bring about), w = p_n if all count were taken.
 * T above 1e18 counts as 1e18. T not above 1e-20 (0, negative or NaN) is greedy: p_i is all on the first of the row's
 * largest logits, x_i is taken if it is that token, and draft logits are not read.
 *
 * tokens_out [n_seq][n_draft + 1]: the taken tokens, the next token, then -1;
 * accepted [n_seq]: n; logprobs (may be NULL) [n_seq][n_draft + 1]: log p_i of each
 * token in tokens_out, 0 for those of -1.
 *
 * Masked values: a NaN, or a value at or below -1e30, counts as -inf. A row without
 * any other value, or with one of +inf, has no distribution: p_i (q_i) is 0
 * everywhere. x_i is then refused for p_i, and where p_n is 0 everywhere the next token
 * is -1, with log-probability 0. A drafted token outside the vocabulary is refused. Counts
 * are taken to [0, n_draft] and uniform numbers to [0, 1] (NaN: 0).
 *
 * Probabilities that decide (p and q of a draft near its border, all of the row that is
 * drawn from) are made to about 2^-29 of themselves and summed as whole numbers, in units
 * that cut off less than 2^-28 of a sum (those below 2^-70 of the row's largest count as 0,
 * and where q is taken off, those below 2^-62; what is left of p then has the errors of both).
 * So neither a row's address nor the launch's shape changes a token; the sums of taken drafts'
 * logprobs are f32.
 *
 * target: row i of sequence s lies at s * target_seq + i * target_row elements, vocab
 * contiguous values; draft likewise (NULL: none), n_draft rows. dtype F32 or BF16 for
 * both. tokens int32 [n_seq][n_draft], counts int32 [n_seq] or NULL, uniforms f32
 * [n_seq][n_draft + 1], temperatures f32 [n_seq] or NULL (1). Outputs must not overlap
 * inputs. n_draft <= 64, vocab <= 2^26, n_seq <= 65535.
 * scratch: talker_draft_scratch bytes, 16-byte aligned (may be NULL when that is 0); it need not
 * hold anything on entry, and calls that may run at the same time need their own.
 * Errors: EINVAL, ECUDA. */
size_t talker_draft_scratch(int n_seq, int n_draft, int vocab);
talker_status talker_draft_verify(const void *target, int64_t target_seq, int64_t target_row, const void *draft,
                                  int64_t draft_seq, int64_t draft_row, int dtype, const int32_t *tokens,
                                  const int32_t *counts, const float *uniforms, const float *temperatures, int n_seq,
                                  int n_draft, int vocab, int32_t *tokens_out, int32_t *accepted, float *logprobs,
                                  void *scratch, size_t scratch_bytes, void *cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* TALKER_DRAFT_H */
