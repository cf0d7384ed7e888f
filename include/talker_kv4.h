/*
 * talker_kv4.h — C-ABI of the 4-bit paged KV cache and of beam selection.
 *
 * These entry points need no handle: the caller owns every buffer, and a call
 * enqueues its kernels on cuda_stream (NULL = legacy stream) of the current
 * device and returns. A talker handle with kv_dtype TALKER_DTYPE_Q4_0 keeps its
 * cache in the same layout and runs the same kernels.
 *
 * Storage, Q4_0 blocks: 32 consecutive dims of a head row share one scale.
 *   m = the dims' value of largest magnitude (the lowest dim on ties), clamped
 *       to +-524032; d = fp16(-m / 8), nearest even;
 *   n = clamp(floor(8.5 - 8 x / m), 0, 15), decided exactly (8 where m = 0);
 *   the code n stands for (n - 8) d.
 * A block that holds a NaN or an infinity stores d = NaN: all of it reads back
 * as NaN, and attention over it gives NaN, instead of a wrong finite value.
 *
 * Page: 64 positions of every (layer, KV head), one tile of 36 * head_dim bytes
 * each, [n_layers][n_kv_heads][tile]; K and V in pools of their own. A tile is
 * 64 rows of head_dim / 2 code bytes, then 64 rows of head_dim / 32 fp16 scales.
 * With NB = head_dim / 32, byte p of a row holds the dims (low nibble, high):
 *   K: p = c * 4 NB + 4 b + j (c, j < 4, b < NB): 32 b + 8 c + 2 j, and the next;
 *   V: p = g * 2 NB + 2 b + e (g < 8, e < 2):     32 b + 4 g + 2 e, and the next.
 * (The order in which the tensor-core fragments of the attention take them.)
 *
 * Conventions: all pointers are device pointers unless a comment says "host".
 * Argument checks run before anything is enqueued. What only the device can see
 * (lengths, page numbers, parents) is checked there: what is out of range is
 * skipped as described and sets a bit of *status (when status is not NULL):
 * 1 << 0 a position or length outside the stream's pages, 1 << 1 a copy that did
 * not arrive within a second (its row is NaN, and so are those that its CTA had yet
 * to attend), 1 << 3 a page number or parent out of range. Nothing is allocated; every call may be captured into
 * a CUDA graph; scratch need not hold anything on entry, and calls that may run
 * at the same time need scratch of their own.
 */
#ifndef TALKER_KV4_H
#define TALKER_KV4_H

#include "talker.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A cache in the caller's memory: pools k and v of n_pages pages each (16-byte
 * aligned), and the page table [n_streams][pages_per_stream] of page numbers.
 * head_dim is 64 or 128. */
typedef struct {
    void *k, *v;
    const int32_t *page_table;
    int32_t *status; /* or NULL */
    int32_t n_pages, n_streams, pages_per_stream;
    int32_t n_layers, n_kv_heads, head_dim;
} talker_kv4;

/* Bytes of one page of one pool; 0 for sizes that are not supported. */
size_t talker_kv4_page_bytes(int n_layers, int n_kv_heads, int head_dim);

/* Dense rows: the element of layer l, stream s, row i, head h, dim d (counted
 * from the call's first layer, stream and row) lies at
 * l * layer + s * stream + i * row + h * head + d elements from the pointer. */
typedef struct {
    int64_t layer, stream, row, head;
} talker_kv4_strides;

/* Write rows i < T of streams [stream0, stream0 + n_streams) of layers [layer0,
 * layer0 + n_layers): row i of stream s goes to position start[s] + i (start
 * NULL: 0). With count, rows i >= count[s] are not written (a padded batch). k
 * and v are dtype TALKER_DTYPE_F32 or _BF16, in the same strides. Streams that
 * share a page (talker_kv4_reorder) must not write it. A row outside the
 * stream's pages is skipped (status 1 << 0), as is one whose page number is out
 * of range (status 1 << 3).
 * Errors: EINVAL (null pointers, sizes, layers or streams out of range, T < 0,
 * T * n_kv_heads >= 2^31), ECUDA. */
talker_status talker_kv4_write(const talker_kv4 *c, int layer0, int n_layers, int stream0, int n_streams,
                               const int32_t *start, const int32_t *count, int T, const void *k, const void *v,
                               int dtype, const talker_kv4_strides *strides, void *cuda_stream);

/* Read the same rows back as the values they stand for, rounded once to dtype.
 * Rows that are not read (past count, or out of range) are left as they are. */
talker_status talker_kv4_read(const talker_kv4 *c, int layer0, int n_layers, int stream0, int n_streams,
                              const int32_t *start, const int32_t *count, int T, void *k, void *v, int dtype,
                              const talker_kv4_strides *strides, void *cuda_stream);

/* Decode attention: for streams b = 0..B-1 and query heads h (KV head h /
 * (n_q_heads / n_kv_heads), at most 8 query heads per KV head),
 *   out[b][h] = sum_j softmax_j(scale q[b][h] . K_j) V_j
 * over the stream's cached rows j < lens[b] of `layer` and, with k_new / v_new,
 * one more row that is attended as given (the step's own row, before or without
 * being written). q [B][n_q_heads][head_dim] and k_new, v_new [B][n_kv_heads]
 * [head_dim] are dense per head, with row strides q_row and new_row in
 * elements; out is contiguous; all are dtype (F32 or BF16). Scores, maxima and
 * sums are f32, and codes are exact. Probabilities, times their value's scale, enter
 * the tensor cores as two fp16 parts (22 bits, down to 2^-31 of the largest
 * probability times the largest scale of the block of dims, for scales from 2^-13);
 * so does q with F32, and with BF16 exactly (values below 2^-26 of a head's largest
 * lose bits). Values of q are to lie below 2^116, those of k_new and v_new where
 * products and sums stay finite.
 * A stream without rows gives zeros. A length outside the stream's pages sets
 * status 1 << 0 and gives zeros; keys of a page whose number is out of range
 * are not attended (status 1 << 3).
 * max_len is a host-side estimate of the longest length that only shapes the
 * launch; any lens give right results. scratch: talker_kv4_attend_scratch
 * bytes, 16-byte aligned, for the same B, heads and max_len (may be NULL when that is 0).
 * Errors: EINVAL, ECUDA. */
size_t talker_kv4_attend_scratch(const talker_kv4 *c, int B, int n_q_heads, int max_len);
talker_status talker_kv4_attend(const talker_kv4 *c, int layer, int B, const int32_t *lens, int max_len, int n_q_heads,
                                float scale, const void *q, int64_t q_row, const void *k_new, const void *v_new,
                                int64_t new_row, int dtype, void *out, void *scratch, size_t scratch_bytes,
                                void *cuda_stream);

/* Test support: the form that a Talker's steps on the tensor cores run, f32 q
 * [B][n_q_heads][head_dim] with bf16 results, over layer 0. Scratch and errors as above. */
talker_status talker_test_kv4_attend_mixed(const talker_kv4 *c, int B, const int32_t *lens, int max_len, int n_q_heads,
                                           float scale, const float *q, void *out_bf16, void *scratch,
                                           size_t scratch_bytes, void *cuda_stream);

/* Reorder the streams (beam search): afterwards, under table_out and lens_out,
 * stream i < R holds what stream parents[i] holds under c->page_table and lens
 * (streams i >= R hold their own). Full pages are shared, by page number; the
 * page that the next row goes to is copied for every stream but the first one
 * that takes it over, so each stream's writable pages are its own. The page
 * table must follow the rule that talker_kv4_reorder keeps: column j holds page
 * numbers r * pages_per_stream + j, r < n_streams, and n_pages >= n_streams *
 * pages_per_stream (the table r * pages_per_stream + j follows it). Streams that
 * nobody has as a parent are given up: the old table must not be used any more
 * once rows are written through the new one, but reordering again from the old
 * table with the same parents gives the same result. A program that cuts streams
 * which share pages (writes fewer into lens) calls it with R = 0 before it writes to
 * them: every stream keeps its rows, and the page that its next row goes to is its own.
 * table_out [n_streams][pages_per_stream] and lens_out [n_streams] must not
 * overlap the inputs. Lens in [0, 64 * pages_per_stream]; parents in
 * [0, n_streams). A bad parent (status 1 << 3) counts as the stream itself, a bad
 * length (status 1 << 0) as the nearest allowed one.
 * Errors: EINVAL (n_streams > 1024 among others), ECUDA. */
talker_status talker_kv4_reorder(const talker_kv4 *c, const int32_t *parents, int R, const int32_t *lens,
                                 int32_t *table_out, int32_t *lens_out, void *cuda_stream);

/* Beam selection. For each of n_seq sequences with `width` beams w, candidates
 *   c[w][v] = scores[w] + logits[w][v] - log(sum_u exp(logits[w][u])),  v < vocab
 * of which the best `width` are chosen, in descending order, equal ones by the
 * lowest w * vocab + v. Masked values: a NaN, or a value at or below -1e30 (the
 * lowest value of a type), counts as -inf, in logits and scores; a score of +inf
 * too, and every candidate of a row with a logit of +inf. Where fewer than
 * width candidates are above -inf, those at -inf follow in the same order. With
 * `ended`, a beam whose flag is not 0 has one candidate, eos_id, at its unchanged
 * score (all others -inf). A row's sum of exponentials is made in f32 (off by about
 * 2^-22 of itself), in an order that the row's values set and not its address: equal
 * rows have equal sums. From there on candidates are compared in 64 bits.
 * logits: [n_seq * width] rows of vocab elements, row_stride elements apart,
 * dtype F32 or BF16; scores f32 [n_seq][width]; ended int32 [n_seq][width] or
 * NULL (eos_id may then be negative: no token ends a beam). Outputs
 * [n_seq][width]: tokens, parents (the row seq * width + w that is continued),
 * scores_out, and ended_out (may be NULL): the parent had ended, or the token is
 * eos_id. Outputs must not overlap the inputs. width <= 32, width <= vocab,
 * vocab <= 2^30, n_seq * width < 2^26.
 * scratch: talker_beam_scratch bytes, 16-byte aligned (may be NULL when that is 0).
 * Errors: EINVAL, ECUDA. */
size_t talker_beam_scratch(int n_seq, int width, int vocab);
talker_status talker_beam_select(const void *logits, int64_t row_stride, int dtype, const float *scores,
                                 const int32_t *ended, int n_seq, int width, int vocab, int eos_id, int32_t *tokens,
                                 int32_t *parents, float *scores_out, int32_t *ended_out, void *scratch,
                                 size_t scratch_bytes, void *cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* TALKER_KV4_H */
