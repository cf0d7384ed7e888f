/*
 * talker_layer.h — C-ABI of the operators that a decoder layer needs around its
 * attention, over the caller's memory: residual addition with RMSNorm, rotary
 * positions, and products with 4-bit weights. With talker_kv4.h (rows written to
 * a cache and attended) they make up a layer.
 *
 * These entry points need no handle: the caller owns every buffer, and a call
 * enqueues its kernels on cuda_stream (NULL = legacy stream) of the current
 * device and returns. Nothing is allocated, and every call may be captured into a
 * CUDA graph. All pointers are device pointers unless a comment says "host"; each
 * is aligned to its element. All argument checks run before anything is enqueued;
 * calls without rows do nothing. Element types are talker_dtype; sums, norms and
 * products are f32 or more inside, and each result is rounded once.
 */
#ifndef TALKER_LAYER_H
#define TALKER_LAYER_H

#include "talker.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Residual addition and RMSNorm of `rows` rows of `width` values:
 *   s = x + residual             (without residual: s = x)
 *   y = s / sqrt(mean(s^2) + eps) * gain
 * The norm is that of the f32 sum, before it is rounded into sum_out. x and
 * residual are F32 or BF16, each its own; gain is f32 [width]. sum_out (NULL: not
 * written) has res_dtype and needs a residual. Row r lies at (r / inner) * outer_stride +
 * (r % inner) * inner_stride elements of each tensor (inner 1: rows at one stride;
 * heads of a row: inner = heads). Values in a row are contiguous.
 * y is F32, BF16 or E4M3. With E4M3 each row is cut into blocks of `block` values
 * (32, 64 or 128; 0: the row is one block), the last one shorter where width is no
 * multiple:
 *   scales[r][b] = max|y| / 448 over block b; code = e4m3(y * (448 / max|y|)), to
 *   the nearest, ties to even; y stands for code * scale.
 * scales is f32 [rows][ceil(width / block)], contiguous. Blocks with max|y| below
 * 2^-100 (or max|s * gain| below it) store zeros; one with an infinity reads back as NaN.
 * A NaN in s makes its row NaN, blocks of zeros too; the sum of a row's squares is to stay in f32's range.
 * sum_out may be residual or x, and y may be x or residual, with the same strides
 * and type; other overlaps are not allowed, nor are rows of sum_out or y at a stride of 0.
 * Errors: EINVAL (null x, gain or y; types; width not in 1..2^24; rows not in 0..2^30;
 * inner < 1; eps not at least 0; a block that is not offered; scales missing with
 * E4M3; results at a stride of 0), ECUDA. */
typedef struct {
    int64_t outer, inner; /* strides in elements */
} talker_row_strides;
talker_status talker_rms_norm(const void *x, int x_dtype, const talker_row_strides *x_at, const void *residual,
                              int res_dtype, const talker_row_strides *res_at, const float *gain, float eps, int rows,
                              int inner, int width, void *sum_out, const talker_row_strides *sum_at, void *y,
                              int y_dtype, const talker_row_strides *y_at, int block, float *scales,
                              void *cuda_stream);

/* Rotary positions. Pair i of a head's first rotary_dim dims, i < rotary_dim / 2, is
 * dims (i, i + rotary_dim / 2), or with `interleaved` dims (2 i, 2 i + 1); at position p
 * its values (a, b) become
 *   (a cos - b sin, a sin + b cos) of the angle p f_i, times the amplitude.
 * Dims from rotary_dim on stay. The frequencies f_i, in radians a position, of
 * theta_i = theta^(-2 i / rotary_dim), by `scaling`:
 *   NONE    theta_i
 *   LINEAR  theta_i / factor
 *   NTK     theta_i of the base theta * factor^(rotary_dim / (rotary_dim - 2))
 *   SMOOTH  theta_i (k + (1 - k) / factor), k = clamp((w - low) / (high - low), 0, 1) with
 *           w = original theta_i / (2 pi), the pair's turns over the original context
 *   YARN    theta_i ((1 - r) + r / factor), r = clamp((i - lo) / max(hi - lo, 0.001), 0, 1),
 *           lo = max(0, floor(d(high))), hi = min(rotary_dim - 1, ceil(d(low))),
 *           d(b) = rotary_dim log(original / (2 pi b)) / (2 log theta); the amplitude is
 *           `amplitude`, or 0.1 log(factor) + 1 where that is 0
 * and the amplitude is 1 but for YARN.
 *
 * A plan of a rope is the table turns[i] = f_i / (2 pi) in units of 2^-64 turn: a position
 * times it, modulo 2^64, is the angle's place in a turn, without error at any position
 * but that of the table (f64: 2^-54 turn a position). */
typedef enum {
    TALKER_ROPE_NONE = 0,
    TALKER_ROPE_LINEAR = 1,
    TALKER_ROPE_NTK = 2,
    TALKER_ROPE_SMOOTH = 3,
    TALKER_ROPE_YARN = 4
} talker_rope_scaling;
typedef struct {
    int32_t rotary_dim;  /* even, 2 to 512 (NTK: at least 4) */
    int32_t scaling;     /* talker_rope_scaling */
    double theta;        /* above 1 */
    double factor;       /* at least 1 */
    double original;     /* SMOOTH, YARN: positions of the original context */
    double low, high;    /* SMOOTH, YARN (its beta_slow and beta_fast, above 0): turns, low < high */
    double amplitude;    /* YARN: 0 for the rule above */
} talker_rope;
/* The table (HOST array of rotary_dim / 2) and amplitude (HOST) of a rope. A host function:
 * the caller copies the table to the device. Errors: EINVAL. */
talker_status talker_rope_turns(const talker_rope *rope, uint64_t *turns, float *amplitude);

/* A Talker with a scaled rope (talker.h): its positions turn with these frequencies and amplitude, in
 * prefills, decodes and frames. Before talker_kv_init_batched (ESTATE after it: cached rows
 * are turned already). rotary_dim must be the handle's head_dim, theta its rope_theta (pairs
 * are halves). rope is a HOST struct. Errors: EINVAL, ESTATE. */
talker_status talker_set_rope_scaling(talker_t *t, const talker_rope *rope);

/* Heads of rows: head h of row t of stream s lies at s * stream + t * row + h * head
 * elements; its dims are contiguous. */
typedef struct {
    const void *in;
    void *out; /* may be `in`, with the same strides; no other overlap */
    int32_t heads;
    int64_t in_stream, in_row, in_head;
    int64_t out_stream, out_row, out_head;
} talker_heads;
/* Rotate the heads of n_sets (1 or 2, for example q and k; HOST array) sets of heads of
 * the same rows. positions: int32 [streams][rows], any value (negative ones rotate back). turns: device table.
 * dtype F32 or BF16 for all. Errors: EINVAL (null pointers, sizes below 0, head_dim not in 2..512,
 * rotary_dim odd or above head_dim, more than 16384 heads in a set, streams * rows above 2^30, several
 * heads written at a stride of 0), ECUDA. */
talker_status talker_rotate(const uint64_t *turns, float amplitude, int head_dim, int rotary_dim, int interleaved,
                            const int32_t *positions, int streams, int rows, const talker_heads *sets, int n_sets,
                            int dtype, void *cuda_stream);

/* Products with 4-bit weights. A matrix W of n outputs and k inputs is cut into groups of
 * `group` consecutive inputs (32, 64 or 128; the last one shorter where k is no multiple),
 * each with a scale d (fp16) and, with zeros, a whole number z in 0..15 (8 without): the code
 * c in 0..15 stands for (c - z) d. A gated matrix is two of the same sizes, W and U, for
 * silu(W x) * (U x).
 *
 * Exchange format (what quantizers write): codes uint8 [n][ceil(k / 2)], input 2 i in the low
 * four bits of byte i and input 2 i + 1 in the high ones; scales fp16 [n][ceil(k / group)];
 * zeros uint8 of the same shape, or NULL. talker_w4_pack lays them out as the kernels read
 * them, in `tiles`: 16 rows to a tile (rows past n are zeros; of a gated matrix 8 rows of W,
 * then the same 8 of U), inputs padded to a multiple of 128. For each tile and 128 inputs one
 * record, in the order of spans of 32 tiles (the last may have fewer), in a span of inputs,
 * then of tiles. In a record twice 512 bytes for 64 inputs: 16 of lane l = 4 g + t, words
 * j = 0..3, whose 4-bit fields 0..7 are, with i = 16 j + 4 t: inputs i and i + 1 of row g in
 * fields 0 and 4, i + 2 and i + 3 in fields 1 and 5, and the same of row g + 8 in fields 2, 6,
 * 3, 7 (the operand's registers of a tensor-core product, one mask away). Then for each group
 * 8 pairs of scales of rows (g, g + 8), and, with zeros, for each group 8 pairs of bytes; a
 * record is padded to 32 bytes. */
typedef struct {
    void *tiles; /* talker_w4_bytes bytes, 16-byte aligned */
    int32_t n, k, group;
    int32_t zeros, gated; /* 0 or 1 */
} talker_w4;
/* Bytes of the tiles (`tiles` is not looked at); 0 for sizes that are not supported: n in
 * 1..2^27, k in 1..2^20. */
size_t talker_w4_bytes(const talker_w4 *w);
/* Lay out a matrix; codes2, scales2 and zeros2 are U's of a gated one (else not looked at).
 * Bits of zeros above the low four are not looked at. Errors: EINVAL, ECUDA. */
talker_status talker_w4_pack(const talker_w4 *w, const uint8_t *codes, const void *scales, const uint8_t *zeros,
                             const uint8_t *codes2, const void *scales2, const uint8_t *zeros2, void *cuda_stream);
/* Quantize a dense matrix, n rows of k values (F32 or BF16, row_stride elements apart), to the
 * exchange format without zeros, by the rule of the 4-bit cache (talker_kv4.h) over groups: m
 * the group's value of largest magnitude (the first on ties), clamped to +-524032; d =
 * fp16(-m / 8); code = clamp(floor(8.5 - 8 x / m), 0, 15), decided exactly, 8 where m = 0. A
 * group with a NaN or an infinity gets codes 8 and d = NaN. Errors: EINVAL, ECUDA. */
talker_status talker_w4_quantize(const void *w, int dtype, int64_t row_stride, int n, int k, int group, uint8_t *codes,
                                 void *scales, void *cuda_stream);
/* out[r] = W x[r] for r < rows, or silu(W x[r]) * (U x[r]) of a gated matrix, plus residual[r]
 * where it is given; silu(g) = g / (1 + exp(-g)).
 * x: rows of k values, x_row elements apart, F32, BF16, or E4M3 with x_scales f32
 * [rows][ceil(k / x_block)] (x_block 32, 64 or 128; 0: a scale a row), as talker_rms_norm
 * writes them. out: rows of n values, out_row apart, F32 or BF16; residual likewise, res_row
 * apart, in out's type; it may be out itself (same stride). Other overlaps are not allowed.
 * Products of codes and x are made by the tensor cores with f32 sums: bf16 x enters exactly
 * (values below 2^-31 of a row's largest lose bits), others with 22 bits in two parts (values
 * below 2^-16 of a row's largest with fewer, down to 2^-39 of it). The order
 * of a sum depends on n, k, rows and types alone. A row of x with a NaN or an infinity gives
 * NaN. (So would a copy of weights that does not arrive within a second, from there on.)
 * Made for few rows: 32 columns of x, one a bf16 row and two any other, in one pass over the
 * weights; more are taken in several, at most 2^16 rows.
 * scratch: talker_w4_scratch bytes, 16-byte aligned, for the same sizes and types; it need not
 * hold anything on entry, and calls that may run at the same time need their own.
 * Errors: EINVAL, ECUDA. */
size_t talker_w4_scratch(const talker_w4 *w, int x_dtype, int rows);
talker_status talker_w4_matmul(const talker_w4 *w, const void *x, int x_dtype, int64_t x_row, const float *x_scales,
                               int x_block, int rows, const void *residual, int64_t res_row, void *out, int out_dtype,
                               int64_t out_row, void *scratch, size_t scratch_bytes, void *cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* TALKER_LAYER_H */
