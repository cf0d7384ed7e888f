// The 4-bit paged cache (Q4_0 blocks, include/talker_kv4.h): tile layout, quantizer and the host
// launchers that the C-ABI entry points and the talker runtime share.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.cuh"
#include "talker_kv4.h"

namespace talker_k {

// Tile of one (page, layer, KV head): 64 code rows, then 64 scale rows.
template <int HD>
struct Kv4Tile {
    static constexpr int NB = HD / 32;                    // blocks of 32 dims per row
    static constexpr int kRow = HD / 2;                   // code bytes per row
    static constexpr int kScales = talker_dev::kPage * kRow;   // byte offset of the scales
    static constexpr int kBytes = kScales + talker_dev::kPage * NB * 2;
};
constexpr int kv4_tile_bytes(int hd) { return hd * 36; }
constexpr int kPage4 = talker_dev::kPage;

// Two f32 values in one 64-bit register, each instruction computing both.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float f2_lo(F2 x) { return __uint_as_float((uint32_t)x.v); }
__device__ __forceinline__ float f2_hi(F2 x) { return __uint_as_float((uint32_t)(x.v >> 32)); }
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// The largest and the smallest of three, NaN if one is NaN.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ float min3_nan(float a, float b, float c) {
    float y;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// Quantizes one block of 32 values. The four lanes of an aligned group hold dims 8 c .. 8 c + 7
// of the block, c = lane & 3; every lane of the warp has to take part. Returns the lane's eight
// codes (dim i in bits 4 i ..) and the block's scale bits.
//
// code = clamp(floor(8.5 - 8 x / m), 0, 15) has to be exact (a neighbouring code is off by a
// whole step, and values exactly between two codes are common in bf16). The whole number k nearest to
// 8.5 - 8 x / m comes from fp32, off by less than 4e-6; the code is k, or k - 1 where
// (17 - 2 k) |m| < 16 x sign(m): the sign of one fma, which rounds that difference only once. Blocks
// with tiny |m| are scaled by 2^60 first (exact), so that neither 8 / m nor the sign can be lost.
//
// BF16: the values are bf16 numbers. A difference 16 x - (17 - 2 k) m other than 0 is then at least
// half the last place of m where it matters (|x| >= |m| / 32), or 2^8 where m is clamped: 8.5 - 8 x / m is
// a whole number or more than 2^-12 away from one, and fp32 plus 2^-13 decides, without that fma.
template <bool BF16>
__device__ __forceinline__ uint32_t q4_codes8(const float (&x)[8], unsigned short &d_bits) {
    const int lane = threadIdx.x & 31;
    float hi = max3_nan(x[0], x[1], x[2]), lo = min3_nan(x[0], x[1], x[2]);
    hi = max3_nan(hi, x[3], x[4]), lo = min3_nan(lo, x[3], x[4]);
    hi = max3_nan(hi, x[5], x[6]), lo = min3_nan(lo, x[5], x[6]);
    hi = max3_nan(hi, x[7], __shfl_xor_sync(0xffffffffu, max3_nan(hi, x[7], x[7]), 1));
    lo = min3_nan(lo, x[7], __shfl_xor_sync(0xffffffffu, min3_nan(lo, x[7], x[7]), 1));
    const float hi2 = __shfl_xor_sync(0xffffffffu, hi, 2), lo2 = __shfl_xor_sync(0xffffffffu, lo, 2);
    hi = max3_nan(hi, hi2, hi2), lo = min3_nan(lo, lo2, lo2);
    const bool bad = !(hi < INFINITY && lo > -INFINITY);
    float m = hi > -lo ? hi : lo;
    if (__any_sync(0xffffffffu, hi == -lo)) {   // both signs: the first one's
        float first = 0.f;
#pragma unroll
        for (int i = 7; i >= 0; --i)
            if (fabsf(x[i]) == hi) first = x[i];
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            const float other = __shfl_xor_sync(0xffffffffu, first, o), a = lane & o ? other : first, b = lane & o ? first : other;
            first = a != 0.f ? a : b;
        }
        const float x0 = __shfl_sync(0xffffffffu, x[0], lane & ~3);   // (of zeros)
        if (hi == -lo) m = hi > 0.f ? first : x0;
    }
    float y[8], up = 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i];
    if (fabsf(m) > 524032.f || fabsf(m) < 1e-30f) {
        m = fminf(fmaxf(m, -524032.f), 524032.f);
        up = fabsf(m) < 1.f ? 1152921504606846976.f : 1.f;   // 2^60
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fminf(fmaxf(y[i], -524032.f), 524032.f) * up;
    }
    const bool none = bad || m == 0.f;
    d_bits = bad ? 0x7e00 : __half_as_ushort(__float2half_rn(m * -0.125f));
    m *= up;
    float inv;   // 1 / |m|, to 2^-23
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(fabsf(m)));
    constexpr float kRound = 12582912.f;   // 1.5 2^23: x + kRound holds the nearest whole number to x
    uint32_t w = 0;                        // modulo 2^32 the eight bit patterns of kRound add up to a constant
    if (BF16) {   // 8 - 8 x / m + 2^-13 in units of kTop, which rounds to 15
        constexpr float kTop = 15.4375f;
        const float s = copysignf(inv * (8.f / kTop), -m);
#pragma unroll
        for (int i = 6; i >= 0; i -= 2) {
            const F2 u = f2(__saturatef(fmaf(y[i], s, (8.f + 0x1p-13f) / kTop)), __saturatef(fmaf(y[i + 1], s, (8.f + 0x1p-13f) / kTop)));
            const F2 r = fma2(u, f2(kTop, kTop), f2(kRound, kRound));
            w = w * 256 + (__float_as_uint(f2_hi(r)) * 16 + __float_as_uint(f2_lo(r)));
        }
    } else {
        const float M = fabsf(m), s = copysignf(16.f, -m), id = 0.5f * inv;
        const int top = __float_as_int(kRound) + 15;
#pragma unroll
        for (int i = 6; i >= 0; i -= 2) {
            const F2 z = f2(y[i], y[i + 1]) * f2(s, s), r = fma2(z, f2(id, id), f2(8.5f, 8.5f)) + f2(kRound, kRound);
            const F2 side = fma2(fma2(f2(-2.f, -2.f), r + f2(-kRound, -kRound), f2(17.f, 17.f)), f2(M, M), z);
            const int n1 = __float_as_int(f2_hi(r)) + (__float_as_int(f2_hi(side)) >> 31);
            const int n0 = __float_as_int(f2_lo(r)) + (__float_as_int(f2_lo(side)) >> 31);
            w = w * 256 + ((uint32_t)min(n1, top) * 16 + (uint32_t)min(n0, top));
        }
    }
    return none ? 0x88888888u : w - 0x4b400000u * 0x11111111u;
}

// The code of x in a block with M = |m| > 0, s = -16 sign(m), both times 2^60 if m is tiny, id = 0.5 / M.
__device__ __forceinline__ int q4_code(float x, float M, float s, float id) {
    constexpr float kRound = 12582912.f;
    const float z = x * s, k = (fmaf(z, id, 8.5f) + kRound) - kRound;
    return min((int)k - (fmaf(fmaf(-2.f, k, 17.f), M, z) < 0.f ? 1 : 0), 15);
}

// Quantizes and stores block b of row `row` of a tile, held one dim per lane of a warp.
__device__ __forceinline__ void q4_store_block(unsigned char *tile, int hd, int row, bool is_v, int b, float x, int lane) {
    const int nb = hd / 32;
    const uint32_t bits = __float_as_uint(x) & 0x7fffffffu, top = __reduce_max_sync(0xffffffffu, bits);
    const bool bad = top >= 0x7f800000u;
    float m = __shfl_sync(0xffffffffu, x, __ffs(__ballot_sync(0xffffffffu, bits == top)) - 1);
    m = fminf(fmaxf(m, -524032.f), 524032.f);
    int n = 8;
    if (!bad && m != 0.f) {
        const float up = fabsf(m) < 1e-30f ? 1152921504606846976.f : 1.f, M = fabsf(m) * up;   // 2^60
        n = q4_code(fminf(fmaxf(x, -524032.f), 524032.f), M, m > 0.f ? -16.f * up : 16.f * up, 0.5f / M);
    }
    const int pair = n | __shfl_down_sync(0xffffffffu, n, 1) << 4;
    if (lane % 2 == 0)   // dims lane and lane + 1 of the block
        tile[row * (hd / 2) + (is_v ? lane / 4 * 2 * nb + 2 * b + lane % 4 / 2 : lane / 8 * 4 * nb + 4 * b + lane % 8 / 2)] =
            (unsigned char)pair;
    if (lane == 0)
        *reinterpret_cast<unsigned short *>(tile + kPage4 * (hd / 2) + (row * nb + b) * 2) =
            bad ? 0x7e00 : __half_as_ushort(__float2half_rn(m * -0.125f));
}

// The 32-bit word of a row that lane (b, c), four lanes to a block, writes or reads. K: its own
// eight codes. V: the codes of two neighbouring blocks for group g = 2 c + b % 2, which lanes b and
// b ^ 1 (lane ^ 4) exchange: v_word turns a lane's codes into its word, and back.
template <int NB>
__device__ __forceinline__ int q4_word_at(bool is_v, int b, int c) {
    return is_v ? (2 * c + (b & 1)) * 2 * NB + 2 * (b & ~1) : c * 4 * NB + 4 * b;
}
__device__ __forceinline__ uint32_t v_word(uint32_t w, int b) {
    const uint32_t other = __shfl_xor_sync(0xffffffffu, w, 4);
    return b & 1 ? __byte_perm(other, w, 0x7632) : __byte_perm(w, other, 0x5410);
}
// The eight values of a lane's codes.
__device__ __forceinline__ void q4_values8(uint32_t w, float d, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)   // the code goes under the exponent of 2^23
        x[i] = (__int_as_float((int)((w >> (4 * i) & 15u) | 0x4b000000u)) - 8388616.f) * d;
}

// Rows of a call to the cache (or back), see talker_kv4_write.
struct Kv4Rows {
    talker_kv4 c;
    int layer0, n_layers, stream0, n_streams;
    const int32_t *start, *count;
    int T;
    void *k, *v;
    talker_kv4_strides st;
};
bool kv4_cache_ok(const talker_kv4 *c);   // the host-side checks of a caller-owned cache
cudaError_t launch_kv4_rows(const Kv4Rows &r, int dtype, bool read, cudaStream_t s);

// Decode attention over the 4-bit cache, see talker_kv4_attend.
struct Kv4Attend {
    talker_kv4 c;
    int layer, B, n_q;
    const int32_t *lens;
    const void *q, *k_new, *v_new;
    int64_t q_row, new_row;
    void *out;
    float scale;
    int grid, one_unit, ctas;   // Kv4AttendShape
    float *scratch;
};
// CTAs of a launch, and whether each (stream, KV head) row is one CTA's work (no scratch then).
struct Kv4AttendShape {
    int grid, one_unit;
    int ctas;        // CTAs that a multiprocessor holds
    int full_grid;   // the grid of any more work than this
};
Kv4AttendShape kv4_attend_shape(int B, int n_kv, int hd, int max_len, int n_sm);
size_t kv4_attend_scratch(const Kv4AttendShape &p, int head_dim);
size_t kv4_attend_scratch(int grid, int head_dim);
cudaError_t prepare_kv4_attend();   // shared-memory limits, on the current device
int kv4_multiprocessors();          // of the current device, prepared as above (0: an error)
// pdl: starts while the kernel before it drains, which must not write lengths, page numbers or rows below
// the lengths.
cudaError_t launch_kv4_attend(const Kv4Attend &a, int in_bf16, int out_bf16, bool pdl, cudaStream_t s);

// Streams reordered by sharing pages (talker_kv4_reorder), for any page layout of n_tiles tiles a
// pool page, each of 64 code rows of row_bytes and, behind them, 64 rows of scale_bytes.
struct KvReorder {
    unsigned char *k, *v;
    size_t page_bytes;
    int n_tiles, row_bytes, scale_bytes, tile_bytes;
    const int32_t *table, *lens, *parents;
    int32_t *table_out, *lens_out, *status;
    int n_streams, pps, R;
    int group;    // > 0: a parent lies in its stream's group of this many consecutive streams
};
constexpr int kReorderMaxStreams = 1024;
cudaError_t launch_kv_reorder(const KvReorder &r, cudaStream_t s);

}  // namespace talker_k
