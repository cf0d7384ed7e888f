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

// Quantizes one block of 32 values. The four lanes of an aligned group hold dims 8 c .. 8 c + 7
// of the block, c = lane & 3; every lane of the warp has to take part. Returns the lane's eight
// codes (dim i in bits 4 i ..) and the block's scale bits.
//
// code = clamp(floor(8.5 - 8 x / m), 0, 15) has to be exact (a neighbouring code is off by a
// whole step): with y = -x sign(m), M = |m| the code is at least k iff 16 y >= (2 k - 17) M.
// fp32 finds the nearest such border k, and the sign of one fma, which rounds 16 y - (2 k - 17) M
// only once, says on which side y lies. Blocks with tiny M are scaled by 2^60 first (exact), so
// that neither 8 / M nor the sign can be lost.
__device__ __forceinline__ uint32_t q4_codes8(const float (&x)[8], unsigned short &d_bits) {
    float m = x[0];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        bad |= !(fabsf(x[i]) <= 3.402823466e38f);
        if (fabsf(x[i]) > fabsf(m)) m = x[i];
    }
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, m, o);
        if (fabsf(other) > fabsf(m) || (fabsf(other) == fabsf(m) && (lane & o))) m = other;
        bad |= __shfl_xor_sync(0xffffffffu, (int)bad, o) != 0;
    }
    m = fminf(fmaxf(m, -524032.f), 524032.f);
    d_bits = bad ? 0x7e00 : __half_as_ushort(__float2half_rn(m * -0.125f));
    const float up = fabsf(m) < 1e-30f ? 1152921504606846976.f : 1.f;   // 2^60
    const float M = fabsf(m) * up;
    if (bad || M == 0.f) return 0x88888888u;
    const float s = m > 0.f ? -up : up, id = 8.f / M;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float y = x[i] * s;
        const float k = rintf(fminf(fmaxf(fmaf(y, id, 8.5f), 0.f), 17.f));
        const float side = fmaf(fmaf(-2.f, k, 17.f), M, 16.f * y);
        const int n = (int)k - (side < 0.f ? 1 : 0);
        w |= (uint32_t)min(max(n, 0), 15) << (4 * i);
    }
    return w;
}

// The eight codes of dims 8 c .. 8 c + 7 of block b of a row, in the order of the K and V rows
// (the K row keeps them in one word, the V row in two halves).
template <int NB>
__device__ __forceinline__ void q4_store_codes(unsigned char *row, bool is_v, int b, int c, uint32_t w) {
    if (!is_v) {
        *reinterpret_cast<uint32_t *>(row + c * 4 * NB + 4 * b) = w;
    } else {
        *reinterpret_cast<uint16_t *>(row + (2 * c) * 2 * NB + 2 * b) = (uint16_t)w;
        *reinterpret_cast<uint16_t *>(row + (2 * c + 1) * 2 * NB + 2 * b) = (uint16_t)(w >> 16);
    }
}
template <int NB>
__device__ __forceinline__ uint32_t q4_load_codes(const unsigned char *row, bool is_v, int b, int c) {
    if (!is_v) return *reinterpret_cast<const uint32_t *>(row + c * 4 * NB + 4 * b);
    return (uint32_t)*reinterpret_cast<const uint16_t *>(row + (2 * c) * 2 * NB + 2 * b) |
           (uint32_t)*reinterpret_cast<const uint16_t *>(row + (2 * c + 1) * 2 * NB + 2 * b) << 16;
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
    int grid, one_unit;   // Kv4AttendShape
    float *scratch;
};
// CTAs of a launch, and whether each (stream, KV head) row is one CTA's work (no scratch then).
struct Kv4AttendShape {
    int grid, one_unit;
};
Kv4AttendShape kv4_attend_shape(int B, int n_kv, int max_len, int n_sm);
size_t kv4_attend_scratch(const Kv4AttendShape &p, int head_dim);
cudaError_t prepare_kv4_attend();   // shared-memory limits, on the current device
int kv4_multiprocessors();          // of the current device, prepared as above (0: an error)
cudaError_t launch_kv4_attend(const Kv4Attend &a, int in_bf16, int out_bf16, cudaStream_t s);

// Streams reordered by sharing pages (talker_kv4_reorder), for any page layout of n_tiles tiles a
// pool page, each of 64 code rows of row_bytes and, behind them, 64 rows of scale_bytes.
struct KvReorder {
    unsigned char *k, *v;
    size_t page_bytes;
    int n_tiles, row_bytes, scale_bytes, tile_bytes;
    const int32_t *table, *lens, *parents;
    int32_t *table_out, *lens_out, *status;
    int n_streams, pps, R;
};
constexpr int kReorderMaxStreams = 1024;
cudaError_t launch_kv_reorder(const KvReorder &r, cudaStream_t s);

}  // namespace talker_k
