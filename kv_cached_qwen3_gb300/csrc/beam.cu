// Beam selection (talker_beam_select): per sequence the best `width` of width * vocab continuations.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "talker_kv4.h"

using namespace talker_dev;

namespace {

constexpr int kThreads = 256;
constexpr int kMaxWidth = 32;
constexpr float kMasked = -1e30f;   // at or below: counts as -inf

// Masked values as -inf, and -0 as 0 (equal values are ordered by their index).
__device__ __forceinline__ float unmask(float x) { return x > kMasked ? x + 0.f : -INFINITY; }

// Order of (value, index): the larger value first, then the lower index.
__device__ __forceinline__ unsigned long long key_of(float x, unsigned i) {
    const uint32_t u = __float_as_uint(x);
    return (unsigned long long)(u & 0x80000000u ? ~u : u | 0x80000000u) << 32 | (0xffffffffu - i);
}
__device__ __forceinline__ float key_value(unsigned long long k) {
    const uint32_t u = (uint32_t)(k >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ unsigned key_index(unsigned long long k) { return 0xffffffffu - (uint32_t)k; }

__device__ __forceinline__ unsigned long long warp_max_key(unsigned long long k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long t = __shfl_xor_sync(0xffffffffu, k, o);
        k = t > k ? t : k;
    }
    return k;
}

struct Args {
    const void *logits;
    int64_t row_stride;
    const float *scores;
    const int32_t *ended;
    int width, vocab, eos;
    int32_t *tokens, *parents, *ended_out;
    float *scores_out;
    // scratch per row: width keys (best first), the maximum and the sum of exp(x - maximum)
    unsigned long long *keys;
    float2 *sums;
};

// One CTA per row: the row's maximum and sum, then its `width` best logits one after another.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_beam_rows(const Args a) {
    __shared__ float red[kThreads / 32];
    __shared__ unsigned long long best[kThreads / 32];
    const int row = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const T *x = static_cast<const T *>(a.logits) + row * a.row_stride;
    float m = -INFINITY;
    for (int v = threadIdx.x; v < a.vocab; v += kThreads) m = fmaxf(m, unmask((float)x[v]));
    m = warp_max(m);
    if (lane == 0) red[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, red[w]);
    __syncthreads();
    float sum = 0.f;
    for (int v = threadIdx.x; v < a.vocab; v += kThreads) {
        const float t = unmask((float)x[v]);
        sum += t == -INFINITY ? 0.f : expf(t - m);
    }
    sum = warp_sum(sum);
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        sum = 0.f;
        for (int w = 0; w < kThreads / 32; ++w) sum += red[w];
        a.sums[row] = make_float2(m, sum);
    }
    unsigned long long last = ~0ull;
    for (int j = 0; j < a.width; ++j) {
        unsigned long long k = 0;
        for (int v = threadIdx.x; v < a.vocab; v += kThreads) {
            const unsigned long long t = key_of(unmask((float)x[v]), v);
            if (t < last && t > k) k = t;
        }
        k = warp_max_key(k);
        if (lane == 0) best[warp] = k;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) k = best[w] > k ? best[w] : k;
        __syncthreads();
        if (threadIdx.x == 0) a.keys[(size_t)row * a.width + j] = k;
        last = k;
    }
}

// One warp per sequence: lane w walks beam w's best logits, and the best of the lanes' heads is
// chosen `width` times. Candidates are compared in 64 bits.
__global__ void __launch_bounds__(32) k_beam_merge(const Args a) {
    const int seq = blockIdx.x, lane = threadIdx.x, row = seq * a.width + lane;
    const bool on = lane < a.width;
    float score = -INFINITY;
    bool old = false, dead = true;
    double base = 0.0;
    if (on) {
        score = unmask(a.scores[row]);
        old = a.ended != nullptr && a.ended[row] != 0;
        const float2 ms = a.sums[row];
        // no candidate above -inf: a masked score, or a row without a finite maximum
        dead = score == -INFINITY || score == INFINITY || (!old && !(fabsf(ms.x) < INFINITY));
        if (!dead && !old) base = (double)ms.x + log((double)ms.y);
    }
    int at = 0;   // of this beam's candidates, in order
    for (int j = 0; j < a.width; ++j) {
        double c = -INFINITY;
        int v = 0x7fffffff;
        if (on && at < a.width) {
            if (dead) {
                v = at;
            } else if (old) {   // eos, then the others in order
                v = at == 0 ? a.eos : at - 1 + (at - 1 >= a.eos);
                if (at == 0) c = score;
            } else {
                const unsigned long long k = a.keys[(size_t)row * a.width + at];
                v = (int)key_index(k);
                c = (double)key_value(k) - base + (double)score;
            }
        }
        double bc = c;
        int bw = lane;
        bool bon = v != 0x7fffffff;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double tc = __shfl_xor_sync(0xffffffffu, bc, o);
            const int tw = __shfl_xor_sync(0xffffffffu, bw, o);
            const bool ton = __shfl_xor_sync(0xffffffffu, (int)bon, o) != 0;
            if (ton && (!bon || tc > bc || (tc == bc && tw < bw))) bc = tc, bw = tw, bon = true;
        }
        if (bw == lane) {
            const int out = seq * a.width + j;
            a.tokens[out] = v;
            a.parents[out] = row;
            a.scores_out[out] = (float)c;
            if (a.ended_out != nullptr) a.ended_out[out] = old || v == a.eos;
            ++at;
        }
    }
}

size_t align16(size_t n) { return (n + 15) / 16 * 16; }

bool sizes_ok(int n_seq, int width, int vocab) {
    return n_seq >= 0 && width >= 1 && width <= kMaxWidth && vocab >= width && (long long)n_seq * width <= 0x7fffffffll;
}

}  // namespace

extern "C" {

size_t talker_beam_scratch(int n_seq, int width, int vocab) {
    if (!sizes_ok(n_seq, width, vocab)) return 0;
    const size_t rows = (size_t)n_seq * width;
    return align16(rows * width * sizeof(unsigned long long)) + rows * sizeof(float2);
}

talker_status talker_beam_select(const void *logits, int64_t row_stride, int dtype, const float *scores,
                                 const int32_t *ended, int n_seq, int width, int vocab, int eos_id, int32_t *tokens,
                                 int32_t *parents, float *scores_out, int32_t *ended_out, void *scratch,
                                 size_t scratch_bytes, void *cuda_stream) {
    if (!sizes_ok(n_seq, width, vocab) || !logits || !scores || !tokens || !parents || !scores_out) return TALKER_EINVAL;
    if (dtype != TALKER_DTYPE_F32 && dtype != TALKER_DTYPE_BF16) return TALKER_EINVAL;
    if (row_stride < vocab || reinterpret_cast<uintptr_t>(logits) % (dtype == TALKER_DTYPE_F32 ? 4 : 2)) return TALKER_EINVAL;
    if (eos_id >= vocab || (ended && eos_id < 0)) return TALKER_EINVAL;
    if (scores_out == scores || (ended_out && ended_out == ended)) return TALKER_EINVAL;
    if (n_seq == 0) return TALKER_OK;
    if (!scratch || scratch_bytes < talker_beam_scratch(n_seq, width, vocab) || (reinterpret_cast<uintptr_t>(scratch) & 15u))
        return TALKER_EINVAL;
    const int rows = n_seq * width;
    Args a{logits, row_stride, scores, ended, width, vocab, eos_id, tokens, parents, ended_out, scores_out};
    a.keys = static_cast<unsigned long long *>(scratch);
    a.sums = reinterpret_cast<float2 *>(static_cast<char *>(scratch) + align16((size_t)rows * width * sizeof(unsigned long long)));
    cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
    if (dtype == TALKER_DTYPE_F32) k_beam_rows<float><<<rows, kThreads, 0, s>>>(a);
    else k_beam_rows<__nv_bfloat16><<<rows, kThreads, 0, s>>>(a);
    k_beam_merge<<<n_seq, 32, 0, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return TALKER_ECUDA;
    return TALKER_OK;
}

}  // extern "C"
