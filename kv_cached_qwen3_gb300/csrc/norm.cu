// Residual addition and RMSNorm of rows, with results in f32, bf16 or e4m3 blocks (include/talker_layer.h).
#include <cuda_fp8.h>

#include <algorithm>

#include "rows.cuh"
#include "talker_layer.h"

using namespace talker_dev;

namespace {

struct Place {
    long long outer, inner;
};
struct NormArgs {
    const void *x, *res;
    const float *gain;
    void *sum, *y;
    float *scales;
    Place x_at, res_at, sum_at, y_at;
    float eps;
    int rows, inner, width;
    int block, block_shift, blocks;   // in values (0: a row), its log2, blocks of a row
    float inv_width;
    bool vec;   // eight neighbouring values by one access, in all tensors
};

__device__ __forceinline__ long long at(const Place &p, int outer, int inner) {
    return inner < 0 ? outer * p.outer : outer * p.outer + inner * p.inner;
}

// A thread's eight values of a chunk: neighbours from `at` on, or, where rows do not lie on whole accesses, every 32nd (a
// warp has the same 256 either way, and reads them in whole sectors).
template <typename T>
__device__ __forceinline__ void load_row8(const T *p, int at, int width, bool vec, float (&v)[8]) {
    if (vec && at + 8 <= width) {
        load8(p + at, true, v);
    } else {
        const int step = vec ? 1 : 32;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = at + j * step < width ? Elem<T>::load(p, at + j * step) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void store_row8(T *p, int at, int width, bool vec, const float (&v)[8]) {
    if (vec && at + 8 <= width) {
        store8(p + at, true, v);
    } else {
        const int step = vec ? 1 : 32;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (at + j * step < width) Elem<T>::store(p, at + j * step, v[j]);
    }
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
           (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3) << 16;
}
__device__ __forceinline__ float max_abs8(const float (&v)[8]) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));   // (a NaN shows in the norm's factor)
    return m;
}

// A row's sum or maximum over its blockDim.x threads, in every one of them. All threads of the CTA take part.
template <bool MAX>
__device__ __forceinline__ float row_all(float v, float *red) {
    if (MAX) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    } else {
        v = warp_sum(v);
    }
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float w = lane < warps ? red[lane] : 0.f;
    if (MAX) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, o));
        return w;
    }
    return warp_sum(w);
}

// 1 / sqrt(x): the hardware's (2^-23 off) and a step of Newton's method; of 0 and infinity as it is.
__device__ __forceinline__ float root(float x) {
    float r;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    const float better = fmaf(r * 0.5f, fmaf(-x * r, r, 1.f), r);
    return r > 0.f && r < INFINITY ? better : r;
}

// Eight values of a row as they lie in memory, so that nothing waits for them until they are used.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
    float v[8];
    __device__ __forceinline__ void load(const float *p, int i, int width, bool vec) { load_row8(p, i, width, vec, v); }
    __device__ __forceinline__ float at(int j) const { return v[j]; }
};
template <>
struct Raw<__nv_bfloat16> {
    uint32_t w[4];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, int i, int width, bool vec) {
        if (vec && i + 8 <= width) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p + i);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else {
            const unsigned short *q = reinterpret_cast<const unsigned short *>(p);
            const int step = vec ? 1 : 32;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = (i + 2 * j * step < width ? q[i + 2 * j * step] : 0u) |
                       (i + (2 * j + 1) * step < width ? (uint32_t)q[i + (2 * j + 1) * step] : 0u) << 16;
        }
    }
    __device__ __forceinline__ float at(int j) const { return j & 1 ? bf16hi(w[j / 2]) : bf16lo(w[j / 2]); }
};

// blockDim.x threads a row, blockDim.y rows at a time; a thread has eight consecutive values of every chunk of 8 *
// blockDim.x. C chunks stay in registers between the sum and the result, and the next rows' are on their way meanwhile; with
// C = 0 (rows of more than 16384 values) they are read again. For E4M3 the norm's factor cancels: a code is that of s gain
// over the largest of its block.
// Threads of a CTA at most. Few threads with several chunks each: what a thread does for a row once is shared by more
// values, and more CTAs are out of step with one another (4096 x 5120: one chunk of 640 threads 57 us, two of 320 54, four of
// 160 42).
constexpr int most_threads(int c) { return c == 0 ? 1024 : c == 4 ? 512 : 128; }
template <typename TX, typename TR, typename TY, int C>
__global__ void __launch_bounds__(most_threads(C), 1) k_rms_norm(const NormArgs a) {
    constexpr bool kRes = !std::is_same<TR, void>::value, k8 = std::is_same<TY, __nv_fp8_storage_t>::value;
    constexpr int H = C > 0 ? C : 1;   // chunks in registers
    constexpr bool kAhead = C == 4;    // (65536 rows of 128: 29 us without, 39 with)
    using R = typename std::conditional<kRes, TR, float>::type;
    using Y = typename std::conditional<k8, float, TY>::type;
    __shared__ float sums[2][32], tops[2][32];   // of a row's warps; of every other turn, so that one wait a turn is enough
    const int lane = threadIdx.x & 31, step = 8 * blockDim.x, per = blockDim.y * gridDim.x;
    const int first = a.vec ? 8 * threadIdx.x : 8 * (threadIdx.x - lane) + lane;
    const int chunks = C > 0 ? C : (a.width + step - 1) / step, warps = blockDim.x >> 5;
    struct Row {
        int outer, inner, width;   // inner -1: rows at one stride; width 0: none
    };
    auto row_of = [&](int row) -> Row {
        if (row >= a.rows) return {0, -1, 0};
        if (a.inner == 1) return {row, -1, a.width};
        const int outer = (unsigned)row / (unsigned)a.inner;
        return {outer, row - outer * a.inner, a.width};
    };
    Raw<TX> x[H];
    Raw<R> r[H];
    auto fetch = [&](const Row &w, int c, Raw<TX> &x, Raw<R> &r) {
        const int i = c * step + first;
        x.load(static_cast<const TX *>(a.x) + at(a.x_at, w.outer, w.inner), i, w.width, a.vec);
        if (kRes) r.load(static_cast<const R *>(a.res) + at(a.res_at, w.outer, w.inner), i, w.width, a.vec);
    };
    auto sum_of = [&](const Raw<TX> &x, const Raw<R> &r, float (&v)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = kRes ? x.at(j) + r.at(j) : x.at(j);
    };
    int row = blockIdx.x * blockDim.y + threadIdx.y;
    Row now = row_of(row);
    if (kAhead) {
#pragma unroll
        for (int c = 0; c < H; ++c) fetch(now, c, x[c], r[c]);
    }
    for (int turn = 0; row - (int)threadIdx.y < a.rows; row += per, turn ^= 1) {   // (all of a CTA's threads together)
        float *const red = sums[turn] + threadIdx.y * warps, *const top = tops[turn] + threadIdx.y * warps;
        float held[H][8];
        float sum = 0.f;
        auto add = [&](const float (&v)[8]) {
            float t = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) t = fmaf(v[j], v[j], t);
            sum += t;
        };
        const Row next = row_of(row + per < a.rows ? row + per : a.rows);
        if (C > 0) {
            if (!kAhead) fetch(now, 0, x[0], r[0]);
#pragma unroll
            for (int c = 0; c < H; ++c) sum_of(x[c], r[c], held[c]);
            if (kAhead) {
#pragma unroll
                for (int c = 0; c < H; ++c) fetch(next, c, x[c], r[c]);
            }
#pragma unroll
            for (int c = 0; c < H; ++c) add(held[c]);
        } else {
            for (int c = 0; c < chunks; ++c) {
                fetch(now, c, x[0], r[0]);
                sum_of(x[0], r[0], held[0]);
                add(held[0]);
            }
        }
        const float scale = root(fmaf(row_all<false>(sum, red), a.inv_width, a.eps));
        auto take = [&](int c, float (&v)[8], float (&g)[8]) {   // s and s gain
            if (C == 0) {
                fetch(now, c, x[0], r[0]);
                sum_of(x[0], r[0], v);
            }
            load_row8(a.gain, c * step + first, a.width, a.vec, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] *= v[j];
        };
        float most = 0.f;   // of the row
        if (k8 && a.block == 0) {
#pragma unroll(C > 0 ? C : 1)
            for (int c = 0; c < chunks; ++c) {
                float g[8];
                take(c, held[C > 0 ? c : 0], g);
                most = fmaxf(most, max_abs8(g));
            }
            most = row_all<true>(most, top);
        }
#pragma unroll(C > 0 ? C : 1)
        for (int c = 0; c < chunks; ++c) {
            float(&v)[8] = held[C > 0 ? c : 0];
            float g[8];
            take(c, v, g);
            const int i = c * step + first;
            if (kRes && a.sum != nullptr) store_row8(static_cast<R *>(a.sum) + at(a.sum_at, now.outer, now.inner), i, now.width, a.vec, v);
            if (k8) {
                uint8_t *out = static_cast<uint8_t *>(a.y) + at(a.y_at, now.outer, now.inner);
                // the factor of codes in a block with max|s gain| m, whose scale the thread that is told to writes
                auto factor = [&](float m, bool writes, int i) -> float {
                    const float d = m * scale;   // max|y|
                    const bool none = d < 0x1p-100f || m < 0x1p-100f;
                    float inv;
                    asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(m));
                    if (writes && i < now.width) a.scales[(size_t)row * a.blocks + (a.block == 0 ? 0 : i >> a.block_shift)] = none ? 0.f : d * (1.f / 448.f);
                    return none ? 0.f : d < INFINITY ? 448.f * inv : NAN;
                };
                if (a.vec) {
                    float m = most;
                    if (a.block != 0) {   // its threads are neighbours in a warp
                        m = max_abs8(g);
                        for (int o = a.block / 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                    }
                    const float inv = factor(m, a.block == 0 ? i == 0 : (i & (a.block - 1)) == 0, i);
                    const uint2 w = make_uint2(e4m3x4(g[0] * inv, g[1] * inv, g[2] * inv, g[3] * inv),
                                               e4m3x4(g[4] * inv, g[5] * inv, g[6] * inv, g[7] * inv));
                    if (i + 8 <= now.width) {
                        *reinterpret_cast<uint2 *>(out + i) = w;
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (i + j < now.width) out[i + j] = (uint8_t)((j < 4 ? w.x : w.y) >> (8 * (j % 4)));
                    }
                } else {   // a block is the whole warp's, of one to four of a thread's values
                    float m[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) m[j] = fabsf(g[j]);
                    if (a.block >= 64) {
#pragma unroll
                        for (int j = 0; j < 8; j += 2) m[j] = m[j + 1] = fmaxf(m[j], m[j + 1]);
                    }
                    if (a.block == 128) {
#pragma unroll
                        for (int j = 0; j < 8; j += 4) m[j] = m[j + 1] = m[j + 2] = m[j + 3] = fmaxf(m[j], m[j + 2]);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int at = i + 32 * j;
                        const float t = a.block == 0 ? most : warp_max(m[j]);
                        const float inv = factor(t, a.block == 0 ? at == 0 : (at & (a.block - 1)) == 0, at);
                        if (at < now.width) out[at] = (uint8_t)e4m3x4(g[j] * inv, 0.f, 0.f, 0.f);
                    }
                }
            } else {
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = g[j] * scale;
                store_row8(static_cast<Y *>(a.y) + at(a.y_at, now.outer, now.inner), i, now.width, a.vec, y);
            }
        }
        now = next;
    }
}

using Kernel = void (*)(NormArgs);
template <typename TX, typename TR, typename TY>
Kernel by_chunks(int c) {
    return c == 1 ? k_rms_norm<TX, TR, TY, 1> : c == 4 ? k_rms_norm<TX, TR, TY, 4> : k_rms_norm<TX, TR, TY, 0>;
}
template <typename TX, typename TR>
Kernel by_y(int y, int c) {
    return y == TALKER_DTYPE_F32 ? by_chunks<TX, TR, float>(c)
                                 : y == TALKER_DTYPE_BF16 ? by_chunks<TX, TR, __nv_bfloat16>(c) : by_chunks<TX, TR, __nv_fp8_storage_t>(c);
}
template <typename TX>
Kernel by_res(bool res, int r, int y, int c) {
    return !res ? by_y<TX, void>(y, c) : r == TALKER_DTYPE_F32 ? by_y<TX, float>(y, c) : by_y<TX, __nv_bfloat16>(y, c);
}

bool dense_type(int t) { return t == TALKER_DTYPE_F32 || t == TALKER_DTYPE_BF16; }
int size_of(int t) { return t == TALKER_DTYPE_F32 ? 4 : t == TALKER_DTYPE_BF16 ? 2 : 1; }
bool aligned(const void *p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Strides of dimensions of one element do not count.
Place place(const void *p, int dtype, const talker_row_strides *s, int rows, int inner, bool &vec) {
    const Place r{rows > inner ? s->outer : 0, inner > 1 ? s->inner : 0};
    vec = vec && aligned(p, 8 * size_of(dtype)) && r.outer % 8 == 0 && r.inner % 8 == 0;
    return r;
}

}  // namespace

extern "C" talker_status talker_rms_norm(const void *x, int x_dtype, const talker_row_strides *x_at, const void *residual,
                                         int res_dtype, const talker_row_strides *res_at, const float *gain, float eps, int rows,
                                         int inner, int width, void *sum_out, const talker_row_strides *sum_at, void *y,
                                         int y_dtype, const talker_row_strides *y_at, int block, float *scales,
                                         void *cuda_stream) {
    if (!x || !x_at || !gain || !y || !y_at || rows < 0 || rows > 1 << 30 || inner < 1 || width < 1 || width > 1 << 24 || !(eps >= 0.f)) return TALKER_EINVAL;
    if (!dense_type(x_dtype) || !(dense_type(y_dtype) || y_dtype == TALKER_DTYPE_E4M3)) return TALKER_EINVAL;
    if (residual ? !dense_type(res_dtype) || !res_at : sum_out != nullptr) return TALKER_EINVAL;
    if (sum_out && !sum_at) return TALKER_EINVAL;
    if (y_dtype == TALKER_DTYPE_E4M3 && (!scales || !aligned(scales, 4) || (block != 0 && block != 32 && block != 64 && block != 128)))
        return TALKER_EINVAL;
    if (!aligned(x, size_of(x_dtype)) || !aligned(gain, 4) || !aligned(y, size_of(y_dtype))) return TALKER_EINVAL;
    if (residual && (!aligned(residual, size_of(res_dtype)) || !aligned(sum_out, size_of(res_dtype)))) return TALKER_EINVAL;
    if (rows == 0) return TALKER_OK;
    NormArgs a{};
    a.x = x, a.res = residual, a.gain = gain, a.sum = sum_out, a.y = y, a.scales = scales;
    a.eps = eps, a.rows = rows, a.inner = inner, a.width = width, a.block = y_dtype == TALKER_DTYPE_E4M3 ? block : 0;
    a.block_shift = a.block == 32 ? 5 : a.block == 64 ? 6 : 7, a.blocks = a.block == 0 ? 1 : (width + a.block - 1) / a.block;
    a.inv_width = (float)(1.0 / width);
    a.vec = aligned(gain, 32);
    a.x_at = place(x, x_dtype, x_at, rows, inner, a.vec);
    if (residual) a.res_at = place(residual, res_dtype, res_at, rows, inner, a.vec);
    if (sum_out) a.sum_at = place(sum_out, res_dtype, sum_at, rows, inner, a.vec);
    a.y_at = place(y, y_dtype, y_at, rows, inner, a.vec);
    const int c = width <= 256 ? 1 : width <= 4 * 8 * most_threads(4) ? 4 : 0;
    const int threads = c == 0 ? 1024 : (width + 256 * c - 1) / (256 * c) * 32;
    const int per = std::max(1, 128 / threads);
    const dim3 block_dim(threads, per);
    const Kernel k = x_dtype == TALKER_DTYPE_F32 ? by_res<float>(residual != nullptr, res_dtype, y_dtype, c)
                                                 : by_res<__nv_bfloat16>(residual != nullptr, res_dtype, y_dtype, c);
    // as many CTAs as the multiprocessors hold, each with several rows where there are more
    const int all = (rows + per - 1) / per, most = 152 * std::max(1, 65536 / (c == 4 ? 128 : 64) / (threads * per));
    k<<<std::min(all, most), block_dim, 0, static_cast<cudaStream_t>(cuda_stream)>>>(a);
    if (cudaGetLastError() != cudaSuccess) return TALKER_ECUDA;
    return TALKER_OK;
}
