// Residual addition and RMSNorm of rows, with results in f32, bf16 or e4m3 blocks (include/talker_layer.h).
#include <cuda_fp8.h>

#include <algorithm>

#include "rows.cuh"
#include "talker_layer.h"

using namespace talker_dev;

namespace {

struct Place {
    long long outer, inner;
    bool vec;   // eight values of a row by one access
};
struct NormArgs {
    const void *x, *res;
    const float *gain;
    void *sum, *y;
    float *scales;
    Place x_at, res_at, sum_at, y_at;
    float eps;
    int rows, inner, width, block;   // block: in values, 0: a row
    bool gain_vec;
};

__device__ __forceinline__ long long at(const Place &p, int outer, int inner) { return outer * p.outer + inner * p.inner; }

template <typename T>
__device__ __forceinline__ void load_row8(const T *p, int i, int width, bool vec, float (&v)[8]) {
    if (i + 8 <= width) {
        load8(p + i, vec, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = i + j < width ? Elem<T>::load(p, i + j) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void store_row8(T *p, int i, int width, bool vec, const float (&v)[8]) {
    if (i + 8 <= width) {
        store8(p + i, vec, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (i + j < width) Elem<T>::store(p, i + j, v[j]);
    }
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
           (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3) << 16;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ float max_abs8(const float (&v)[8]) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max_nan(m, fabsf(v[j]));
    return m;
}

// A row's sum or maximum over its blockDim.x threads, in every one of them. All threads of the CTA take part.
template <bool MAX>
__device__ __forceinline__ float row_all(float v, float *red) {
    if (MAX) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
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
        for (int o = 16; o > 0; o >>= 1) w = max_nan(w, __shfl_xor_sync(0xffffffffu, w, o));
        return w;
    }
    return warp_sum(w);
}

// blockDim.x threads a row, blockDim.y rows a CTA; a thread has eight consecutive values of every chunk of 8 *
// blockDim.x. C chunks stay in registers between the sum and the result; with C = 0 (rows of more) they are read again.
template <typename TX, typename TR, typename TY, int C>
__global__ void __launch_bounds__(1024) k_rms_norm(const NormArgs a) {
    constexpr bool kRes = !std::is_same<TR, void>::value, k8 = std::is_same<TY, __nv_fp8_storage_t>::value;
    using R = typename std::conditional<kRes, TR, float>::type;
    using Y = typename std::conditional<k8, float, TY>::type;
    __shared__ float sums[32], tops[32];   // of a row's warps
    const int row = blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = row < a.rows;
    const int outer = live ? row / a.inner : 0, inner = live ? row - outer * a.inner : 0;
    const TX *x = static_cast<const TX *>(a.x) + at(a.x_at, outer, inner);
    const R *res = kRes ? static_cast<const R *>(a.res) + at(a.res_at, outer, inner) : nullptr;
    const int width = live ? a.width : 0, step = 8 * blockDim.x, first = 8 * threadIdx.x;
    const int chunks = C > 0 ? C : (a.width + step - 1) / step;
    float *const red = sums + threadIdx.y * (blockDim.x >> 5), *const top = tops + threadIdx.y * (blockDim.x >> 5);

    auto take = [&](int c, float (&v)[8]) {
        const int i = c * step + first;
        load_row8(x, i, width, a.x_at.vec, v);
        if (kRes) {
            float r[8];
            load_row8(res, i, width, a.res_at.vec, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += r[j];
        }
    };
    float held[C > 0 ? C : 1][8];
    float sum = 0.f;
#pragma unroll(C > 0 ? C : 1)
    for (int c = 0; c < chunks; ++c) {
        float(&v)[8] = held[C > 0 ? c : 0];
        take(c, v);
        float t = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) t = fmaf(v[j], v[j], t);
        sum += t;
    }
    const float scale = 1.0f / sqrtf(row_all<false>(sum, red) / (float)a.width + a.eps);
    auto result = [&](int c, float (&v)[8], float (&y)[8]) {
        if (C == 0) take(c, v);
        const int i = c * step + first;
        float g[8];
        load_row8(a.gain, i, width, a.gain_vec, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = v[j] * scale * g[j];
    };
    float most = 0.f;   // of the row
    if (k8 && a.block == 0) {
#pragma unroll(C > 0 ? C : 1)
        for (int c = 0; c < chunks; ++c) {
            float y[8];
            result(c, held[C > 0 ? c : 0], y);
            most = max_nan(most, max_abs8(y));
        }
        most = row_all<true>(most, top);
    }
#pragma unroll(C > 0 ? C : 1)
    for (int c = 0; c < chunks; ++c) {
        float(&v)[8] = held[C > 0 ? c : 0];
        float y[8];
        result(c, v, y);
        const int i = c * step + first;
        if (kRes && a.sum != nullptr) store_row8(static_cast<R *>(a.sum) + at(a.sum_at, outer, inner), i, width, a.sum_at.vec, v);
        if (k8) {
            float m = most;
            if (a.block != 0) {   // its threads are neighbours in a warp
                m = max_abs8(y);
                for (int o = a.block / 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            }
            const bool none = m < 0x1p-100f;
            const float inv = none ? 0.f : 448.f / m;
            const int blocks = a.block == 0 ? 1 : (a.width + a.block - 1) / a.block;
            if (a.block == 0 ? i == 0 : i % a.block == 0 && i < width)
                if (live) a.scales[(size_t)row * blocks + (a.block == 0 ? 0 : i / a.block)] = none ? 0.f : m / 448.f;
            uint8_t *out = static_cast<uint8_t *>(a.y) + at(a.y_at, outer, inner);
            const uint2 w = make_uint2(e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                                       e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
            if (a.y_at.vec && i + 8 <= width) {
                *reinterpret_cast<uint2 *>(out + i) = w;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (i + j < width) out[i + j] = (uint8_t)((j < 4 ? w.x : w.y) >> (8 * (j % 4)));
            }
        } else {
            store_row8(static_cast<Y *>(a.y) + at(a.y_at, outer, inner), i, width, a.y_at.vec, y);
        }
    }
}

using Kernel = void (*)(NormArgs);
template <typename TX, typename TR, typename TY>
Kernel by_chunks(int c) {
    return c == 1 ? k_rms_norm<TX, TR, TY, 1> : c == 2 ? k_rms_norm<TX, TR, TY, 2> : k_rms_norm<TX, TR, TY, 0>;
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
Place place(const void *p, int dtype, const talker_row_strides *s, int rows, int inner) {
    Place r{rows > inner ? s->outer : 0, inner > 1 ? s->inner : 0, false};
    r.vec = aligned(p, 8 * size_of(dtype)) && r.outer % 8 == 0 && r.inner % 8 == 0;
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
    a.x_at = place(x, x_dtype, x_at, rows, inner);
    if (residual) a.res_at = place(residual, res_dtype, res_at, rows, inner);
    if (sum_out) a.sum_at = place(sum_out, res_dtype, sum_at, rows, inner);
    a.y_at = place(y, y_dtype, y_at, rows, inner);
    a.gain_vec = aligned(gain, 32);
    const int c = width <= 8192 ? 1 : width <= 16384 ? 2 : 0;
    const int threads = c == 0 ? 1024 : (width + 256 * c - 1) / (256 * c) * 32;
    const int per = std::max(1, 128 / threads);
    const dim3 block_dim(threads, per);
    const Kernel k = x_dtype == TALKER_DTYPE_F32 ? by_res<float>(residual != nullptr, res_dtype, y_dtype, c)
                                                 : by_res<__nv_bfloat16>(residual != nullptr, res_dtype, y_dtype, c);
    k<<<(rows + per - 1) / per, block_dim, 0, static_cast<cudaStream_t>(cuda_stream)>>>(a);
    if (cudaGetLastError() != cudaSuccess) return TALKER_ECUDA;
    return TALKER_OK;
}
