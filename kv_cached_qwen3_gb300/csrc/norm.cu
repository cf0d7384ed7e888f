// Residual addition and RMSNorm of rows, with results in f32, bf16 or e4m3 blocks (include/talker_layer.h).
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

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
};

__device__ __forceinline__ long long at(const Place &p, int outer, int inner) {
    return inner < 0 ? outer * p.outer : outer * p.outer + inner * p.inner;
}

struct Row {
    int outer, inner, width;   // inner -1: rows at one stride; width 0: none
};
__device__ __forceinline__ Row place_of(const NormArgs &a, int row) {
    if (row >= a.rows) return {0, -1, 0};
    if (a.inner == 1) return {row, -1, a.width};
    const int outer = (unsigned)row / (unsigned)a.inner;
    return {outer, row - outer * a.inner, a.width};
}

// Eight neighbouring values of a row, at its end those that it has.
template <typename T>
__device__ __forceinline__ void load_row8(const T *p, int at, int width, float (&v)[8]) {
    if (at + 8 <= width) {
        load8(p + at, true, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = at + j < width ? Elem<T>::load(p, at + j) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void store_row8(T *p, int at, int width, const float (&v)[8]) {
    if (at + 8 <= width) {
        store8(p + at, true, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (at + j < width) Elem<T>::store(p, at + j, v[j]);
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

// A row's sum or maximum over its blockDim.x threads (4, 8, 16 or whole warps), in every one of them. All threads of the CTA
// take part.
template <bool MAX>
__device__ __forceinline__ float lanes_all(float v, int lanes) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (o >= lanes) continue;
        const float w = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? fmaxf(v, w) : v + w;
    }
    return v;
}
template <bool MAX>
__device__ __forceinline__ float row_all(float v, float *red) {
    v = lanes_all<MAX>(v, blockDim.x);
    const int warps = blockDim.x >> 5;
    if (warps <= 1) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return lanes_all<MAX>(lane < warps ? red[lane] : 0.f, 32);
}

// 1 / sqrt(x): the hardware's (2^-23 off) and a step of Newton's method; of 0 and infinity as it is.
__device__ __forceinline__ float root(float x) {
    float r;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    const float better = fmaf(r * 0.5f, fmaf(-x * r, r, 1.f), r);
    return r > 0.f && r < INFINITY ? better : r;
}

// Of a block with max|s gain| m, in a row whose norm's factor is `norm`: its scale, and what s gain is multiplied by for codes.
struct Scale {
    float scale, codes;
    __device__ __forceinline__ Scale(float m, float norm) {
        const float d = m * norm;   // max|y|
        const bool none = d < 0x1p-100f || (m < 0x1p-100f && norm == norm);   // (a NaN in the row: in all its blocks, of zeros too)
        scale = none ? 0.f : d * (1.f / 448.f);
        codes = none ? 0.f : d < INFINITY ? __fdiv_rn(448.f, m) : NAN;   // (to the last place: an error here is all of a block's)
    }
};

// Eight values of a row as they lie in memory, so that nothing waits for them until they are used.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
    float v[8];
    __device__ __forceinline__ void load(const float *p, int i, int width) { load_row8(p, i, width, v); }
    __device__ __forceinline__ float at(int j) const { return v[j]; }
};
template <>
struct Raw<__nv_bfloat16> {
    uint32_t w[4];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p, int i, int width) {
        if (i + 8 <= width) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p + i);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else {
            const unsigned short *q = reinterpret_cast<const unsigned short *>(p);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = (i + 2 * j < width ? q[i + 2 * j] : 0u) | (i + 2 * j + 1 < width ? (uint32_t)q[i + 2 * j + 1] : 0u) << 16;
        }
    }
    __device__ __forceinline__ float at(int j) const { return j & 1 ? bf16hi(w[j / 2]) : bf16lo(w[j / 2]); }
};

// Rows that lie on whole accesses. What bounds them is memory: a value is read once and written once. blockDim.x threads a
// row, blockDim.y rows at a time; a thread has eight consecutive values of every chunk of 8 * blockDim.x. C chunks stay in
// registers between the sum and the result, and the next rows' are on their way meanwhile (4096 x 5120 bf16 + f32 to e4m3:
// 62 us without); with C = 0 (rows of more than 16384 values) they are read again. For e4m3 the norm's factor cancels: a
// code is that of s gain over the largest of its block.
// Few threads with several chunks each: what a thread does for a row once is shared by more values, and more CTAs are out
// of step with one another (4096 x 5120: one chunk of 640 threads 57 us, two of 320 54, four of 160 41, which is 83% of the
// copy rate; 65536 x 1024 bf16 to bf16 47.5, 83%, 89% with a residual). Narrow rows take 4 to 16 threads, so that a warp has
// several (65536 x 128 bf16, a call by itself: a warp each 31 us, four threads each 12; one of many 7.6). In blocks of 128
// they take sixteen, and three of their four chunks are empty: 131072 x 128 to e4m3 93 us, 29%. A lone row of 1024: 3 us, all of
// it latency.
constexpr int most_threads(int c) { return c == 0 ? 1024 : 512; }
template <typename TX, typename TR, typename TY, int C>
__global__ void __launch_bounds__(most_threads(C), 1) k_rms_norm(const NormArgs a) {
    constexpr bool kRes = !std::is_same<TR, void>::value, k8 = std::is_same<TY, __nv_fp8_storage_t>::value;
    constexpr int H = C > 0 ? C : 1;   // chunks in registers
    using R = typename std::conditional<kRes, TR, float>::type;
    using Y = typename std::conditional<k8, float, TY>::type;
    __shared__ float sums[2][32], tops[2][32];   // of a row's warps; of every other turn, so that one wait a turn is enough
    const int step = 8 * blockDim.x, per = blockDim.y * gridDim.x;
    const int first = 8 * threadIdx.x;
    const int chunks = C > 0 ? C : (a.width + step - 1) / step, warps = blockDim.x >> 5;
    auto row_of = [&](int row) { return place_of(a, row); };
    Raw<TX> x[H];
    Raw<R> r[H];
    auto fetch = [&](const Row &w, int c, Raw<TX> &x, Raw<R> &r) {
        const int i = c * step + first;
        x.load(static_cast<const TX *>(a.x) + at(a.x_at, w.outer, w.inner), i, w.width);
        if (kRes) r.load(static_cast<const R *>(a.res) + at(a.res_at, w.outer, w.inner), i, w.width);
    };
    auto sum_of = [&](const Raw<TX> &x, const Raw<R> &r, float (&v)[8]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = kRes ? x.at(j) + r.at(j) : x.at(j);
    };
    int row = blockIdx.x * blockDim.y + threadIdx.y;
    Row now = row_of(row);
    if (C > 0) {
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
#pragma unroll
            for (int c = 0; c < H; ++c) sum_of(x[c], r[c], held[c]);
#pragma unroll
            for (int c = 0; c < H; ++c) fetch(next, c, x[c], r[c]);
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
            load_row8(a.gain, c * step + first, a.width, g);
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
            if (kRes && a.sum != nullptr) store_row8(static_cast<R *>(a.sum) + at(a.sum_at, now.outer, now.inner), i, now.width, v);
            if (k8) {
                uint8_t *out = static_cast<uint8_t *>(a.y) + at(a.y_at, now.outer, now.inner);
                float m = most;
                if (a.block != 0) {   // its threads are neighbours in a warp
                    m = max_abs8(g);
                    for (int o = a.block / 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                }
                const Scale f(m, scale);
                if (i < now.width && (a.block == 0 ? i == 0 : (i & (a.block - 1)) == 0)) a.scales[(size_t)row * a.blocks + (a.block == 0 ? 0 : i >> a.block_shift)] = f.scale;
                const uint2 w = make_uint2(e4m3x4(g[0] * f.codes, g[1] * f.codes, g[2] * f.codes, g[3] * f.codes),
                                           e4m3x4(g[4] * f.codes, g[5] * f.codes, g[6] * f.codes, g[7] * f.codes));
                if (i + 8 <= now.width) {
                    *reinterpret_cast<uint2 *>(out + i) = w;
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (i + j < now.width) out[i + j] = (uint8_t)((j < 4 ? w.x : w.y) >> (8 * (j % 4)));
                }
            } else {
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = g[j] * scale;
                store_row8(static_cast<Y *>(a.y) + at(a.y_at, now.outer, now.inner), i, now.width, y);
            }
        }
        now = next;
    }
}

// Rows that no vector access fits (odd widths, strides or starts). blockDim.x threads share a row: a warp reads 32
// neighbouring values of it at a time, so that loads and stores touch whole sectors. STAGED: rows pass through shared
// memory, where the next ones arrive while these are worked on, in whole 16 bytes but for their ends; otherwise (two rows
// of more than 220 KB) they are read twice. What bounds it are the instructions, a value at a time (60 each; 69% of the
// issue slots): 4001 x 5003 bf16 + f32 to e4m3 in blocks 51 us, 64% of the copy rate. As calls by themselves, 2 to 7 us
// more: 53 (148 from registers, without shared memory; 74 with a thread's values as far apart as a row has threads, whose
// addresses take instructions), 2000 x 10001 bf16 + bf16 to f32 49 (207). A thread for 16 values (74 us then; for 8: 84, for 32: 82); of narrow rows 8 or 16 threads
// (100000 x 47: a warp each 57 us, eight threads each 22), unless a warp's lanes have to be blocks.
constexpr int kOddThreads = 512;
constexpr int kMostStaged = 220 * 1024;
__host__ __device__ constexpr int slot_bytes(int width, int size) { return (width * size + 31) & ~15; }   // at any offset in 16 bytes

__device__ __forceinline__ void copy_async(uint32_t to, const char *from, bool sixteen) {
    if (sixteen)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
// One value of two bytes at a row's odd end: loaded when the row's copies begin, stored when they are waited for.
struct End {
    unsigned short value;
    int to = -1;   // in shared memory
};
// A row of n bytes to a slot, by `threads` threads; two of them take its odd ends.
__device__ __forceinline__ void stage_row(char *smem, int slot, const char *p, int n, int t, int threads, bool ends, End &end) {
    const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15);
    const int low = min((16 - off) & 15, n), high = max(low, ((off + n) & ~15) - off);   // whole 16 bytes
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(smem + slot + off);
    for (int u = low + 16 * t; u < high; u += 16 * threads) copy_async(to + u, p + u, true);
    // words before and after
    if (t < 8) {
        const int u = t < 4 ? ((4 - off) & 3) + 4 * t : high + (t - 4) * 4;
        const int first = (4 - off) & 3;
        if (t < 4 ? u + 4 <= low : u + 4 <= n && u >= first) copy_async(to + u, p + u, false);
    }
    if (ends) {
        const int u = t & 1 ? n - 2 : 0;
        if ((off + (t & 1 ? n : 0)) & 2) end.value = *reinterpret_cast<const unsigned short *>(p + u), end.to = slot + off + u;
    }
}

template <typename TX, typename TR, typename TY, bool STAGED>
__global__ void __launch_bounds__(kOddThreads, 2) k_rms_norm_odd(const NormArgs a, const int tile) {
    constexpr bool kRes = !std::is_same<TR, void>::value, k8 = std::is_same<TY, __nv_fp8_storage_t>::value;
    using R = typename std::conditional<kRes, TR, float>::type;
    using Y = typename std::conditional<k8, float, TY>::type;
    extern __shared__ __align__(16) char smem[];
    __shared__ float sums[2][32], tops[2][32];
    const int t = threadIdx.x, threads = blockDim.x, warps = threads >> 5, width = a.width;
    const int x_slot = slot_bytes(width, sizeof(TX)), slot = x_slot + (kRes ? slot_bytes(width, sizeof(R)) : 0);
    const int per = blockDim.y * tile * gridDim.x;
    End x_end, r_end;
    auto x_of = [&](const Row &w) { return static_cast<const TX *>(a.x) + at(a.x_at, w.outer, w.inner); };
    auto r_of = [&](const Row &w) { return static_cast<const R *>(a.res) + at(a.res_at, w.outer, w.inner); };
    auto slot_of = [&](int turn, int k) { return (((turn & 1) * (int)blockDim.y + (int)threadIdx.y) * tile + k) * slot; };
    auto issue = [&](int first, int turn) {
        for (int k = 0; k < tile && first + k < a.rows; ++k) {
            const Row w = place_of(a, first + k);
            const bool ends = t >> 1 == k;
            stage_row(smem, slot_of(turn, k), reinterpret_cast<const char *>(x_of(w)), width * (int)sizeof(TX), t, threads, sizeof(TX) == 2 && ends, x_end);
            if (kRes) stage_row(smem, slot_of(turn, k) + x_slot, reinterpret_cast<const char *>(r_of(w)), width * (int)sizeof(R), t, threads, sizeof(R) == 2 && ends, r_end);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int first = (blockIdx.x * blockDim.y + threadIdx.y) * tile;
    if (STAGED) issue(first, 0);
    for (int turn = 0; first - (int)threadIdx.y * tile < a.rows; first += per, ++turn) {   // (all of a CTA's threads together)
        if (STAGED) {
            if (x_end.to >= 0) *reinterpret_cast<unsigned short *>(smem + x_end.to) = x_end.value;
            if (kRes && r_end.to >= 0) *reinterpret_cast<unsigned short *>(smem + r_end.to) = r_end.value;
            x_end.to = r_end.to = -1;
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            if (warps <= 1) __syncwarp();
            else __syncthreads();
            issue(first + per, turn + 1);   // to the slots that the last turn is done with
        }
        for (int k = 0; k < tile; ++k) {
            const Row now = place_of(a, first + k);
            const TX *x = x_of(now);
            const R *r = kRes ? r_of(now) : nullptr;
            if (STAGED) {   // (a place of 16 bytes in global memory is one in shared memory)
                r = reinterpret_cast<const R *>(smem + slot_of(turn, k) + x_slot + (reinterpret_cast<uintptr_t>(r) & 15));
                x = reinterpret_cast<const TX *>(smem + slot_of(turn, k) + (reinterpret_cast<uintptr_t>(x) & 15));
            }
            auto value = [&](int i) { return Elem<TX>::load(x, i) + (kRes ? Elem<R>::load(r, i) : 0.f); };
            float sum = 0.f, most = 0.f;
            float *const red = sums[turn & 1] + threadIdx.y * warps, *const top = tops[turn & 1] + threadIdx.y * warps;
            R *const s_out = !kRes || a.sum == nullptr ? nullptr : static_cast<R *>(a.sum) + at(a.sum_at, now.outer, now.inner);
            Y *const y = static_cast<Y *>(a.y) + (k8 ? 0 : at(a.y_at, now.outer, now.inner));
            uint8_t *const codes = static_cast<uint8_t *>(a.y) + (k8 ? at(a.y_at, now.outer, now.inner) : 0);
            float *const scales = a.scales + (size_t)(first + k) * a.blocks;
            auto spread = [&](auto apart_) {   // a thread's values are `apart` from one another, at offsets that instructions hold
                constexpr int apart = decltype(apart_)::value;
                const int own = t % apart, from = t - own;
                for (int i = 8 * from + own; i < now.width; i += 8 * threads) {
                    float s8 = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const bool in = i + j * apart < now.width;
                        const float v = in ? value(i + j * apart) : 0.f;
                        s8 = fmaf(v, v, s8);
                        if (k8 && a.block == 0) most = fmaxf(most, in ? fabsf(v * a.gain[i + j * apart]) : 0.f);
                    }
                    sum += s8;
                }
                const float scale = root(fmaf(row_all<false>(sum, red), a.inv_width, a.eps));
                // four values: s to its place, s gain to g (0 behind the row)
                auto four = [&](int i, float (&g)[4]) {
                    float v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool in = i + apart * j < now.width;
                        v[j] = in ? value(i + apart * j) : 0.f;
                        g[j] = in ? a.gain[i + apart * j] : 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (kRes && s_out != nullptr && i + apart * j < now.width) Elem<R>::store(s_out, i + apart * j, v[j]);
                        g[j] *= v[j];
                    }
                };
                if (!k8 || a.block == 0) {
                    const Scale f(k8 ? row_all<true>(most, top) : 0.f, scale);
                    if (k8 && t == 0 && now.width > 0) *scales = f.scale;
                    for (int i = 4 * from + own; i < now.width; i += 4 * threads) {
                        float g[4];
                        four(i, g);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int p = i + j * apart;
                            if (p >= now.width) continue;
                            if (k8) codes[p] = __nv_cvt_float_to_fp8(g[j] * f.codes, __NV_SATFINITE, __NV_E4M3);
                            else Elem<Y>::store(y, p, g[j] * scale);
                        }
                    }
                    return;
                }
                if constexpr (apart == 32) {   // (rows in blocks have whole warps)
                    auto blocks = [&](auto values) {   // of so many values: a warp has four, two or one
                        constexpr int B = decltype(values)::value, per = B / 32;
                        for (int i = 4 * from + own; i - own < now.width; i += 4 * threads) {
                            float g[4];
                            four(i, g);
#pragma unroll
                            for (int j = 0; j < 4; j += per) {
                                float m = 0.f;
#pragma unroll
                                for (int l = 0; l < per; ++l) m = fmaxf(m, fabsf(g[j + l]));
                                const Scale f(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m))), scale);   // (not negative: ordered as whole numbers)
                                if (own == 0 && i + 32 * j < now.width) scales[(i + 32 * j) / B] = f.scale;
#pragma unroll
                                for (int l = j; l < j + per; ++l)
                                    if (i + 32 * l < now.width) codes[i + 32 * l] = __nv_cvt_float_to_fp8(g[l] * f.codes, __NV_SATFINITE, __NV_E4M3);
                            }
                        }
                    };
                    if (a.block == 32) blocks(std::integral_constant<int, 32>());
                    else if (a.block == 64) blocks(std::integral_constant<int, 64>());
                    else blocks(std::integral_constant<int, 128>());
                }
            };
            if (threads >= 32) spread(std::integral_constant<int, 32>());
            else if (threads == 16) spread(std::integral_constant<int, 16>());
            else spread(std::integral_constant<int, 8>());
        }
    }
}

// Kernels by what they do: -1 and -2 rows without vector accesses, staged and read twice; else chunks in registers.
template <typename TX, typename TR, typename TY>
cudaError_t launch(const NormArgs &a, int kind, dim3 grid, dim3 block, int tile, int shared, cudaStream_t st) {
    if (kind == 4) {
        k_rms_norm<TX, TR, TY, 4><<<grid, block, 0, st>>>(a);
    } else if (kind == 0) {
        k_rms_norm<TX, TR, TY, 0><<<grid, block, 0, st>>>(a);
    } else if (kind == -2) {
        k_rms_norm_odd<TX, TR, TY, false><<<grid, block, 0, st>>>(a, 1);
    } else {
        static std::atomic<unsigned long long> raised{0};   // devices whose limit of shared memory is raised
        int device = 0;
        cudaError_t e = cudaGetDevice(&device);
        const unsigned long long bit = device < 64 ? 1ull << device : 0;
        if (e == cudaSuccess && !(raised.load() & bit)) {
            e = cudaFuncSetAttribute(k_rms_norm_odd<TX, TR, TY, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostStaged);
            if (e == cudaSuccess) raised |= bit;
        }
        if (e != cudaSuccess) return e;
        k_rms_norm_odd<TX, TR, TY, true><<<grid, block, shared, st>>>(a, tile);
    }
    return cudaGetLastError();
}
using Launch = cudaError_t (*)(const NormArgs &, int, dim3, dim3, int, int, cudaStream_t);
template <typename TX, typename TR>
Launch by_y(int y) {
    return y == TALKER_DTYPE_F32 ? launch<TX, TR, float> : y == TALKER_DTYPE_BF16 ? launch<TX, TR, __nv_bfloat16> : launch<TX, TR, __nv_fp8_storage_t>;
}
template <typename TX>
Launch by_res(bool res, int r, int y) {
    return !res ? by_y<TX, void>(y) : r == TALKER_DTYPE_F32 ? by_y<TX, float>(y) : by_y<TX, __nv_bfloat16>(y);
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
// Rows of a result lie in places of their own.
bool apart(const Place &p, int rows, int inner) { return (rows <= inner || p.outer != 0) && (std::min(rows, inner) <= 1 || p.inner != 0); }

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
    bool vec = aligned(gain, 32);
    a.x_at = place(x, x_dtype, x_at, rows, inner, vec);
    if (residual) a.res_at = place(residual, res_dtype, res_at, rows, inner, vec);
    if (sum_out) a.sum_at = place(sum_out, res_dtype, sum_at, rows, inner, vec);
    a.y_at = place(y, y_dtype, y_at, rows, inner, vec);
    if (!apart(a.y_at, rows, inner) || (sum_out && !apart(a.sum_at, rows, inner))) return TALKER_EINVAL;
    // (both kernels' sides are beside them)
    const int row_bytes = slot_bytes(width, size_of(x_dtype)) + (residual ? slot_bytes(width, size_of(res_dtype)) : 0);
    const int kind = !vec ? 2 * row_bytes <= kMostStaged ? -1 : -2 : width <= 4 * 8 * most_threads(4) ? 4 : 0;
    int threads = kind == 0 ? 1024 : (width + 1023) / 1024 * 32, tile = 1, ctas = 0, shared = 0;
    if (kind == 4 && width <= 512)   // several rows a warp; a block's threads are neighbours
        for (threads = std::max(4, a.block / 8); threads * 32 < width;) threads *= 2;
    if (kind < 0) threads = a.block == 0 && width <= 128 ? width <= 64 ? 8 : 16 : std::min(kOddThreads, (width + 511) / 512 * 32);
    const int per = std::max(1, 128 / threads);
    if (kind == -1) {
        if (threads <= 32) tile = std::max(1, std::min({threads / 2, 8, 8192 / (per * row_bytes), rows / (152 * 8 * per)}));
        shared = 2 * per * tile * row_bytes;
        ctas = std::max(1, std::min(1024 / (threads * per), 227 * 1024 / (shared + 1536)));
    } else {
        ctas = std::max(1, (kind == -2 ? 1024 : 512) / (threads * per));
    }
    // as many CTAs as the multiprocessors hold, each with several rows where there are more
    const long long all = ((long long)rows + per * tile - 1) / (per * tile);
    const Launch go = x_dtype == TALKER_DTYPE_F32 ? by_res<float>(residual != nullptr, res_dtype, y_dtype)
                                                  : by_res<__nv_bfloat16>(residual != nullptr, res_dtype, y_dtype);
    const cudaError_t e = go(a, kind, dim3((unsigned)std::min<long long>(all, 152 * ctas)), dim3(threads, per), tile, shared,
                             static_cast<cudaStream_t>(cuda_stream));
    return e == cudaSuccess ? TALKER_OK : TALKER_ECUDA;
}
