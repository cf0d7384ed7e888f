// Products with 4-bit weights in groups (include/talker_layer.h).
#include <cuda_fp8.h>

#include <algorithm>

#include "rows.cuh"
#include "talker_layer.h"

using namespace talker_dev;

namespace {

constexpr int kUnit = 128;              // inputs: what k is padded to, and what one warp takes at a time
constexpr int kUnitBytes = 16 * kUnit / 2;

struct Sizes {
    int tiles, units, groups;           // row tiles, units of inputs, groups (of the padded inputs)
    size_t scales_at, zeros_at, bytes;  // in the tiles' memory
};
__host__ __device__ inline Sizes sizes_of(int n, int k, int group, int zeros, int gated) {
    Sizes s;
    s.tiles = gated ? (n + 7) / 8 : (n + 15) / 16;
    s.units = (k + kUnit - 1) / kUnit;
    s.groups = s.units * (kUnit / group);
    s.scales_at = (size_t)s.tiles * s.units * kUnitBytes;
    s.zeros_at = s.scales_at + (size_t)s.tiles * s.groups * 32;
    s.bytes = s.zeros_at + (zeros ? (size_t)s.tiles * s.groups * 16 : 0);
    return s;
}

// ---- layout

struct PackArgs {
    const uint8_t *codes[2], *zeros[2];
    const __half *scales[2];
    unsigned char *tiles;
    Sizes s;
    int n, k, group, gated;
};
__device__ __forceinline__ int row_of(const PackArgs &a, int tile, int r, int &matrix) {
    matrix = a.gated && r >= 8;
    return a.gated ? tile * 8 + (r & 7) : tile * 16 + r;
}
// A thread per word of codes.
__global__ void __launch_bounds__(256) k_w4_pack_codes(const PackArgs a, long long words) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= words) return;
    const int j = (int)(i & 3), lane = (int)(i >> 2) & 31, g = lane >> 2, t = lane & 3;
    const long long chunk = i >> 7;
    const int tile = (int)(chunk / (2 * a.s.units)), k0 = (int)(chunk % (2 * a.s.units)) * 64 + 16 * j + 4 * t;
    const int row_bytes = (a.k + 1) / 2;
    uint32_t w = 0;
    for (int half = 0; half < 2; ++half) {
        int m;
        const int row = row_of(a, tile, g + 8 * half, m);
        if (row >= a.n) continue;
        for (int e = 0; e < 4; ++e) {
            const int k = k0 + e;
            if (k >= a.k) continue;
            const uint32_t c = a.codes[m][(size_t)row * row_bytes + k / 2] >> (4 * (k & 1)) & 15;
            w |= c << 4 * ((e & 1) * 4 + (e >> 1) + 2 * half);
        }
    }
    reinterpret_cast<uint32_t *>(a.tiles)[i] = w;
}
// A thread per scale (and zero) of a tile's row.
__global__ void __launch_bounds__(256) k_w4_pack_scales(const PackArgs a, long long scales) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= scales) return;
    const int r = (int)(i & 15), g = r >> 1, half = r & 1;
    const long long at = i >> 4;
    const int tile = (int)(at / a.s.groups), group = (int)(at % a.s.groups), groups = (a.k + a.group - 1) / a.group;
    int m;
    const int row = row_of(a, tile, g + 8 * half, m);
    const bool there = row < a.n && group < groups;
    const size_t from = (size_t)row * groups + group;
    reinterpret_cast<__half *>(a.tiles + a.s.scales_at)[i] = there ? a.scales[m][from] : __float2half_rn(0.f);
    if (a.zeros[0]) (a.tiles + a.s.zeros_at)[i] = there ? a.zeros[m][from] & 15 : 0;
}

// A warp per group of a row. The code of x is the largest n <= 15 with 16 x sign(m) <= (17 - 2 n) |m| (0 if there
// is none), a comparison that 64 bits make exactly; one division finds it but for the last step.
template <typename T>
__global__ void __launch_bounds__(256) k_w4_quantize(const T *w, long long row_stride, int n, int k, int group, uint8_t *codes, __half *scales) {
    const int groups = (k + group - 1) / group, lane = threadIdx.x & 31;
    const long long at = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (at >= (long long)n * groups) return;
    const int row = (int)(at / groups), k0 = (int)(at % groups) * group, k1 = min(k, k0 + group);
    float top = -1.f, m = 0.f;
    int first = 0x7fffffff;
    bool bad = false;
    for (int i = k0 + lane; i < k1; i += 32) {
        const float x = Elem<T>::load(w + row * row_stride, i);
        bad |= !(fabsf(x) < INFINITY);
        if (fabsf(x) > top) top = fabsf(x), m = x, first = i;
    }
    bad = __any_sync(0xffffffffu, bad);
    const float most = warp_max(top);
    const int who = __reduce_min_sync(0xffffffffu, top == most ? first : 0x7fffffff);
    m = __shfl_sync(0xffffffffu, m, __ffs(__ballot_sync(0xffffffffu, first == who)) - 1);
    m = fminf(fmaxf(m, -524032.f), 524032.f);
    const bool none = bad || !(most > 0.f);
    if (lane == 0) scales[at] = bad ? __ushort_as_half(0x7fff) : __float2half_rn(m * -0.125f);   // (zeros keep the first one's sign)
    const double am = fabs((double)m);
    for (int i = k0 + 2 * lane; i < k1; i += 64) {   // (groups begin at even inputs)
        uint32_t two = 0;
        for (int e = 0; e < 2; ++e) {
            int c = 8;
            if (i + e < k1 && !none) {
                const float x = Elem<T>::load(w + row * row_stride, i + e);
                const double v = 16.0 * (m > 0.f ? (double)x : -(double)x);
                c = (int)fmin(fmax(floor(8.5 - v / (2.0 * am)), -1.0), 16.0);
                if (v > (17 - 2 * c) * am) --c;
                else if (v <= (15 - 2 * c) * am) ++c;
                c = min(max(c, 0), 15);
            }
            if (i + e < k1) two |= c << 4 * e;
        }
        codes[(size_t)row * ((k + 1) / 2) + i / 2] = (uint8_t)two;
    }
}

// ---- rows of x as the tensor cores' operand

// x enters as fp16 in columns: bf16 rows one column each, others two (the nearest fp16 and what is left), of x times
// 2^e with the row's largest magnitude in [2^14, 2^15). Codes enter as the whole numbers c - z.
struct XArgs {
    const void *x;
    const float *scales;
    long long row;
    int block, k, rows;
};
struct Prepared {
    uint4 *frags;     // [unit][tile of 8 columns][4 quarters of 32 inputs][lane]: steps of 16 inputs 2 q, 2 q + 1
    float *back;      // [row]: 2^-e, or NaN
};
template <typename T>
__device__ __forceinline__ float load_x(const XArgs &a, int r, int k) {
    return Elem<T>::load(static_cast<const T *>(a.x) + r * a.row, k);
}
template <>
__device__ __forceinline__ float load_x<__nv_fp8_storage_t>(const XArgs &a, int r, int k) {
    const __nv_fp8_storage_t c = static_cast<const __nv_fp8_storage_t *>(a.x)[r * a.row + k];
    const float v = __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
    const int blocks = a.block ? (a.k + a.block - 1) / a.block : 1;
    return v * a.scales[(size_t)r * blocks + (a.block ? k / a.block : 0)];
}

// A CTA per row.
template <typename T, int PARTS>
__global__ void __launch_bounds__(256) k_w4_rows(const XArgs a, const Prepared to, int units, int col_tiles) {
    __shared__ float red[8];
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
    float most = 0.f;
    bool bad = false;
    for (int k = tid; k < a.k; k += 256) {
        const float v = fabsf(load_x<T>(a, r, k));
        bad |= !(v < INFINITY);
        most = fmaxf(most, v);
    }
    most = warp_max(most);
    if (lane == 0) red[tid >> 5] = most;
    bad = __syncthreads_or(bad);
    for (int i = 0; i < 8; ++i) most = fmaxf(most, red[i]);
    int e = most > 0.f ? ilogbf(most) : 0;     // 2^e <= most
    e = min(max(14 - e, -113), 120);
    const float up = ldexpf(1.f, e);           // (most below 2^-106 keeps fewer bits)
    if (tid == 0) to.back[r] = bad ? NAN : ldexpf(1.f, -e);
    // eight threads make 32 inputs, four each
    for (int k = 4 * tid; k < units * kUnit; k += 1024) {
        __half h[PARTS][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = k + i < a.k && !bad ? load_x<T>(a, r, k + i) * up : 0.f;
            h[0][i] = __float2half_rn(v);
            if (PARTS == 2) h[PARTS - 1][i] = __float2half_rn(v - __half2float(h[0][i]));
        }
        const int unit = k / kUnit, q = k % kUnit / 32, step = k % 32 / 16, t = k % 16 / 4;
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
            const int col = r * PARTS + p;
            uint2 *at = reinterpret_cast<uint2 *>(to.frags + (((size_t)unit * col_tiles + col / 8) * 4 + q) * 32 + (col & 7) * 4 + t) + step;
            *at = make_uint2(__half_as_ushort(h[p][0]) | (uint32_t)__half_as_ushort(h[p][1]) << 16,
                             __half_as_ushort(h[p][2]) | (uint32_t)__half_as_ushort(h[p][3]) << 16);
        }
    }
}

// ---- the product

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes of one word as the operand's registers: fields 0 and 4 of v (or of v >> 8) under 1024, whose last place is 1, are
// 1024 + c; fields 1 and 5 are 1024 + 16 c. Taking off 1024 + z, or 64 + z after a sixteenth, leaves c - z, exactly.
struct Zero {
    uint32_t a, b;   // -(1024 + z) and -(64 + z), twice each
};
__device__ __forceinline__ Zero zero_of(uint32_t z) { return {(0xe400u | z) * 0x10001u, (0xd400u | z << 4) * 0x10001u}; }
__device__ __forceinline__ uint32_t centred(uint32_t v, Zero z) {
    uint32_t y;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"((v & 0x000f000fu) | 0x64006400u), "r"(z.a));
    return y;
}
__device__ __forceinline__ uint32_t centred16(uint32_t v, Zero z) {
    uint32_t y;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"((v & 0x00f000f0u) | 0x64006400u), "r"(0x2c002c00u), "r"(z.b));
    return y;
}

struct MatmulArgs {
    const unsigned char *tiles;
    Sizes s;
    Prepared x;
    const void *res;
    void *out;
    long long res_row, out_row;
    int n, rows, col_tiles;   // col_tiles: of all rows' columns
    bool zeros, gated, bf16;
};

// A CTA per row tile and NT column tiles: its warps share the units of inputs; their sums meet in shared memory. A warp
// multiplies 16 rows of codes with 8 NT columns; a group's sum is added to the total times the group's scale.
template <int GROUP, int PARTS, int NT>
__global__ void __launch_bounds__(256) k_w4_matmul(const MatmulArgs a) {
    extern __shared__ float4 red[];   // [warp][NT][lane]
    const int tile = blockIdx.x, ct0 = blockIdx.y * NT, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint4 *codes = reinterpret_cast<const uint4 *>(a.tiles) + (size_t)tile * a.s.units * 64 + lane;
    const uint32_t *scales = reinterpret_cast<const uint32_t *>(a.tiles + a.s.scales_at) + (size_t)tile * a.s.groups * 8 + g;
    const uint16_t *zeros = reinterpret_cast<const uint16_t *>(a.tiles + a.s.zeros_at) + (size_t)tile * a.s.groups * 8 + g;
    float total[NT][4], c[NT][4];
    Zero z0 = zero_of(8), z1 = z0;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) total[i][j] = c[i][j] = 0.f;
    for (int u = warp; u < a.s.units; u += 8) {
        const uint4 w[2] = {codes[(size_t)u * 64], codes[(size_t)u * 64 + 32]};
#pragma unroll
        for (int q = 0; q < 4; ++q) {   // 32 inputs
            if (q * 32 % GROUP == 0) {
                const int grp = u * (kUnit / GROUP) + q * 32 / GROUP;
                if (a.zeros) {
                    const uint16_t z = zeros[(size_t)grp * 8];
                    z0 = zero_of(z & 15), z1 = zero_of(z >> 8);
                }
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) c[i][j] = 0.f;
            }
            uint4 b[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i)
                b[i] = ct0 + i < a.col_tiles ? a.x.frags[(((size_t)u * a.col_tiles + ct0 + i) * 4 + q) * 32 + lane] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int step = 0; step < 2; ++step) {
                const uint4 ww = w[q / 2];
                const uint32_t v = q % 2 ? (step ? ww.w : ww.z) : (step ? ww.y : ww.x), v8 = v >> 8;
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    mma_f16(c[i], centred(v, z0), centred(v8, z1), centred16(v, z0), centred16(v8, z1), step ? b[i].z : b[i].x, step ? b[i].w : b[i].y);
            }
            if ((q + 1) * 32 % GROUP == 0) {
                const int grp = u * (kUnit / GROUP) + q * 32 / GROUP;
                const uint32_t d = scales[(size_t)grp * 8];
                const float d0 = __half2float(__ushort_as_half((unsigned short)d)), d1 = __half2float(__ushort_as_half((unsigned short)(d >> 16)));
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    total[i][0] = fmaf(d0, c[i][0], total[i][0]), total[i][1] = fmaf(d0, c[i][1], total[i][1]);
                    total[i][2] = fmaf(d1, c[i][2], total[i][2]), total[i][3] = fmaf(d1, c[i][3], total[i][3]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) red[(warp * NT + i) * 32 + lane] = make_float4(total[i][0], total[i][1], total[i][2], total[i][3]);
    __syncthreads();
    // a thread per lane of the tensor cores' result: rows g and g + 8 of two columns
    for (int j = threadIdx.x; j < NT * 32; j += 256) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        for (int w = 0; w < 8; ++w) {
            const float4 p = red[w * NT * 32 + j];
            v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
        }
        const int l = j & 31, gg = l >> 2, col = (ct0 + (j >> 5)) * 8 + 2 * (l & 3);
#pragma unroll
        for (int e = 0; e < (PARTS == 2 ? 1 : 2); ++e) {
            const int r = PARTS == 2 ? col / 2 : col + e;
            if (r >= a.rows) continue;
            const float back = a.x.back[r];
            const float y0 = (PARTS == 2 ? v[0] + v[1] : v[e]) * back, y1 = (PARTS == 2 ? v[2] + v[3] : v[2 + e]) * back;
            for (int half = 0; half < (a.gated ? 1 : 2); ++half) {
                const int row = a.gated ? tile * 8 + gg : tile * 16 + gg + 8 * half;
                if (row >= a.n) continue;
                float y = a.gated ? y0 / (1.f + expf(-y0)) * y1 : half ? y1 : y0;
                if (a.bf16) {
                    if (a.res) y += Elem<__nv_bfloat16>::load(static_cast<const __nv_bfloat16 *>(a.res) + r * a.res_row, row);
                    Elem<__nv_bfloat16>::store(static_cast<__nv_bfloat16 *>(a.out) + r * a.out_row, row, y);
                } else {
                    if (a.res) y += static_cast<const float *>(a.res)[r * a.res_row + row];
                    static_cast<float *>(a.out)[r * a.out_row + row] = y;
                }
            }
        }
    }
}

template <int GROUP, int PARTS>
void launch_matmul(const MatmulArgs &a, cudaStream_t st) {
    const int nt = a.col_tiles >= 5 ? 8 : a.col_tiles >= 3 ? 4 : a.col_tiles;
    const dim3 grid(a.s.tiles, (a.col_tiles + nt - 1) / nt);
    const size_t smem = (size_t)8 * nt * 32 * sizeof(float4);
    if (nt == 8) k_w4_matmul<GROUP, PARTS, 8><<<grid, 256, smem, st>>>(a);
    else if (nt == 4) k_w4_matmul<GROUP, PARTS, 4><<<grid, 256, smem, st>>>(a);
    else if (nt == 2) k_w4_matmul<GROUP, PARTS, 2><<<grid, 256, smem, st>>>(a);
    else k_w4_matmul<GROUP, PARTS, 1><<<grid, 256, smem, st>>>(a);
}

bool matrix_ok(const talker_w4 *w) {
    return w && w->n >= 1 && w->n <= 1 << 27 && w->k >= 1 && w->k <= 1 << 20 && (w->group == 32 || w->group == 64 || w->group == 128) &&
           (w->zeros == 0 || w->zeros == 1) && (w->gated == 0 || w->gated == 1);
}
bool packed_ok(const talker_w4 *w) { return matrix_ok(w) && w->tiles && reinterpret_cast<uintptr_t>(w->tiles) % 16 == 0; }
Sizes sizes_of(const talker_w4 *w) { return sizes_of(w->n, w->k, w->group, w->zeros, w->gated); }
int size_of(int t) { return t == TALKER_DTYPE_F32 ? 4 : t == TALKER_DTYPE_BF16 ? 2 : 1; }
bool aligned(const void *p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
talker_status status_of(cudaError_t e) { return e == cudaSuccess ? TALKER_OK : TALKER_ECUDA; }

struct Scratch {
    int col_tiles;
    size_t back_at, bytes;
};
Scratch scratch_of(const Sizes &s, int x_dtype, int rows) {
    Scratch r;
    r.col_tiles = (int)(((long long)rows * (x_dtype == TALKER_DTYPE_BF16 ? 1 : 2) + 7) / 8);
    r.back_at = (size_t)s.units * r.col_tiles * 128 * sizeof(uint4);
    r.bytes = r.back_at + (size_t)rows * 4;
    return r;
}

}  // namespace

extern "C" {

size_t talker_w4_bytes(const talker_w4 *w) { return matrix_ok(w) ? sizes_of(w).bytes : 0; }

talker_status talker_w4_pack(const talker_w4 *w, const uint8_t *codes, const void *scales, const uint8_t *zeros,
                             const uint8_t *codes2, const void *scales2, const uint8_t *zeros2, void *cuda_stream) {
    if (!packed_ok(w) || !codes || !scales || (w->zeros && !zeros)) return TALKER_EINVAL;
    if (w->gated && (!codes2 || !scales2 || (w->zeros && !zeros2))) return TALKER_EINVAL;
    if (!aligned(scales, 2) || (w->gated && !aligned(scales2, 2))) return TALKER_EINVAL;
    const PackArgs a{{codes, codes2},
                     {w->zeros ? zeros : nullptr, w->zeros ? zeros2 : nullptr},
                     {static_cast<const __half *>(scales), static_cast<const __half *>(scales2)},
                     static_cast<unsigned char *>(w->tiles), sizes_of(w), w->n, w->k, w->group, w->gated};
    const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    const long long words = (long long)a.s.scales_at / 4, n = (long long)a.s.tiles * a.s.groups * 16;
    if ((words + 255) / 256 > 0x7fffffffll) return TALKER_EINVAL;
    k_w4_pack_codes<<<(unsigned)((words + 255) / 256), 256, 0, st>>>(a, words);
    k_w4_pack_scales<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(a, n);
    return status_of(cudaGetLastError());
}

talker_status talker_w4_quantize(const void *w, int dtype, int64_t row_stride, int n, int k, int group, uint8_t *codes,
                                 void *scales, void *cuda_stream) {
    const talker_w4 sizes{nullptr, n, k, group, 0, 0};
    if (!matrix_ok(&sizes) || !w || !codes || !scales || (dtype != TALKER_DTYPE_F32 && dtype != TALKER_DTYPE_BF16)) return TALKER_EINVAL;
    if (!aligned(w, size_of(dtype)) || !aligned(scales, 2) || (n > 1 && row_stride < k)) return TALKER_EINVAL;
    const long long blocks = ((long long)n * ((k + group - 1) / group) + 7) / 8;
    if (blocks > 0x7fffffffll) return TALKER_EINVAL;
    const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    if (dtype == TALKER_DTYPE_F32)
        k_w4_quantize<<<(unsigned)blocks, 256, 0, st>>>(static_cast<const float *>(w), row_stride, n, k, group, codes, static_cast<__half *>(scales));
    else
        k_w4_quantize<<<(unsigned)blocks, 256, 0, st>>>(static_cast<const __nv_bfloat16 *>(w), row_stride, n, k, group, codes, static_cast<__half *>(scales));
    return status_of(cudaGetLastError());
}

size_t talker_w4_scratch(const talker_w4 *w, int x_dtype, int rows) {
    return matrix_ok(w) && rows > 0 ? scratch_of(sizes_of(w), x_dtype, rows).bytes : 0;
}

talker_status talker_w4_matmul(const talker_w4 *w, const void *x, int x_dtype, int64_t x_row, const float *x_scales,
                               int x_block, int rows, const void *residual, int64_t res_row, void *out, int out_dtype,
                               int64_t out_row, void *scratch, size_t scratch_bytes, void *cuda_stream) {
    if (!packed_ok(w) || !x || !out || rows < 0 || rows > 1 << 20) return TALKER_EINVAL;
    const bool f8 = x_dtype == TALKER_DTYPE_E4M3, bf16 = x_dtype == TALKER_DTYPE_BF16;
    if ((!f8 && !bf16 && x_dtype != TALKER_DTYPE_F32) || (out_dtype != TALKER_DTYPE_F32 && out_dtype != TALKER_DTYPE_BF16)) return TALKER_EINVAL;
    if (f8 && (!x_scales || !aligned(x_scales, 4) || (x_block != 0 && x_block != 32 && x_block != 64 && x_block != 128))) return TALKER_EINVAL;
    if (!aligned(x, size_of(x_dtype)) || !aligned(out, size_of(out_dtype)) || !aligned(residual, size_of(out_dtype))) return TALKER_EINVAL;
    if (rows > 1 && (out_row < w->n || (residual == out && residual && res_row != out_row))) return TALKER_EINVAL;
    if (rows == 0) return TALKER_OK;
    const Sizes s = sizes_of(w);
    const Scratch sc = scratch_of(s, x_dtype, rows);
    if (!scratch || scratch_bytes < sc.bytes || !aligned(scratch, 16)) return TALKER_EINVAL;
    char *base = static_cast<char *>(scratch);
    const Prepared p{reinterpret_cast<uint4 *>(base), reinterpret_cast<float *>(base + sc.back_at)};
    const XArgs xa{x, x_scales, x_row, x_block, w->k, rows};
    const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    if (bf16) k_w4_rows<__nv_bfloat16, 1><<<rows, 256, 0, st>>>(xa, p, s.units, sc.col_tiles);
    else if (f8) k_w4_rows<__nv_fp8_storage_t, 2><<<rows, 256, 0, st>>>(xa, p, s.units, sc.col_tiles);
    else k_w4_rows<float, 2><<<rows, 256, 0, st>>>(xa, p, s.units, sc.col_tiles);
    const MatmulArgs a{static_cast<const unsigned char *>(w->tiles), s, p, residual, out, res_row, out_row, w->n, rows, sc.col_tiles,
                       w->zeros != 0, w->gated != 0, out_dtype == TALKER_DTYPE_BF16};
    if (w->group == 32) bf16 ? launch_matmul<32, 1>(a, st) : launch_matmul<32, 2>(a, st);
    else if (w->group == 64) bf16 ? launch_matmul<64, 1>(a, st) : launch_matmul<64, 2>(a, st);
    else bf16 ? launch_matmul<128, 1>(a, st) : launch_matmul<128, 2>(a, st);
    return status_of(cudaGetLastError());
}

}  // extern "C"
