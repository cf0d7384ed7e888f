// Products with 4-bit weights in groups (include/talker_layer.h).
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>

#include "rows.cuh"
#include "talker_layer.h"

using namespace talker_dev;

namespace {

constexpr int kUnit = 128;              // inputs: what k is padded to, and what one warp takes at a time
constexpr int kUnitBytes = 16 * kUnit / 2;
constexpr int kMostRows = 1 << 19;

struct Sizes {
    int tiles, units, groups;   // row tiles, units of inputs, groups of a unit
    int record;                 // bytes of a tile's unit: codes, scales, zeros
    size_t bytes;
};
__host__ __device__ inline Sizes sizes_of(int n, int k, int group, int zeros, int gated) {
    Sizes s;
    s.tiles = gated ? (n + 7) / 8 : (n + 15) / 16;
    s.units = (k + kUnit - 1) / kUnit;
    s.groups = kUnit / group;
    s.record = kUnitBytes + 32 * s.groups + (zeros ? (s.groups == 1 ? 32 : 16 * s.groups) : 0);   // (whole sectors of 32 bytes)
    s.bytes = (size_t)s.tiles * s.units * s.record;
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
    const int tile = (int)(chunk / (2 * a.s.units)), own = (int)(chunk % (2 * a.s.units)), k0 = own * 64 + 16 * j + 4 * t;
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
    reinterpret_cast<uint32_t *>(a.tiles + ((size_t)tile * a.s.units + own / 2) * a.s.record + own % 2 * 512)[i & 127] = w;
}
// A thread per scale (and zero) of a tile's row.
__global__ void __launch_bounds__(256) k_w4_pack_scales(const PackArgs a, long long scales) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= scales) return;
    const int r = (int)(i & 15), g = r >> 1, half = r & 1;
    const long long at = i >> 4;
    const int all = a.s.units * a.s.groups, tile = (int)(at / all), group = (int)(at % all), groups = (a.k + a.group - 1) / a.group;
    int m;
    const int row = row_of(a, tile, g + 8 * half, m), in_unit = group % a.s.groups;
    const bool there = row < a.n && group < groups;
    const size_t from = (size_t)row * groups + group;
    unsigned char *record = a.tiles + ((size_t)tile * a.s.units + group / a.s.groups) * a.s.record + kUnitBytes;
    reinterpret_cast<__half *>(record + in_unit * 32)[r] = there ? a.scales[m][from] : __float2half_rn(0.f);
    if (a.zeros[0]) (record + 32 * a.s.groups + in_unit * 16)[r] = there ? a.zeros[m][from] & 15 : 0;
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
// Fragments: [32 inputs][column][t] 16 bytes: the inputs 4 t .. 4 t + 3 of the two steps of 16.
struct XArgs {
    const void *x;
    const float *scales;
    long long row;
    int dtype, block, k, rows;
    bool vec;         // four values by one access
};
template <typename T>
__device__ __forceinline__ void load_x4(const XArgs &a, int r, int k, float (&v)[4]) {
    const T *p = static_cast<const T *>(a.x) + r * a.row + k;
    if (a.vec && k + 4 <= a.k) {
        if (sizeof(T) == 4) {
            const float4 u = *reinterpret_cast<const float4 *>(p);
            v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(p);
            v[0] = bf16lo(u.x), v[1] = bf16hi(u.x), v[2] = bf16lo(u.y), v[3] = bf16hi(u.y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = k + i < a.k ? Elem<T>::load(p, i) : 0.f;
    }
}
template <>
__device__ __forceinline__ void load_x4<__nv_fp8_storage_t>(const XArgs &a, int r, int k, float (&v)[4]) {
    const __nv_fp8_storage_t *p = static_cast<const __nv_fp8_storage_t *>(a.x) + r * a.row + k;
    const int blocks = a.block ? (a.k + a.block - 1) / a.block : 1;
    uint32_t u = 0;
    if (a.vec && k + 4 <= a.k) {
        u = *reinterpret_cast<const uint32_t *>(p);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) u |= (k + i < a.k ? (uint32_t)p[i] : 0u) << (8 * i);
    }
    const float d = k < a.k ? a.scales[(size_t)r * blocks + (a.block ? k / a.block : 0)] : 0.f;   // (blocks are multiples of 4)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)(u >> (8 * i)), __NV_E4M3))) * d;
}

// Rows first .. first + rows - 1 (at most as many as warps) by the CTA, each by as many warps as there are for it: their columns to frags
// (of `cols` columns, the first row's at `col`), and what undoes the scaling to back. red: a float for each warp.
template <typename T, int PARTS>
__device__ __forceinline__ void prepare_rows(const XArgs &a, int first, int rows, uint2 *frags, int cols, int col, int units, float *back, float *red) {
    const int tid = threadIdx.x, warps = blockDim.x >> 5, warp = tid >> 5;
    int each = warps;
    while (each * rows > warps) each >>= 1;
    const int own = warp / each, lane = tid - own * each * 32, step = 4 * 32 * each;
    const bool busy = own < rows;
    const int r = first + own;
    float most = 0.f;
    bool bad = false;
    if (busy) {
#pragma unroll 4
        for (int k = 4 * lane; k < a.k; k += step) {
            float v[4];
            load_x4<T>(a, r, k, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                bad |= !(fabsf(v[i]) < INFINITY);
                most = fmaxf(most, fabsf(v[i]));
            }
        }
    }
    most = warp_max(most);
    bad = __any_sync(0xffffffffu, bad);
    if ((tid & 31) == 0) red[warp] = bad ? INFINITY : most;
    __syncthreads();
    if (!busy) return;
    for (int i = 0; i < each; ++i) most = fmaxf(most, red[own * each + i]);
    bad = most == INFINITY;
    int e = most > 0.f && !bad ? ilogbf(most) : 0;     // 2^e <= most
    e = min(max(14 - e, -113), 120);
    const float up = ldexpf(1.f, e);                   // (most below 2^-106 keeps fewer bits)
    if (lane == 0) back[own] = bad ? NAN : ldexpf(1.f, -e);
#pragma unroll 4
    for (int k = 4 * lane; k < units * kUnit; k += step) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (k < a.k && !bad) load_x4<T>(a, r, k, v);
        uint32_t h[PARTS][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float v0 = v[2 * i] * up, v1 = v[2 * i + 1] * up;
            const __half2 near = __floats2half2_rn(v0, v1);
            h[0][i] = *reinterpret_cast<const uint32_t *>(&near);
            if (PARTS == 2) {
                const __half2 left = __floats2half2_rn(v0 - __low2float(near), v1 - __high2float(near));
                h[PARTS - 1][i] = *reinterpret_cast<const uint32_t *>(&left);
            }
        }
        const int quarter = k / 32, s = k % 32 / 16, t = k % 16 / 4;
#pragma unroll
        for (int p = 0; p < PARTS; ++p) frags[((quarter * cols + col + own * PARTS + p) * 4 + t) * 2 + s] = make_uint2(h[p][0], h[p][1]);
    }
}
__device__ __forceinline__ void prepare_rows(const XArgs &a, int first, int rows, uint2 *frags, int cols, int col, int units, float *back, float *red) {
    if (a.dtype == TALKER_DTYPE_BF16) prepare_rows<__nv_bfloat16, 1>(a, first, rows, frags, cols, col, units, back, red);
    else if (a.dtype == TALKER_DTYPE_F32) prepare_rows<float, 2>(a, first, rows, frags, cols, col, units, back, red);
    else prepare_rows<__nv_fp8_storage_t, 2>(a, first, rows, frags, cols, col, units, back, red);
}

// How the columns of all rows are taken: in `passes` over the weights, `cols` columns each (the last may have fewer).
struct Columns {
    int passes, cols, parts;   // parts: columns of a row
};

// A CTA per row, for calls whose own CTAs would take too long over it.
constexpr int kRowThreads = 512;
__global__ void __launch_bounds__(kRowThreads) k_w4_rows(const XArgs a, uint2 *frags, float *back, int units, const Columns c) {
    __shared__ float red[kRowThreads / 32];
    const int r = blockIdx.x, pass = r * c.parts / c.cols, col = r * c.parts % c.cols;
    prepare_rows(a, r, 1, frags + (size_t)pass * units * 4 * c.cols * 8, c.cols, col, units, back + r, red);
    pdl_launch_dependents();
}

// ---- the product

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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
__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
// (In their place: what they read arrives by copies that the compiler does not see.)
__device__ __forceinline__ uint4 read16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t read4(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t read2(uint32_t at) {
    unsigned short v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
    return v;
}

constexpr int kWarps = 16, kThreads = kWarps * 32;
constexpr int kMultiprocessors = 152, kMostShared = 227 * 1024;
struct MatmulArgs {
    const unsigned char *tiles;
    Sizes s;
    XArgs x;
    const uint4 *frags;       // null: the CTAs prepare the rows themselves
    const float *back;
    float4 *partial;          // [pass][tile][column tile][lane]: sums of the inputs so far, where they do not fit at once
    const void *res;
    void *out;
    long long res_row, out_row;
    int n, rows;
    Columns c;
    int k_parts;              // warps that share a tile
    int units_at_once;        // of x in shared memory
    int fixed;                // bytes of shared memory before x
    bool zeros, gated, bf16;
};

// A warp's ring of records that are on their way: RT tiles' of a unit a slot, 68 KB in flight a multiprocessor.
constexpr int ring_depth(int rt) { return rt == 1 ? 4 : 2; }
constexpr int fixed_bytes(int nt, int rt, int record) {   // the rings, the sums of one of a warp's tiles, the rows' factors
    return kWarps * (ring_depth(rt) + 1) * rt * record + kWarps * nt * 512 + 1024;
}
static_assert((kMostShared - fixed_bytes(4, 2, kUnitBytes + 4 * 48)) / (32 * 256) >= 8, "room for 8 units of x");

// Persistent CTAs, one a multiprocessor, over groups of row tiles. x lies in shared memory as fragments (all of it, or so many
// units at a time); records come through rings of asynchronous copies, a ring a warp, so that no warp waits for
// another. In a round the warps take kWarps / k_parts tiles (RT of them at once a warp: one fragment of x then serves two
// tiles), k_parts warps share a tile's units, and their sums meet in shared memory, always in the same order. A group's sum
// is added to the total times its scale.
template <int NT, int NG>
__global__ void __launch_bounds__(kThreads, 1) k_w4_matmul(const MatmulArgs a) {
    constexpr int RT = NT >= 3 ? 2 : 1, kDepth = ring_depth(RT), kSlots = kDepth + 1;
    extern __shared__ uint4 smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int units = a.s.units, record = a.s.record, pass = blockIdx.y, parts = a.c.parts;
    const int cols = min(a.c.cols, a.rows * parts - pass * a.c.cols);
    const int slot_bytes = RT * record;
    float4 *sums = reinterpret_cast<float4 *>(smem) + kWarps * kSlots * slot_bytes / 16;
    float *back = reinterpret_cast<float *>(sums + kWarps * NT * 32);   // 32 rows at most, and room for a reduction
    uint4 *xs = smem + a.fixed / 16;
    const int k_part = warp % a.k_parts, slot = warp / a.k_parts, per_round = kWarps / a.k_parts;
    const int groups_of_tiles = (a.s.tiles + RT - 1) / RT;
    const int rounds = (groups_of_tiles + gridDim.x * per_round - 1) / (gridDim.x * per_round);
    // tile group of this warp in a round: neighbours read neighbouring memory
    auto group_of = [&](int round) { return (round * per_round + slot) * (int)gridDim.x + (int)blockIdx.x; };
    const uint32_t mine = smem_u32(smem) + warp * kSlots * slot_bytes;
    const bool extra = lane < (record - kUnitBytes) / 16;

    int first = 0, last = 0, steps = 0;      // the units at hand, and a warp's steps a round
    int at_round = 0, at_unit = 0, end_unit = 0, to_slot = 0;   // of the next copy
    const unsigned char *src = nullptr;
    int second = 0;                          // the other tile's record, from src
    auto begin = [&]() {
        const int tg = group_of(at_round);
        at_unit = first + k_part;
        end_unit = at_round < rounds && tg < groups_of_tiles ? last : 0;
        src = a.tiles + ((size_t)min(tg, groups_of_tiles - 1) * RT * units + at_unit) * record + lane * 16;
        if (RT == 2) second = tg * 2 + 1 < a.s.tiles ? units * record : 0;
    };
    auto copy_next = [&]() {
        if (at_unit < end_unit) {
            const uint32_t to = mine + to_slot * slot_bytes + lane * 16;
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const unsigned char *from = src + (i ? second : 0);
                copy16(to + i * record, from);
                copy16(to + i * record + 512, from + 512);
                if (extra) copy16(to + i * record + 1024, from + 1024);
            }
        }
        src += a.k_parts * record;
        at_unit += a.k_parts;
        if (at_unit - k_part >= first + steps * a.k_parts) ++at_round, begin();
        if (++to_slot == kSlots) to_slot = 0;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    for (first = 0; first < units; first = last) {
        last = min(first + a.units_at_once, units);
        steps = (last - first + a.k_parts - 1) / a.k_parts;
        if (first > 0) {   // the copies before are done and read, and so is x
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncthreads();
        }
        if (a.frags == nullptr) {
            at_round = to_slot = 0;
            begin();
            for (int i = 0; i < kDepth; ++i) copy_next();   // (codes do not wait for x)
            prepare_rows(a.x, 0, a.rows, reinterpret_cast<uint2 *>(xs), cols, 0, units, back, back + 64);
        } else {
            at_round = to_slot = 0;
            begin();
            for (int i = 0; i < kDepth; ++i) copy_next();
            if (first == 0) {
                pdl_wait();
                if (tid < cols / parts) back[tid] = a.back[pass * a.c.cols / parts + tid];
            }
            const uint4 *from = a.frags + ((size_t)pass * units + first) * 4 * a.c.cols * 4;
            const int n = (last - first) * 4 * cols * 4;
            if (cols == a.c.cols) {
#pragma unroll 8
                for (int i = tid; i < n; i += kThreads) xs[i] = from[i];
            } else {
                for (int i = tid; i < n; i += kThreads) {
                    const int quarter = i / (cols * 4);
                    xs[i] = from[quarter * a.c.cols * 4 + i - quarter * cols * 4];
                }
            }
        }
        __syncthreads();
        int from_col[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) from_col[i] = min(i * 8 + g, cols - 1) * 4 + t;   // (columns past the last are not looked at)
        int from_slot = 0;
        for (int round = 0; round < rounds; ++round) {
            const int end = group_of(round) < groups_of_tiles ? last : 0;
            float total[RT][NT][4];
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) total[r][i][j] = 0.f;
            int unit = first + k_part;
            const uint4 *x = xs + k_part * 16 * cols;
            for (int step = 0; step < steps; ++step, unit += a.k_parts, x += a.k_parts * 16 * cols) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
                __syncwarp();   // (other lanes' copies too; and the slot before this one has been read by all)
                copy_next();    // (into that one)
                const uint32_t at = mine + from_slot * slot_bytes;
                if (++from_slot == kSlots) from_slot = 0;
                if (unit >= end) continue;
                uint4 w[RT][2];
#pragma unroll
                for (int r = 0; r < RT; ++r) w[r][0] = read16(at + r * record + lane * 16), w[r][1] = read16(at + r * record + 512 + lane * 16);
                float c[RT][NT][4];
                Zero z0[RT], z1[RT];
#pragma unroll
                for (int q = 0; q < 4; ++q) {   // 32 inputs
                    if (q * NG % 4 == 0) {
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            uint32_t z = 0x0808;
                            if (a.zeros) z = read2(at + r * record + kUnitBytes + 32 * NG + q * NG / 4 * 16 + g * 2);
                            z0[r] = zero_of(z & 15), z1[r] = zero_of(z >> 8);
                        }
                    }
                    uint4 b[NT];
#pragma unroll
                    for (int i = 0; i < NT; ++i) b[i] = x[q * cols * 4 + from_col[i]];
#pragma unroll
                    for (int r = 0; r < RT; ++r)
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            const uint4 ww = w[r][q / 2];
                            const uint32_t v = q % 2 ? (s ? ww.w : ww.z) : (s ? ww.y : ww.x), v8 = v >> 8;
                            const uint32_t a0 = centred(v, z0[r]), a1 = centred(v8, z1[r]), a2 = centred16(v, z0[r]), a3 = centred16(v8, z1[r]);
#pragma unroll
                            for (int i = 0; i < NT; ++i) {
                                if (s == 0 && q * NG % 4 == 0) mma_f16_first(c[r][i], a0, a1, a2, a3, b[i].x, b[i].y);
                                else mma_f16(c[r][i], a0, a1, a2, a3, s ? b[i].z : b[i].x, s ? b[i].w : b[i].y);
                            }
                        }
                    if ((q + 1) * NG % 4 == 0) {
#pragma unroll
                        for (int r = 0; r < RT; ++r) {
                            const uint32_t d = read4(at + r * record + kUnitBytes + q * NG / 4 * 32 + g * 4);
                            const float d0 = __half2float(__ushort_as_half((unsigned short)d)), d1 = __half2float(__ushort_as_half((unsigned short)(d >> 16)));
#pragma unroll
                            for (int i = 0; i < NT; ++i) {
                                total[r][i][0] = fmaf(d0, c[r][i][0], total[r][i][0]), total[r][i][1] = fmaf(d0, c[r][i][1], total[r][i][1]);
                                total[r][i][2] = fmaf(d1, c[r][i][2], total[r][i][2]), total[r][i][3] = fmaf(d1, c[r][i][3], total[r][i][3]);
                            }
                        }
                    }
                }
            }
            // the round's sums: an item is a lane's part of a tile's result, rows g and g + 8 of two columns
#pragma unroll
            for (int r = 0; r < RT; ++r) {
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    sums[(warp * NT + i) * 32 + lane] = make_float4(total[r][i][0], total[r][i][1], total[r][i][2], total[r][i][3]);
                __syncthreads();
                for (int item = tid; item < per_round * NT * 32; item += kThreads) {
                    const int l = item & 31, i = item / 32 % NT, sl = item / (NT * 32);
                    const int tile = ((round * per_round + sl) * (int)gridDim.x + (int)blockIdx.x) * RT + r, col = i * 8 + 2 * (l & 3);
                    if (tile >= a.s.tiles || col >= cols) continue;
                    float v[4] = {0.f, 0.f, 0.f, 0.f};
                    for (int k = 0; k < a.k_parts; ++k) {
                        const float4 p = sums[((sl * a.k_parts + k) * NT + i) * 32 + l];
                        v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
                    }
                    float4 *partial = a.partial + (((size_t)pass * a.s.tiles + tile) * NT + i) * 32 + l;   // (the same thread's every time)
                    if (first > 0) {
                        const float4 p = *partial;
                        v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w;
                    }
                    if (last < units) {
                        *partial = make_float4(v[0], v[1], v[2], v[3]);
                        continue;
                    }
                    const int row0 = a.gated ? tile * 8 + (l >> 2) : tile * 16 + (l >> 2);
                    if (parts == 2) v[0] += v[1], v[2] += v[3];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (col + e >= cols || (e == 1 && parts == 2)) continue;
                        const int own = parts == 2 ? col / 2 : col + e, x_row = pass * a.c.cols / parts + own;
                        const float up = back[own], y0 = v[e] * up, y1 = v[2 + e] * up;
                        for (int half = 0; half < (a.gated ? 1 : 2); ++half) {
                            const int row = row0 + 8 * half;
                            if (row >= a.n) continue;
                            float y = a.gated ? y0 / (1.f + expf(-y0)) * y1 : half ? y1 : y0;
                            if (a.bf16) {
                                if (a.res) y += Elem<__nv_bfloat16>::load(static_cast<const __nv_bfloat16 *>(a.res) + x_row * a.res_row, row);
                                Elem<__nv_bfloat16>::store(static_cast<__nv_bfloat16 *>(a.out) + x_row * a.out_row, row, y);
                            } else {
                                if (a.res) y += static_cast<const float *>(a.res)[x_row * a.res_row + row];
                                static_cast<float *>(a.out)[x_row * a.out_row + row] = y;
                            }
                        }
                    }
                }
                __syncthreads();
            }
        }
    }
}

constexpr int kOwnRows = 4, kOwnValues = 16384;   // of x: up to so many the CTAs prepare themselves

// How a call runs.
struct Plan {
    Columns c;
    int nt, k_parts, ctas, units_at_once, fixed;
    bool own;
    size_t back_at, partial_at, bytes;   // of the scratch
};
Plan plan_of(const Sizes &s, int k, int x_dtype, int rows) {
    Plan p{};
    p.c.parts = x_dtype == TALKER_DTYPE_BF16 ? 1 : 2;
    const long long columns = (long long)rows * p.c.parts, col_tiles = (columns + 7) / 8;
    p.c.passes = (int)((col_tiles + 3) / 4);
    p.nt = (int)((col_tiles + p.c.passes - 1) / p.c.passes);
    p.c.cols = (int)std::min<long long>(columns, p.nt * 8);
    const int rt = p.nt >= 3 ? 2 : 1;
    p.fixed = fixed_bytes(p.nt, rt, s.record);
    const int room = (kMostShared - p.fixed) / (p.c.cols * 256);   // units of x, 8 or more
    p.own = rows <= kOwnRows && (long long)rows * k <= kOwnValues && s.units <= room;
    const int blocks = (s.units + room - 1) / room;
    p.units_at_once = (s.units + blocks - 1) / blocks;
    // the fewest steps: rounds of tiles times a warp's units, and a round's end, which takes about as long as one
    const int groups = (s.tiles + rt - 1) / rt;
    p.ctas = std::min(groups, std::max(1, kMultiprocessors / std::min(p.c.passes, kMultiprocessors)));
    long long best = 1ll << 62;
    for (int k = 1; k <= kWarps; k *= 2) {
        const long long rounds = (groups + (long long)p.ctas * (kWarps / k) - 1) / ((long long)p.ctas * (kWarps / k));
        const long long cost = rounds * ((p.units_at_once + k - 1) / k + 1);
        if (cost < best) best = cost, p.k_parts = k;
    }
    p.back_at = p.own ? 0 : (size_t)p.c.passes * s.units * 16 * p.c.cols * sizeof(uint4);
    p.partial_at = p.own ? 0 : (p.back_at + (size_t)rows * 4 + 15) / 16 * 16;
    p.bytes = p.partial_at + (blocks > 1 ? (size_t)p.c.passes * s.tiles * p.nt * 32 * sizeof(float4) : 0);
    return p;
}

template <int NT, int NG>
cudaError_t launch_one(const MatmulArgs &a, const Plan &p, cudaStream_t st) {
    static std::atomic<unsigned long long> raised{0};   // devices whose limit of shared memory is raised
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    const unsigned long long bit = device < 64 ? 1ull << device : 0;
    if (e == cudaSuccess && !(raised.load() & bit)) {
        e = cudaFuncSetAttribute(k_w4_matmul<NT, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
        if (e == cudaSuccess) raised |= bit;
    }
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(p.ctas, p.c.passes);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = p.fixed + (size_t)p.units_at_once * p.c.cols * 256;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.own ? 0 : 1;
    return cudaLaunchKernelEx(&cfg, k_w4_matmul<NT, NG>, a);
}
template <int NT>
cudaError_t launch_tiles(const MatmulArgs &a, const Plan &p, cudaStream_t st) {
    return a.s.groups == 1 ? launch_one<NT, 1>(a, p, st) : a.s.groups == 2 ? launch_one<NT, 2>(a, p, st) : launch_one<NT, 4>(a, p, st);
}
cudaError_t launch_matmul(const MatmulArgs &a, const Plan &p, char *scratch, cudaStream_t st) {
    if (!p.own) {
        k_w4_rows<<<a.rows, kRowThreads, 0, st>>>(a.x, reinterpret_cast<uint2 *>(scratch), reinterpret_cast<float *>(scratch + p.back_at), a.s.units, p.c);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return p.nt == 1 ? launch_tiles<1>(a, p, st) : p.nt == 2 ? launch_tiles<2>(a, p, st) : p.nt == 3 ? launch_tiles<3>(a, p, st) : launch_tiles<4>(a, p, st);
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
    const long long words = (long long)a.s.tiles * a.s.units * (kUnitBytes / 4), n = (long long)a.s.tiles * a.s.units * a.s.groups * 16;
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
    return matrix_ok(w) && rows > 0 && rows <= kMostRows ? plan_of(sizes_of(w), w->k, x_dtype, rows).bytes : 0;
}

talker_status talker_w4_matmul(const talker_w4 *w, const void *x, int x_dtype, int64_t x_row, const float *x_scales,
                               int x_block, int rows, const void *residual, int64_t res_row, void *out, int out_dtype,
                               int64_t out_row, void *scratch, size_t scratch_bytes, void *cuda_stream) {
    if (!packed_ok(w) || !x || !out || rows < 0 || rows > kMostRows) return TALKER_EINVAL;
    const bool f8 = x_dtype == TALKER_DTYPE_E4M3;
    if ((!f8 && x_dtype != TALKER_DTYPE_BF16 && x_dtype != TALKER_DTYPE_F32) || (out_dtype != TALKER_DTYPE_F32 && out_dtype != TALKER_DTYPE_BF16)) return TALKER_EINVAL;
    if (f8 && (!x_scales || !aligned(x_scales, 4) || (x_block != 0 && x_block != 32 && x_block != 64 && x_block != 128))) return TALKER_EINVAL;
    if (!aligned(x, size_of(x_dtype)) || !aligned(out, size_of(out_dtype)) || !aligned(residual, size_of(out_dtype))) return TALKER_EINVAL;
    if (rows > 1 && (out_row < w->n || (residual == out && residual && res_row != out_row))) return TALKER_EINVAL;
    if (rows == 0) return TALKER_OK;
    const Sizes s = sizes_of(w);
    const Plan p = plan_of(s, w->k, x_dtype, rows);
    if (p.bytes > 0 && (!scratch || scratch_bytes < p.bytes || !aligned(scratch, 16))) return TALKER_EINVAL;
    char *base = static_cast<char *>(scratch);
    MatmulArgs a{};
    a.tiles = static_cast<const unsigned char *>(w->tiles), a.s = s;
    a.x = {x, x_scales, x_row, x_dtype, x_block, w->k, rows, aligned(x, 4 * size_of(x_dtype)) && (rows == 1 || x_row % 4 == 0)};
    if (!p.own) a.frags = reinterpret_cast<const uint4 *>(base), a.back = reinterpret_cast<const float *>(base + p.back_at);
    a.partial = reinterpret_cast<float4 *>(base + p.partial_at);
    a.res = residual, a.out = out, a.res_row = res_row, a.out_row = out_row;
    a.n = w->n, a.rows = rows, a.c = p.c;
    a.k_parts = p.k_parts, a.units_at_once = p.units_at_once, a.fixed = p.fixed;
    a.zeros = w->zeros != 0, a.gated = w->gated != 0, a.bf16 = out_dtype == TALKER_DTYPE_BF16;
    const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = launch_matmul(a, p, base, st);
    if (e == cudaSuccess) return TALKER_OK;
    cudaGetLastError();
    return TALKER_ECUDA;
}

}  // extern "C"
