// Products with 4-bit weights in groups (include/talker_layer.h).
#include <cuda_fp8.h>

#include <algorithm>
#include <atomic>

#include "rows.cuh"
#include "talker_layer.h"
#include "w4_ring.cuh"

using namespace talker_dev;
using namespace talker_k;

namespace {

constexpr int kUnit = 128;              // inputs: what k is padded to, and what one warp takes at a time
constexpr int kUnitBytes = 16 * kUnit / 2;
constexpr int kMostRows = 1 << 16;

constexpr int kSpan = 32;               // row tiles whose records of a unit are neighbours

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
// Where a tile's unit lies: a span's records of one unit are neighbours.
__host__ __device__ inline size_t record_at(const Sizes &s, int tile, int unit) {
    const int span = tile / kSpan, first = span * kSpan, of_span = s.tiles - first < kSpan ? s.tiles - first : kSpan;
    return ((size_t)first * s.units + (size_t)unit * of_span + (tile - first)) * s.record;
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
    reinterpret_cast<uint32_t *>(a.tiles + record_at(a.s, tile, own / 2) + own % 2 * 512)[i & 127] = w;
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
    unsigned char *record = a.tiles + record_at(a.s, tile, group / a.s.groups) + kUnitBytes;
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

// How the columns of all rows are taken: in `passes` over the weights, `cols` columns each (the last may have fewer).
struct Columns {
    int passes, cols, parts;   // parts: columns of a row
};

// A CTA per row: its columns to frags, and what undoes the scaling to back. A row's values are read once where eight quads
// a thread hold them (k <= 16384). Bound by latency (6.8 us by itself for one row of 8192, of which the product's CTAs, which
// may begin at once and bring weights in until they need this, hide all but 3).
constexpr int kRowThreads = 512, kHeld = 8;
template <typename T, int PARTS>
__device__ __forceinline__ void prepare_row(const XArgs &a, int r, uint2 *frags, int cols, int col, int units, float *back) {
    __shared__ float red[kRowThreads / 32];
    const int tid = threadIdx.x;
    float held[kHeld][4];
    float most = 0.f;
    bool bad = false;
    auto see = [&](const float (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            bad |= !(fabsf(v[i]) < INFINITY);
            most = fmaxf(most, fabsf(v[i]));
        }
    };
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        const int k = 4 * (tid + j * kRowThreads);
#pragma unroll
        for (int i = 0; i < 4; ++i) held[j][i] = 0.f;
        if (k < a.k) load_x4<T>(a, r, k, held[j]);
    }
#pragma unroll
    for (int j = 0; j < kHeld; ++j) see(held[j]);
    for (int k = 4 * (tid + kHeld * kRowThreads); k < a.k; k += 4 * kRowThreads) {
        float v[4];
        load_x4<T>(a, r, k, v);
        see(v);
    }
    most = warp_max(most);
    if ((tid & 31) == 0) red[tid >> 5] = most;
    bad = __syncthreads_or(bad);
    most = warp_max(red[tid & 15]);
    int e = most > 0.f && !bad ? ilogbf(most) : 0;     // 2^e <= most
    e = min(max(14 - e, -113), 120);
    const float up = ldexpf(1.f, e);                   // (most below 2^-106 keeps fewer bits)
    if (tid == 0) *back = bad ? NAN : ldexpf(1.f, -e);
    auto store = [&](int k, const float (&v)[4]) {
        uint32_t h[PARTS][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float v0 = bad ? 0.f : v[2 * i] * up, v1 = bad ? 0.f : v[2 * i + 1] * up;
            const __half2 near = __floats2half2_rn(v0, v1);
            h[0][i] = *reinterpret_cast<const uint32_t *>(&near);
            if (PARTS == 2) {
                const __half2 left = __floats2half2_rn(v0 - __low2float(near), v1 - __high2float(near));
                h[PARTS - 1][i] = *reinterpret_cast<const uint32_t *>(&left);
            }
        }
        const int quarter = k / 32, s = k % 32 / 16, t = k % 16 / 4;
#pragma unroll
        for (int p = 0; p < PARTS; ++p) frags[((quarter * cols + col + p) * 4 + t) * 2 + s] = make_uint2(h[p][0], h[p][1]);
    };
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        const int k = 4 * (tid + j * kRowThreads);
        if (k < units * kUnit) store(k, held[j]);
    }
    for (int k = 4 * (tid + kHeld * kRowThreads); k < units * kUnit; k += 4 * kRowThreads) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (k < a.k) load_x4<T>(a, r, k, v);
        store(k, v);
    }
}
__global__ void __launch_bounds__(kRowThreads) k_w4_rows(const XArgs a, uint2 *frags, float *back, int units, const Columns c) {
    pdl_launch_dependents();
    const int r = blockIdx.x, pass = r * c.parts / c.cols, col = r * c.parts % c.cols;
    frags += (size_t)pass * units * 4 * c.cols * 8;
    if (a.dtype == TALKER_DTYPE_BF16) prepare_row<__nv_bfloat16, 1>(a, r, frags, c.cols, col, units, back + r);
    else if (a.dtype == TALKER_DTYPE_F32) prepare_row<float, 2>(a, r, frags, c.cols, col, units, back + r);
    else prepare_row<__nv_fp8_storage_t, 2>(a, r, frags, c.cols, col, units, back + r);
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
// Codes of one word as the operand's registers, by a widely published method (an integer under an fp16 power of two): fields
// 0 and 4 of v (or of v >> 8) under 1024, whose last place is 1, are 1024 + c; fields 1 and 5 are 1024 + 16 c. Taking off
// 1024 + z, or 64 + z after a sixteenth, leaves c - z, exactly.
struct Zero {
    uint32_t a, b;   // -(1024 + z) and -(64 + z), twice each
};
__device__ __forceinline__ Zero zero_of(uint32_t z) { return {(0xe400u | z) * 0x10001u, (0xd400u | z << 4) * 0x10001u}; }
__device__ __forceinline__ uint32_t centred(uint32_t v, Zero z) {
    uint32_t y;
    asm("{.reg .b32 t;\n\t"
        "lop3.b32 t, %1, 0x000f000f, 0x64006400, 0xea;\n\t"   // (v & ..) | ..: one instruction, two as the compiler makes it
        "add.rn.f16x2 %0, t, %2;}"
        : "=r"(y) : "r"(v), "r"(z.a));
    return y;
}
__device__ __forceinline__ uint32_t centred16(uint32_t v, Zero z) {
    uint32_t y;
    asm("{.reg .b32 t, s;\n\t"
        "lop3.b32 t, %1, 0x00f000f0, 0x64006400, 0xea;\n\t"
        "mov.b32 s, 0x2c002c00;\n\t"
        "fma.rn.f16x2 %0, t, s, %2;}"
        : "=r"(y) : "r"(v), "r"(z.b));
    return y;
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

constexpr int kMultiprocessors = 152, kMostShared = 227 * 1024;
constexpr int kTiles = 2;                        // of a warp: one fragment of x, and one turn of the loop, serve both
constexpr int kSlots = kW4Slots;                 // 135 KB a multiprocessor
// Warps that multiply (one more makes the copies). With three or four column tiles a warp needs more registers than
// sixteen leave it, and has enough to do for the tensor cores by itself.
constexpr int warps_of(int nt) { return nt <= 2 ? 16 : 8; }
constexpr int tiles_of(int nt) { return warps_of(nt) * kTiles; }   // of a step: a span, or half of one
static_assert(kSpan % tiles_of(1) == 0 && kSpan % tiles_of(4) == 0, "steps within spans");

// A product is `all` steps, in the order of passes, blocks of tiles_of(nt) row tiles, and units: a step is a unit of a block's tiles
// for a pass's columns. CTA c takes the steps from start(c) to start(c + 1), so all have the same number, give or take one. A
// stretch of steps of one pass and block is a segment, whose sums go to the place c + pass * blocks + block.
struct Steps {
    long long all;
    int ctas, units;
    __host__ __device__ long long start(int c) const { return all * c / ctas; }
    __host__ __device__ int cta_of(long long step) const { return (int)(((step + 1) * ctas - 1) / all); }
};
struct MatmulArgs {
    const unsigned char *tiles;
    Sizes s;
    Steps steps;
    XArgs x;
    const uint4 *frags;
    const float *back;              // [row]: what undoes the rows' scaling
    float4 *sums;             // [place][warp][tile][column tile][lane]
    const void *res;
    void *out;
    long long res_row, out_row;
    int n, blocks;
    Columns c;
    int rows, x_bytes;        // of x in a slot
    bool zeros, gated, bf16;
};

// The phase of `parity` of a barrier, waited for up to a second: false if it did not come.
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
    return true;
}

// One CTA a multiprocessor, all with the same number of steps. A thread of its own brings each step into a ring of slots by
// two bulk copies: a span's records of a unit lie together, and so do its fragments of x. Warps run on their own, up to a
// ring's length apart. Nothing is joined in here: a segment's sums go to memory, and the kernel after adds them up. A group
// of inputs' sum is added to the total times its scale. A copy that does not arrive within a second makes its warps' sums NaN
// from there on.
// Few rows are bound by the instructions that make codes operands, nine for the four registers of an MMA. 24576 x 8192,
// groups of 128, one row: 26 us for 104 MB (59% of the copy rate, 59% of the issue slots, a quarter of the tensor cores'
// cycles), 30 with the kernels around it; 8 bf16 rows 29, 16 36, 32 53 (MMAs and their operands), 64 in two passes 94. Equal
// steps: with whole tiles to a CTA the last ones run alone (49 us); a ring and warps of their own
// instead of a barrier a step: 36; codes as whole numbers under a scale a group instead of scaled ones: 31. Codes that keep
// their offset of 8, taken off the sum: an instruction less for two, but errors of 1e-6 instead of 9e-8.
template <int NT, int NG>
__global__ void __launch_bounds__((warps_of(NT) + 1) * 32, 1) k_w4_matmul(const MatmulArgs a) {
    constexpr int kWarps = warps_of(NT), kBlock = tiles_of(NT);
    extern __shared__ uint4 smem[];
    __shared__ uint64_t full[kSlots], empty[kSlots];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int units = a.s.units, record = a.s.record, parts = a.c.parts;
    const int slot_bytes = kBlock * record + a.x_bytes;
    const uint32_t slots = smem_u32(smem);
    const long long first = a.steps.start(blockIdx.x);
    const int count = (int)(a.steps.start(blockIdx.x + 1) - first);
    // where a step is: place = pass * blocks + block, the block's tiles and the first of them
    struct At {
        int place, unit, pass, first, tiles;
    };
    auto enter = [&](At &p) {
        p.pass = p.place / a.blocks, p.first = (p.place - p.pass * a.blocks) * kBlock;
        p.tiles = min(a.s.tiles - p.first, kBlock);
    };
    auto next = [&](At &p) {
        if (++p.unit < units) return;
        p.unit = 0, ++p.place;
        enter(p);
    };
    At at;
    at.place = (int)(first / units), at.unit = (int)(first - (long long)at.place * units);
    enter(at);
    auto copy_codes = [&](const At &p, int slot) {
        const uint32_t bytes = p.tiles * record;
        mbar_arrive_expect_tx(&full[slot], bytes + a.x_bytes);
        bulk_g2s(reinterpret_cast<char *>(smem) + slot * slot_bytes, a.tiles + record_at(a.s, p.first, p.unit), bytes, &full[slot]);
    };
    auto copy_x = [&](const At &p, int slot) {   // (also columns past the last pass's: they are not looked at)
        bulk_g2s(reinterpret_cast<char *>(smem) + slot * slot_bytes + kBlock * record, a.frags + ((size_t)p.pass * units + p.unit) * 16 * a.c.cols,
                 a.x_bytes, &full[slot]);
    };
    At ahead = at;
    if (tid == kWarps * 32) {
        for (int i = 0; i < kSlots; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], kWarps);
        fence_barrier_init();
        fence_proxy_async();
        // codes do not wait for the kernel before, x does
        for (int i = 0; i < min(kSlots, count); ++i, next(ahead)) copy_codes(ahead, i);
    }
    __syncthreads();
    if (warp == kWarps) {
        if (lane != 0) return;
        pdl_wait();
        At x = at;
        for (int i = 0; i < min(kSlots, count); ++i, next(x)) copy_x(x, i);
        int i = kSlots;
        for (; i < count; ++i, next(ahead)) {
            if (!wait_for(&empty[w4_slot(i)], w4_empty_parity(i))) break;
            copy_codes(ahead, w4_slot(i));
            copy_x(ahead, w4_slot(i));
        }
        for (int k = max(0, min(i, count) - kSlots); k < min(i, count); ++k) wait_for(&full[w4_slot(k)], w4_full_parity(k));   // (nothing is on its way when the CTA ends)
        return;
    }

    const uint32_t mine = warp * kTiles * record + lane * 16;   // in a slot
    W4Ring ring;
    float total[kTiles][NT][4];
    bool fresh = true;
    int from_col[NT];
    for (int step = 0; step < count; ++step) {
        const int slot = w4_slot(step), tiles = at.tiles - warp * kTiles;   // tiles of this warp
        if (fresh) {
            fresh = false;
            const int cols = min(a.c.cols, a.rows * parts - at.pass * a.c.cols);
#pragma unroll
            for (int r = 0; r < kTiles; ++r)
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) total[r][i][j] = ring.lost ? NAN : 0.f;
#pragma unroll
            for (int i = 0; i < NT; ++i) from_col[i] = (min(i * 8 + g, cols - 1) * 4 + t) * 16;   // (columns past the last are not looked at)
        }
        if (ring.waits()) {
            ring.waited(__all_sync(0xffffffffu, wait_for(&full[slot], w4_full_parity(step))));   // (a warp's lanes agree)
            if (ring.lost) {
#pragma unroll
                for (int r = 0; r < kTiles; ++r)
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) total[r][i][j] = NAN;
            }
        }
        if (tiles > 0 && ring.reads()) {
            const uint32_t now = slots + slot * slot_bytes;
            const uint32_t x = now + kBlock * record, tail = now + mine - lane * 16 + kUnitBytes;   // scales, then zeros
            uint4 w[kTiles][2];
#pragma unroll
            for (int r = 0; r < kTiles; ++r) w[r][0] = read16(now + mine + r * record), w[r][1] = read16(now + mine + r * record + 512);
            float c[kTiles][NT][4];
            Zero z0[kTiles], z1[kTiles];
#pragma unroll
            for (int q = 0; q < 4; ++q) {   // 32 inputs
                if (q * NG % 4 == 0) {
#pragma unroll
                    for (int r = 0; r < kTiles; ++r) {
                        if (a.zeros) {
                            const uint32_t z = read2(tail + r * record + 32 * NG + q * NG / 4 * 16 + g * 2);
                            z0[r] = zero_of(z & 15), z1[r] = zero_of(z >> 8 & 15);
                        } else {
                            z0[r] = z1[r] = zero_of(8);
                        }
                    }
                }
                uint4 b[NT];
#pragma unroll
                for (int i = 0; i < NT; ++i) b[i] = read16(x + q * 64 * a.c.cols + from_col[i]);
#pragma unroll
                for (int r = 0; r < kTiles; ++r)
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
                    for (int r = 0; r < kTiles; ++r) {
                        const uint32_t d = read4(tail + r * record + q * NG / 4 * 32 + g * 4);
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
        __syncwarp();
        if (lane == 0 && ring.releases()) mbar_arrive(&empty[slot]);   // (all of it has been read)
        if (step + 1 == count || at.unit + 1 == units) {   // the segment's end
            float4 *place = a.sums + ((size_t)(blockIdx.x + at.place) * kWarps + warp) * kTiles * NT * 32 + lane;
#pragma unroll
            for (int r = 0; r < kTiles; ++r)
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    if (r < tiles) place[(r * NT + i) * 32] = make_float4(total[r][i][0], total[r][i][1], total[r][i][2], total[r][i][3]);
            fresh = true;
        }
        next(at);
    }
    pdl_launch_dependents();
}

// A CTA per row tile and pass: the segments' sums in their order, and the result. A thread adds up one number of a lane's
// four: rows g (0, 1) and g + 8 (2, 3) of two columns. Where there are many segments, groups of 128 threads take a range each.
// Bound by latency: 3 to 4 us after the product. (Adding in the product, by whoever is last, needs counters that are zero
// on entry, and its chain at the end is as long.)
__global__ void __launch_bounds__(1024) k_w4_join(const MatmulArgs a, int nt) {
    __shared__ float sums[7 * 128];
    const int per = tiles_of(nt), pass = blockIdx.y, tile = blockIdx.x, place = pass * a.blocks + tile / per, parts = a.c.parts;
    const int id = threadIdx.x & 127, j = id & 3, l = id >> 2, own = threadIdx.x >> 7, ranges = blockDim.x >> 7;
    const int cols = min(a.c.cols, a.rows * parts - pass * a.c.cols);
    const int c0 = a.steps.cta_of((long long)place * a.steps.units), all = a.steps.cta_of((long long)(place + 1) * a.steps.units - 1) + 1 - c0;
    const int from = all * own / ranges, to = all * (own + 1) / ranges;
    const int row = a.gated ? tile * 8 + (l >> 2) : tile * 16 + (l >> 2) + 8 * (j >> 1);
    const size_t segment = (size_t)per * nt * 128;
    const float *at = reinterpret_cast<const float *>(a.sums) + (size_t)(c0 + place + from) * segment + (size_t)(tile % per) * nt * 128 + id;
    pdl_wait();
    for (int i = 0; i < nt; ++i, at += 128) {
        const int col = i * 8 + 2 * (l & 3) + (j & 1);
        float v = 0.f;
#pragma unroll 8
        for (int c = 0; c < to - from; ++c) v += at[c * segment];
        if (ranges > 1) {
            __syncthreads();
            if (own > 0) sums[(own - 1) * 128 + id] = v;
            __syncthreads();
            if (own > 0) continue;
            for (int k = 1; k < ranges; ++k) v += sums[(k - 1) * 128 + id];
        }
        if (parts == 2) v += __shfl_xor_sync(0xffffffffu, v, 1);
        const int x_row = pass * a.c.cols / parts + col / parts;
        float y = v * (col < cols ? a.back[x_row] : 0.f);
        const float up = __shfl_xor_sync(0xffffffffu, y, 2);   // (U's row of a gated matrix)
        if (a.gated) y = y / (1.f + expf(-y)) * up;
        if (row >= a.n || col >= cols || (parts == 2 && j & 1) || (a.gated && j & 2)) continue;
        if (a.bf16) {
            if (a.res) y += Elem<__nv_bfloat16>::load(static_cast<const __nv_bfloat16 *>(a.res) + x_row * a.res_row, row);
            Elem<__nv_bfloat16>::store(static_cast<__nv_bfloat16 *>(a.out) + x_row * a.out_row, row, y);
        } else {
            if (a.res) y += static_cast<const float *>(a.res)[x_row * a.res_row + row];
            static_cast<float *>(a.out)[x_row * a.out_row + row] = y;
        }
    }
}

// How a call runs.
struct Plan {
    Columns c;
    Steps steps;
    int nt, blocks, x_bytes, join_threads;
    size_t shared, back_at, sums_at, bytes;   // (the last three: of the scratch)
};
Plan plan_of(const Sizes &s, int x_dtype, int rows) {
    Plan p{};
    p.c.parts = x_dtype == TALKER_DTYPE_BF16 ? 1 : 2;
    const long long columns = (long long)rows * p.c.parts, col_tiles = (columns + 7) / 8;
    p.c.passes = (int)((col_tiles + 3) / 4);
    p.nt = (int)((col_tiles + p.c.passes - 1) / p.c.passes);
    p.c.cols = (int)std::min<long long>(columns, p.nt * 8);
    p.x_bytes = p.c.cols * 256;
    p.shared = (size_t)kSlots * (tiles_of(p.nt) * s.record + p.x_bytes);
    p.blocks = (s.tiles + tiles_of(p.nt) - 1) / tiles_of(p.nt);
    p.steps.units = s.units;
    p.steps.all = (long long)p.c.passes * p.blocks * s.units;
    p.steps.ctas = (int)std::min<long long>(p.steps.all, kMultiprocessors);
    const long long segments = (s.units * (long long)p.steps.ctas + p.steps.all - 1) / p.steps.all;   // of a place, about
    p.join_threads = segments <= 8 ? 128 : segments <= 16 ? 256 : segments <= 32 ? 512 : 1024;
    p.back_at = (size_t)p.c.passes * s.units * 16 * p.c.cols * sizeof(uint4);
    p.sums_at = (p.back_at + (size_t)rows * 4 + 15) / 16 * 16;
    p.bytes = p.sums_at + ((size_t)p.c.passes * p.blocks + p.steps.ctas - 1) * tiles_of(p.nt) * p.nt * 32 * sizeof(float4);
    return p;
}
// The most shared memory that a plan asks for.
static_assert(kSlots * (tiles_of(2) * (kUnitBytes + 4 * 48) + 16 * 256) <= kMostShared - 256, "slots");
static_assert(kSlots * (tiles_of(4) * (kUnitBytes + 4 * 48) + 32 * 256) <= kMostShared - 256, "slots");

// After the kernel before it on the stream, of this call: it may begin earlier and waits for what it needs.
template <typename... A>
cudaError_t launch_after(void (*kernel)(A...), dim3 grid, int threads, size_t shared, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <int NT, int NG>
cudaError_t launch_one(const MatmulArgs &a, const Plan &p, cudaStream_t st) {
    static std::atomic<unsigned long long> raised{0};   // devices whose limit of shared memory is raised
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    const unsigned long long bit = device < 64 ? 1ull << device : 0;
    if (e == cudaSuccess && !(raised.load() & bit)) {
        e = cudaFuncSetAttribute(k_w4_matmul<NT, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared - 256);
        if (e == cudaSuccess) raised |= bit;
    }
    if (e != cudaSuccess) return e;
    return launch_after(k_w4_matmul<NT, NG>, dim3(p.steps.ctas), (warps_of(NT) + 1) * 32, p.shared, st, a);
}
template <int NT>
cudaError_t launch_tiles(const MatmulArgs &a, const Plan &p, cudaStream_t st) {
    return a.s.groups == 1 ? launch_one<NT, 1>(a, p, st) : a.s.groups == 2 ? launch_one<NT, 2>(a, p, st) : launch_one<NT, 4>(a, p, st);
}
cudaError_t launch_matmul(const MatmulArgs &a, const Plan &p, char *scratch, cudaStream_t st) {
    k_w4_rows<<<a.rows, kRowThreads, 0, st>>>(a.x, reinterpret_cast<uint2 *>(scratch), reinterpret_cast<float *>(scratch + p.back_at), a.s.units, p.c);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess)
        e = p.nt == 1 ? launch_tiles<1>(a, p, st) : p.nt == 2 ? launch_tiles<2>(a, p, st) : p.nt == 3 ? launch_tiles<3>(a, p, st) : launch_tiles<4>(a, p, st);
    if (e == cudaSuccess) e = launch_after(k_w4_join, dim3(a.s.tiles, p.c.passes), p.join_threads, 0, st, a, p.nt);
    return e;
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
    return matrix_ok(w) && rows > 0 && rows <= kMostRows ? plan_of(sizes_of(w), x_dtype, rows).bytes : 0;
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
    const Plan p = plan_of(s, x_dtype, rows);
    if (!scratch || scratch_bytes < p.bytes || !aligned(scratch, 16)) return TALKER_EINVAL;
    char *base = static_cast<char *>(scratch);
    MatmulArgs a{};
    a.tiles = static_cast<const unsigned char *>(w->tiles), a.s = s, a.steps = p.steps;
    a.x = {x, x_scales, x_row, x_dtype, x_block, w->k, rows, aligned(x, 4 * size_of(x_dtype)) && (rows == 1 || x_row % 4 == 0)};
    a.frags = reinterpret_cast<const uint4 *>(base), a.back = reinterpret_cast<const float *>(base + p.back_at), a.sums = reinterpret_cast<float4 *>(base + p.sums_at);
    a.res = residual, a.out = out, a.res_row = res_row, a.out_row = out_row;
    a.n = w->n, a.blocks = p.blocks, a.c = p.c, a.rows = rows, a.x_bytes = p.x_bytes;
    a.zeros = w->zeros != 0, a.gated = w->gated != 0, a.bf16 = out_dtype == TALKER_DTYPE_BF16;
    const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = launch_matmul(a, p, base, st);
    if (e == cudaSuccess) return TALKER_OK;
    cudaGetLastError();
    return TALKER_ECUDA;
}

}  // extern "C"
