// Decode attention over the 4-bit paged cache (talker_kv4_attend).
#include <algorithm>
#include <atomic>
#include <math.h>

#include "kv4.cuh"
#include "kv4_ring.cuh"

using namespace talker_dev;

namespace talker_k {

namespace {

constexpr int kWarps = 4;
constexpr int kFewCtas = 3, kManyCtas = 4;   // CTAs a multiprocessor holds, by units (kv4_attend_shape)
// Tiles that a warp has in shared memory. 3: a page's K, its V, the next page's K ...; 2: K and V, each refilled once used.
constexpr int slots_of(int ctas) { return ctas == kManyCtas ? 2 : 3; }
constexpr int kMaxG = 8;
constexpr int kMaxGrid = 1024;            // CTAs of a launch
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTopBits = 11;              // probabilities stay below 2^11 ...
constexpr int kNewBits = 6;               // ... and the largest is brought to 2^6 when one would pass it
constexpr int kTopScale = 4;              // value scales stay below 2^4, times their block's power of two ...
constexpr int kNewScale = 2;              // ... which brings the largest to [2^2, 2^3) when one would pass it

__device__ __forceinline__ float ex2(float x) {   // relative error about 2^-22, 0 at -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = a b
__device__ __forceinline__ void mma16816_new(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// The same over 8 instead of 16.
__device__ __forceinline__ void mma1688_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%7,%7,%7,%7};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(b), "f"(0.f));
}
// (lo, hi) as an fp16 pair, rounded to nearest
__device__ __forceinline__ uint32_t pack_rn(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_half(__half lo, __half hi) {
    return (uint32_t)__half_as_ushort(lo) | ((uint32_t)__half_as_ushort(hi) << 16);
}
__device__ __forceinline__ float half_lo(uint32_t u) { return __half2float(__ushort_as_half((unsigned short)u)); }
__device__ __forceinline__ float half_hi(uint32_t u) { return __half2float(__ushort_as_half((unsigned short)(u >> 16))); }

// Two codes share a byte. As they are: its nibbles n0 and 16 n1 by an AND each, exact as fp16 subnormals
// (times 2^-24).
__device__ __forceinline__ uint32_t bytes13(uint32_t w) { return __byte_perm(w, 0, 0x4341); }
__device__ __forceinline__ uint32_t low_nibbles(uint32_t bytes) { return bytes & 0x000f000fu; }
__device__ __forceinline__ uint32_t high_nibbles(uint32_t bytes) { return bytes & 0x00f000f0u; }
// Centred: bytes 0 and 2, or 1 and 3, are raised under the fp16 exponent of 1024, and 1024 + 8 is taken off
// their low nibbles, 1024 + 136 (8 + 16 8) off the bytes n0 + 16 n1, whose product takes n0's part along (the
// other operand, or the result, takes it off again).
__device__ __forceinline__ uint32_t raised02(uint32_t w) { return __byte_perm(w, 0x64646464u, 0x4240); }
__device__ __forceinline__ uint32_t raised13(uint32_t w) { return __byte_perm(w, 0x64646464u, 0x4341); }
__device__ __forceinline__ uint32_t centred(uint32_t x, uint32_t mid) {
    uint32_t r;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(mid));
    return r;
}
__device__ __forceinline__ uint32_t centred_nibbles(uint32_t raised) { return centred(raised & 0xff0fff0fu, 0x64086408u); }
__device__ __forceinline__ uint32_t centred_bytes(uint32_t raised) { return centred(raised, 0x64886488u); }

// Transposes an 8 x 8 matrix of fp16 pairs: from row r, columns 2 c and 2 c + 1 to rows 2 c and 2 c + 1, column r.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Two numbers p = ph + pl times half `hi` of d, as two fp16 parts again: x = ph d rounded, y the rest.
struct HalfParts {
    uint32_t x, y;
};
__device__ __forceinline__ HalfParts mul_parts(uint32_t ph, uint32_t pl, uint32_t d, bool hi) {
    HalfParts r;
    asm("{.reg .b16 h0, h1; .reg .b32 t, u;\n\t"
        "mov.b32 {h0, h1}, %4;\n\t"
        "mov.b32 t, {h0, h0};\n\t"
        "mul.rn.f16x2 %0, %2, t;\n\t"
        "neg.f16x2 u, %0;\n\t"
        "fma.rn.f16x2 u, %2, t, u;\n\t"
        "fma.rn.f16x2 %1, %3, t, u;}"
        : "=&r"(r.x), "=r"(r.y) : "r"(ph), "r"(pl), "r"(hi ? d >> 16 : d));
    return r;
}
// Half i of the words of a key's scales.
__device__ __forceinline__ float scale_at(const uint32_t *w, int i) { return i & 1 ? half_hi(w[i / 2]) : half_lo(w[i / 2]); }

__device__ __forceinline__ uint32_t lds_u1(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
template <int N>
struct Words;
template <>
struct Words<4> {
    uint32_t w[4];
    __device__ __forceinline__ void load(uint32_t at) {
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
    }
};
template <>
struct Words<2> {
    uint32_t w[2];
    __device__ __forceinline__ void load(uint32_t at) {
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
    }
};
template <>
struct Words<1> {
    uint32_t w[1];
    __device__ __forceinline__ void load(uint32_t at) {
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at) : "memory");
    }
};

__device__ __forceinline__ bool bounded_wait(uint64_t *bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
    return true;
}

constexpr size_t attend_smem(int hd, int ctas) {
    return (size_t)kWarps * slots_of(ctas) * kv4_tile_bytes(hd) + (size_t)kWarps * kMaxG * hd * 4;
}

// Eight dims of a query head; vec: rows lie on 16-byte boundaries.
__device__ __forceinline__ void load_dims8(const float *p, bool vec, float (&x)[8]) {
    if (vec) {
        const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = p[i];
    }
}
__device__ __forceinline__ void load_dims8(const __nv_bfloat16 *p, bool vec, float (&x)[8]) {
    if (vec) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = bf16lo(w[i]), x[2 * i + 1] = bf16hi(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __bfloat162float(p[i]);
    }
}

// The work of a call in units of one page for every warp of a CTA: each (stream, KV head) row has
// a unit for every kWarps pages, at least one, or (one_unit) a single unit of all its pages. Rows
// lie behind one another, streams outermost, and CTA i of n takes units [i U / n, (i + 1) U / n).
__device__ __forceinline__ int checked_len(const Kv4Attend &a, int b) {
    const int len = a.lens[b];
    return len >= 0 && len <= a.c.pages_per_stream * kPage ? len : -1;
}
__device__ __forceinline__ int pages_of(int len) { return len > 0 ? (len + kPage - 1) / kPage : 0; }
__device__ __forceinline__ int units_of(const Kv4Attend &a, int len) {
    return a.one_unit ? 1 : max(1, (pages_of(len) + kWarps - 1) / kWarps);
}
// Units of one KV head of all streams, and of those before stream `upto` (one warp).
__device__ __forceinline__ long long count_units(const Kv4Attend &a, int upto, long long &before) {
    const int lane = threadIdx.x & 31;
    long long all = 0, part = 0;
    for (int b = lane; b < a.B; b += 32) {
        const int u = units_of(a, checked_len(a, b));
        all += u;
        if (b < upto) part += u;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, o);
        part += __shfl_xor_sync(0xffffffffu, part, o);
    }
    before = part;
    return all;
}
// The stream of unit x and the number of units before its first row.
__device__ __forceinline__ int stream_of(const Kv4Attend &a, long long x, long long &first) {
    const int lane = threadIdx.x & 31;
    long long sum = 0;
    for (int base = 0; base < a.B; base += 32) {
        const long long u = base + lane < a.B ? (long long)units_of(a, checked_len(a, base + lane)) * a.c.n_kv_heads : 0;
        long long to = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, to, o);
            if (lane >= o) to += t;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, sum + to > x);
        if (past != 0) {
            const int at = __ffs(past) - 1;
            first = sum + __shfl_sync(0xffffffffu, to - u, at);
            return base + at;
        }
        sum += __shfl_sync(0xffffffffu, to, 31);
    }
    first = sum;
    return a.B;
}

// Each CTA walks its units row by row. Within a row, each warp takes every kWarps-th page through a
// ring of its own: bulk copies, no barrier between warps; the warps' parts are merged at the row's
// (or the range's) end. A row that lies in one CTA's range is finished there, else its parts go to
// scratch: a CTA has at most two such parts, one that begins its range and one that ends it.
//
// A lane is (r = lane / 4, c = lane % 4). Scores of 16 keys, S[keys x 8] = K Q^T by m16n8k16 per
// block of 32 dims; q is scaled by a power of two so that its largest value lies in [2^13, 2^14). The
// results times the key's scales are added in f32.
// Values, O^T[dims x 8] += V^T P^T, P being the probabilities p times the value's scale of each block,
// transposed between lanes as fp16. p = ph + pl, and P = ph d rounded, plus what that leaves and pl d: three fp16
// instructions. Two things keep P in fp16's range and bits. The exponents' reference m follows the largest
// score: where a p would pass 2^11, O and l are rescaled so that the largest is 2^6. And each block of 32 dims
// has a power of two, up to 2^15, that brings its largest value scale so far to [2^2, 2^3) and under which its
// O is summed; where a scale would pass 2^4, that block's O is rescaled. So the parts hold a
// P to 2^-31 of the largest of its own block. An accumulator's columns are its lane's heads throughout.
// V codes are centred in fp16 before the MMA. P is held in two fp16 parts (22 bits): for up to 4 query heads in
// columns h and h + 4 of one MMA, above that (WIDE) by two MMAs. So is q where it is f32 (QTWO); a bf16 q is exact
// in one part. f32 results (PREC): K codes centred too. bf16 results: K codes as they are, times 2^-24, and the scores'
// offset, -8 sum(q) of each block times its scale, by one more MMA over blocks. (f32 results would lose bits to
// that: an error of 2e-6 of the result instead of 3e-7 for 128 dims and G = 2.)
// The MMA cuts its sums off instead of rounding them, so a long chain of them shrinks: over 8192 rows a CTA
// f32 results were 1e-6 off, with WIDE 3e-6 (2e-5 for 20000 values of one sign). So theirs start from zero every 16
// keys, and 2 to 3e-7 is left at any length (G = 2 135 instead of 129 us below, G = 8 172 instead of 161). bf16
// results, whose step is 2^-8, keep the chain.
//
// 64 streams x 8192 rows x 8 KV heads of 128 dims (604 MB of tiles, 89 us at the measured copy rate):
// bf16, G = 8 139 us, G = 2 122; f32, G = 2 135, G = 8 (WIDE) 172; bf16 with 64 dims, G = 8 90 (floor 44.5).
// (P in one fp16 part: 111 us in bf16 with G = 8, terms off by up to 2^-10.) Not DRAM, but
// instructions: 1340 a page and warp in bf16 with G = 8 at 2.3 per cycle and multiprocessor, over a quarter on
// the ALU pipe (masks and byte permutations of codes), which takes one in two cycles; the rest is the latency that
// its 12 or 16 warps do not hide (kv4_attend_shape). One wave of CTAs over balanced ranges instead of a CTA per
// split of a row: 144 instead of 164 us, at that time.
template <int HD, bool WIDE, typename TI, typename TO, int CTAS>
__global__ void __launch_bounds__(kWarps * 32, CTAS) k_kv4_attend(const Kv4Attend a) {
    using Tile = Kv4Tile<HD>;
    constexpr bool PREC = sizeof(TO) == 4;
    constexpr int NB = Tile::NB, kSlots = slots_of(CTAS);
    constexpr int kParts = WIDE ? 1 : 2;                // columns of P per query head
    constexpr bool QTWO = sizeof(TI) == 4;              // q has two parts, in WIDE's second MMA or in columns of their own
    constexpr int kQParts = QTWO ? kParts : 1;
    constexpr int kCorrBits = 10;
    extern __shared__ __align__(128) unsigned char ring_all[];
    __shared__ __align__(8) uint64_t bars[kWarps][kSlots];
    __shared__ float wm[kWarps + 1][kMaxG], wl[kWarps + 1][kMaxG];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int G = a.n_q / a.c.n_kv_heads;
    if (!a.one_unit) pdl_launch_dependents();   // (the joining kernel; at the end 2 us more for 32768 rows;
                                                // another would only take room)
    unsigned char *ring = ring_all + warp * kSlots * Tile::kBytes;
    if (lane == 0) {
        for (int i = 0; i < kSlots; ++i) mbar_init(&bars[warp][i], 1);
        fence_barrier_init();
    }
    __syncwarp();
    long long before;
    const long long U = count_units(a, 0, before) * a.c.n_kv_heads;
    const long long n = min(U, (long long)gridDim.x);
    if (blockIdx.x >= n) return;
    const long long x_begin = blockIdx.x * U / n, x_end = (blockIdx.x + 1) * U / n;
    const int b0 = stream_of(a, x_begin, before), len0 = checked_len(a, b0), nu0 = units_of(a, len0);
    int slot = 0;   // where the next K tile goes
    Kv4Ring state;
    // Of 8 keys, row 2 c of the scores (and so slot 2 c of P) is key c and row 2 c + 1 key c2: the
    // two rows of codes that eight lanes load together lie in other banks.
    const int c2 = 4 + (c ^ 1), key_r = r & 1 ? 4 + ((r >> 1) ^ 1) : r >> 1;

    // Units [u0, u1) of the row of stream b and KV head g, which has nu; `left` units of the CTA's follow.
    // Kept in shared memory, a copy for each warp, so that the loop over pages has the registers.
    struct Range {
        int b, g, len, nu, u0, u1;
        long long left;
    };
    __shared__ Range ranges[kWarps];
    Range &at = ranges[warp];
    auto good = [&](int page) { return page >= 0 && page < a.c.n_pages; };
    // a tile to a slot, by one lane, behind what the warp read there; a bad page number copies page 0, which is not used
    auto issue = [&](int to, const void *pool, int page, int g) {
        state.issued(to);
        if (lane != 0) return;
        fence_proxy_async();
        const size_t tile = ((size_t)(good(page) ? page : 0) * a.c.n_layers + a.layer) * a.c.n_kv_heads + g;
        mbar_arrive_expect_tx(&bars[warp][to], Tile::kBytes);
        bulk_g2s(ring + to * Tile::kBytes, static_cast<const unsigned char *>(pool) + tile * Tile::kBytes, Tile::kBytes,
                 &bars[warp][to]);
    };
    auto wait = [&](int at) {
        const bool ok = !__any_sync(0xffffffffu, !bounded_wait(&bars[warp][at], state.parity(at)));
        if (ok) state.landed(at);
        return ok;
    };
    auto after = [](int at) { return at == kSlots - 1 ? 0 : at + 1; };
    // of the warp's pages: how many, the numbers of 32 j + lane, of this one and of the next
    int n_it = 0, rows = 0, pages = 0, ahead = 0, page = 0, page1 = 0;
    auto page_of = [&](int it) {
        const int *p = a.c.page_table + (size_t)at.b * a.c.pages_per_stream + at.u0 * kWarps + warp;
        return it < n_it ? p[it * kWarps] : 0;
    };
    auto open = [&](int b, int g, int len, int nu, int u0, long long left) {   // ... and its first copies
        const int u1 = (int)min((long long)nu, u0 + left), pb = u0 * kWarps + warp, pe = u1 == nu ? pages_of(len) : u1 * kWarps;
        n_it = pb < pe && !state.lost() ? (pe - pb + kWarps - 1) / kWarps : 0;
        rows = len - pb * kPage;
        if (lane == 0) at = {b, g, len, nu, u0, u1, left - (u1 - u0)};
        __syncwarp();
        pages = page_of(lane);
        ahead = page_of(32 + lane);
        page = __shfl_sync(0xffffffffu, pages, 0);
        page1 = __shfl_sync(0xffffffffu, pages, 1);
        if (n_it > 0) issue(slot, a.c.k, page, g), issue(after(slot), a.c.v, page, g);
        if (kSlots == 3 && n_it > 1) issue(after(after(slot)), a.c.k, page1, g);
    };
    open(b0, (int)((x_begin - before) / nu0), len0, nu0, (int)((x_begin - before) % nu0), x_end - x_begin);
    pdl_wait();   // before it: lengths, page numbers and cached rows, which the kernel before does not write

    for (bool begins = true;; begins = false) {
        if (at.len < 0 && threadIdx.x == 0 && a.c.status != nullptr) atomicOr(a.c.status, ST_BAD_POSITION);

        // this lane's query head (rows beyond G compute on zeros)
        const int hq = kParts == 2 ? r & 3 : r;
        const bool q_vec = (reinterpret_cast<uintptr_t>(a.q) & 15u) == 0 && a.q_row * sizeof(TI) % 16 == 0;
        const float cs = a.scale * kLog2e;
        uint32_t qf[NB][2][2], ql[NB][2][2];       // (ql: WIDE and QTWO)
        uint32_t qc = 0;                           // (unless PREC) -8 sum(q) of two blocks, times 2^kCorrBits: lanes
                                                   // c < H have a first part, lanes c - H its rest
        F2 fs;                                     // from these units to scores in base 2, of this lane's columns 2 c, 2 c + 1
        {
            float x[NB][8], top = 0.f;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                if (hq < G) {
                    load_dims8(static_cast<const TI *>(a.q) + at.b * a.q_row + (size_t)(at.g * G + hq) * HD + nb * 32 + c * 8, q_vec, x[nb]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[nb][i] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[nb][i]));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = min((int)(__float_as_uint(top) >> 23), 254);        // biased exponent of the largest
            const int up = min(13 + 127 - e, 120);                            // 2^up brings it to [2^13, 2^14)
            const float qs = __uint_as_float((uint32_t)(up + 127) << 23);
            const float unit = cs * exp2f((float)((PREC ? 0 : 24) - up));
            fs = f2(__shfl_sync(0xffffffffu, unit, 8 * c), __shfl_sync(0xffffffffu, unit, 8 * c + 4));
            float corr[NB];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                float sum = 0.f;
                __half hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // of the byte that holds dims i and i + 1: n0's part, and that of 16 n1 (PREC: of n0 + 16 n1)
                    const float y = i & 1 ? x[nb][i] * qs * 0.0625f
                                          : PREC ? fmaf(x[nb][i + 1], qs * -0.0625f, x[nb][i] * qs) : x[nb][i] * qs;
                    hi[i] = __float2half_rn(y);
                    lo[i] = __float2half_rn(y - __half2float(hi[i]));
                    if (kQParts == 2 && r >= 4) hi[i] = lo[i];
                    if (!PREC) sum = fmaf(__half2float(hi[i]) + (WIDE && QTWO ? __half2float(lo[i]) : 0.f), i & 1 ? 16.f : 1.f, sum);
                }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        qf[nb][t][i] = pack_half(hi[2 * t + i], hi[2 * t + 4 + i]);
                        ql[nb][t][i] = pack_half(lo[2 * t + i], lo[2 * t + 4 + i]);
                    }
                if (PREC) continue;
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                corr[nb] = sum * (-8.f / 16777216.f * (1 << kCorrBits));
            }
#pragma unroll
            for (int i = 0; i < NB / 2 && !PREC; ++i) {
                const __half h0 = __float2half_rn(corr[2 * i]), h1 = __float2half_rn(corr[2 * i + 1]);
                if (c == i) qc = pack_half(h0, h1);
                if (c == i + NB / 2)
                    qc = pack_half(__float2half_rn(corr[2 * i] - __half2float(h0)), __float2half_rn(corr[2 * i + 1] - __half2float(h1)));
            }
        }

        constexpr int H = NB / 2;
        uint32_t up[H];                           // the powers of two of blocks 2 i, 2 i + 1 (fp16), and
#pragma unroll
        for (int i = 0; i < H; ++i) up[i] = 0x78007800u;   // ... 2^15 at first, the largest
        float m0 = -INFINITY, m1 = -INFINITY;     // references of the exponents of this lane's columns
        F2 l2 = f2(0.f, 0.f);                     // its keys' parts of their sums
        // dim 32 (t / 2) + 4 r + 2 (t % 2), and it plus 16 times the next one (e >= 2), of heads 2 c, 2 c + 1
        float o[2 * NB][4];
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[t][e] = 0.f;

        for (int it = 0; it < n_it; ++it) {
            if ((it + 2) % 32 == 0) {
                pages = ahead;
                ahead = page_of(it + 34 + lane);
            }
            const int page2 = __shfl_sync(0xffffffffu, pages, (it + 2) % 32), vslot = after(slot);
            const int valid = min(kPage, rows - it * kWarps * kPage);
            const uint32_t kt = smem_u32(ring) + slot * Tile::kBytes, vt = smem_u32(ring) + vslot * Tile::kBytes;
            if (!wait(slot)) {
                state.lose();
                break;
            }
            F2 sc[4][2];   // scores in base 2: of keys 16 i + key_r and 16 i + 8 + key_r
            if (!good(page)) {
                if (lane == 0 && a.c.status != nullptr) atomicOr(a.c.status, ST_BAD_ARG);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    Words<NB> k0, k1;
                    Words<H> d0, d1;
                    k0.load(kt + (16 * i + key_r) * Tile::kRow + c * 4 * NB);
                    k1.load(kt + (16 * i + 8 + key_r) * Tile::kRow + c * 4 * NB);
                    d0.load(kt + Tile::kScales + (16 * i + key_r) * NB * 2);
                    d1.load(kt + Tile::kScales + (16 * i + 8 + key_r) * NB * 2);
                    F2 s0, s1;
                    if (PREC) {
                        s0 = s1 = f2(0.f, 0.f);
                    } else {
                        // scales of blocks 2 (c % H) and the next (columns past the parts meet zeros)
                        float acc[4];
                        mma1688_new(acc, lds_u1(kt + Tile::kScales + (16 * i + key_r) * NB * 2 + 4 * (c & (H - 1))),
                                    lds_u1(kt + Tile::kScales + (16 * i + 8 + key_r) * NB * 2 + 4 * (c & (H - 1))), qc);
                        const F2 down = f2(1.f / (1 << kCorrBits), 1.f / (1 << kCorrBits));
                        s0 = f2(acc[0], acc[1]) * down, s1 = f2(acc[2], acc[3]) * down;
                    }
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        float acc[4];
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            uint32_t codes[4];
                            if (!PREC) {
                                const uint32_t w0 = t ? bytes13(k0.w[nb]) : k0.w[nb], w1 = t ? bytes13(k1.w[nb]) : k1.w[nb];
                                codes[0] = low_nibbles(w0), codes[1] = low_nibbles(w1);
                                codes[2] = high_nibbles(w0), codes[3] = high_nibbles(w1);
                            } else {
                                const uint32_t x0 = t ? raised13(k0.w[nb]) : raised02(k0.w[nb]);
                                const uint32_t x1 = t ? raised13(k1.w[nb]) : raised02(k1.w[nb]);
                                codes[0] = centred_nibbles(x0), codes[1] = centred_nibbles(x1);
                                codes[2] = centred_bytes(x0), codes[3] = centred_bytes(x1);
                            }
                            if (t == 0) mma16816_new(acc, codes, qf[nb][0][0], qf[nb][0][1]);
                            else mma16816(acc, codes, qf[nb][1][0], qf[nb][1][1]);
                            if (WIDE && QTWO) mma16816(acc, codes, ql[nb][t][0], ql[nb][t][1]);
                        }
                        const float e0 = scale_at(d0.w, nb), e1 = scale_at(d1.w, nb);
                        s0 = f2(fmaf(e0, acc[0], f2_lo(s0)), fmaf(e0, acc[1], f2_hi(s0)));
                        s1 = f2(fmaf(e1, acc[2], f2_lo(s1)), fmaf(e1, acc[3], f2_hi(s1)));
                    }
                    sc[i][0] = s0, sc[i][1] = s1;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        F2 &x = sc[i][u];
                        if (kQParts == 2)   // the parts of head h: columns h and h + 4
                            x = x + f2(__shfl_xor_sync(0xffffffffu, f2_lo(x), 2), __shfl_xor_sync(0xffffffffu, f2_hi(x), 2));
                        x = x * fs;
                    }
                if (valid < kPage) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (8 * i + key_r >= valid) sc[i >> 1][i & 1] = f2(-INFINITY, -INFINITY);
                }
            }
            __syncwarp();
            if (it + 1 < n_it) issue(slot, kSlots == 3 ? a.c.v : a.c.k, page1, at.g);   // the next page's V (of two slots: K) over this K
            if (!wait(vslot)) {
                state.lose();
                break;
            }
            if (good(page)) {
                if (valid < kPage) {   // value scales past the length: zero (a row's last page: never refilled)
                    unsigned char *d = ring + vslot * Tile::kBytes + Tile::kScales;
                    for (int i = valid * NB + lane; i < kPage * NB; i += 32) reinterpret_cast<unsigned short *>(d)[i] = 0;
                    __syncwarp();
                }
                // the page's value scales under their blocks' powers of two (a NaN is no size)
                {
                    __half2 top[H];
                    bool past = false;
#pragma unroll
                    for (int i = 0; i < H; ++i) top[i] = __float2half2_rn(0.f);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        Words<H> d;
                        d.load(vt + Tile::kScales + (2 * lane + u) * NB * 2);
#pragma unroll
                        for (int i = 0; i < H; ++i)
                            top[i] = __hmax2(top[i], __habs2(*reinterpret_cast<__half2 *>(&d.w[i])));
                    }
                    const __half2 most = __float2half2_rn((float)(1 << kTopScale));
#pragma unroll
                    for (int i = 0; i < H; ++i)
                        past |= !__hble2(__hmul2(top[i], *reinterpret_cast<const __half2 *>(&up[i])), most);
                    if (__any_sync(0xffffffffu, past)) {
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) {
                            const uint32_t bits = *reinterpret_cast<const uint32_t *>(&top[nb / 2]), at = 16 * (nb & 1);
                            const uint32_t e = __reduce_max_sync(0xffffffffu, bits >> at & 0xffffu) >> 10;   // biased by 15
                            const uint32_t old = up[nb / 2] >> (at + 10) & 31u;
                            const uint32_t now = min(old, min(30u, kNewScale + 30u - max(e, 1u)));
                            const float by = __uint_as_float((127u + now - old) << 23);
                            up[nb / 2] += (now - old) << (at + 10);
#pragma unroll
                            for (int t = 2 * nb; t < 2 * nb + 2; ++t)
#pragma unroll
                                for (int i = 0; i < 4; ++i) o[t][i] *= by;
                        }
                    }
                }
                F2 mx = f2(-INFINITY, -INFINITY);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int u = 0; u < 2; ++u) mx = f2(fmaxf(f2_lo(mx), f2_lo(sc[i][u])), fmaxf(f2_hi(mx), f2_hi(sc[i][u])));
#pragma unroll
                for (int j = 4; j < 32; j <<= 1)
                    mx = f2(fmaxf(f2_lo(mx), __shfl_xor_sync(0xffffffffu, f2_lo(mx), j)),
                            fmaxf(f2_hi(mx), __shfl_xor_sync(0xffffffffu, f2_hi(mx), j)));
                if (__any_sync(0xffffffffu, f2_lo(mx) > m0 + kTopBits || f2_hi(mx) > m1 + kTopBits)) {
                    const float n0 = fmaxf(m0, f2_lo(mx) - kNewBits), n1 = fmaxf(m1, f2_hi(mx) - kNewBits);
                    const F2 al = f2(m0 == n0 ? 1.f : ex2(m0 - n0), m1 == n1 ? 1.f : ex2(m1 - n1));
                    m0 = n0;
                    m1 = n1;
                    l2 = l2 * al;
#pragma unroll
                    for (int t = 0; t < 2 * NB; ++t)
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const F2 x = f2(o[t][e], o[t][e + 1]) * al;
                            o[t][e] = f2_lo(x), o[t][e + 1] = f2_hi(x);
                        }
                }
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    F2 p[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const F2 x = sc[ks][i] + f2(-m0, -m1);
                        p[i] = f2(ex2(f2_lo(x)), ex2(f2_hi(x)));
                        l2 = l2 + p[i];
                    }
                    uint32_t ph[2], pl[2];
                    Words<H> v[4], d[2];   // codes of slots 2 c, 2 c + 1 and 8 further, scales of p's keys
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = 16 * ks + 8 * (i >> 1) + (i & 1 ? c2 : c);
                        v[i].load(vt + key * Tile::kRow + r * 2 * NB);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        d[i].load(vt + Tile::kScales + (16 * ks + 8 * i + key_r) * NB * 2);
#pragma unroll
                        for (int u = 0; u < H; ++u) d[i].w[u] = mul_half2(d[i].w[u], up[u]);
                        ph[i] = pack_rn(f2_lo(p[i]), f2_hi(p[i]));
                        const F2 rest = fma2(f2(half_lo(ph[i]), half_hi(ph[i])), f2(-1.f, -1.f), p[i]);
                        pl[i] = pack_rn(f2_lo(rest), f2_hi(rest));
                    }
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        const uint32_t sel = nb & 1 ? 0x7632 : 0x5410;   // halves nb % 2 of two keys' words
                        uint32_t bh[2], bl[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const HalfParts y = mul_parts(ph[i], pl[i], d[i].w[nb / 2], nb & 1);
                            bh[i] = transpose8(WIDE || c < 2 ? y.x : y.y);   // (else columns h and h + 4 have head h's parts)
                            if (WIDE) bl[i] = transpose8(y.y);
                        }
                        const uint32_t u0 = __byte_perm(v[0].w[nb / 2], v[1].w[nb / 2], sel);
                        const uint32_t u1 = __byte_perm(v[2].w[nb / 2], v[3].w[nb / 2], sel);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float(&acc)[4] = o[2 * nb + e];
                            const uint32_t x0 = e ? raised13(u0) : raised02(u0), x1 = e ? raised13(u1) : raised02(u1);
                            const uint32_t codes[4] = {centred_nibbles(x0), centred_bytes(x0), centred_nibbles(x1), centred_bytes(x1)};
                            if (PREC) {   // the 16 keys' sums on their own, then to the others' by rounded additions
                                float part[4];
                                mma16816_new(part, codes, WIDE ? bl[0] : bh[0], WIDE ? bl[1] : bh[1]);
                                if (WIDE) mma16816(part, codes, bh[0], bh[1]);
#pragma unroll
                                for (int i = 0; i < 4; i += 2) {
                                    const F2 x = f2(acc[i], acc[i + 1]) + f2(part[i], part[i + 1]);
                                    acc[i] = f2_lo(x), acc[i + 1] = f2_hi(x);
                                }
                            } else {
                                mma16816(acc, codes, bh[0], bh[1]);
                                if (WIDE) mma16816(acc, codes, bl[0], bl[1]);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (it + (kSlots == 3 ? 2 : 1) < n_it)   // the K after the next (V of the next) over this V
                issue(vslot, kSlots == 3 ? a.c.k : a.c.v, kSlots == 3 ? page2 : page1, at.g);
            slot = after(vslot);
            page = page1;
            page1 = page2;
        }
        if (n_it > 0 && state.lost()) {   // report, and give the copies in flight their chance to land; no more follow
            if (lane == 0 && a.c.status != nullptr) atomicOr(a.c.status, ST_WAIT_TIMEOUT);
            for (int i = 0; i < kSlots; ++i)
                if (state.in_flight(i)) wait(i);
        }

        // The next range's first copies go out now. (This warp's reads and writes of its ring lie behind it.)
        const Range done = at;
        const int b = done.b, g = done.g;
        if (done.left > 0) {
            const bool row_ends = g == a.c.n_kv_heads - 1;
            const int nb = row_ends ? b + 1 : b, nl = row_ends ? checked_len(a, nb) : done.len;
            fence_proxy_async();
            __syncwarp();
            open(nb, row_ends ? 0 : g + 1, nl, row_ends ? units_of(a, nl) : done.nu, 0, done.left);
        }

        // the warp's (m, l, O) to shared memory
#pragma unroll
        for (int j = 4; j < 32; j <<= 1)
            l2 = l2 + f2(__shfl_xor_sync(0xffffffffu, f2_lo(l2), j), __shfl_xor_sync(0xffffffffu, f2_hi(l2), j));
        if (state.lost()) {   // this row and the rest of the CTA's
            m0 = m1 = __int_as_float(0x7fc00000);
            l2 = f2(m0, m0);
        }
        __syncthreads();
        float *wo = reinterpret_cast<float *>(ring_all + kWarps * kSlots * Tile::kBytes);   // [kWarps][kMaxG][HD]
        if (r == 0 && (kParts == 1 || c < 2)) {
            wm[warp][2 * c] = m0, wm[warp][2 * c + 1] = m1;
            wl[warp][2 * c] = f2_lo(l2), wl[warp][2 * c + 1] = f2_hi(l2);
        }
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float y = e < 2 ? o[t][e] : (o[t][e] - o[t][e - 2]) * 0.0625f;
                y *= __uint_as_float((127u + 15u - (up[t / 4] >> (t & 2 ? 26 : 10) & 31u)) << 23);   // (less its block's power of two)
                if (kParts == 2) y += __shfl_xor_sync(0xffffffffu, y, 2);   // the parts of head h: columns h and h + 4
                const int h = 2 * c + (e & 1), dim = 32 * (t >> 1) + 4 * r + 2 * (t & 1) + (e >> 1);
                if (kParts == 1 || c < 2) wo[(warp * kMaxG + h) * HD + dim] = y;
            }
        // the step's own row, as one more part of the row's first units
        const bool fresh = done.u0 == 0 && done.len >= 0 && a.k_new != nullptr;
        if (fresh) {
            const TI *kn = static_cast<const TI *>(a.k_new) + b * a.new_row + (size_t)g * HD;
            for (int h = warp; h < G; h += kWarps) {
                const TI *q = static_cast<const TI *>(a.q) + b * a.q_row + (size_t)(g * G + h) * HD;
                float t = 0.f;
#pragma unroll
                for (int i = 0; i < HD / 32; ++i) t = fmaf((float)q[32 * i + lane], (float)kn[32 * i + lane], t);
                t = warp_sum(t);
                if (lane == 0) wm[kWarps][h] = t * cs, wl[kWarps][h] = 1.f;
            }
        }
        __syncthreads();
        const bool whole = done.u0 == 0 && done.u1 == done.nu;
        for (int idx = threadIdx.x; idx < G * HD; idx += kWarps * 32) {
            const int h = idx / HD, d = idx % HD;
            float M = fresh ? wm[kWarps][h] : -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w][h]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float e = wm[w][h] == -INFINITY ? 0.f : ex2(wm[w][h] - M);
                L = fmaf(wl[w][h], e, L);
                O = fmaf(wo[(w * kMaxG + h) * HD + d], e, O);
            }
            if (fresh) {
                const float e = ex2(wm[kWarps][h] - M);
                L += e;
                O = fmaf((float)static_cast<const TI *>(a.v_new)[b * a.new_row + (size_t)g * HD + d], e, O);
            }
            if (whole) {
                static_cast<TO *>(a.out)[((size_t)b * a.n_q + g * G + h) * HD + d] = (TO)(L == 0.f ? 0.f : O / L);
            } else {
                float *ws = a.scratch + (((size_t)blockIdx.x * 2 + !begins) * kMaxG + h) * (HD + 4);
                ws[4 + d] = O;
                if (d == 0) ws[0] = M, ws[1] = L;
            }
        }
        if (done.left == 0) break;
    }
}

// The parts of a row that several CTAs shared: CTAs [first, last] have one each (first == last: none).
struct Parts {
    int first, last, tail;   // tail: the first CTA's range began with another row
};
__device__ __forceinline__ Parts parts_of(const Kv4Attend &a, int grid, int b, int g) {
    long long before;
    const long long U = count_units(a, b, before) * a.c.n_kv_heads;
    const int nu = units_of(a, checked_len(a, b));
    const long long n = min(U, (long long)grid), x0 = before * a.c.n_kv_heads + (long long)g * nu;
    Parts p{(int)(((x0 + 1) * n - 1) / U), (int)(((x0 + nu) * n - 1) / U), 0};   // CTAs of the row's ends
    p.tail = p.first * U / n != x0;
    return p;
}
template <int HD>
__device__ __forceinline__ const float *part_at(const Kv4Attend &a, const Parts &p, int i, int h) {
    return a.scratch + (((size_t)i * 2 + (i == p.first ? p.tail : 0)) * kMaxG + h) * (HD + 4);
}

// Many rows have about two parts each. Grid (KV heads, B), HD x kJoinHeads threads: a thread has one dim of
// every kJoinHeads-th head of the group, and reads all it needs at once.
constexpr int kJoinHeads = 4, kJoinAhead = 4;
template <int HD, typename TO>
__global__ void __launch_bounds__(HD * kJoinHeads) k_kv4_join(const Kv4Attend a, const int grid) {
    const int b = blockIdx.y, g = blockIdx.x, G = a.n_q / a.c.n_kv_heads, d = threadIdx.x % HD;
    const Parts p = parts_of(a, grid, b, g);   // (lengths were there before the kernel that this one follows)
    pdl_wait();
    if (p.first == p.last) return;
    for (int h = threadIdx.x / HD; h < G; h += kJoinHeads) {
        float m = -INFINITY, L = 0.f, O = 0.f;
        for (int i0 = p.first; i0 <= p.last; i0 += kJoinAhead) {
            float2 ml[kJoinAhead];
            float o[kJoinAhead];
#pragma unroll
            for (int i = 0; i < kJoinAhead; ++i)
                if (i0 + i <= p.last) {
                    const float *part = part_at<HD>(a, p, i0 + i, h);
                    ml[i] = *reinterpret_cast<const float2 *>(part), o[i] = part[4 + d];
                } else {
                    ml[i] = make_float2(-INFINITY, 0.f), o[i] = 0.f;
                }
            float top = m;
#pragma unroll
            for (int i = 0; i < kJoinAhead; ++i) top = fmaxf(top, ml[i].x);
            const float old = m == -INFINITY ? 0.f : ex2(m - top);
            L *= old, O *= old, m = top;
#pragma unroll
            for (int i = 0; i < kJoinAhead; ++i) {
                const float e = ml[i].x == -INFINITY ? 0.f : ex2(ml[i].x - top);
                L = fmaf(ml[i].y, e, L), O = fmaf(o[i], e, O);
            }
        }
        static_cast<TO *>(a.out)[((size_t)b * a.n_q + g * G + h) * HD + d] = (TO)(L == 0.f ? 0.f : O / L);
    }
}

// A few rows have many parts each. Grid (n_q, B): the maxima and sums of all parts are read at once, then each
// group of HD threads adds up every kGroups-th part, several in flight.
constexpr int kCombineThreads = 512;
template <int HD, typename TO>
__global__ void __launch_bounds__(kCombineThreads) k_kv4_combine(const Kv4Attend a, const int grid) {
    constexpr int kThreads = kCombineThreads, kGroups = kThreads / HD, kAhead = 8, kWarpsHere = kThreads / 32;
    __shared__ float weight[kMaxGrid], red[2][kWarpsHere], sums[kGroups][HD];
    const int b = blockIdx.y, G = a.n_q / a.c.n_kv_heads, g = blockIdx.x / G, h = blockIdx.x % G;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = threadIdx.x % HD, group = threadIdx.x / HD;
    const Parts p = parts_of(a, grid, b, g);
    const int first = p.first, last = p.last;
    pdl_wait();
    if (first == last) return;
    auto part = [&](int i) { return part_at<HD>(a, p, i, h); };
    float m = -INFINITY;
    for (int i = first + threadIdx.x; i <= last; i += kThreads) m = fmaxf(m, part(i)[0]);
    m = warp_max(m);
    if (lane == 0) red[0][warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarpsHere; ++w) m = fmaxf(m, red[0][w]);
    float L = 0.f;
    for (int i = first + threadIdx.x; i <= last; i += kThreads) {
        const float2 ml = *reinterpret_cast<const float2 *>(part(i));
        const float e = ml.x == -INFINITY ? 0.f : ex2(ml.x - m);
        weight[i - first] = e;
        L = fmaf(ml.y, e, L);
    }
    L = warp_sum(L);
    if (lane == 0) red[1][warp] = L;
    __syncthreads();
    L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarpsHere; ++w) L += red[1][w];
    float O = 0.f;
    for (int i0 = first + group; i0 <= last; i0 += kGroups * kAhead) {
        float o[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) o[i] = i0 + i * kGroups <= last ? part(i0 + i * kGroups)[4 + d] : 0.f;
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i0 + i * kGroups <= last) O = fmaf(o[i], weight[i0 + i * kGroups - first], O);
    }
    sums[group][d] = O;
    __syncthreads();
    if (group != 0) return;
    O = 0.f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) O += sums[i][d];
    static_cast<TO *>(a.out)[((size_t)b * a.n_q + blockIdx.x) * HD + d] = (TO)(L == 0.f ? 0.f : O / L);
}

// Parts of a row, if all are alike, from which on it is k_kv4_combine (a CTA per query head) that joins them. With
// k_kv4_join / with it, bf16: 64 streams of 8192 rows x 8 heads (2 parts) 122 / 130 us, 16 streams of up to 2048 (5) 13.2 /
// 14.6, 7 streams of up to 5001 x 5 heads (13) 13.4 / 11.1, 1 stream of 32768 x 8 heads (57) 22.4 / 18.3.
constexpr int kManyParts = 8;
template <int HD, typename TI, typename TO>
cudaError_t launch_t(Kv4Attend a, bool pdl, cudaStream_t s) {
    const bool wide = a.n_q / a.c.n_kv_heads > 4;
    void (*kernel)(Kv4Attend) = k_kv4_attend<HD, false, TI, TO, kFewCtas>;
    if constexpr (HD == 128)
        if (a.ctas == kManyCtas) kernel = k_kv4_attend<HD, false, TI, TO, kManyCtas>;
    // With three / four CTAs (128 registers, which spill), G = 8 in bf16: 64 x 8192 rows 139 / 139 us, 32 x 4096 49 / 52,
    // 16 x 2048 23.2 / 27.5, 16 of up to 2048 22.8 / 18.5, 32 of up to 4096 36.6 / 36.5; f32 172 / 172 and 56.8 / 60.7.
    if (wide) {
        if (a.ctas == kManyCtas) a.grid = std::max(1, a.grid * kFewCtas / kManyCtas);
        a.ctas = kFewCtas;
        kernel = k_kv4_attend<HD, true, TI, TO, kFewCtas>;
    }
    const size_t smem = attend_smem(HD, a.ctas);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    if (pdl) {
        cfg.gridDim = dim3(a.grid);
        cfg.blockDim = dim3(kWarps * 32);
        cfg.dynamicSmemBytes = smem;
        e = cudaLaunchKernelEx(&cfg, kernel, a);
        cfg.dynamicSmemBytes = 0;
    } else {
        kernel<<<a.grid, kWarps * 32, smem, s>>>(a);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess || a.one_unit) return e;
    const bool many = a.grid >= (long long)kManyParts * a.B * a.c.n_kv_heads;
    cfg.gridDim = dim3(many ? a.n_q : a.c.n_kv_heads, a.B);
    cfg.blockDim = dim3(many ? kCombineThreads : HD * kJoinHeads);
    return cudaLaunchKernelEx(&cfg, many ? k_kv4_combine<HD, TO> : k_kv4_join<HD, TO>, a, a.grid);
}

template <int HD>
cudaError_t launch_hd(const Kv4Attend &a, int in_bf16, int out_bf16, bool pdl, cudaStream_t s) {
    if (in_bf16) return out_bf16 ? launch_t<HD, __nv_bfloat16, __nv_bfloat16>(a, pdl, s) : cudaErrorInvalidValue;
    return out_bf16 ? launch_t<HD, float, __nv_bfloat16>(a, pdl, s) : launch_t<HD, float, float>(a, pdl, s);
}

}  // namespace

// CTAs of a launch and whether rows are left whole: with at most kWholePages pages (one or two per
// warp) the second launch costs more than splitting wins. A Talker step over one stream of 300 / 480 / 700 /
// 1000 rows with 4: 658 / 688 / 681 / 693 us, 8: 625 / 679 / 679 / 693, 12: 625 / 677 / 690 / 694, 16: 626 / 678 /
// 690 / 818.
constexpr int kWholePages = 8;

// Three or four CTAs a multiprocessor, up to 4 query heads a KV head: four hide more latency and finish more units
// at once, but have two tiles in flight per warp instead of three. us with 3 / 4, 8 KV heads of 128 dims, G = 2, bf16:
// 64 streams of 8192 rows 127 / 122; 32 of up to 4096 30.8 / 29.6 (all of 4096: 43.7 / 43.9); 16 of up to 2048 17.7 /
// 13.2 (all of 2048: 19.5 / 20.5); 2 of 16384 20.1 / 18.3; 1 of 32768 18.3 / 19.1, of 131072 41.0 / 41.3; with a row to
// a CTA, 100 streams of 500 22.0 / 26.1. (With 64 dims four were slower too: 13.6 / 15.3 for 7 of up to 5001.)
Kv4AttendShape kv4_attend_shape(int B, int n_kv, int hd, int max_len, int n_sm) {
    const long long rows = (long long)B * n_kv, pages = ((long long)max_len + kPage - 1) / kPage;
    Kv4AttendShape p;
    p.one_unit = pages <= kWholePages;
    const long long units = p.one_unit ? rows : rows * ((pages + kWarps - 1) / kWarps);
    const bool many = hd == 128 && B > 1 && !p.one_unit && units > (long long)kFewCtas * n_sm;
    p.ctas = many ? kManyCtas : kFewCtas;
    p.full_grid = std::min(p.ctas * n_sm, kMaxGrid);
    p.grid = (int)std::max<long long>(1, std::min<long long>(units, p.full_grid));
    return p;
}

size_t kv4_attend_scratch(const Kv4AttendShape &p, int head_dim) {
    return p.one_unit ? 0 : kv4_attend_scratch(p.grid, head_dim);
}
size_t kv4_attend_scratch(int grid, int head_dim) {
    return (size_t)grid * 2 * kMaxG * (head_dim + 4) * sizeof(float);
}

template <int HD, bool WIDE, typename TI, typename TO, int CTAS>
cudaError_t raise_one() {
    return cudaFuncSetAttribute(k_kv4_attend<HD, WIDE, TI, TO, CTAS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)attend_smem(HD, CTAS));
}
template <int HD, bool WIDE, int CTAS>
cudaError_t raise_types() {
    cudaError_t e = raise_one<HD, WIDE, float, float, CTAS>();
    e = e ? e : raise_one<HD, WIDE, float, __nv_bfloat16, CTAS>();
    return e ? e : raise_one<HD, WIDE, __nv_bfloat16, __nv_bfloat16, CTAS>();
}

cudaError_t prepare_kv4_attend() {
    cudaError_t e = raise_types<128, false, kFewCtas>();
    e = e ? e : raise_types<128, false, kManyCtas>();
    e = e ? e : raise_types<64, false, kFewCtas>();
    e = e ? e : raise_types<128, true, kFewCtas>();
    return e ? e : raise_types<64, true, kFewCtas>();
}

int kv4_multiprocessors() {
    // once per device: the kernels' shared-memory limits and the number of multiprocessors
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return 0;
    }
    n = known[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || prepare_kv4_attend() != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    known[dev].store(n, std::memory_order_relaxed);
    return n;
}

cudaError_t launch_kv4_attend(const Kv4Attend &a, int in_bf16, int out_bf16, bool pdl, cudaStream_t s) {
    if (a.B == 0) return cudaSuccess;
    return a.c.head_dim == 128 ? launch_hd<128>(a, in_bf16, out_bf16, pdl, s) : launch_hd<64>(a, in_bf16, out_bf16, pdl, s);
}

}  // namespace talker_k

using namespace talker_k;

namespace {

bool attend_sizes_ok(const talker_kv4 *c, int B, int n_q, int max_len) {
    return kv4_cache_ok(c) && B >= 0 && B <= c->n_streams && B <= 65535 && c->n_kv_heads <= 65535 && max_len >= 0 && n_q >= 1 &&
           n_q % c->n_kv_heads == 0 && n_q / c->n_kv_heads <= kMaxG;
}

Kv4AttendShape shape_here(const talker_kv4 *c, int B, int max_len) {
    const int n_sm = std::max(kv4_multiprocessors(), 1);
    return kv4_attend_shape(B, c->n_kv_heads, c->head_dim, std::min(max_len, c->pages_per_stream * kPage), n_sm);
}

talker_status attend_call(const talker_kv4 *c, int layer, int B, const int32_t *lens, int max_len, int n_q_heads, float scale,
                          const void *q, int64_t q_row, const void *k_new, const void *v_new, int64_t new_row, int in_dtype,
                          int out_dtype, void *out, void *scratch, size_t scratch_bytes, void *cuda_stream) {
    if (!attend_sizes_ok(c, B, n_q_heads, max_len) || layer < 0 || layer >= c->n_layers) return TALKER_EINVAL;
    if (!lens || !q || !out || (k_new == nullptr) != (v_new == nullptr)) return TALKER_EINVAL;
    if (in_dtype != TALKER_DTYPE_F32 && in_dtype != TALKER_DTYPE_BF16) return TALKER_EINVAL;
    const uintptr_t size = in_dtype == TALKER_DTYPE_F32 ? 4 : 2, out_size = out_dtype == TALKER_DTYPE_F32 ? 4 : 2;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) % size ||
        reinterpret_cast<uintptr_t>(out) % out_size)
        return TALKER_EINVAL;
    const Kv4AttendShape shape = shape_here(c, B, max_len);
    const size_t need = kv4_attend_scratch(shape, c->head_dim);
    if (need > 0 && (!scratch || scratch_bytes < need || (reinterpret_cast<uintptr_t>(scratch) & 15u))) return TALKER_EINVAL;
    const Kv4Attend a{*c, layer, B, n_q_heads, lens, q, k_new, v_new, q_row, new_row, out, scale, shape.grid, shape.one_unit, shape.ctas,
                      static_cast<float *>(scratch)};
    if (launch_kv4_attend(a, in_dtype == TALKER_DTYPE_BF16, out_dtype == TALKER_DTYPE_BF16, false,
                          static_cast<cudaStream_t>(cuda_stream)) != cudaSuccess) {
        cudaGetLastError();
        return TALKER_ECUDA;
    }
    return TALKER_OK;
}

}  // namespace

extern "C" {

size_t talker_kv4_attend_scratch(const talker_kv4 *c, int B, int n_q_heads, int max_len) {
    if (!attend_sizes_ok(c, B, n_q_heads, max_len)) return 0;
    return kv4_attend_scratch(shape_here(c, B, max_len), c->head_dim);
}

talker_status talker_kv4_attend(const talker_kv4 *c, int layer, int B, const int32_t *lens, int max_len, int n_q_heads,
                                float scale, const void *q, int64_t q_row, const void *k_new, const void *v_new,
                                int64_t new_row, int dtype, void *out, void *scratch, size_t scratch_bytes,
                                void *cuda_stream) {
    return attend_call(c, layer, B, lens, max_len, n_q_heads, scale, q, q_row, k_new, v_new, new_row, dtype, dtype, out, scratch,
                       scratch_bytes, cuda_stream);
}

talker_status talker_test_kv4_attend_mixed(const talker_kv4 *c, int B, const int32_t *lens, int max_len, int n_q_heads,
                                           float scale, const float *q, void *out_bf16, void *scratch, size_t scratch_bytes,
                                           void *cuda_stream) {
    if (!c) return TALKER_EINVAL;
    return attend_call(c, 0, B, lens, max_len, n_q_heads, scale, q, (int64_t)n_q_heads * c->head_dim, nullptr, nullptr, 0,
                       TALKER_DTYPE_F32, TALKER_DTYPE_BF16, out_bf16, scratch, scratch_bytes, cuda_stream);
}

}  // extern "C"
