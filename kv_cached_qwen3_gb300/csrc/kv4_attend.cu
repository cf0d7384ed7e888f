// Decode attention over the 4-bit paged cache (talker_kv4_attend).
#include <algorithm>
#include <math.h>

#include "kv4.cuh"

using namespace talker_dev;

namespace talker_k {

namespace {

constexpr int kWarps = 4;
constexpr int kSlots = 2;                 // pages (K and V tile) a warp has in shared memory
constexpr int kMaxG = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 4.f;             // how far (base 2) scores may pass the reference before O is rescaled
constexpr float kTop = 1024.f;            // scaled value scales stay below this

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
// (lo, hi) as an fp16 pair, rounded towards zero
__device__ __forceinline__ uint32_t pack_rz(float lo, float hi) {
    uint32_t r;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// what is left of x after its first 11 bits (the fp16 part that pack_rz keeps)
__device__ __forceinline__ float rest11(float x, uint32_t mask) { return x - __uint_as_float(__float_as_uint(x) & mask); }
__device__ __forceinline__ uint32_t pack_half(__half lo, __half hi) {
    return (uint32_t)__half_as_ushort(lo) | ((uint32_t)__half_as_ushort(hi) << 16);
}
__device__ __forceinline__ float half_lo(uint32_t u) { return __half2float(__ushort_as_half((unsigned short)u)); }
__device__ __forceinline__ float half_hi(uint32_t u) { return __half2float(__ushort_as_half((unsigned short)(u >> 16))); }

// Nibbles 0 and 4 of u as an fp16 pair of (code - 8), and nibbles 1 and 5: the code goes under the
// exponent of 1024 (or as 16 code), where fp16 holds it exactly.
__device__ __forceinline__ uint32_t codes_even(uint32_t u) {
    const uint32_t x = (u & 0x000f000fu) | 0x64006400u;
    uint32_t r;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(0x64086408u));           // - 1032
    return r;
}
__device__ __forceinline__ uint32_t codes_odd(uint32_t u) {
    const uint32_t x = (u & 0x00f000f0u) | 0x64006400u;
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0x2c002c00u), "r"(0xd480d480u));   // / 16 - 72
    return r;
}

template <int N>
struct Words;
template <>
struct Words<4> {
    uint32_t w[4];
    __device__ __forceinline__ void load(uint32_t at) {
        const uint4 u = lds_u4(at);
        w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    }
};
template <>
struct Words<2> {
    uint32_t w[2];
    __device__ __forceinline__ void load(uint32_t at) {
        const uint2 u = lds_u2(at);
        w[0] = u.x, w[1] = u.y;
    }
};
template <>
struct Words<1> {
    uint32_t w[1];
    __device__ __forceinline__ void load(uint32_t at) { asm("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(at)); }
};

__device__ __forceinline__ bool bounded_wait(uint64_t *bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
    return true;
}

constexpr size_t attend_smem(int hd) {
    const size_t ring = (size_t)kWarps * kSlots * 2 * kv4_tile_bytes(hd), merge = (size_t)kWarps * kMaxG * hd * 4;
    return ring > merge ? ring : merge;
}

template <typename T>
__device__ __forceinline__ void load_dims8(const T *p, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)p[i];
}

// Pages of one stream per split: at least one for each warp.
__device__ __forceinline__ int pages_per_split(int npages, int splits) {
    return max(kWarps, (npages + splits - 1) / splits);
}
__device__ __forceinline__ int checked_len(const Kv4Attend &a, int b, bool report) {
    const int len = a.lens[b];
    if (len >= 0 && len <= a.c.pages_per_stream * kPage) return len;
    if (report && a.c.status != nullptr) atomicOr(a.c.status, ST_BAD_POSITION);
    return -1;
}

// Grid (splits, n_kv, B). Each warp of CTA (s, g, b) takes every fourth page of the CTA's range of
// stream b and KV head g through a ring of its own: bulk copies, no barrier between warps.
//
// A lane is (r = lane / 4, c = lane % 4). Scores of 8 keys, S[16 x 8] = Q K^T by m16n8k16: rows
// r and r + 8 of Q are the two fp16 parts of one query head, scaled by a power of two so that its
// largest value lies in [2^13, 2^14). K codes n enter as the fp16 subnormals n 2^-24 (and 16 n
// 2^-24, against q / 16): a nibble is its own operand after one AND. The accumulator starts at
// -8 sum(q) 2^-24 per block of 32 dims, and its two rows, added and multiplied by the key's scale,
// make the block's part of the score in f32.
// Values, O^T[dims x heads] += V^T P^T: V codes are centred in fp16 ((n - 8) exactly: with n as it
// is, 8 sum(p) would cancel), and the probabilities, times the value's scale of each block and a
// power of two, enter as two fp16 parts: with up to 4 query heads in columns h and h + 4 of one
// MMA (SPLIT 1), else by two MMAs. The score's layout is the P operand's: a lane keeps its keys.
template <int HD, bool WIDE, typename TI, typename TO>
__global__ void __launch_bounds__(kWarps * 32, 3) k_kv4_attend(const Kv4Attend a) {
    using Tile = Kv4Tile<HD>;
    constexpr int NB = Tile::NB;
    constexpr int kSlotBytes = 2 * Tile::kBytes;
    extern __shared__ __align__(128) unsigned char ring_all[];
    __shared__ __align__(8) uint64_t bars[kWarps][kSlots];
    __shared__ float wm[kWarps + 1][kMaxG], wl[kWarps + 1][kMaxG];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const int s = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
    const int G = a.n_q / a.c.n_kv_heads;
    pdl_launch_dependents();
    const int len = checked_len(a, b, threadIdx.x == 0 && s == 0);
    const int npages = len > 0 ? (len + kPage - 1) / kPage : 0;
    const int per = pages_per_split(npages, a.splits);
    const int pb = s * per, pe = min(pb + per, npages);
    if (s > 0 && pb >= pe) return;   // not among the stream's splits

    unsigned char *ring = ring_all + warp * kSlots * kSlotBytes;
    const int *ptab = a.c.page_table + (size_t)b * a.c.pages_per_stream;
    const size_t head_off = ((size_t)a.layer * a.c.n_kv_heads + g) * Tile::kBytes;
    const size_t page_bytes = (size_t)a.c.n_layers * a.c.n_kv_heads * Tile::kBytes;
    const int n_it = pb + warp < pe ? (pe - pb - warp + kWarps - 1) / kWarps : 0;
    // lane i holds the page number of iteration 32 j + i
    auto page_of = [&](int it) { return it < n_it ? ptab[pb + warp + it * kWarps] : 0; };
    auto good = [&](int page) { return page >= 0 && page < a.c.n_pages; };
    auto issue = [&](int slot, int page) {   // one lane; a bad page number copies page 0, which is not used
        const size_t off = (good(page) ? page : 0) * page_bytes + head_off;
        unsigned char *dst = ring + slot * kSlotBytes;
        mbar_arrive_expect_tx(&bars[warp][slot], kSlotBytes);
        bulk_g2s(dst, static_cast<const unsigned char *>(a.c.k) + off, Tile::kBytes, &bars[warp][slot]);
        bulk_g2s(dst + Tile::kBytes, static_cast<const unsigned char *>(a.c.v) + off, Tile::kBytes, &bars[warp][slot]);
    };
    int pages = page_of(lane), ahead = page_of(32 + lane);
    if (lane == 0) {
        for (int i = 0; i < kSlots; ++i) mbar_init(&bars[warp][i], 1);
        fence_barrier_init();
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        const int page = __shfl_sync(0xffffffffu, pages, i);
        if (lane == 0 && i < n_it) issue(i, page);
    }

    // this lane's query head (rows beyond G compute on zeros)
    const int hq = WIDE ? r : r & 3;
    const float cs = a.scale * kLog2e;
    uint32_t qf[NB][2][4];
    float corr[NB][2], fs;
    {
        float x[NB][8], top = 0.f;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            if (hq < G) {
                load_dims8(static_cast<const TI *>(a.q) + b * a.q_row + (size_t)(g * G + hq) * HD + nb * 32 + c * 8, x[nb]);
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
        fs = cs * exp2f((float)(24 - up));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float sh = 0.f, sl = 0.f;
            __half hi[8], lo[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = x[nb][i] * qs * (i & 1 ? 0.0625f : 1.f);
                hi[i] = __float2half_rn(y);
                lo[i] = __float2half_rn(y - __half2float(hi[i]));
                sh = fmaf(__half2float(hi[i]), i & 1 ? 16.f : 1.f, sh);
                sl = fmaf(__half2float(lo[i]), i & 1 ? 16.f : 1.f, sl);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                qf[nb][t][0] = pack_half(hi[2 * t], hi[2 * t + 4]);
                qf[nb][t][1] = pack_half(lo[2 * t], lo[2 * t + 4]);
                qf[nb][t][2] = pack_half(hi[2 * t + 1], hi[2 * t + 5]);
                qf[nb][t][3] = pack_half(lo[2 * t + 1], lo[2 * t + 5]);
            }
            sh += __shfl_xor_sync(0xffffffffu, sh, 1);
            sl += __shfl_xor_sync(0xffffffffu, sl, 1);
            sh += __shfl_xor_sync(0xffffffffu, sh, 2);
            sl += __shfl_xor_sync(0xffffffffu, sl, 2);
            corr[nb][0] = sh * (-8.f / 16777216.f);
            corr[nb][1] = sl * (-8.f / 16777216.f);
        }
    }

    float m = -INFINITY, l = 0.f;             // reference of the exponents, this lane's part of the sum
    float vs = 274877906944.f;                // 2^38: the power of two on value scales
    float o[2 * NB][4];                       // dims 32 (t / 2) + 4 r + 2 (t % 2) (+ 1 in the upper pair), heads 2 c, 2 c + 1
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
    const uint32_t lo_mask = WIDE || r >= 4 ? 0xffffe000u : 0u;
    const int krow = (r >> 1) + 4 * (r & 1);   // the key whose codes this lane loads, of the 8 of a score tile

    bool failed = false;
    for (int it = 0; it < n_it; ++it) {
        const int slot = it % kSlots;
        if (it > 0 && it % 32 == 0) {
            pages = ahead;
            ahead = page_of(it + 32 + lane);
        }
        if (__any_sync(0xffffffffu, !bounded_wait(&bars[warp][slot], (it / kSlots) & 1))) {
            // report, give the copies in flight their chance to land, and leave with a NaN
            if (lane == 0 && a.c.status != nullptr) atomicOr(a.c.status, ST_WAIT_TIMEOUT);
            for (int j = it; j < it + kSlots && j < n_it; ++j) bounded_wait(&bars[warp][j % kSlots], (j / kSlots) & 1);
            failed = true;
            m = __int_as_float(0x7fc00000);
            break;
        }
        const int page = __shfl_sync(0xffffffffu, pages, it % 32);
        const int valid = min(kPage, len - (pb + warp + it * kWarps) * kPage);
        if (!good(page)) {
            if (lane == 0 && a.c.status != nullptr) atomicOr(a.c.status, ST_BAD_ARG);
        } else {
            const uint32_t kt = smem_u32(ring + slot * kSlotBytes), vt = kt + Tile::kBytes;
            if (valid < kPage) {   // value scales past the length: zero (a stream's last page: never refilled)
                for (int i = valid * NB + lane; i < kPage * NB; i += 32)
                    *reinterpret_cast<unsigned short *>(ring + slot * kSlotBytes + Tile::kBytes + Tile::kScales + 2 * i) = 0;
                __syncwarp();
            }
            // scores, in base 2: key 8 j + c and 8 j + 4 + c
            float sc[8][2];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                Words<NB> k;
                k.load(kt + (8 * j + krow) * Tile::kRow + c * 4 * NB);
                Words<NB / 2> d0, d1;
                d0.load(kt + Tile::kScales + (8 * j + c) * NB * 2);
                d1.load(kt + Tile::kScales + (8 * j + 4 + c) * NB * 2);
                float s0 = 0.f, s1 = 0.f;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    float acc[4] = {corr[nb][0], corr[nb][0], corr[nb][1], corr[nb][1]};
                    const uint32_t w = k.w[nb], w8 = w >> 8;
                    mma16816(acc, qf[nb][0], w & 0x000f000fu, w & 0x00f000f0u);
                    mma16816(acc, qf[nb][1], w8 & 0x000f000fu, w8 & 0x00f000f0u);
                    s0 = fmaf(nb & 1 ? half_hi(d0.w[nb / 2]) : half_lo(d0.w[nb / 2]), acc[0] + acc[2], s0);
                    s1 = fmaf(nb & 1 ? half_hi(d1.w[nb / 2]) : half_lo(d1.w[nb / 2]), acc[1] + acc[3], s1);
                }
                sc[j][0] = s0 * fs;
                sc[j][1] = s1 * fs;
            }
            if (valid < kPage) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (8 * j + c >= valid) sc[j][0] = -INFINITY;
                    if (8 * j + 4 + c >= valid) sc[j][1] = -INFINITY;
                }
            }
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 8; ++j) mx = fmaxf(mx, fmaxf(sc[j][0], sc[j][1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // the largest value scale of the page (a NaN is no size)
            float dmax;
            {
                Words<NB / 2> d;
                __half2 h = __float2half2_rn(0.f);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    d.load(vt + Tile::kScales + (2 * lane + i) * NB * 2);
#pragma unroll
                    for (int u = 0; u < NB / 2; ++u) h = __hmax2(h, __habs2(*reinterpret_cast<__half2 *>(&d.w[u])));
                }
                const float t = fmaxf(__low2float(h), __high2float(h));
                dmax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(t)));
            }
            const bool grow = mx > m + kSlack, wider = dmax * vs >= kTop;
            if (__any_sync(0xffffffffu, grow) || wider) {
                const float mn = fmaxf(m, mx);
                float al = m == mn ? 1.f : ex2(m - mn);
                m = mn;
                l *= al;
                if (wider) {   // dmax vs goes to [2^9, 2^10)
                    const float nv = __uint_as_float((uint32_t)(127 + 9 + 127 - (int)(__float_as_uint(dmax) >> 23)) << 23);
                    al *= nv / vs;
                    vs = nv;
                }
                const float a0 = __shfl_sync(0xffffffffu, al, 8 * c), a1 = __shfl_sync(0xffffffffu, al, 8 * c + 4);
#pragma unroll
                for (int t = 0; t < 2 * NB; ++t) {
                    o[t][0] *= a0, o[t][1] *= a1;
                    o[t][2] *= a0, o[t][3] *= a1;
                }
            }
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {   // 16 keys: c, c + 4, c + 8, c + 12
                float p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p[i] = ex2(sc[2 * ks + (i >> 1)][i & 1] - m);
                    l += p[i];
                    p[i] *= vs;
                }
                Words<NB / 2> v[4], d[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i].load(vt + (16 * ks + 4 * i + c) * Tile::kRow + r * 2 * NB);
                    d[i].load(vt + Tile::kScales + (16 * ks + 4 * i + c) * NB * 2);
                }
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    float y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = p[i] * (nb & 1 ? half_hi(d[i].w[nb / 2]) : half_lo(d[i].w[nb / 2]));
                    uint32_t ph[2], pl[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (WIDE) ph[i] = pack_rz(y[2 * i], y[2 * i + 1]);
                        pl[i] = pack_rz(rest11(y[2 * i], lo_mask), rest11(y[2 * i + 1], lo_mask));
                    }
                    // bytes 2 (nb % 2) and the next of the four keys' words
                    const uint32_t sel = nb & 1 ? 0x7632 : 0x5410;
                    uint32_t u0 = __byte_perm(v[0].w[nb / 2], v[1].w[nb / 2], sel);
                    uint32_t u1 = __byte_perm(v[2].w[nb / 2], v[3].w[nb / 2], sel);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t va[4] = {codes_even(u0), codes_odd(u0), codes_even(u1), codes_odd(u1)};
                        if (WIDE) mma16816(o[2 * nb + e], va, ph[0], ph[1]);
                        mma16816(o[2 * nb + e], va, pl[0], pl[1]);
                        u0 >>= 8;
                        u1 >>= 8;
                    }
                }
            }
        }
        __syncwarp();
        const int next = it + kSlots;
        const int np = __shfl_sync(0xffffffffu, next / 32 == it / 32 ? pages : ahead, next % 32);
        if (lane == 0 && next < n_it) {
            fence_proxy_async();
            issue(slot, np);
        }
    }

    // the warp's (m, l, O) to shared memory, over the ring
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (failed) l = m;
    __syncthreads();
    float *wo = reinterpret_cast<float *>(ring_all);   // [kWarps][kMaxG][HD]
    const float down = 1.f / vs;
    if (c == 0 && r == hq) wm[warp][hq] = m, wl[warp][hq] = l;
#pragma unroll
    for (int t = 0; t < 2 * NB; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float x = o[t][e] * down;
            if (!WIDE) x += __shfl_xor_sync(0xffffffffu, x, 2);   // the parts of head h: columns h and h + 4
            const int h = 2 * c + (e & 1), dim = 32 * (t >> 1) + 4 * r + 2 * (t & 1) + (e >> 1);
            if (WIDE || c < 2) wo[(warp * kMaxG + h) * HD + dim] = x;
        }
    // the step's own row, as one more part of split 0
    const bool fresh = s == 0 && len >= 0 && a.k_new != nullptr;
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
    const int nact = (npages + per - 1) / per;
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
        const size_t row = (size_t)b * a.n_q + g * G + h;
        if (nact <= 1) {
            static_cast<TO *>(a.out)[row * HD + d] = (TO)(L == 0.f ? 0.f : O / L);
        } else {
            float *ws = a.scratch + (row * a.splits + s) * (HD + 4);
            ws[4 + d] = O;
            if (d == 0) ws[0] = M, ws[1] = L;
        }
    }
}

// Grid (n_q, B), HD threads: the splits' partials joined in split order.
template <int HD, typename TO>
__global__ void __launch_bounds__(HD) k_kv4_combine(const Kv4Attend a) {
    pdl_wait();
    const int b = blockIdx.y;
    const int npages = (max(checked_len(a, b, false), 0) + kPage - 1) / kPage;
    const int per = pages_per_split(npages, a.splits), nact = (npages + per - 1) / per;
    if (nact <= 1) return;   // written by its only split
    const size_t row = (size_t)b * a.n_q + blockIdx.x;
    const float *ws = a.scratch + row * a.splits * (HD + 4);
    float M = -INFINITY, L = 0.f, O = 0.f;
    for (int s = 0; s < nact; ++s) M = fmaxf(M, ws[s * (HD + 4)]);
    for (int s = 0; s < nact; ++s) {
        const float m = ws[s * (HD + 4)], e = m == -INFINITY ? 0.f : ex2(m - M);
        L = fmaf(ws[s * (HD + 4) + 1], e, L);
        O = fmaf(ws[s * (HD + 4) + 4 + threadIdx.x], e, O);
    }
    static_cast<TO *>(a.out)[row * HD + threadIdx.x] = (TO)(L == 0.f ? 0.f : O / L);
}

template <int HD, typename TI, typename TO>
cudaError_t launch_t(const Kv4Attend &a, cudaStream_t s) {
    const bool wide = a.n_q / a.c.n_kv_heads > 4;
    void (*kernel)(Kv4Attend) = wide ? k_kv4_attend<HD, true, TI, TO> : k_kv4_attend<HD, false, TI, TO>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)attend_smem(HD));
    if (e != cudaSuccess) return e;
    kernel<<<dim3(a.splits, a.c.n_kv_heads, a.B), kWarps * 32, attend_smem(HD), s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess || a.splits == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.n_q, a.B);
    cfg.blockDim = dim3(HD);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_kv4_combine<HD, TO>, a);
}

template <int HD>
cudaError_t launch_hd(const Kv4Attend &a, int in_bf16, int out_bf16, cudaStream_t s) {
    if (in_bf16) return out_bf16 ? launch_t<HD, __nv_bfloat16, __nv_bfloat16>(a, s) : cudaErrorInvalidValue;
    return out_bf16 ? launch_t<HD, float, __nv_bfloat16>(a, s) : launch_t<HD, float, float>(a, s);
}

}  // namespace

int kv4_attend_splits(int B, int n_kv, int head_dim, int max_len, int n_sm) {
    const long long rows = (long long)B * n_kv;
    const int pages = std::max(1, (int)(((long long)max_len + kPage - 1) / kPage));
    return (int)std::min<long long>(std::min(64, pages), std::max<long long>(1, (4ll * n_sm + rows - 1) / rows));
}

size_t kv4_attend_scratch(int B, int n_q, int head_dim, int splits) {
    return splits > 1 ? (size_t)B * n_q * splits * (head_dim + 4) * sizeof(float) : 0;
}

cudaError_t launch_kv4_attend(const Kv4Attend &a, int in_bf16, int out_bf16, cudaStream_t s) {
    if (a.B == 0) return cudaSuccess;
    return a.c.head_dim == 128 ? launch_hd<128>(a, in_bf16, out_bf16, s) : launch_hd<64>(a, in_bf16, out_bf16, s);
}

}  // namespace talker_k

using namespace talker_k;

namespace {

bool attend_sizes_ok(const talker_kv4 *c, int B, int n_q, int max_len) {
    return kv4_cache_ok(c) && B >= 0 && B <= c->n_streams && B <= 65535 && c->n_kv_heads <= 65535 && max_len >= 0 && n_q >= 1 &&
           n_q % c->n_kv_heads == 0 && n_q / c->n_kv_heads <= kMaxG;
}

int splits_here(const talker_kv4 *c, int B, int max_len) {
    int dev = 0, n_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        n_sm = 152;
    }
    return kv4_attend_splits(std::max(B, 1), c->n_kv_heads, c->head_dim, std::min(max_len, c->pages_per_stream * kPage), n_sm);
}

}  // namespace

extern "C" {

size_t talker_kv4_attend_scratch(const talker_kv4 *c, int B, int n_q_heads, int max_len) {
    if (!attend_sizes_ok(c, B, n_q_heads, max_len)) return 0;
    return kv4_attend_scratch(B, n_q_heads, c->head_dim, splits_here(c, B, max_len));
}

talker_status talker_kv4_attend(const talker_kv4 *c, int layer, int B, const int32_t *lens, int max_len, int n_q_heads,
                                float scale, const void *q, int64_t q_row, const void *k_new, const void *v_new,
                                int64_t new_row, int dtype, void *out, void *scratch, size_t scratch_bytes,
                                void *cuda_stream) {
    if (!attend_sizes_ok(c, B, n_q_heads, max_len) || layer < 0 || layer >= c->n_layers) return TALKER_EINVAL;
    if (!lens || !q || !out || (k_new == nullptr) != (v_new == nullptr)) return TALKER_EINVAL;
    if (dtype != TALKER_DTYPE_F32 && dtype != TALKER_DTYPE_BF16) return TALKER_EINVAL;
    const uintptr_t size = dtype == TALKER_DTYPE_F32 ? 4 : 2;
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(k_new) |
         reinterpret_cast<uintptr_t>(v_new)) % size)
        return TALKER_EINVAL;
    const int splits = splits_here(c, B, max_len);
    const size_t need = kv4_attend_scratch(B, n_q_heads, c->head_dim, splits);
    if (need > 0 && (!scratch || scratch_bytes < need || (reinterpret_cast<uintptr_t>(scratch) & 15u))) return TALKER_EINVAL;
    const Kv4Attend a{*c, layer, B, n_q_heads, lens, q, k_new, v_new, q_row, new_row, out, scale, splits,
                      static_cast<float *>(scratch)};
    const int bf16 = dtype == TALKER_DTYPE_BF16;
    if (launch_kv4_attend(a, bf16, bf16, static_cast<cudaStream_t>(cuda_stream)) != cudaSuccess) {
        cudaGetLastError();
        return TALKER_ECUDA;
    }
    return TALKER_OK;
}

}  // extern "C"
