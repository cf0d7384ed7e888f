// Beam selection (talker_beam_select): per sequence the best `width` of width * vocab continuations.
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "kv4.cuh"
#include "talker_kv4.h"

namespace cg = cooperative_groups;
using namespace talker_dev;
using namespace talker_k;

namespace {

constexpr int kWarps = 8;
constexpr int kMaxWidth = 32;
constexpr int kMaxChunks = 32;      // parts of a row: the lists that one warp joins, a lane each
constexpr int kCluster = 8;
constexpr int kRowEntries = 544;    // best logits of a row's parts, at most (k_beam_choose holds a row's for each warp)
constexpr int kClusterTasks = 128, kClusterEntries = 3200;   // parts of a sequence and their best logits, in a cluster
constexpr float kMasked = -1e30f;   // at or below: counts as -inf
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLeastRef = -9.9999994e29f;   // reference of a row's exponents without a logit: the next value above kMasked
static_assert(kLeastRef > kMasked && kLeastRef - kMasked < 1e23f, "next to one another");

// Masked values (and NaN) as kMasked, the lowest value that is told apart.
__device__ __forceinline__ float unmask(float x) { return fmaxf(x, kMasked); }

// A logit and where it is in its row. rank: its value as a whole number of the same order, above 0.
struct Entry {
    uint32_t rank, index;
};
__device__ __forceinline__ uint32_t rank_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);   // (-0 ranks as 0: equal values are ordered by their index)
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t rank) {
    return __uint_as_float(rank & 0x80000000u ? rank & 0x7fffffffu : ~rank);
}
__device__ __forceinline__ float ex2(float x) {   // relative error about 2^-22, 0 at -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {   // NaN only if all are
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
// log2(x) for a normal x, to about 1e-10: x = 2^k f with f in [0.7, 1.5), log f = 2 atanh(z) by its
// series in z = (f - 1) / (f + 1), |z| < 0.2, a quotient in f32 and its remainder. (Sums of exponentials meet here; scores next to one
// another are told apart in 64 bits, in which the general logarithm would take most of a small call.)
__device__ __forceinline__ double log2_near(float x) {
    const int bits = __float_as_int(x), k = (bits - 0x3f333333) >> 23;
    const float f = __int_as_float(bits - (k << 23)), r = __frcp_rn(f + 1.f), near = (f - 1.f) * r;
    const double z = fma(fma(-(double)near, (double)f + 1.0, (double)f - 1.0), (double)r, (double)near), q = z * z;
    double t = 1.0 / 15.0;
    t = fma(t, q, 1.0 / 13.0);
    t = fma(t, q, 1.0 / 11.0);
    t = fma(t, q, 1.0 / 9.0);
    t = fma(t, q, 1.0 / 7.0);
    t = fma(t, q, 1.0 / 5.0);
    t = fma(t, q, 1.0 / 3.0);
    t = fma(t, q, 1.0);
    return fma(2.885390081777926814 * z, t, (double)k);   // 2 / log 2
}

struct Args {
    const void *logits;
    int64_t row_stride;
    const float *scores;
    const int32_t *ended;
    int width, vocab, eos;
    int32_t *tokens, *parents, *ended_out;
    float *scores_out;
    int chunks;       // parts of a row
    Entry *best;      // scratch: [row][chunk][width], best first
    float2 *sums;     // scratch: [row][chunk] (reference c, sum of e^(x - c))
};

// What a warp has seen of a row: lane i < width holds the i-th best logit (-inf: none yet); every lane
// has its part of the sum of e^(x - c) and its reference c, its largest logit (at least kLeastRef, below
// which masked values, and lanes that have none, add nothing). The difference comes before the factor log2 e:
// for logits of any size it is exact or of its own size's bits, while kLog2e x - c in one multiply-add would leave
// half a step of kLog2e x, 2^16 where x is 1e12. A logit that is not above `least` is not among the best any more.
struct Seen {
    float value;
    uint32_t index;
    float least, c, sum;

    __device__ __forceinline__ Entry entry() const { return {value == -INFINITY ? 0 : rank_of(value), index}; }
    __device__ __forceinline__ void insert(float x, uint32_t i, int width) {   // the same in all lanes
        const int lane = threadIdx.x & 31;
        const int at = __popc(__ballot_sync(0xffffffffu, value > x || (value == x && index < i)));
        const float v = __shfl_up_sync(0xffffffffu, value, 1);
        const uint32_t k = __shfl_up_sync(0xffffffffu, index, 1);
        if (lane > at) value = v, index = k;
        if (lane == at) value = x, index = i;
        if (lane >= width) value = -INFINITY, index = 0xffffffffu;
        least = fmaxf(least, __shfl_sync(0xffffffffu, value, width - 1));
    }
};

// kVecs vectors of N logits per lane; tops: each one's largest, on(v): it exists; at(v, l): the index
// of lane l's first. Those above `least` are inserted, in the order of their indexes, so a later equal
// one never replaces another.
template <int N, int kVecs, typename At>
__device__ __forceinline__ void insert_all(Seen &s, const float (&x)[N * kVecs], const float (&tops)[kVecs], At at, int width) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        uint32_t lanes = __ballot_sync(0xffffffffu, tops[v] > s.least);
        while (lanes != 0) {
            const int from = __ffs(lanes) - 1;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float y = __shfl_sync(0xffffffffu, x[v * N + i], from);
                if (y > s.least) s.insert(y, at(v, from) + i, width);
            }
            lanes &= lanes - 1;
            lanes &= __ballot_sync(0xffffffffu, tops[v] > s.least);
        }
    }
}
__device__ __forceinline__ void refer(Seen &s, float top) {   // the lane's reference to at least top
    if (top > s.c) {
        s.sum *= ex2((s.c - top) * kLog2e);
        s.c = top;
    }
}
// Any logits: masked values count as kMasked, and are inserted while there are too few others.
template <int N, int kVecs, typename On, typename At>
__device__ __forceinline__ void take(Seen &s, const float (&raw)[N * kVecs], On on, At at, int width) {
    float x[N * kVecs], tops[kVecs], top = kMasked;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        tops[v] = kMasked;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[v * N + i] = unmask(raw[v * N + i]);
            tops[v] = fmaxf(tops[v], x[v * N + i]);
        }
        top = fmaxf(top, tops[v]);
        if (!on(v)) tops[v] = -INFINITY;
    }
    refer(s, top);
#pragma unroll
    for (int i = 0; i < N * kVecs; ++i) s.sum += ex2((x[i] - s.c) * kLog2e);
    insert_all<N, kVecs>(s, x, tops, at, width);
}
// The same where `least` is at least kMasked (and vectors that do not exist hold masked values): those
// are not inserted any more, and add nothing to the sum as they are, but for NaN.
template <int N, int kVecs, typename At>
__device__ __forceinline__ void take_above(Seen &s, const float (&x)[N * kVecs], At at, int width) {
    float tops[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        tops[v] = max3(x[v * N], x[v * N + 1], x[v * N + 2]);
#pragma unroll
        for (int i = 3; i + 1 < N; i += 2) tops[v] = max3(tops[v], x[v * N + i], x[v * N + i + 1]);
        tops[v] = fmaxf(tops[v], x[v * N + N - 1]);
    }
    float top = fmaxf(tops[0], tops[1]);
#pragma unroll
    for (int v = 2; v < kVecs; ++v) top = fmaxf(top, tops[v]);
    refer(s, top);
    const F2 log2e = f2(kLog2e, kLog2e), c = f2(-s.c, -s.c);
    F2 sum = f2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N * kVecs; i += 2) {
        const F2 y = (f2(x[i], x[i + 1]) + c) * log2e;
        sum = sum + f2(ex2(f2_lo(y)), ex2(f2_hi(y)));
    }
    float both = f2_lo(sum) + f2_hi(sum);
    if (both != both) {
        both = 0.f;
#pragma unroll
        for (int i = 0; i < N * kVecs; ++i) both += ex2((unmask(x[i]) - s.c) * kLog2e);
    }
    s.sum += both;
    if (__any_sync(0xffffffffu, top > s.least)) insert_all<N, kVecs>(s, x, tops, at, width);
}

template <typename T>
struct Vec;   // 16 bytes of logits; pieces(p): those at p where p is a multiple of 4 but not of 16
template <>
struct Vec<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ void get(const uint4 &u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
    }
    __device__ static __forceinline__ uint4 pieces(const float *p) {
        if (reinterpret_cast<uintptr_t>(p) % 8 == 0) {   // (the same in all lanes)
            const uint2 a = __ldg(reinterpret_cast<const uint2 *>(p)), b = __ldg(reinterpret_cast<const uint2 *>(p) + 1);
            return make_uint4(a.x, a.y, b.x, b.y);
        }
        const uint32_t *w = reinterpret_cast<const uint32_t *>(p);
        return make_uint4(__ldg(w), __ldg(w + 1), __ldg(w + 2), __ldg(w + 3));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static __forceinline__ void get(const uint4 &u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = bf16lo(w[i]), x[2 * i + 1] = bf16hi(w[i]);
    }
    __device__ static __forceinline__ uint4 pieces(const __nv_bfloat16 *p) {
        return Vec<float>::pieces(reinterpret_cast<const float *>(p));
    }
};
// Eight bf16 logits at an odd place: the three words between the first and the last one, and the last; the first.
__device__ __forceinline__ uint4 odd_pieces(const void *p, uint32_t &first) {
    const unsigned short *h = static_cast<const unsigned short *>(p);
    const uint32_t *w = reinterpret_cast<const uint32_t *>(h + 1);
    first = __ldg(h);
    return make_uint4(__ldg(w), __ldg(w + 1), __ldg(w + 2), __ldg(h + 7));
}
__device__ __forceinline__ uint4 odd_joined(const uint4 &u, uint32_t first) {
    return make_uint4(__byte_perm(first, u.x, 0x5410), __byte_perm(u.x, u.y, 0x5432), __byte_perm(u.y, u.z, 0x5432),
                      __byte_perm(u.z, u.w, 0x5432));
}

// Of n <= 32 * kPer ranks, the width-th highest (0 if there are fewer), by one warp: so many logits rank
// at least as high, and nothing below it is among the best. Without such a floor most of a part's first
// logits would be inserted and pushed out again.
template <int kPer>
__device__ __forceinline__ uint32_t floor_of(uint32_t (&r)[kPer], int width) {
    const int lane = threadIdx.x & 31;
    uint32_t floor = 0;
    for (int j = 0; j < width; ++j) {
        uint32_t top = r[0];
#pragma unroll
        for (int i = 1; i < kPer; ++i) top = max(top, r[i]);
        floor = __reduce_max_sync(0xffffffffu, top);
        if (lane == __ffs(__ballot_sync(0xffffffffu, top == floor)) - 1) {
            bool gone = false;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (!gone && r[i] == floor) r[i] = 0, gone = true;
        }
    }
    return floor;
}

// One warp reads part `chunk` of a row once, by 16-byte loads where the row lies on 16 bytes. The row's
// maximum and sum of exponentials come from the same pass as its best logits. Parts, vectors and lanes are
// counted from the row's first logit wherever it lies, so that the sum's rounding depends on the row's values alone: equal
// beams have equal scores. (Parts of aligned vectors, with the logits before the first one for themselves, gave
// equal rows sums that differed in their last bits.) tops: where the CTA's warps all read parts of one row,
// shared memory for their lanes' largest logits of the first vectors, from which they take one floor.
template <typename T>
__device__ Seen read_part(const Args &a, int row, int chunk, uint32_t *tops) {
    constexpr int N = Vec<T>::N, kAhead = 16 / N;
    const int lane = threadIdx.x & 31;
    const T *x = static_cast<const T *>(a.logits) + row * a.row_stride;
    const bool aligned = reinterpret_cast<uintptr_t>(x) % 16 == 0, odd = sizeof(T) == 2 && reinterpret_cast<uintptr_t>(x) % 4 != 0;
    const int vectors = a.vocab / N;                            // whole ones
    const int v0 = (int)((long long)vectors * chunk / a.chunks), v1 = (int)((long long)vectors * (chunk + 1) / a.chunks);
    Seen s{-INFINITY, 0xffffffffu, -INFINITY, kLeastRef, 0.f};
    uint4 next[kAhead];
    uint32_t first[kAhead];   // (odd rows)
    auto request = [&](int v) {
        if (aligned) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (v + 32 * i + lane < v1) next[i] = ldg_stream(x + (size_t)(v + 32 * i + lane) * N);
        } else if (odd) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (v + 32 * i + lane < v1) next[i] = odd_pieces(x + (size_t)(v + 32 * i + lane) * N, first[i]);
        } else {
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (v + 32 * i + lane < v1) next[i] = Vec<T>::pieces(x + (size_t)(v + 32 * i + lane) * N);
        }
    };
    request(v0);
#pragma unroll 1
    for (int v = v0; v < v1 || (v == v0 && tops != nullptr); v += 32 * kAhead) {
        uint4 u[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) u[i] = odd ? odd_joined(next[i], first[i]) : next[i];
        request(v + 32 * kAhead);
        float f[kAhead * N];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            float g[N];
            Vec<T>::get(u[i], g);
#pragma unroll
            for (int e = 0; e < N; ++e) f[i * N + e] = g[e];
        }
        if (v + 32 * kAhead > v1) {   // the last ones
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (v + 32 * i + lane >= v1) {
#pragma unroll
                    for (int e = 0; e < N; ++e) f[i * N + e] = kMasked;
                }
        }
        if (v == v0) {
            float m = kMasked;
#pragma unroll
            for (int i = 0; i < kAhead * N; ++i) m = fmaxf(m, f[i]);
            const uint32_t top = v + lane < v1 ? rank_of(m) : 0;
            uint32_t floor;
            if (tops != nullptr) {
                uint32_t r[kWarps];
                tops[threadIdx.x] = top;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kWarps; ++i) r[i] = tops[32 * i + lane];
                __syncthreads();
                floor = floor_of(r, a.width);
            } else {
                uint32_t r[1] = {top};
                floor = floor_of(r, a.width);
            }
            // the next value below it (below 0 that is not -0)
            if (floor > 0) s.least = fmaxf(s.least, value_of(floor - (floor == 0x80000000u ? 2 : 1)));
        }
        const auto at = [&](int i, int l) { return (uint32_t)((v + 32 * i + l) * N); };
        if (s.least >= kMasked) take_above<N, kAhead>(s, f, at, a.width);
        else take<N, kAhead>(s, f, [&](int i) { return v + 32 * i + lane < v1; }, at, a.width);
    }
    const int t = vectors * N;
    if (chunk == a.chunks - 1 && t < a.vocab) {   // fewer than a vector
        const float one[1] = {t + lane < a.vocab ? (float)x[t + lane] : kMasked};
        take<1, 1>(s, one, [&](int) { return t + lane < a.vocab; }, [&](int, int l) { return (uint32_t)(t + l); }, a.width);
    }
    const float c = warp_max(s.c);
    s.sum = warp_sum(s.sum * ex2((s.c - c) * kLog2e));
    s.c = c;
    return s;
}

// A row's beam, as its candidates see it. They score their logit less `ref`, the row's largest (exactly, so that
// a score is not lost beside large logits), plus `offset`, the beam's score less the logarithm of the row's sum; an
// ended beam goes on with the end token alone, at its own score (which is the offset then); all of a dead
// one's are at -inf.
struct Beam {
    double offset;
    float ref;
    bool dead, ended;
};
struct Choice {   // shared memory of choose()
    Beam beams[kMaxWidth];
    unsigned long long ranks[kMaxWidth * kMaxWidth];   // of the candidates; before, the joined lists: rank << 32 | index
    int tokens[kMaxWidth * kMaxWidth];
};

// The scores and end marks of the rows that a warp joins: lane i has those of row warp + kWarps i.
struct Given {
    float score = 0.f;
    int ended = 0;
};
__device__ __forceinline__ Given given(const Args &a, int seq) {
    Given g;
    const int w = (threadIdx.x >> 5) + kWarps * (threadIdx.x & 31);
    if (w < a.width) {
        g.score = a.scores[seq * a.width + w];
        if (a.ended != nullptr) g.ended = a.ended[seq * a.width + w];
    }
    return g;
}

// The parts of a sequence's rows joined and its continuations chosen, by one CTA of kWarps warps. best,
// sums: [row of the sequence][part]; stage: room for a row's lists for each warp, or null. Where a
// sequence has more than a warp's lists, a warp joins each row's first (into c.ranks). All candidates'
// scores are then made at once, in 64 bits, as whole numbers of the same order; and one warp, a lane to
// a list, takes the best of the lists' heads `width` times.
__device__ void choose(const Args &a, int seq, const Given &g, const Entry *best, const float2 *sums, Choice &c, Entry *stage) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool join = a.width * a.chunks > 32;
    const int lists = join ? 1 : a.chunks;   // of a row
    for (int w = warp; w < a.width; w += kWarps) {
        const bool part = lane < a.chunks;
        const Entry *list = best + (size_t)w * a.chunks * a.width;
        const float2 cs = part ? sums[w * a.chunks + lane] : make_float2(kLeastRef, 0.f);
        if (join && stage != nullptr) {   // from global memory: all at once, not a list's entries one after another
            Entry *mine = stage + warp * a.chunks * a.width;
            __syncwarp();
            for (int i = lane; i < a.chunks * a.width; i += 32) mine[i] = list[i];
            __syncwarp();
            list = mine;
        }
        const float ref = warp_max(cs.x), sum = warp_sum(cs.y * ex2((cs.x - ref) * kLog2e));
        const float score = __shfl_sync(0xffffffffu, g.score, w / kWarps);
        const int ended = __shfl_sync(0xffffffffu, g.ended, w / kWarps);
        if (lane == 0) {
            // no candidate above -inf: a masked score, or a row of masked logits (whose sum is 0) or with an infinite one
            const bool dead = !(score > kMasked && score < INFINITY) || (!ended && !(sum > 0.f && ref < INFINITY));
            const double ls = dead || ended ? 0.0 : log2_near(sum) * 0.69314718055994530942;
            c.beams[w] = {(double)score - ls, ref, dead, ended != 0};
        }
        if (!join) continue;
        list += lane * a.width;
        int at = 0;
        Entry head = part ? list[0] : Entry{0, 0};
        for (int j = 0; j < a.width; ++j) {
            const uint32_t rank = __reduce_max_sync(0xffffffffu, head.rank);
            const uint32_t index = __reduce_min_sync(0xffffffffu, head.rank == rank ? head.index : 0xffffffffu);
            if (lane == 0) c.ranks[w * a.width + j] = (unsigned long long)rank << 32 | index;
            if (head.rank == rank && head.index == index && rank != 0) head = ++at < a.width ? list[at] : Entry{0, 0};
        }
    }
    __syncthreads();
    const int n = a.width * lists;   // lists, in the order of rows and indexes
    for (int i = threadIdx.x; i < n * a.width; i += kWarps * 32) {
        const int l = i / a.width, at = i - l * a.width;
        const Beam b = c.beams[l / lists];
        Entry e = join ? Entry{(uint32_t)(c.ranks[i] >> 32), (uint32_t)c.ranks[i]} : best[i];
        double score = -INFINITY;
        bool there = e.rank != 0;
        if (!b.dead && !b.ended) {
            const float x = value_of(e.rank);
            if (x > kMasked) score = ((double)x - (double)b.ref) + b.offset;
        } else {   // one list, in order of tokens after the end token
            there = l % lists == 0;
            e.index = b.dead ? at : at == 0 ? a.eos : at - 1 + (at - 1 >= a.eos);
            if (!b.dead && at == 0) score = b.offset;
        }
        const unsigned long long u = (unsigned long long)__double_as_longlong(score + 0.0);
        c.ranks[i] = !there ? 0 : u >> 63 ? ~u : u | 1ull << 63;   // 0: none
        c.tokens[i] = (int)e.index;
    }
    __syncthreads();
    if (warp != 0) return;
    int at = lane * a.width;
    const int end = at + (lane < n ? a.width : 0);
    unsigned long long rank = at < end ? c.ranks[at] : 0;
    for (int j = 0; j < a.width; ++j) {
        const uint32_t hi = (uint32_t)(rank >> 32), top = __reduce_max_sync(0xffffffffu, hi);
        const uint32_t lo = hi == top ? (uint32_t)rank : 0, low = __reduce_max_sync(0xffffffffu, lo);
        if (lane == __ffs(__ballot_sync(0xffffffffu, hi == top && lo == low)) - 1) {
            const int out = seq * a.width + j, w = lane / lists, token = c.tokens[at];
            const unsigned long long u = rank >> 63 ? rank & ~(1ull << 63) : ~rank;
            a.tokens[out] = token;
            a.parents[out] = seq * a.width + w;
            a.scores_out[out] = (float)__longlong_as_double((long long)u);
            if (a.ended_out != nullptr) a.ended_out[out] = c.beams[w].ended || token == a.eos;
            rank = ++at < end ? c.ranks[at] : 0;
        }
    }
}

// One cluster per sequence (gridDim.x / n_seq CTAs): its warps share the parts, whose results go to
// the first CTA's shared memory, which joins them. No scratch, one launch. Bound by latencies: 4 rows of 2048
// take 7.0 us, of which a launch is 2.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_beam_cluster(const Args a) {
    __shared__ Entry best[kClusterEntries];
    __shared__ Choice choice;
    __shared__ float2 sums[kClusterTasks];
    __shared__ uint32_t tops[kWarps * 32];
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = cluster.num_blocks(), rank = cluster.block_rank(), seq = blockIdx.x / ctas;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Entry *best0 = cluster.map_shared_rank(best, 0);
    float2 *sums0 = cluster.map_shared_rank(sums, 0);
    Given g;
    if (rank == 0) g = given(a, seq);
    cluster.sync();   // every CTA's shared memory is there
    for (int t = rank * kWarps + warp; t < a.width * a.chunks; t += ctas * kWarps) {
        const Seen s = read_part<T>(a, seq * a.width + t / a.chunks, t % a.chunks, a.chunks % kWarps == 0 ? tops : nullptr);
        if (lane < a.width) best0[(size_t)t * a.width + lane] = s.entry();
        if (lane == 0) sums0[t] = make_float2(s.c, s.sum);
    }
    cluster.sync();
    if (rank == 0) choose(a, seq, g, best, sums, choice, nullptr);
}

// Larger calls: a warp per part over the whole GPU, the results in scratch; then a CTA per sequence. 24 x 8
// rows of 100003 f32 logits (77 MB, 11.3 us at the measured copy rate) take 28: about 20 for the parts, whose
// warps spend over half of their 3700 instructions finding and inserting the best logits, 6 for the joining CTAs. Rows
// off 16 bytes, three of four here, cost 2 of them (of 100000 logits: 26); in bf16 29.5 (28).
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_beam_parts(const Args a, long long parts) {
    __shared__ uint32_t tops[kWarps * 32];
    const int lane = threadIdx.x & 31;
    const long long t = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= parts) return;
    const Seen s = read_part<T>(a, (int)(t / a.chunks), (int)(t % a.chunks), a.chunks % kWarps == 0 ? tops : nullptr);
    if (lane < a.width) a.best[t * a.width + lane] = s.entry();
    if (lane == 0) a.sums[t] = make_float2(s.c, s.sum);
    pdl_launch_dependents();   // (at the start 11 us more for 24 x 8 rows of 100003: its CTAs take the parts' room)
}
__global__ void __launch_bounds__(kWarps * 32) k_beam_choose(const Args a) {
    extern __shared__ Entry stage[];   // a row's lists for each warp
    __shared__ Choice choice;
    const Given g = given(a, blockIdx.x);   // (written before the parts began)
    pdl_wait();
    const size_t first = (size_t)blockIdx.x * a.width * a.chunks;
    choose(a, blockIdx.x, g, a.best + first * a.width, a.sums + first, choice, stage);
}

// How a call runs. A cluster serves a sequence until its CTAs would read over kClusterLogits each;
// then the parts are spread over the GPU, at least kPartLogits each. us by a cluster / over the GPU, of
// (sequences, beams, vocabulary) in f32: (1, 4, 2048) 7.4 / 7.5, (24, 8, 8000) 14.0 / 13.4, (1, 4, 32000) 9.9 / 9.2 (and
// a second launch for the host, about 3 us), (1, 4, 65000) 12.2 / 10.5, (64, 4, 50257) 26.2 / 23.7,
// (1, 8, 100003) 27.3 / 17.0, (1, 32, 32000) 95 / 47. Parts of 256 / 1024 / 4096 logits: (1, 4, 2048) 7.3 / 8.8 / 9.8,
// (4, 8, 4099) 10.9 / 14.3 / 20.6, (24, 8, 8000) 14.0 / 17.5 / 25.9.
struct Shape {
    int ctas;     // of the cluster, or 0: two launches
    int chunks;
};
constexpr int kClusterLogits = 16384, kPartLogits = 256;
constexpr int kTargetParts = 152 * 20;   // 24 x 8 rows of 100003: 28.2 us; 152 * 16: 28.2, 152 * 24: 28.5, 152 * 32: 34.1

Shape shape_of(int n_seq, int width, int vocab) {
    const long long logits = (long long)width * vocab;
    Shape p{1, 1};
    while (p.ctas < kCluster && logits > (long long)p.ctas * kWarps * kPartLogits) p.ctas *= 2;
    long long parts = (long long)p.ctas * kWarps;   // per sequence
    if (logits > (long long)kCluster * kClusterLogits) {
        p.ctas = 0;
        parts = (kTargetParts + n_seq - 1) / n_seq;
    }
    const long long most = std::max(1, std::min(kMaxChunks, vocab / kPartLogits));
    long long chunks = std::min(most, std::max(1ll, (parts + width - 1) / width));
    if (chunks > kWarps / 2) chunks = std::min(most, (chunks + kWarps / 2) / kWarps * kWarps);   // a CTA's warps in one row
    chunks = std::min<long long>(chunks, kRowEntries / width);
    if (p.ctas > 0) chunks = std::min<long long>(chunks, std::min(kClusterTasks, kClusterEntries / width) / width);
    if (chunks >= kWarps) chunks -= chunks % kWarps;
    p.chunks = (int)chunks;
    return p;
}

size_t align16(size_t n) { return (n + 15) / 16 * 16; }

bool sizes_ok(int n_seq, int width, int vocab) {
    return n_seq >= 0 && width >= 1 && width <= kMaxWidth && vocab >= width && vocab <= 1 << 30 && (long long)n_seq * width <= 0x7fffffffll / kMaxChunks;
}

}  // namespace

extern "C" {

size_t talker_beam_scratch(int n_seq, int width, int vocab) {
    if (!sizes_ok(n_seq, width, vocab)) return 0;
    const Shape p = shape_of(n_seq, width, vocab);
    const size_t parts = (size_t)n_seq * width * p.chunks;
    return p.ctas > 0 ? 0 : align16(parts * width * sizeof(Entry)) + parts * sizeof(float2);
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
    const size_t need = talker_beam_scratch(n_seq, width, vocab);
    if (need > 0 && (!scratch || scratch_bytes < need || (reinterpret_cast<uintptr_t>(scratch) & 15u))) return TALKER_EINVAL;
    const Shape p = shape_of(n_seq, width, vocab);
    Args a{logits, row_stride, scores, ended, width, vocab, eos_id, tokens, parents, ended_out, scores_out, p.chunks};
    const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    const bool f32 = dtype == TALKER_DTYPE_F32;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    if (p.ctas == 1) {
        if (f32) k_beam_cluster<float><<<n_seq, kWarps * 32, 0, st>>>(a);
        else k_beam_cluster<__nv_bfloat16><<<n_seq, kWarps * 32, 0, st>>>(a);
        e = cudaGetLastError();
    } else if (p.ctas > 1) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = p.ctas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3((unsigned)(n_seq * p.ctas));
        e = cudaLaunchKernelEx(&cfg, f32 ? k_beam_cluster<float> : k_beam_cluster<__nv_bfloat16>, a);
    } else {
        const long long parts = (long long)n_seq * width * p.chunks;
        const unsigned blocks = (unsigned)((parts + kWarps - 1) / kWarps);
        a.best = static_cast<Entry *>(scratch);
        a.sums = reinterpret_cast<float2 *>(static_cast<char *>(scratch) + align16((size_t)parts * width * sizeof(Entry)));
        if (f32) k_beam_parts<float><<<blocks, kWarps * 32, 0, st>>>(a, parts);
        else k_beam_parts<__nv_bfloat16><<<blocks, kWarps * 32, 0, st>>>(a, parts);
        e = cudaGetLastError();
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3((unsigned)n_seq);
        static_assert(sizeof(Choice) + kWarps * kRowEntries * sizeof(Entry) <= 48 * 1024, "k_beam_choose's shared memory");
        cfg.dynamicSmemBytes = width * p.chunks > 32 ? (size_t)kWarps * p.chunks * width * sizeof(Entry) : 0;
        if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, k_beam_choose, a);
    }
    if (e == cudaSuccess) return TALKER_OK;
    cudaGetLastError();
    return TALKER_ECUDA;
}

}  // extern "C"
