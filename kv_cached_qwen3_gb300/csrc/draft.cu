// Verification of drafted tokens (include/talker_draft.h).
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <utility>

#include "common.cuh"
#include "kv4.cuh"
#include "talker_draft.h"

namespace cg = cooperative_groups;
using namespace talker_dev;
using namespace talker_k;

namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kCluster = 16;            // CTAs of a sequence, at most
constexpr int kMaxDraft = 64, kMaxRows = 2 * kMaxDraft + 1;
constexpr int kMaxParts = 32;           // of a row: a lane each where they are joined
constexpr int kOwnParts = kMaxRows + kCluster * kWarps;   // of a sequence, where its cluster reads its rows itself
constexpr float kMasked = -1e30f;       // at or below: counts as -inf
constexpr float kLeastRef = -9.9999994e29f;   // the next value above kMasked: the least reference of exponents, below which masked ones add nothing
constexpr float kGreedy = 1e-20f;       // a temperature not above it
constexpr float kHottest = 1e18f;       // a temperature above it counts as this one (masked logits still add nothing)
// Of f32 sums: decisions nearer to their border are made again, exactly. A p above 1e-30 has an exponent of at most 100, whose
// three roundings are 1.3e-5 of it; the terms of a sum that count have 46 at most (6e-6), and their additions add 1e-6 however
// long the row is (Lane). With ex2's own 2^-22, p and q are off by 2.5e-5 each at most.
constexpr float kNear = 1e-4f;
constexpr float kAbove = 16.f;          // a lane's reference is moved by terms of more than 2^16

struct Args {
    const void *target, *draft;
    long long target_seq, target_row, draft_seq, draft_row;
    const int32_t *tokens, *counts;
    const float *uniforms, *temperatures;
    int n_draft, vocab;
    int32_t *tokens_out, *accepted;
    float *logprobs;
    int parts;              // of a row
    int ctas;               // of a sequence's cluster
    struct Seen *seen;      // scratch: [sequence][row][part]
};

template <typename T>
__device__ __forceinline__ float load_logit(const T *p, int i) { return Elem<T>::load(p, i); }
__device__ __forceinline__ bool masked(float x) { return !(x > kMasked); }

// What is read of a sequence: target rows 0 .. count, then draft rows 0 .. count - 1, unless it is greedy.
struct Sequence {
    int count;
    float temperature;
    bool greedy, drafted;
    __device__ __forceinline__ int targets() const { return count + 1; }
    __device__ __forceinline__ int rows() const { return targets() + (drafted ? count : 0); }
};
__device__ __forceinline__ Sequence sequence(const Args &a, int seq) {
    Sequence s;
    s.count = a.counts ? min(max(a.counts[seq], 0), a.n_draft) : a.n_draft;
    s.temperature = a.temperatures ? fminf(a.temperatures[seq], kHottest) : 1.f;
    if (a.temperatures && isnan(a.temperatures[seq])) s.temperature = 0.f;
    s.greedy = !(s.temperature > kGreedy);
    s.drafted = a.draft != nullptr && !s.greedy;
    return s;
}
template <typename T>
__device__ __forceinline__ const T *row_at(const Args &a, const Sequence &s, int seq, int r) {
    return r < s.targets() ? static_cast<const T *>(a.target) + seq * a.target_seq + r * a.target_row
                           : static_cast<const T *>(a.draft) + seq * a.draft_seq + (r - s.targets()) * a.draft_row;
}

// A row's largest logit (kMasked where none counts), the first place that has it (of greedy sequences), and the sum of
// e^((x - ref) / T) (of others).
struct Seen {
    float most, sum;
    int first;
    __device__ __forceinline__ float ref() const { return fmaxf(most, kLeastRef); }
    __device__ __forceinline__ bool alive() const { return most > kMasked && most < INFINITY; }
};
__device__ __forceinline__ float ex2(float x) {   // relative error about 2^-22, 0 at -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// s.sum counts from `ref`.
__device__ __forceinline__ Seen warp_join(Seen s, float ref, float c) {
    Seen all;
    all.most = warp_max(s.most);
    all.sum = warp_sum(s.sum * ex2((ref - all.ref()) * c));
    all.first = (int)__reduce_min_sync(0xffffffffu, s.most == all.most ? (uint32_t)s.first : 0x7fffffffu);
    return all;
}

template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ void unpack(const uint4 u, float *x) {
        x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static __forceinline__ void unpack(const uint4 u, float *x) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = bf16lo(w[i]), x[2 * i + 1] = bf16hi(w[i]);
    }
};

// What a lane has seen, with sums whose error does not grow with the row: `lost` is what their roundings took off (Kahan), and
// `ref`, from which exponents count, is moved only by a term of more than 2^16, next to which an earlier sum's errors, the
// factor's own among them, are below 2^-16 of what they were. (One f32 sum, scaled anew whenever a larger logit came, was off by
// up to 2^-22 for each of a row's 2^14 vectors.)
struct Lane {
    Seen seen{kMasked, 0.f, 0x7fffffff};
    float ref = kLeastRef, lost = 0.f;
};
// n values, the first of them logit `at` of its row.
template <int N>
__device__ __forceinline__ void take(Lane &l, float (&x)[N], int at, float c, bool greedy) {
    Seen &s = l.seen;
    float top = kMasked;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = fmaxf(x[i], kMasked);   // NaN too
        top = fmaxf(top, x[i]);
    }
    if (greedy) {
        if (top > s.most) {
            s.most = top;
            int first = 0;
#pragma unroll
            for (int i = N - 1; i >= 0; --i)
                if (x[i] == top) first = i;
            s.first = at + first;
        }
        return;
    }
    s.most = fmaxf(s.most, top);
    if ((top - l.ref) * c > kAbove) {
        const float less = ex2((l.ref - top) * c);
        s.sum *= less, l.lost *= less;
        l.ref = top;
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) sum += ex2((x[i] - l.ref) * c);
    const float part = sum - l.lost, all = s.sum + part;
    l.lost = (all - s.sum) - part;
    s.sum = all;
}

// Part `part` of `parts` of a row, by one warp; c = log2 e / T. A part is so many of the row's vectors of 16 bytes; logits
// before the first and after the last are the first and the last part's.
template <typename T>
__device__ Seen see_part(const T *row, int vocab, int part, int parts, float c, bool greedy) {
    constexpr int N = Vec<T>::N, kAhead = 4;
    const int lane = threadIdx.x & 31;
    const int lead = min(vocab, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) % 16 / sizeof(T)));
    const int vecs = (vocab - lead) / N;
    const int from = (unsigned)vecs * part / parts, to = (unsigned)vecs * (part + 1) / parts;   // (2^24 times 32 at most)
    Lane s;
    if (part == 0 && lane < lead) {
        float x[1] = {load_logit(row, lane)};
        take(s, x, lane, c, greedy);
    }
    const uint4 *v = reinterpret_cast<const uint4 *>(row + lead);
    int i = from + lane;
    for (; i + (kAhead - 1) * 32 < to; i += kAhead * 32) {
        uint4 u[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) u[j] = ldg_stream(v + i + j * 32);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            float x[N];
            Vec<T>::unpack(u[j], x);
            take(s, x, lead + (i + j * 32) * N, c, greedy);
        }
    }
    for (; i < to; i += 32) {
        float x[N];
        Vec<T>::unpack(ldg_stream(v + i), x);
        take(s, x, lead + i * N, c, greedy);
    }
    const int tail = lead + vecs * N + lane;
    if (part == parts - 1 && tail < vocab) {
        float x[1] = {load_logit(row, tail)};
        take(s, x, tail, c, greedy);
    }
    return warp_join(s.seen, s.ref, c);
}

// e^((x - most) / T) = m 2^(-30 - shift), m in [2^30, 2^31), for x <= most, to about 2^-29 of itself. With
// t = (x - most) log2 e / T in two floats, t = k / 32 + f, |f| <= 1/64: m = 2^30 2^(k % 32 / 32) e^y, y = f log 2, by the
// series of e^y - 1, whose terms after y^4 / 24 are below 2^-39. Below 2^-70, and of masked logits: 0, by a shift that
// leaves nothing.
struct Exact {
    uint32_t m;
    int shift;
};
// v 2^32 >> s for any s (shifts of 32 or more give 0): five instructions, a 64-bit shift takes nine.
__device__ __forceinline__ unsigned long long place(uint32_t v, int s) {
    uint32_t hi, up, down;
    asm("shr.u32 %0, %1, %2;" : "=r"(hi) : "r"(v), "r"(s));
    asm("shl.b32 %0, %1, %2;" : "=r"(up) : "r"(v), "r"(32 - s));
    asm("shr.u32 %0, %1, %2;" : "=r"(down) : "r"(v), "r"(s - 32));
    return (unsigned long long)hi << 32 | (up | down);
}
struct Scale {   // log2 e / T in two floats
    float hi, lo;
};
__device__ __forceinline__ Scale scale_of(float temperature) {
    constexpr float kHi = 1.44269502162933349609375f, kLo = 1.92596299112661746887e-08f;   // log2 e
    const float hi = kHi / temperature;
    return {hi, (fmaf(-hi, temperature, kHi) + kLo) / temperature};
}
__constant__ uint32_t kRoots[32] = {   // 2^(31 + j / 32), to the nearest
    2147483648u, 2194507417u, 2242560872u, 2291666561u, 2341847524u, 2393127307u, 2445529972u, 2499080105u,
    2553802834u, 2609723834u, 2666869345u, 2725266179u, 2784941738u, 2845924021u, 2908241642u, 2971923842u,
    3037000500u, 3103502151u, 3171459999u, 3240905930u, 3311872529u, 3384393094u, 3458501653u, 3534232978u,
    3611622603u, 3690706840u, 3771522796u, 3854108391u, 3938502376u, 4024744348u, 4112874773u, 4202935003u};
// Two of them at once, in packed f32 arithmetic (half the instructions), with -most of each. Whole numbers come from f32
// sums with 1.5 2^23, whose last place is 1: conversions are a quarter as fast. Where the result is 0 what is made on the
// way means nothing. A difference of logits may not fit f32 (of bf16 ones neither: 16 and -2^-20), so what is left of it is
// carried along.
__device__ __forceinline__ void exact_exp2(float x0, float x1, F2 less, const Scale c, const uint32_t *roots, Exact &e0, Exact &e1) {
    constexpr float kWhole = 12582912.f;
    constexpr uint32_t kWholeBits = 0x4b400000u;
    constexpr float kLn2 = 0.693147182464599609375f, kLn2Lo = -1.904654299957768e-09f;   // log 2 in two floats
    // (what is named n... is the negative, so that no sign has to be changed)
    const F2 minus = f2(-1.f, -1.f), hi = f2(c.hi, c.hi), nhi = f2(-c.hi, -c.hi), nlo = f2(-c.lo, -c.lo);
    const F2 ln2 = f2(kLn2, kLn2), nln2 = f2(-kLn2, -kLn2), whole = f2(kWhole, kWhole), nwhole = f2(-kWhole, -kWhole);
    const F2 x = f2(x0, x1), d = x + less, t = d * hi;
    const F2 b = fma2(d, minus, x), dl = fma2(d + b, minus, x) + (b + less);   // x - most = d + dl, exactly
    const F2 nt = fma2(dl, nhi, fma2(d, nlo, fma2(d, nhi, t)));
    const F2 k = fma2(t, f2(32.f, 32.f), whole), f0 = fma2(k + nwhole, f2(-1.f / 32.f, -1.f / 32.f), t);
    const F2 f = fma2(nt, minus, f0), nf = nt + fma2(f0, minus, f);
    const F2 y = f * ln2, ny = fma2(f, f2(-kLn2Lo, -kLn2Lo), fma2(nf, ln2, fma2(f, nln2, y)));
    const F2 q = (y * y) * fma2(y, fma2(y, f2(1.f / 24.f, 1.f / 24.f), f2(1.f / 6.f, 1.f / 6.f)), f2(0.5f, 0.5f));
    // (e^y - 1) 2^31 = (y + q - ny) 2^31: y 2^15 as a whole number, what is left of it, and the rest
    const F2 y15 = fma2(y, f2(32768.f, 32768.f), whole), over = fma2(y, f2(-32768.f, -32768.f), y15 + nwhole);
    const F2 rest = fma2(ny, f2(-0x1p31f, -0x1p31f), fma2(q, f2(0x1p31f, 0x1p31f), fma2(over, f2(-65536.f, -65536.f), whole)));
    auto make = [&](float t, float k, float y15, float rest) -> Exact {
        constexpr uint32_t kOne = 0x80000000u - kWholeBits * 65536u - kWholeBits;   // 2^31 less the two sums' own bits
        const uint32_t e = __float_as_uint(y15) * 65536u + __float_as_uint(rest) + kOne, bits = __float_as_uint(k);   // 2^31 e^y
        return {__umulhi(roots[bits & 31], e), t > -70.f ? (int)((kWholeBits >> 5) - (bits >> 5)) : 256};
    };
    e0 = make(f2_lo(t), f2_lo(k), f2_lo(y15), f2_lo(rest));
    e1 = make(f2_hi(t), f2_hi(k), f2_hi(y15), f2_hi(rest));
}

__device__ __forceinline__ unsigned long long warp_sum64(unsigned long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The rows' parts, a warp each, for calls that a sequence's cluster would read too slowly. One pass: the running largest
// and the sum of exponentials. 24 sequences of up to 5 drafts of 100003 tokens, f32, both models' logits (58 MB): 14 us,
// 61% of the copy rate; a multiply-add, an exponential and two maxima a value, and a few additions a vector that keep the sum.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_draft_rows(const Args a) {
    const int seq = blockIdx.y, t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const Sequence q = sequence(a, seq);
    if (t < q.rows() * a.parts) {
        const int r = t / a.parts;
        const Seen s = see_part(row_at<T>(a, q, seq, r), a.vocab, t - r * a.parts, a.parts, scale_of(q.temperature).hi, q.greedy);
        if ((threadIdx.x & 31) == 0) a.seen[(size_t)seq * (2 * a.n_draft + 1) * a.parts + t] = s;
    }
    pdl_launch_dependents();
}

enum Verdict : int { kTake = 0, kRefuse = 1, kUnsure = 2 };

struct Shared {
    uint32_t roots[32];                        // 2^(31 + j / 32)
    Seen parts[kOwnParts];
    Seen rows[kMaxRows];                       // joined
    int verdict[kMaxDraft];
    unsigned long long warp[kWarps][2];
    unsigned long long cta[kCluster][2];       // every CTA's sums
};

// A row of probabilities: p = (m factor >> 32) 2^32 >> (down + shift), in units of 2^-62, of an Exact. (A row's largest has 2^(62 - bits) units
// of z: no shift to the left.)
struct Row {
    float most;
    uint32_t factor;        // 0: no distribution
    int down;
    unsigned long long z;   // the sum of e^((x - most) / T), in units of 2^(bits - 62); 0: not made
    int bits;
    __device__ __forceinline__ bool alive() const { return most > kMasked; }
    __device__ __forceinline__ void has(unsigned long long sum);
};
// 2^95 / z for z in [2^63, 2^64), in [2^31, 2^32), to about 2^-31 of itself: an f32 reciprocal and one step of Newton's
// method on the upper 32 bits. (f64 divisions by all threads of a CTA would take 3 us.)
__device__ __forceinline__ uint32_t reciprocal(unsigned long long z) {
    const uint32_t top = (uint32_t)(z >> 32);
    const uint32_t r = (uint32_t)fminf(0x1p63f / (float)top, 4294967040.f);
    const long long left = (long long)((1ull << 63) - (unsigned long long)r * top);   // 2^63 times what is missing of r, relative
    const long long better = (long long)r + (((long long)r * (left >> 31)) >> 32);
    return (uint32_t)min(better, 0xffffffffll);
}

__device__ __forceinline__ void Row::has(unsigned long long sum) {
    if (sum == 0) return;
    const int zeros = __clzll(sum);
    z = sum, factor = reciprocal(sum << zeros), down = 1 + bits - zeros;
}

// A cluster per sequence. f32 sums decide which drafts are surely taken and which first one is not; that one's rows, and
// those that the next token is drawn from, are gone over by all CTAs, each a range of the vocabulary, with exponentials of
// 29 bits and sums in whole numbers: which token a uniform number meets is a question of sums of 10^5 terms next to one
// another, where f32 would err once in some hundred draws.
// Small calls are a chain of latencies: a cluster's start, two or three of its barriers (a microsecond or two each), a
// draw (one sequence of 4 drafts of 2048 tokens: 9 us). Large ones make an exponential of some 25 instructions twice a token, once
// for the sums and once for the draw (the batch above: 30 us of 43 with its rows), but are bound by waits, not by their issue:
// with 28% of a multiprocessor's warps there (64 registers, clusters of unequal work) instructions are issued in 38% of the
// cycles, and most stalls are on loads and barriers. With f64, and the rows read by the cluster: 376 us; rows by the whole
// GPU 79; exponentials in packed f32 and sixteen CTAs 52; every CTA deciding by itself 46.
template <typename T, bool OWN>
__global__ void __launch_bounds__(kThreads, 4) k_draft_choose(const Args a) {
    __shared__ Shared s;
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = a.ctas, rank = cluster.block_rank(), seq = blockIdx.x / ctas;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int K = a.n_draft, V = a.vocab;
    auto arrived = cluster.barrier_arrive();
    const Sequence sq = sequence(a, seq);
    const int count = sq.count, n_rows = sq.rows();
    const bool greedy = sq.greedy, drafted = sq.drafted;
    const float temperature = sq.temperature;
    const Scale c = greedy ? Scale{1.f, 0.f} : scale_of(sq.temperature);
    const float *u = a.uniforms + (size_t)seq * (K + 1);
    const int32_t *tokens = a.tokens + (size_t)seq * K;
    if (tid < 32) s.roots[tid] = kRoots[tid];
    // a thread per draft
    int x = -1;
    float x_target = -INFINITY, x_draft = -INFINITY, x_u = 0.f;
    if (tid < count) {
        x = tokens[tid];
        x_u = fminf(fmaxf(u[tid], 0.f), 1.f);
        if (x >= 0 && x < V) {
            x_target = load_logit(row_at<T>(a, sq, seq, tid), x);
            if (drafted) x_draft = load_logit(row_at<T>(a, sq, seq, sq.targets() + tid), x);
        } else {
            x = -1;
        }
    }
    const float u_draw = fminf(fmaxf(u[K], 0.f), 1.f);
    cluster.barrier_wait(std::move(arrived));   // every CTA's shared memory is there

    if (OWN) {
        Shared *other = cluster.map_shared_rank(&s, lane < ctas ? lane : 0);
        for (int t = rank * kWarps + warp; t < n_rows * a.parts; t += ctas * kWarps) {
            const int r = t / a.parts;
            const Seen seen = see_part(row_at<T>(a, sq, seq, r), V, t - r * a.parts, a.parts, c.hi, greedy);
            if (lane < ctas) other->parts[t] = seen;
        }
        cluster.sync();
    } else {
        pdl_wait();
    }
    // every CTA makes the same decisions: a wait for one that tells them to the others takes 2 to 4 us
    {
        const Seen *parts = OWN ? s.parts : a.seen + (size_t)seq * (2 * K + 1) * a.parts;
        for (int r = warp; r < n_rows; r += kWarps) {
            const Seen one = lane < a.parts ? parts[r * a.parts + lane] : Seen{kMasked, 0.f, 0x7fffffff};
            const Seen seen = warp_join(one, one.ref(), c.hi);
            if (lane == 0) s.rows[r] = seen;
        }
        __syncthreads();
        if (tid < count) {
            const Seen p = s.rows[tid];
            int v = kRefuse;
            if (greedy) {
                v = p.alive() && x == p.first ? kTake : kRefuse;
            } else if (p.alive() && !masked(x_target)) {
                const float px = ex2((x_target - p.most) * c.hi) / p.sum;
                float qx = 1.f;
                if (drafted) {
                    const Seen q = s.rows[sq.targets() + tid];
                    qx = masked(x_draft) || !q.alive() ? 0.f : ex2((x_draft - q.most) * c.hi) / q.sum;
                }
                const float need = x_u * qx;
                // (an exponential that f32 cannot tell from 0 decides nothing)
                v = px > 1e-30f && need < px * (1.f - kNear) ? kTake : need > px * (1.f + kNear) && need > 1e-30f ? kRefuse : kUnsure;
            }
            s.verdict[tid] = v;
        }
        __syncthreads();
    }

    int n = 0, verdict;
    bool spent = false;   // s.cta may still be read
    Row p{}, q{};
    // Sums are of exponentials in units of 2^(bits - 62), m 2^32 >> bits + shift of an Exact, with what is left cut off. V of them fit
    // 64 bits with `whole`. Where what was cut off may be more than 2^-28 of a sum z (few tokens have most of a long row, or
    // the one that does is left out), the sum is made again in units that it needs; a whole number, it is the same
    // whatever the launch's shape, and so are the units.
    const int whole = 31 - __clz(max(V - 1, 1));
    auto finer = [&](unsigned long long z, int bits) {   // (z + V units are more than the sum)
        return z >> 28 >= (unsigned)V || bits <= -70 ? bits : max(-70, bits + 2 - __clzll(z + V));
    };
    // this CTA's range, and its warps'
    const int slice = (V + ctas - 1) / ctas, from = min(rank * slice, V), to = min(from + slice, V);
    const int each = (slice + kWarps - 1) / kWarps;
    const int w0 = min(from + warp * each, to), w1 = min(w0 + each, to);
    const T *rp = nullptr, *rq = nullptr;
    // a value or two of each thread, summed over every CTA, to all CTAs
    auto spread = [&](unsigned long long v0, unsigned long long v1) {
        v0 = warp_sum64(v0), v1 = warp_sum64(v1);
        if (lane == 0) s.warp[warp][0] = v0, s.warp[warp][1] = v1;
        __syncthreads();
        if (tid < 2 * ctas) {
            unsigned long long v = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += s.warp[w][tid & 1];
            cluster.map_shared_rank(&s, tid >> 1)->cta[rank][tid & 1] = v;
        }
        cluster.sync();
    };
    // f(exponential of token i of p, i), or f(p's, q's), for the warp's range
    auto over_one = [&](auto f) {
        const F2 less = f2(-p.most, -p.most);
#pragma unroll 2
        for (int i = w0 + lane; i < w1; i += 64) {
            Exact e, g;
            exact_exp2(load_logit(rp, i), i + 32 < w1 ? load_logit(rp, i + 32) : -INFINITY, less, c, s.roots, e, g);
            f(e, i);
            f(g, i + 32);
        }
    };
    auto over_both = [&](auto f) {
        const F2 less = f2(-p.most, -q.most);
#pragma unroll 2
        for (int i = w0 + lane; i < w1; i += 32) {
            Exact e, g;
            exact_exp2(load_logit(rp, i), load_logit(rq, i), less, c, s.roots, e, g);
            f(e, g);
        }
    };
    while (true) {
        while (n < count && s.verdict[n] == kTake) ++n;
        if (greedy) break;
        verdict = n < count ? s.verdict[n] : kRefuse;
        const bool has_q = drafted && n < count;
        p = Row{kMasked, 0, 0, 0, whole}, q = p;
        if (s.rows[n].alive()) p.most = s.rows[n].most;
        if (has_q && s.rows[sq.targets() + n].alive()) q.most = s.rows[sq.targets() + n].most;
        rp = row_at<T>(a, sq, seq, n);
        rq = has_q ? row_at<T>(a, sq, seq, sq.targets() + n) : nullptr;
        if (rq == nullptr && verdict == kRefuse) break;   // (drawn from p alone: its sum is the draw's)
        while (true) {
            unsigned long long sums[2] = {0, 0};
            if (p.alive() && q.alive())
                over_both([&](Exact e, Exact g) { sums[0] += place(e.m, p.bits + e.shift), sums[1] += place(g.m, q.bits + g.shift); });
            else if (p.alive())
                over_one([&](Exact e, int) { sums[0] += place(e.m, p.bits + e.shift); });
            if (spent) cluster.sync();   // (s.cta is free again)
            spread(sums[0], sums[1]);
            spent = true;
            unsigned long long z0 = 0, z1 = 0;
            for (int i = 0; i < ctas; ++i) z0 += s.cta[i][0], z1 += s.cta[i][1];
            const int bits0 = z0 ? finer(z0, p.bits) : p.bits, bits1 = z1 ? finer(z1, q.bits) : q.bits;
            if (bits0 == p.bits && bits1 == q.bits) {
                p.has(z0), q.has(z1);
                break;
            }
            p.bits = bits0, q.bits = bits1;
        }
        if (verdict == kRefuse) break;
        if (tid == n) {   // an unsure draft: the same in every CTA
            auto of = [&](float logit, const Row &r) {   // (of values that the draw takes for 0 too)
                return r.factor && !masked(logit) ? exp(((double)logit - (double)r.most) / (double)temperature) / ((double)r.z * exp2(r.bits - 62.0)) : 0.0;
            };
            s.verdict[n] = (double)x_u * (rq != nullptr ? of(x_draft, q) : 1.0) < of(x_target, p) ? kTake : kRefuse;
        }
        cluster.sync();   // (s.cta is free again)
        spent = false;
        // a draft that is refused after all: its rows' sums are made once more by the next turn
    }

    // the draw
    const size_t out = (size_t)seq * (K + 1);
    const bool minus_q = rq != nullptr && q.factor != 0;
    const int gone = n < count && a.draft == nullptr ? tokens[n] : -1;   // (without draft logits all of q is on the draft)
    int units = p.z ? p.bits : whole;   // of the sum of p, where q is not taken off
    auto weight = [&](Exact e, int i, bool plain) { return i == gone && !plain ? 0 : place(e.m, units + e.shift); };
    auto left = [&](Exact e, Exact g, bool plain) {   // of p without q, in units of 2^-62
        const unsigned long long w = place(__umulhi(e.m, p.factor), p.down + e.shift);
        const unsigned long long v = plain ? 0 : place(__umulhi(g.m, q.factor), q.down + g.shift);
        return w > v ? w - v : 0;
    };
    bool plain = n == count;
    unsigned long long total = 0, before = 0;
    while (!greedy && p.alive()) {
        if (spent) cluster.sync();   // (s.cta is free again)
        spent = true;
        unsigned long long sum = 0;
        if (minus_q) over_both([&](Exact e, Exact g) { sum += left(e, g, plain); });
        else over_one([&](Exact e, int i) { sum += weight(e, i, plain); });
        spread(sum, 0);
        total = before = 0;
        for (int i = 0; i < ctas; ++i) {
            if (i < rank) before += s.cta[i][0];
            total += s.cta[i][0];
        }
        const int bits = minus_q ? units : finer(total, units);
        if (bits != units) {
            units = bits;
            continue;
        }
        if (total != 0 || plain) break;
        plain = true;
        units = p.z ? p.bits : whole;
    }
    if (total != 0) {
        const unsigned long long un64 = u_draw >= 1.f ? ~0ull : (unsigned long long)(u_draw * 0x1p64f);
        const unsigned long long border = __umul64hi(un64, total);   // the first token whose sum is above it
        if (border >= before && border - before < s.cta[rank][0]) {
            // its warp's tokens, then a thread's, then itself
            int w = 0;
            while (border - before >= s.warp[w][0]) before += s.warp[w++][0];
            const int b0 = min(from + w * each, to), b1 = min(b0 + each, to), own = (b1 - b0 + kThreads - 1) / kThreads;
            const int i0 = min(b0 + tid * own, b1), i1 = min(i0 + own, b1);
            auto at_token = [&](int i) {
                Exact e, g;
                exact_exp2(load_logit(rp, i), minus_q ? load_logit(rq, i) : 0.f, f2(-p.most, -q.most), c, s.roots, e, g);
                return minus_q ? left(e, g, plain) : weight(e, i, plain);
            };
            unsigned long long sum = 0;
            for (int i = i0; i < i1; ++i) sum += at_token(i);
            unsigned long long up = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long v = __shfl_up_sync(0xffffffffu, up, o);
                if (lane >= o) up += v;
            }
            if (lane == 31) s.warp[warp][1] = up;
            __syncthreads();
            unsigned long long at = before + up - sum;
            for (int i = 0; i < warp; ++i) at += s.warp[i][1];
            if (border >= at && border - at < sum) {
                int i = i0;
                for (unsigned long long v; border - at >= (v = at_token(i)); ++i) at += v;
                a.tokens_out[out + n] = i;
                if (a.logprobs) {
                    float z = (float)p.z * exp2f((float)(p.bits - 62));
                    if (p.z == 0) {   // (no sum of p alone was made: it is the draw's, and the token's that was left out)
                        z = (float)total * exp2f((float)(units - 62));
                        if (gone >= 0 && gone < V && !plain) {
                            Exact e, g;
                            exact_exp2(load_logit(rp, gone), 0.f, f2(-p.most, 0.f), c, s.roots, e, g);
                            z += (float)e.m * exp2f((float)(-30 - e.shift));
                        }
                    }
                    a.logprobs[out + n] = (load_logit(rp, i) - p.most) / temperature - logf(z);
                }
            }
        }
    }
    if (rank != 0) return;
    // the rest of the results
    for (int i = tid; i <= K; i += kThreads) {
        int token = -1;
        if (i < n) token = tokens[i];
        else if (i == n && greedy && s.rows[n].alive()) token = s.rows[n].first;
        else if (i == n && total != 0) continue;
        a.tokens_out[out + i] = token;
        if (a.logprobs) {
            float lp = 0.f;
            if (i < n && !greedy) lp = (load_logit(row_at<T>(a, sq, seq, i), token) - s.rows[i].most) / temperature - logf(s.rows[i].sum);
            a.logprobs[out + i] = lp;
        }
    }
    if (tid == 0) a.accepted[seq] = n;
}

bool sizes_ok(int n_seq, int n_draft, int vocab) {
    return n_seq >= 0 && n_seq <= 65535 && n_draft >= 0 && n_draft <= kMaxDraft && vocab >= 1 && vocab <= 1 << 26;
}

// How a call runs. A sequence's own cluster reads its rows while they are few logits; else the whole GPU does, in a launch
// before (bf16, 4 drafts, one sequence: 8192 tokens 9.2 against 10.9 us, 32768 tokens 13.7 against 12). CTAs of a cluster: each
// has something to do, and all clusters are soon there, which take longer to begin the more CTAs they have (4 drafts of 2048
// tokens: one sequence 9.0 us with eight, 9.6 with four; 64 sequences 13.1 with eight, 11.2 with two; 8 sequences of 8
// drafts of 100003 tokens: 40 with eight, 33.7 with sixteen).
constexpr int kOwnLogits = 1 << 17;
struct Shape {
    bool own;
    int parts, ctas;
};
Shape shape_of(int n_seq, int n_draft, int vocab) {
    const int rows = 2 * n_draft + 1;
    const long long logits = (long long)rows * vocab;
    Shape p;
    p.own = logits <= kOwnLogits;
    p.ctas = 1;
    while (p.ctas < kCluster && (long long)n_seq * p.ctas * 2 <= (p.own ? 256 : 512) &&
           (p.own ? logits > (p.ctas < 8 ? 4096ll : 12288ll) * p.ctas : vocab > p.ctas * 1024ll))
        p.ctas *= 2;
    const long long warps = p.own ? p.ctas * kWarps : std::max(1ll, 152ll * 64 / std::max(1, n_seq));   // for a sequence
    p.parts = (int)std::max(1ll, std::min<long long>(std::min(kMaxParts, vocab / 256), warps / rows));
    return p;
}

// Clusters of 16 are allowed once for each device.
template <typename T, bool OWN>
cudaError_t allow() {
    return cudaFuncSetAttribute(k_draft_choose<T, OWN>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}
cudaError_t allow_clusters() {
    static std::atomic<unsigned long long> done{0};
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    const unsigned long long bit = device < 64 ? 1ull << device : 0;
    if (e != cudaSuccess || (done.load() & bit)) return e;
    if ((e = allow<float, true>()) != cudaSuccess || (e = allow<float, false>()) != cudaSuccess ||
        (e = allow<__nv_bfloat16, true>()) != cudaSuccess || (e = allow<__nv_bfloat16, false>()) != cudaSuccess)
        return e;
    done |= bit;
    return cudaSuccess;
}

}  // namespace

extern "C" {

size_t talker_draft_scratch(int n_seq, int n_draft, int vocab) {
    if (!sizes_ok(n_seq, n_draft, vocab)) return 0;
    const Shape p = shape_of(n_seq, n_draft, vocab);
    return p.own ? 0 : (size_t)n_seq * (2 * n_draft + 1) * p.parts * sizeof(Seen);
}

talker_status talker_draft_verify(const void *target, int64_t target_seq, int64_t target_row, const void *draft,
                                  int64_t draft_seq, int64_t draft_row, int dtype, const int32_t *tokens,
                                  const int32_t *counts, const float *uniforms, const float *temperatures, int n_seq,
                                  int n_draft, int vocab, int32_t *tokens_out, int32_t *accepted, float *logprobs,
                                  void *scratch, size_t scratch_bytes, void *cuda_stream) {
    if (!sizes_ok(n_seq, n_draft, vocab) || !target || !uniforms || !tokens_out || !accepted) return TALKER_EINVAL;
    if (n_draft > 0 && !tokens) return TALKER_EINVAL;
    if (dtype != TALKER_DTYPE_F32 && dtype != TALKER_DTYPE_BF16) return TALKER_EINVAL;
    if ((reinterpret_cast<uintptr_t>(target) | reinterpret_cast<uintptr_t>(draft)) % (dtype == TALKER_DTYPE_F32 ? 4 : 2)) return TALKER_EINVAL;
    for (const void *p : {static_cast<const void *>(tokens), static_cast<const void *>(counts), static_cast<const void *>(uniforms), static_cast<const void *>(temperatures),
                          static_cast<const void *>(tokens_out), static_cast<const void *>(accepted), static_cast<const void *>(logprobs)})
        if (reinterpret_cast<uintptr_t>(p) % 4) return TALKER_EINVAL;
    if (n_seq == 0) return TALKER_OK;
    const size_t need = talker_draft_scratch(n_seq, n_draft, vocab);
    if (need > 0 && (!scratch || scratch_bytes < need || reinterpret_cast<uintptr_t>(scratch) % 16)) return TALKER_EINVAL;
    const Shape p = shape_of(n_seq, n_draft, vocab);
    const Args a{target, draft, target_seq, target_row, draft_seq, draft_row, tokens, counts, uniforms, temperatures, n_draft, vocab,
                 tokens_out, accepted, logprobs, p.parts, p.ctas, static_cast<Seen *>(scratch)};
    const bool f32 = dtype == TALKER_DTYPE_F32;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.blockDim = dim3(kThreads);
    cfg.gridDim = dim3((unsigned)(n_seq * p.ctas));
    cfg.stream = static_cast<cudaStream_t>(cuda_stream);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.own ? 1 : 2;
    cudaError_t e = allow_clusters();
    if (e != cudaSuccess) {
        cudaGetLastError();
        return TALKER_ECUDA;
    }
    if (!p.own) {
        const dim3 grid((unsigned)(((2 * n_draft + 1) * p.parts + kWarps - 1) / kWarps), (unsigned)n_seq);
        if (f32) k_draft_rows<float><<<grid, kWarps * 32, 0, cfg.stream>>>(a);
        else k_draft_rows<__nv_bfloat16><<<grid, kWarps * 32, 0, cfg.stream>>>(a);
        e = cudaGetLastError();
        if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, f32 ? k_draft_choose<float, false> : k_draft_choose<__nv_bfloat16, false>, a);
    } else {
        e = cudaLaunchKernelEx(&cfg, f32 ? k_draft_choose<float, true> : k_draft_choose<__nv_bfloat16, true>, a);
    }
    if (e == cudaSuccess) return TALKER_OK;
    cudaGetLastError();
    return TALKER_ECUDA;
}

}  // extern "C"
