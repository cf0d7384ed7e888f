// Verification of drafted tokens (include/talker_draft.h).
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "talker_draft.h"

namespace cg = cooperative_groups;
using namespace talker_dev;

namespace {

constexpr int kWarps = 16, kThreads = kWarps * 32;   // of the CTAs that choose
constexpr int kRowWarps = 8;            // of those that read rows for them
constexpr int kCluster = 8;
constexpr int kMaxDraft = 64, kMaxRows = 2 * kMaxDraft + 1;
constexpr int kMaxParts = 32;           // of a row: a lane each where they are joined
constexpr int kOwnParts = kMaxRows + kCluster * kWarps;   // of a sequence, where its cluster reads its rows itself
constexpr float kMasked = -1e30f;       // at or below: counts as -inf
constexpr float kLeastRef = -9.9999994e29f;   // reference of a row's exponents without a logit: the next value above kMasked
constexpr float kGreedy = 1e-20f;       // a temperature not above it
constexpr float kHottest = 1e18f;       // a temperature above it counts as this one (masked logits still add nothing)
constexpr float kNear = 1e-4f;          // of f32 sums: decisions nearer to their border are made again, exactly
constexpr double kLog2e = 1.4426950408889634074;

struct Args {
    const void *target, *draft;
    long long target_seq, target_row, draft_seq, draft_row;
    const int32_t *tokens, *counts;
    const float *uniforms, *temperatures;
    int n_draft, vocab;
    int32_t *tokens_out, *accepted;
    float *logprobs;
    int parts;              // of a row
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

// A row's largest logit (at least kLeastRef, below which masked ones add nothing), the first place that has it (of greedy
// sequences), and the sum of e^((x - most) / T) (of others).
struct Seen {
    float most, sum;
    int first;
    __device__ __forceinline__ bool alive() const { return most > kLeastRef && most < INFINITY; }
};
__device__ __forceinline__ float ex2(float x) {   // relative error about 2^-22, 0 at -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ Seen warp_join(Seen s, float c) {
    const float most = warp_max(s.most);
    s.sum = warp_sum(s.sum * ex2((s.most - most) * c));
    s.first = (int)__reduce_min_sync(0xffffffffu, s.most == most ? (uint32_t)s.first : 0x7fffffffu);
    s.most = most;
    return s;
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

// n values, the first of them logit `at` of its row.
template <int N>
__device__ __forceinline__ void take(Seen &s, float (&x)[N], int at, float c, bool greedy) {
    float top = kLeastRef;
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
    if (top > s.most) {
        s.sum *= ex2((s.most - top) * c);
        s.most = top;
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) sum += ex2((x[i] - s.most) * c);
    s.sum += sum;
}

// Part `part` of `parts` of a row, by one warp; c = log2 e / T. A part is so many of the row's vectors of 16 bytes; logits
// before the first and after the last are the first and the last part's.
template <typename T>
__device__ Seen see_part(const T *row, int vocab, int part, int parts, float c, bool greedy) {
    constexpr int N = Vec<T>::N, kAhead = 4;
    const int lane = threadIdx.x & 31;
    const int lead = min(vocab, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) % 16 / sizeof(T)));
    const int vecs = (vocab - lead) / N;
    const int from = (int)((long long)vecs * part / parts), to = (int)((long long)vecs * (part + 1) / parts);
    Seen s{kLeastRef, 0.f, 0x7fffffff};
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
    return warp_join(s, c);
}

// e^((x - most) / T) = m 2^(-31 - shift), m in [2^31, 2^32), for x <= most, to about 2^-31 of itself. With
// t = (x - most) log2 e / T in two floats, t = k / 32 + f, |f| <= 1/64: m = 2^31 2^(k % 32 / 32) e^y, y = f log 2, by the
// series of e^y - 1, whose terms after y^4 / 24 are below 2^-39.
struct Exact {
    uint32_t m;
    int shift;   // 64: 0
};
struct Scale {   // log2 e / T in two floats
    float hi, lo;
};
__device__ __forceinline__ Scale scale_of(float temperature) {
    const double c = kLog2e / (double)temperature;
    const float hi = (float)c;
    return {hi, (float)(c - (double)hi)};
}
__device__ __forceinline__ Exact exact_exp(float x, float most, const Scale c, const uint32_t *roots) {
    const float d = x - most, b = d - x, dl = (x - (d - b)) - (most + b);   // x - most = d + dl, exactly
    const float t = d * c.hi;
    if (masked(x) || !(t > -70.f)) return {0u, 64};
    const float tl = fmaf(d, c.hi, -t) + fmaf(d, c.lo, dl * c.hi);
    const float kf = rintf(t * 32.f);
    const int k = (int)kf;
    const float f = fmaf(kf, -1.f / 32.f, t);
    constexpr float kLn2 = 0.693147182464599609375f, kLn2Lo = -1.904654299957768e-09f;   // log 2 in two floats
    const float y = f * kLn2, yl = fmaf(f, kLn2, -y) + fmaf(f, kLn2Lo, tl * kLn2);
    const float q = y * y * fmaf(y, fmaf(y, 1.f / 24.f, 1.f / 6.f), 0.5f) + yl;
    const int rise = __float2int_rn(y * 0x1p32f) + __float2int_rn(q * 0x1p32f);   // (e^y - 1) 2^32
    const uint32_t r = roots[k & 31];
    return {r + (uint32_t)(((long long)r * rise) >> 32), -(k >> 5)};
}

__device__ __forceinline__ unsigned long long warp_sum64(unsigned long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The rows' parts, a warp each, for calls that a sequence's cluster would read too slowly.
template <typename T>
__global__ void __launch_bounds__(kRowWarps * 32) k_draft_rows(const Args a) {
    const int seq = blockIdx.y, t = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
    const Sequence q = sequence(a, seq);
    if (t < q.rows() * a.parts) {
        const int r = t / a.parts;
        const Seen s = see_part(row_at<T>(a, q, seq, r), a.vocab, t - r * a.parts, a.parts, (float)kLog2e / q.temperature, q.greedy);
        if ((threadIdx.x & 31) == 0) a.seen[(size_t)seq * (2 * a.n_draft + 1) * a.parts + t] = s;
    }
    pdl_launch_dependents();
}

enum Verdict : int { kTake = 0, kRefuse = 1, kUnsure = 2 };

struct Shared {
    uint32_t roots[32];                        // 2^(31 + j / 32)
    Seen parts[kOwnParts];                     // of CTA 0
    Seen rows[kMaxRows];                       // joined
    int verdict[kMaxDraft];
    unsigned long long warp[kWarps][2];
    unsigned long long cta[kCluster][2];       // every CTA's sums
    int row;                                   // the row that is looked at; decided: drawn from
};

// A row of probabilities: p = m factor >> (down + shift), in units of 2^-62, of an Exact.
struct Row {
    float most;
    uint32_t factor;   // 0: no distribution
    int down;
    double z;          // the sum of e^((x - most) / T)
};

// A cluster per sequence. Its first CTA decides by f32 sums which drafts are surely taken and which first one is
// not; that one's rows, and those that the next token is drawn from, are gone over by all CTAs, each a range of the vocabulary, with
// exponentials of 31 bits and sums in whole numbers: which token a uniform number meets is a question of sums of
// 10^5 terms next to one another, where f32 would err once in some hundred draws.
template <typename T, bool OWN>
__global__ void __launch_bounds__(kThreads, 1) k_draft_choose(const Args a) {
    __shared__ Shared s;
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = cluster.num_blocks(), rank = cluster.block_rank(), seq = blockIdx.x / ctas;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int K = a.n_draft, V = a.vocab;
    const Sequence sq = sequence(a, seq);
    const int count = sq.count, n_rows = sq.rows();
    const bool greedy = sq.greedy, drafted = sq.drafted;
    const double temperature = sq.temperature;
    const Scale c = greedy ? Scale{1.f, 0.f} : scale_of(sq.temperature);
    const float *u = a.uniforms + (size_t)seq * (K + 1);
    const int32_t *tokens = a.tokens + (size_t)seq * K;
    Shared *lead = cluster.map_shared_rank(&s, 0);
    if (tid < 32) s.roots[tid] = (uint32_t)llrint(exp2(31.0 + tid / 32.0));
    cluster.sync();   // every CTA's shared memory is there

    if (OWN) {
        for (int t = rank * kWarps + warp; t < n_rows * a.parts; t += ctas * kWarps) {
            const int r = t / a.parts;
            const Seen seen = see_part(row_at<T>(a, sq, seq, r), V, t - r * a.parts, a.parts, c.hi, greedy);
            if (lane == 0) lead->parts[t] = seen;
        }
        cluster.sync();
    } else {
        pdl_wait();
    }
    if (rank == 0) {
        const Seen *parts = OWN ? s.parts : a.seen + (size_t)seq * (2 * K + 1) * a.parts;
        for (int r = warp; r < n_rows; r += kWarps) {
            const Seen one = lane < a.parts ? parts[r * a.parts + lane] : Seen{kLeastRef, 0.f, 0x7fffffff};
            const Seen seen = warp_join(one, c.hi);
            if (lane == 0) s.rows[r] = seen;
        }
        __syncthreads();
        for (int i = tid; i < count; i += kThreads) {
            const int x = tokens[i];
            int v = kRefuse;
            const Seen p = s.rows[i];
            if (x >= 0 && x < V && p.alive()) {
                const float logit = load_logit(row_at<T>(a, sq, seq, i), x);
                if (greedy) {
                    v = x == p.first ? kTake : kRefuse;
                } else if (!masked(logit)) {
                    const float px = ex2((logit - p.most) * c.hi) / p.sum;
                    float qx = 1.f;
                    if (drafted) {
                        const Seen q = s.rows[sq.targets() + i];
                        const float other = load_logit(row_at<T>(a, sq, seq, sq.targets() + i), x);
                        qx = masked(other) || !q.alive() ? 0.f : ex2((other - q.most) * c.hi) / q.sum;
                    }
                    const float need = fminf(fmaxf(u[i], 0.f), 1.f) * qx;
                    // (an exponential that f32 cannot tell from 0 decides nothing)
                    v = px > 1e-30f && need < px * (1.f - kNear) ? kTake : need > px * (1.f + kNear) && need > 1e-30f ? kRefuse : kUnsure;
                }
            }
            s.verdict[i] = v;
        }
        __syncthreads();
    }

    int n = 0;
    Row p{}, q{};
    const int bits = 32 - __clz(max(V - 1, 1)), lift = 32 - bits;   // a sum of V numbers below 2^(32 + lift) fits 64 bits
    // this CTA's range, and its warps'
    const int from = (int)((long long)V * rank / ctas), to = (int)((long long)V * (rank + 1) / ctas);
    const int each = (to - from + kWarps - 1) / kWarps;
    const int w0 = min(from + warp * each, to), w1 = min(w0 + each, to);
    const T *rp = nullptr, *rq = nullptr;
    // a value from each CTA's sums over its warps to all CTAs
    auto spread = [&](unsigned long long v0, unsigned long long v1) {
        v0 = warp_sum64(v0), v1 = warp_sum64(v1);
        if (lane == 0) s.warp[warp][0] = v0, s.warp[warp][1] = v1;
        __syncthreads();
        if (tid < 2 * ctas) {
            unsigned long long v = 0;
            for (int w = 0; w < kWarps; ++w) v += s.warp[w][tid & 1];
            cluster.map_shared_rank(&s, tid >> 1)->cta[rank][tid & 1] = v;
        }
        cluster.sync();
    };
    auto whole = [&](float x, float most) -> unsigned long long {   // e^((x - most) / T) in units of 2^-(31 + lift)
        const Exact e = exact_exp(x, most, c, s.roots);
        return e.shift < 64 ? (((unsigned long long)e.m << lift) + (1ull << e.shift >> 1)) >> e.shift : 0;
    };
    while (true) {
        if (rank == 0 && tid == 0) {
            while (n < count && s.verdict[n] == kTake) ++n;
            s.row = n;
        }
        cluster.sync();
        n = lead->row;
        const int verdict = n < count ? lead->verdict[n] : kRefuse;   // (read before CTA 0 may change it below)
        if (greedy) break;
        const Seen ps = lead->rows[n], qs = drafted && n < count ? lead->rows[sq.targets() + n] : Seen{kLeastRef, 0.f, 0};
        p.most = ps.most, q.most = qs.most;
        rp = row_at<T>(a, sq, seq, n);
        rq = drafted && n < count ? row_at<T>(a, sq, seq, sq.targets() + n) : nullptr;
        p.factor = q.factor = 0;
        p.z = 0.0;
        if (rq == nullptr && verdict == kRefuse) break;   // (drawn from p alone: its sum is the draw's)
        unsigned long long sums[2] = {0, 0};
        if (ps.alive() && qs.alive()) {
#pragma unroll 4
            for (int i = w0 + lane; i < w1; i += 32) {
                const float x = load_logit(rp, i), y = load_logit(rq, i);
                sums[0] += whole(x, p.most);
                sums[1] += whole(y, q.most);
            }
        } else if (ps.alive()) {
#pragma unroll 4
            for (int i = w0 + lane; i < w1; i += 32) sums[0] += whole(load_logit(rp, i), p.most);
        }
        spread(sums[0], sums[1]);
        for (int w = 0; w < 2; ++w) {
            unsigned long long z = 0;
            for (int i = 0; i < ctas; ++i) z += s.cta[i][w];
            if (z == 0) continue;
            Row &r = w ? q : p;
            const int zeros = __clzll(z);
            // 2^95 / (z 2^zeros), in (2^31, 2^32]
            r.factor = (uint32_t)fmin(0x1p95 / (double)(z << zeros), 4294967295.0);
            r.down = 33 - lift - zeros;
            r.z = (double)z * exp2(-(double)(31 + lift));
        }
        if (verdict == kRefuse) break;
        if (rank == 0 && tid == 0) {   // an unsure draft
            const int x = tokens[n];
            auto of = [&](const T *row, const Row &r) {   // (of values that the draw takes for 0 too)
                const float logit = load_logit(row, x);
                return r.factor && !masked(logit) ? exp(((double)logit - (double)r.most) / temperature) / r.z : 0.0;
            };
            const double px = of(rp, p), qx = rq != nullptr ? of(rq, q) : 1.0;
            s.verdict[n] = (double)fminf(fmaxf(u[n], 0.f), 1.f) * qx < px ? kTake : kRefuse;
        }
        cluster.sync();
        if (lead->verdict[n] == kRefuse) break;
    }

    const size_t out = (size_t)seq * (K + 1);
    if (rank == 0) {   // the drafts that are taken
        for (int i = tid; i <= K; i += kThreads) {
            int token = i < n ? tokens[i] : -1;
            if (greedy && i == n && s.rows[n].alive()) token = s.rows[n].first;
            a.tokens_out[out + i] = token;
            if (a.logprobs) {
                float lp = 0.f;
                if (i < n && !greedy)
                    lp = (float)(((double)load_logit(row_at<T>(a, sq, seq, i), token) - (double)s.rows[i].most) / temperature - log((double)s.rows[i].sum));
                a.logprobs[out + i] = lp;
            }
        }
        if (tid == 0) a.accepted[seq] = n;
    }
    // the draw
    const bool minus_q = rq != nullptr && q.factor != 0;
    const int gone = n < count && a.draft == nullptr ? tokens[n] : -1;   // (without draft logits all of q is on the draft)
    auto weight = [&](float x, float y, int i, bool plain) -> unsigned long long {
        if (!minus_q) return i == gone && !plain ? 0 : whole(x, p.most);
        const Exact e = exact_exp(x, p.most, c, s.roots), g = exact_exp(y, q.most, c, s.roots);
        const int es = p.down + e.shift, gs = q.down + g.shift;
        const unsigned long long w = e.shift < 64 && es < 64 ? (unsigned long long)e.m * p.factor >> es : 0;
        const unsigned long long v = g.shift < 64 && gs < 64 && !plain ? (unsigned long long)g.m * q.factor >> gs : 0;
        return w > v ? w - v : 0;
    };
    bool plain = n == count;
    unsigned long long total = 0, before = 0;
    while (!greedy && lead->rows[n].alive()) {
        cluster.sync();   // (s.cta is free again)
        unsigned long long sum = 0;
        if (minus_q) {
#pragma unroll 4
            for (int i = w0 + lane; i < w1; i += 32) sum += weight(load_logit(rp, i), load_logit(rq, i), i, plain);
        } else {
#pragma unroll 4
            for (int i = w0 + lane; i < w1; i += 32) sum += weight(load_logit(rp, i), 0.f, i, plain);
        }
        spread(sum, 0);
        total = before = 0;
        for (int i = 0; i < ctas; ++i) {
            if (i < rank) before += s.cta[i][0];
            total += s.cta[i][0];
        }
        if (total != 0 || plain) break;
        plain = true;
    }
    if (total != 0) {
        const float un = fminf(fmaxf(u[K], 0.f), 1.f);
        const unsigned long long un64 = un >= 1.f ? ~0ull : (unsigned long long)(un * 0x1p64f);
        const unsigned long long border = __umul64hi(un64, total);   // the first token whose sum is above it
        if (border >= before && border - before < s.cta[rank][0]) {
            // its warp's tokens, then a thread's, then itself
            int w = 0;
            while (border - before >= s.warp[w][0]) before += s.warp[w++][0];
            const int b0 = min(from + w * each, to), b1 = min(b0 + each, to), own = (b1 - b0 + kThreads - 1) / kThreads;
            const int i0 = min(b0 + tid * own, b1), i1 = min(i0 + own, b1);
            auto at_token = [&](int i) { return weight(load_logit(rp, i), minus_q ? load_logit(rq, i) : 0.f, i, plain); };
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
                    double z = p.z;
                    if (z == 0.0) {   // (no sum of p alone was made: it is the draw's, and the token's that was left out)
                        const unsigned long long left = gone >= 0 && gone < V && !plain ? whole(load_logit(rp, gone), p.most) : 0;
                        z = (double)(total + left) * exp2(-(double)(31 + lift));
                    }
                    a.logprobs[out + n] = (float)(((double)load_logit(rp, i) - (double)p.most) / temperature - log(z));
                }
            }
        }
    }
    cluster.sync();   // (nobody leaves while others read its shared memory)
}

bool sizes_ok(int n_seq, int n_draft, int vocab) {
    return n_seq >= 0 && n_seq <= 65535 && n_draft >= 0 && n_draft <= kMaxDraft && vocab >= 1 && vocab <= 1 << 26;
}

// A sequence's own cluster reads its rows while they are few logits; else the whole GPU does, in a launch before.
constexpr int kOwnLogits = 65536;
struct Shape {
    bool own;
    int parts;
};
Shape shape_of(int n_seq, int n_draft, int vocab) {
    const int rows = 2 * n_draft + 1;
    Shape p;
    p.own = (long long)rows * vocab <= kOwnLogits;
    const long long warps = p.own ? kCluster * kWarps : std::max(1ll, 152ll * 32 / std::max(1, n_seq));   // for a sequence
    p.parts = (int)std::max(1ll, std::min<long long>(std::min(kMaxParts, vocab / 256), warps / rows));
    return p;
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
    if (n_seq == 0) return TALKER_OK;
    const size_t need = talker_draft_scratch(n_seq, n_draft, vocab);
    if (need > 0 && (!scratch || scratch_bytes < need || reinterpret_cast<uintptr_t>(scratch) % 16)) return TALKER_EINVAL;
    const Shape p = shape_of(n_seq, n_draft, vocab);
    const Args a{target, draft, target_seq, target_row, draft_seq, draft_row, tokens, counts, uniforms, temperatures, n_draft, vocab,
                 tokens_out, accepted, logprobs, p.parts, static_cast<Seen *>(scratch)};
    const bool f32 = dtype == TALKER_DTYPE_F32;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.blockDim = dim3(kThreads);
    cfg.gridDim = dim3((unsigned)(n_seq * kCluster));
    cfg.stream = static_cast<cudaStream_t>(cuda_stream);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.own ? 1 : 2;
    cudaError_t e = cudaSuccess;
    if (!p.own) {
        const dim3 grid((unsigned)(((2 * n_draft + 1) * p.parts + kRowWarps - 1) / kRowWarps), (unsigned)n_seq);
        if (f32) k_draft_rows<float><<<grid, kRowWarps * 32, 0, cfg.stream>>>(a);
        else k_draft_rows<__nv_bfloat16><<<grid, kRowWarps * 32, 0, cfg.stream>>>(a);
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
