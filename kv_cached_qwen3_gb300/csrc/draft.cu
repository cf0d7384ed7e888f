// Verification of drafted tokens (include/talker_draft.h).
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "talker_draft.h"

namespace cg = cooperative_groups;
using namespace talker_dev;

namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kCluster = 8;
constexpr int kMaxDraft = 64;
constexpr int kMaxParts = 16;           // of a row
constexpr float kMasked = -1e30f;       // at or below: counts as -inf
constexpr float kGreedy = 1e-20f;       // a temperature not above it
constexpr float kNear = 1e-5f;          // of f32 sums: decisions nearer to their border are made again, exactly
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
};

template <typename T>
__device__ __forceinline__ float load_logit(const T *p, int i) { return Elem<T>::load(p, i); }
__device__ __forceinline__ bool masked(float x) { return !(x > kMasked); }

// A row's largest logit, the first place that has it, and the sum of e^((x - most) / T). Without a logit that is not masked:
// -inf, and a sum of 0.
struct Seen {
    float most, sum;
    int first;
};
__device__ __forceinline__ float ex2(float x) {   // relative error about 2^-22, 0 at -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ Seen join(const Seen &a, const Seen &b, float c) {
    Seen r;
    r.most = fmaxf(a.most, b.most);
    r.first = a.most == r.most ? (b.most == r.most ? min(a.first, b.first) : a.first) : b.first;
    // (a difference of -inf from itself is not made)
    r.sum = (a.sum > 0.f ? a.sum * ex2((a.most - r.most) * c) : 0.f) + (b.sum > 0.f ? b.sum * ex2((b.most - r.most) * c) : 0.f);
    return r;
}

// Part `part` of `parts` of a row, by one warp; c = log2 e / T.
template <typename T>
__device__ Seen see_part(const T *row, int vocab, int part, int parts, float c) {
    const int lane = threadIdx.x & 31;
    const int from = (int)((long long)vocab * part / parts), to = (int)((long long)vocab * (part + 1) / parts);
    Seen s{-INFINITY, 0.f, 0x7fffffff};
    for (int i = from + lane; i < to; i += 32) {
        const float x = load_logit(row, i);
        if (masked(x)) continue;
        if (x > s.most) {
            s.sum = (s.sum > 0.f ? s.sum * ex2((s.most - x) * c) : 0.f) + 1.f;
            s.most = x;
            s.first = i;
        } else {
            s.sum += ex2((x - s.most) * c);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const Seen b{__shfl_xor_sync(0xffffffffu, s.most, o), __shfl_xor_sync(0xffffffffu, s.sum, o), __shfl_xor_sync(0xffffffffu, s.first, o)};
        s = join(s, b, c);
    }
    return s;
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

// Sums of whole numbers over the CTA, in every thread.
__device__ __forceinline__ unsigned long long warp_sum64(unsigned long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

enum Verdict : int { kTake = 0, kRefuse = 1, kUnsure = 2 };

struct Shared {
    uint32_t roots[32];                        // 2^(31 + j / 32)
    Seen parts[(2 * kMaxDraft + 1) * kMaxParts];   // of CTA 0: the rows' parts
    Seen rows[2 * kMaxDraft + 1];              // joined; target rows, then draft rows
    int verdict[kMaxDraft];
    unsigned long long warp[kWarps][2];
    unsigned long long cta[kCluster][2];       // every CTA's sums
    float most[kCluster][2];
    int row;                                   // the row that is looked at, decided: drawn from
    int found;
};

// Everything a draw needs to know of a row of probabilities: p = m scale >> (down + shift), in units of 2^-62.
struct Row {
    float most;
    Scale c;
    uint32_t factor;   // 0: no distribution
    int down;
    double z;          // the sum of e^((x - most) / T)
};

template <typename T>
__global__ void __launch_bounds__(kThreads) k_draft_verify(const Args a) {
    extern __shared__ unsigned char raw[];
    Shared &s = *reinterpret_cast<Shared *>(raw);
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = cluster.num_blocks(), rank = cluster.block_rank(), seq = blockIdx.x / ctas;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int K = a.n_draft, V = a.vocab;
    const int count = a.counts ? min(max(a.counts[seq], 0), K) : K;
    const float temperature = a.temperatures ? a.temperatures[seq] : 1.f;
    const bool greedy = !(temperature > kGreedy), drafted = a.draft != nullptr && !greedy;
    const Scale c = greedy ? Scale{1.f, 0.f} : scale_of(temperature);
    const T *target = static_cast<const T *>(a.target) + seq * a.target_seq;
    const T *draft = static_cast<const T *>(a.draft) + seq * a.draft_seq;
    const float *u = a.uniforms + (size_t)seq * (K + 1);
    const int32_t *tokens = a.tokens + (size_t)seq * K;
    Shared *lead = cluster.map_shared_rank(&s, 0);
    if (tid < 32) s.roots[tid] = (uint32_t)llrint(exp2(31.0 + tid / 32.0));
    cluster.sync();   // every CTA's shared memory is there

    // the rows' sums: target rows before the last draft (of greedy sequences the one after too), and draft rows
    const int n_target = count + (greedy ? 1 : 0), n_rows = n_target + (drafted ? count : 0);
    for (int t = rank * kWarps + warp; t < n_rows * a.parts; t += ctas * kWarps) {
        const int r = t / a.parts;
        const T *row = r < n_target ? target + r * a.target_row : draft + (r - n_target) * a.draft_row;
        const Seen seen = see_part(row, V, t - r * a.parts, a.parts, c.hi);
        if (lane == 0) lead->parts[t] = seen;
    }
    cluster.sync();
    if (rank == 0) {
        for (int r = tid; r < n_rows; r += kThreads) {
            Seen seen = s.parts[r * a.parts];
            for (int i = 1; i < a.parts; ++i) seen = join(seen, s.parts[r * a.parts + i], c.hi);
            s.rows[r] = seen;
        }
        __syncthreads();
        for (int i = tid; i < count; i += kThreads) {
            const int x = tokens[i];
            int v = kRefuse;
            if (x >= 0 && x < V) {
                const Seen p = s.rows[i];
                const float logit = load_logit(target + i * a.target_row, x);
                if (greedy) {
                    v = p.most < INFINITY && x == p.first ? kTake : kRefuse;
                } else if (!masked(logit) && p.most < INFINITY) {
                    const float px = ex2((logit - p.most) * c.hi) / p.sum;
                    float qx = 1.f;
                    if (drafted) {
                        const Seen q = s.rows[n_target + i];
                        const float other = load_logit(draft + i * a.draft_row, x);
                        qx = masked(other) || !(q.most < INFINITY) ? 0.f : ex2((other - q.most) * c.hi) / q.sum;
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

    // the first draft that is not surely taken, exactly; then the draw
    int n = 0;
    Row p{}, q{};
    const int bits = 32 - __clz(V - 1 > 0 ? V - 1 : 1), lift = 32 - bits;   // a sum of V numbers below 2^(32 + lift) fits
    const int from = (int)((long long)V * rank / ctas), to = (int)((long long)V * (rank + 1) / ctas);
    while (true) {
        if (rank == 0 && tid == 0) {
            while (n < count && s.verdict[n] == kTake) ++n;
            s.row = n;
        }
        cluster.sync();
        n = lead->row;
        const int verdict = n < count ? lead->verdict[n] : kRefuse;   // (read before CTA 0 may change it below)
        if (greedy) break;
        // the largest logits
        const T *rows[2] = {target + n * a.target_row, draft + n * a.draft_row};
        const int both = drafted && n < count ? 2 : 1;
        if (n < count) {
            p.most = lead->rows[n].most;
            if (both == 2) q.most = lead->rows[n_target + n].most;
        } else {
            float m = -INFINITY;
            for (int i = from + tid; i < to; i += kThreads) {
                const float x = load_logit(rows[0], i);
                if (!masked(x)) m = fmaxf(m, x);
            }
            m = warp_max(m);
            if (lane == 0) s.warp[warp][0] = __float_as_uint(m);
            __syncthreads();
            if (tid < ctas) {
                m = -INFINITY;
                for (int w = 0; w < kWarps; ++w) m = fmaxf(m, __uint_as_float((uint32_t)s.warp[w][0]));
                cluster.map_shared_rank(&s, tid)->most[rank][0] = m;
            }
            cluster.sync();
            p.most = -INFINITY;
            for (int i = 0; i < ctas; ++i) p.most = fmaxf(p.most, s.most[i][0]);
        }
        // their sums
        unsigned long long sums[2] = {0, 0};
        for (int w = 0; w < both; ++w) {
            const float most = w ? q.most : p.most;
            if (!(most > kMasked && most < INFINITY)) continue;
            for (int i = from + tid; i < to; i += kThreads) {
                const Exact e = exact_exp(load_logit(rows[w], i), most, c, s.roots);
                if (e.shift < 64) sums[w] += (((unsigned long long)e.m << lift) + (1ull << e.shift >> 1)) >> e.shift;
            }
        }
        for (int w = 0; w < 2; ++w) {
            sums[w] = warp_sum64(sums[w]);
            if (lane == 0) s.warp[warp][w] = sums[w];
        }
        __syncthreads();
        if (tid < 2 * ctas) {
            unsigned long long v = 0;
            for (int w = 0; w < kWarps; ++w) v += s.warp[w][tid & 1];
            cluster.map_shared_rank(&s, tid >> 1)->cta[rank][tid & 1] = v;
        }
        cluster.sync();
        for (int w = 0; w < 2; ++w) {
            unsigned long long z = 0;
            for (int i = 0; i < ctas; ++i) z += s.cta[i][w];
            Row &r = w ? q : p;
            r.c = c;
            r.factor = 0;
            if (z == 0) continue;
            const int lead_zeros = __clzll(z);
            // 2^95 / (z 2^lead_zeros), in (2^31, 2^32]
            r.factor = (uint32_t)fmin(0x1p95 / (double)(z << lead_zeros), 4294967295.0);
            r.down = 33 - lift - lead_zeros;
            r.z = (double)z * exp2(-(double)(31 + lift));
        }
        if (verdict == kRefuse) break;
        // an unsure draft
        if (rank == 0 && tid == 0) {
            const int x = tokens[n];
            auto of = [&](const T *row, const Row &r) {   // (of values that the draw takes for 0 too)
                const float logit = load_logit(row, x);
                return r.factor && !masked(logit) ? exp(((double)logit - (double)r.most) / (double)temperature) / r.z : 0.0;
            };
            const double px = of(rows[0], p), qx = both == 2 ? of(rows[1], q) : 1.0;
            s.verdict[n] = (double)fminf(fmaxf(u[n], 0.f), 1.f) * qx < px ? kTake : kRefuse;
        }
        cluster.sync();
        if (lead->verdict[n] == kRefuse) break;
    }

    if (rank == 0) {   // the drafts that are taken
        for (int i = tid; i <= K; i += kThreads) {
            a.tokens_out[(size_t)seq * (K + 1) + i] = i < n ? tokens[i] : -1;
            if (a.logprobs) {
                float lp = 0.f;
                if (i < n && !greedy)
                    lp = (float)(((double)load_logit(target + i * a.target_row, tokens[i]) - (double)s.rows[i].most) / (double)temperature -
                                 log((double)s.rows[i].sum));
                a.logprobs[(size_t)seq * (K + 1) + i] = lp;
            }
        }
        if (tid == 0) a.accepted[seq] = n;
        __syncthreads();
    }
    if (greedy) {
        if (rank == 0 && tid == 0) {
            const Seen r = s.rows[n];
            a.tokens_out[(size_t)seq * (K + 1) + n] = r.most > kMasked && r.most < INFINITY ? r.first : -1;
        }
        cluster.sync();   // (CTA 0's shared memory is read until here)
        return;
    }
    // the draw
    const T *rp = target + n * a.target_row, *rq = draft + n * a.draft_row;
    const bool minus_q = n < count && drafted;
    const int gone = n < count && a.draft == nullptr ? tokens[n] : -1;   // (without draft logits: all of q is on the draft)
    auto weight = [&](int i, bool plain) -> unsigned long long {
        if (p.factor == 0) return 0;
        const Exact e = exact_exp(load_logit(rp, i), p.most, c, s.roots);
        const int sh = p.down + e.shift;
        unsigned long long w = e.shift < 64 && sh < 64 ? (unsigned long long)e.m * p.factor >> sh : 0;
        if (plain) return w;
        if (i == gone) return 0;
        if (minus_q && q.factor) {
            const Exact g = exact_exp(load_logit(rq, i), q.most, c, s.roots);
            const int gs = q.down + g.shift;
            const unsigned long long v = g.shift < 64 && gs < 64 ? (unsigned long long)g.m * q.factor >> gs : 0;
            w = w > v ? w - v : 0;
        }
        return w;
    };
    const int each = (to - from + kWarps - 1) / kWarps;   // of a warp
    const int w0 = min(from + warp * each, to), w1 = min(w0 + each, to);
    bool plain = n == count;
    unsigned long long total = 0, before = 0;
    while (true) {
        cluster.sync();   // (s.cta is free again)
        unsigned long long sum = 0;
        for (int i = w0 + lane; i < w1; i += 32) sum += weight(i, plain);
        sum = warp_sum64(sum);
        if (lane == 0) s.warp[warp][0] = sum;
        __syncthreads();
        if (tid < ctas) {
            unsigned long long v = 0;
            for (int w = 0; w < kWarps; ++w) v += s.warp[w][0];
            cluster.map_shared_rank(&s, tid)->cta[rank][0] = v;
        }
        cluster.sync();
        total = before = 0;
        for (int i = 0; i < ctas; ++i) {
            if (i < rank) before += s.cta[i][0];
            total += s.cta[i][0];
        }
        if (total != 0 || plain) break;
        plain = true;
    }
    if (total == 0) {
        cluster.sync();
        return;   // no distribution: -1 is there already
    }
    const float un = fminf(fmaxf(u[K], 0.f), 1.f);
    const unsigned long long un64 = un >= 1.f ? ~0ull : (unsigned long long)(un * 0x1p64f);
    const unsigned long long border = __umul64hi(un64, total);   // the first token whose sum is above it
    if (border >= before && border < before + s.cta[rank][0]) {
        // its warp's tokens, then a thread's, then itself
        int w = 0;
        while (border - before >= s.warp[w][0]) before += s.warp[w++][0];
        const int b0 = min(from + w * each, to), b1 = min(b0 + each, to), own = (b1 - b0 + kThreads - 1) / kThreads;
        const int i0 = min(b0 + tid * own, b1), i1 = min(i0 + own, b1);
        unsigned long long sum = 0;
        for (int i = i0; i < i1; ++i) sum += weight(i, plain);
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
            for (unsigned long long v; border - at >= (v = weight(i, plain)); ++i) at += v;
            a.tokens_out[(size_t)seq * (K + 1) + n] = i;
            if (a.logprobs)
                a.logprobs[(size_t)seq * (K + 1) + n] =
                    (float)(((double)load_logit(rp, i) - (double)p.most) / (double)temperature - log(p.z));
        }
    }
    cluster.sync();   // (nobody leaves while others read its shared memory)
}

bool sizes_ok(int n_seq, int n_draft, int vocab) {
    return n_seq >= 0 && n_seq <= 65536 && n_draft >= 0 && n_draft <= kMaxDraft && vocab >= 1 && vocab <= 1 << 26;
}

}  // namespace

extern "C" {

size_t talker_draft_scratch(int, int, int) { return 0; }

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
    const int rows = 2 * n_draft + 1;
    Args a{target, draft, target_seq, target_row, draft_seq, draft_row, tokens, counts, uniforms, temperatures, n_draft, vocab,
           tokens_out, accepted, logprobs, 1};
    a.parts = std::max(1, std::min(kMaxParts, kCluster * kWarps / rows));
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.blockDim = dim3(kThreads);
    cfg.gridDim = dim3((unsigned)(n_seq * kCluster));
    cfg.dynamicSmemBytes = sizeof(Shared);
    static_assert(sizeof(Shared) <= 48 * 1024, "without a raised limit");
    cfg.stream = static_cast<cudaStream_t>(cuda_stream);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e =
        cudaLaunchKernelEx(&cfg, dtype == TALKER_DTYPE_F32 ? k_draft_verify<float> : k_draft_verify<__nv_bfloat16>, a);
    if (e == cudaSuccess) return TALKER_OK;
    cudaGetLastError();
    return TALKER_ECUDA;
}

}  // extern "C"
