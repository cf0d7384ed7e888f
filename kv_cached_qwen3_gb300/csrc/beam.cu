// Beam selection (talker_beam_select): per sequence the best `width` of width * vocab continuations.
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "talker_kv4.h"

namespace cg = cooperative_groups;
using namespace talker_dev;

namespace {

constexpr int kWarps = 8;
constexpr int kMaxWidth = 32;
constexpr int kMaxChunks = 32;      // parts of a row: the lists that one warp joins, a lane each
constexpr int kCluster = 8;
constexpr int kClusterTasks = kWarps * kCluster + kMaxWidth;
constexpr float kMasked = -1e30f;   // at or below: counts as -inf
constexpr float kLog2e = 1.4426950408889634f;
typedef unsigned long long Key;

// Masked values as -inf, and -0 as 0 (equal values are ordered by their index).
__device__ __forceinline__ float unmask(float x) { return x > kMasked ? x + 0.f : -INFINITY; }

// Order of (value, index): the larger value first, then the lower index. No key is 0.
__device__ __forceinline__ Key key_of(float x, unsigned i) {
    const uint32_t u = __float_as_uint(x);
    return (Key)(u & 0x80000000u ? ~u : u | 0x80000000u) << 32 | (0xffffffffu - i);
}
__device__ __forceinline__ float key_value(Key k) {
    const uint32_t u = (uint32_t)(k >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ unsigned key_index(Key k) { return 0xffffffffu - (uint32_t)k; }

__device__ __forceinline__ Key warp_max_key(Key k) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const Key t = __shfl_xor_sync(0xffffffffu, k, o);
        k = t > k ? t : k;
    }
    return k;
}
__device__ __forceinline__ float ex2(float x) {   // relative error about 2^-22, 0 at -inf
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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
    Key *keys;        // scratch: [row][chunk][width], best first
    float2 *sums;     // scratch: [row][chunk] (maximum, sum of exp(x - maximum))
};

// What a warp has seen of a row: lane i < width holds the i-th best logit, lanes apart their part of
// the maximum and of the sum of exponentials.
struct Seen {
    Key mine;
    float m, sum, least;   // least: the logit a new one has to pass (-inf and not `full` at first)
    bool full;
};

// Values x of consecutive indexes: lane l holds those from at + l * N on, in order; on: how many of
// them exist. Logits come in the order of their indexes, so an equal one never replaces another.
template <int N>
__device__ __forceinline__ void take(Seen &s, const float (&x)[N], unsigned at, int on, int width) {
    const int lane = threadIdx.x & 31;
    float top = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, x[i]);
    if (top > s.m) {
        s.sum = s.m == -INFINITY ? 0.f : s.sum * ex2((s.m - top) * kLog2e);
        s.m = top;
    }
    if (s.m != -INFINITY) {
#pragma unroll
        for (int i = 0; i < N; ++i) s.sum += ex2((x[i] - s.m) * kLog2e);
    }
    if (!__any_sync(0xffffffffu, on > 0 && (top > s.least || !s.full))) return;
    uint32_t left = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) left |= (uint32_t)(i < on) << i;
    while (true) {
        uint32_t pass = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) pass |= (uint32_t)(x[i] > s.least || !s.full) << i;
        left &= pass;
        const uint32_t lanes = __ballot_sync(0xffffffffu, left != 0);
        if (lanes == 0) return;
        const int from = __ffs(lanes) - 1, e = __ffs(left) - 1;
        float v = x[0];
#pragma unroll
        for (int i = 1; i < N; ++i) v = e == i ? x[i] : v;
        const Key k = __shfl_sync(0xffffffffu, key_of(v, at + lane * N + e), from);
        if (lane == from) left &= left - 1;
        const int pos = __popc(__ballot_sync(0xffffffffu, s.mine > k));
        const Key up = __shfl_up_sync(0xffffffffu, s.mine, 1);
        if (lane > pos) s.mine = up;
        if (lane == pos) s.mine = k;
        if (lane >= width) s.mine = 0;
        const Key last = __shfl_sync(0xffffffffu, s.mine, width - 1);
        s.full = last != 0;
        s.least = s.full ? key_value(last) : -INFINITY;
    }
}

template <typename T>
struct Vec;   // 16 bytes of logits
template <>
struct Vec<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ void get(const uint4 &u, float (&x)[4]) {
        x[0] = unmask(__uint_as_float(u.x)), x[1] = unmask(__uint_as_float(u.y));
        x[2] = unmask(__uint_as_float(u.z)), x[3] = unmask(__uint_as_float(u.w));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static __forceinline__ void get(const uint4 &u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = unmask(bf16lo(w[i])), x[2 * i + 1] = unmask(bf16hi(w[i]));
    }
};

// One warp reads part `chunk` of a row once, by 16-byte loads where the row allows: the unaligned
// logits at its ends go to the first and the last part. The row's maximum and sum of exponentials
// come from the same pass as its best logits.
template <typename T>
__device__ Seen read_part(const Args &a, int row, int chunk) {
    constexpr int N = Vec<T>::N, kAhead = 4;
    const int lane = threadIdx.x & 31;
    const T *x = static_cast<const T *>(a.logits) + row * a.row_stride;
    const int head = min((int)((16 - (reinterpret_cast<uintptr_t>(x) & 15u)) % 16 / sizeof(T)), a.vocab);
    const int vectors = (a.vocab - head) / N;                   // whole ones
    const int v0 = (int)((long long)vectors * chunk / a.chunks), v1 = (int)((long long)vectors * (chunk + 1) / a.chunks);
    Seen s{0, -INFINITY, 0.f, -INFINITY, false};
    if (chunk == 0) {
        const float one[1] = {lane < head ? unmask((float)x[lane]) : -INFINITY};
        take<1>(s, one, 0, lane < head, a.width);
    }
    const uint4 *vec = reinterpret_cast<const uint4 *>(x + head);
    for (int v = v0; v < v1; v += 32 * kAhead) {
        uint4 u[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (v + 32 * i + lane < v1) u[i] = ldg_stream(vec + v + 32 * i + lane);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (v + 32 * i >= v1) break;
            const bool in = v + 32 * i + lane < v1;
            float f[N];
            if (in) {
                Vec<T>::get(u[i], f);
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) f[e] = -INFINITY;
            }
            take<N>(s, f, head + (v + 32 * i) * N, in ? N : 0, a.width);
        }
    }
    if (chunk == a.chunks - 1) {
        const int t = head + vectors * N, n = a.vocab - t;       // fewer than a vector
        const float one[1] = {lane < n ? unmask((float)x[t + lane]) : -INFINITY};
        take<1>(s, one, t, lane < n, a.width);
    }
    const float m = warp_max(s.m);
    s.sum = warp_sum(s.m == -INFINITY ? 0.f : s.sum * ex2((s.m - m) * kLog2e));
    s.m = m;
    return s;
}

// The parts of a sequence's rows joined and its continuations chosen, by one CTA of kWarps warps.
// keys, sums: [row of the sequence][part]. A warp joins a row's parts, lane = part; then lane w of
// one warp walks beam w's best logits, and the best of the lanes' heads is chosen `width` times.
// Candidates are compared in 64 bits.
__device__ void choose(const Args &a, int seq, const Key *keys, const float2 *sums, Key *rows, float2 *lse) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int w = warp; w < a.width; w += kWarps) {
        const bool part = lane < a.chunks;
        const Key *list = keys + ((size_t)w * a.chunks + lane) * a.width;
        const float2 ms = part ? sums[w * a.chunks + lane] : make_float2(-INFINITY, 0.f);
        const float m = warp_max(ms.x), sum = warp_sum(ms.x == -INFINITY ? 0.f : ms.y * ex2((ms.x - m) * kLog2e));
        if (lane == 0) lse[w] = make_float2(m, sum);
        int at = 0;
        Key head = part ? list[0] : 0;
        for (int j = 0; j < a.width; ++j) {
            const Key best = warp_max_key(head);
            if (lane == 0) rows[w * a.width + j] = best;
            if (head == best && best != 0) head = ++at < a.width ? list[at] : 0;
        }
    }
    __syncthreads();
    if (warp != 0) return;
    const int row = seq * a.width + lane;
    const bool on = lane < a.width;
    float score = -INFINITY;
    bool old = false, dead = true;
    double base = 0.0;
    if (on) {
        score = unmask(a.scores[row]);
        old = a.ended != nullptr && a.ended[row] != 0;
        const float2 ms = lse[lane];
        // no candidate above -inf: a masked score, or a row without a finite maximum
        dead = score == -INFINITY || score == INFINITY || (!old && !(fabsf(ms.x) < INFINITY));
        if (!dead && !old) base = (double)ms.x + log((double)ms.y);
    }
    int at = 0;   // of this beam's candidates, in order
    for (int j = 0; j < a.width; ++j) {
        double c = -INFINITY;
        int v = 0x7fffffff;
        if (on && at < a.width) {
            if (dead) {
                v = at;
            } else if (old) {   // eos, then the others in order
                v = at == 0 ? a.eos : at - 1 + (at - 1 >= a.eos);
                if (at == 0) c = score;
            } else {
                const Key k = rows[lane * a.width + at];
                v = (int)key_index(k);
                c = (double)key_value(k) - base + (double)score;
            }
        }
        double bc = c;
        int bw = lane;
        bool bon = v != 0x7fffffff;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double tc = __shfl_xor_sync(0xffffffffu, bc, o);
            const int tw = __shfl_xor_sync(0xffffffffu, bw, o);
            const bool ton = __shfl_xor_sync(0xffffffffu, (int)bon, o) != 0;
            if (ton && (!bon || tc > bc || (tc == bc && tw < bw))) bc = tc, bw = tw, bon = true;
        }
        if (bw == lane) {
            const int out = seq * a.width + j;
            a.tokens[out] = v;
            a.parents[out] = row;
            a.scores_out[out] = (float)c;
            if (a.ended_out != nullptr) a.ended_out[out] = old || v == a.eos;
            ++at;
        }
    }
}

// One cluster per sequence (gridDim.x / n_seq CTAs): its warps share the parts, whose results go to
// the first CTA's shared memory, which joins them. No scratch, one launch.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_beam_cluster(const Args a) {
    __shared__ Key keys[kClusterTasks * kMaxWidth], rows[kMaxWidth * kMaxWidth];
    __shared__ float2 sums[kClusterTasks], lse[kMaxWidth];
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = cluster.num_blocks(), rank = cluster.block_rank(), seq = blockIdx.x / ctas;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Key *keys0 = cluster.map_shared_rank(keys, 0);
    float2 *sums0 = cluster.map_shared_rank(sums, 0);
    cluster.sync();   // every CTA's shared memory is there
    for (int t = rank * kWarps + warp; t < a.width * a.chunks; t += ctas * kWarps) {
        const Seen s = read_part<T>(a, seq * a.width + t / a.chunks, t % a.chunks);
        if (lane < a.width) keys0[(size_t)t * a.width + lane] = s.mine;
        if (lane == 0) sums0[t] = make_float2(s.m, s.sum);
    }
    cluster.sync();
    if (rank == 0) choose(a, seq, keys, sums, rows, lse);
}

// Larger calls: a warp per part over the whole GPU, the results in scratch; then a CTA per sequence.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) k_beam_parts(const Args a, long long parts) {
    const int lane = threadIdx.x & 31;
    pdl_launch_dependents();
    const long long t = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= parts) return;
    const Seen s = read_part<T>(a, (int)(t / a.chunks), (int)(t % a.chunks));
    if (lane < a.width) a.keys[t * a.width + lane] = s.mine;
    if (lane == 0) a.sums[t] = make_float2(s.m, s.sum);
}
__global__ void __launch_bounds__(kWarps * 32) k_beam_choose(const Args a) {
    __shared__ Key rows[kMaxWidth * kMaxWidth];
    __shared__ float2 lse[kMaxWidth];
    pdl_wait();
    const size_t first = (size_t)blockIdx.x * a.width * a.chunks;
    choose(a, blockIdx.x, a.keys + first * a.width, a.sums + first, rows, lse);
}

// How a call runs. A cluster serves a sequence until its CTAs would read over kClusterLogits each;
// then the parts are spread over the GPU, at least kPartLogits each.
struct Shape {
    int ctas;     // of the cluster, or 0: two launches
    int chunks;
};
constexpr int kClusterLogits = 32768, kPartLogits = 1024;
constexpr int kTargetParts = 152 * 24;

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
    p.chunks = (int)std::min(most, std::max(1ll, (parts + width - 1) / width));
    return p;
}

size_t align16(size_t n) { return (n + 15) / 16 * 16; }

bool sizes_ok(int n_seq, int width, int vocab) {
    return n_seq >= 0 && width >= 1 && width <= kMaxWidth && vocab >= width && (long long)n_seq * width <= 0x7fffffffll / kMaxChunks;
}

}  // namespace

extern "C" {

size_t talker_beam_scratch(int n_seq, int width, int vocab) {
    if (!sizes_ok(n_seq, width, vocab)) return 0;
    const Shape p = shape_of(n_seq, width, vocab);
    const size_t parts = (size_t)n_seq * width * p.chunks;
    return p.ctas > 0 ? 0 : align16(parts * width * sizeof(Key)) + parts * sizeof(float2);
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
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = static_cast<cudaStream_t>(cuda_stream);
    cudaLaunchAttribute attr[1];
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const bool f32 = dtype == TALKER_DTYPE_F32;
    cudaError_t e;
    if (p.ctas > 0) {
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = p.ctas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3((unsigned)(n_seq * p.ctas));
        e = cudaLaunchKernelEx(&cfg, f32 ? k_beam_cluster<float> : k_beam_cluster<__nv_bfloat16>, a);
    } else {
        const long long parts = (long long)n_seq * width * p.chunks;
        a.keys = static_cast<Key *>(scratch);
        a.sums = reinterpret_cast<float2 *>(static_cast<char *>(scratch) + align16((size_t)parts * width * sizeof(Key)));
        cfg.gridDim = dim3((unsigned)((parts + kWarps - 1) / kWarps));
        cfg.numAttrs = 0;
        e = cudaLaunchKernelEx(&cfg, f32 ? k_beam_parts<float> : k_beam_parts<__nv_bfloat16>, a, parts);
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3((unsigned)n_seq);
        cfg.numAttrs = 1;
        if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, k_beam_choose, a);
    }
    if (e == cudaSuccess) return TALKER_OK;
    cudaGetLastError();
    return TALKER_ECUDA;
}

}  // extern "C"
