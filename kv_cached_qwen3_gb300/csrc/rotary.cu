// Rotary positions of heads (include/talker_layer.h).
#include <algorithm>
#include <cmath>

#include "kernels.cuh"
#include "rows.cuh"
#include "talker_layer.h"

using namespace talker_dev;

namespace {

constexpr double kPi = 3.14159265358979323846;
constexpr int kMostDims = 512;      // of a head
constexpr int kMostThreads = 512;   // groups of a head at most: of one dim and another, or of two neighbours

struct RotateArgs {
    const unsigned long long *turns;
    const int32_t *positions;
    talker_heads set[2];
    float amplitude;
    int all, rows;      // rows of all streams, of a stream
    int heads;          // of both sets
    int per, subs;      // a CTA's rows, and threads for each group of a row: every subs * gridDim.y th head each
    int rotary;         // rotary_dim
    int pair_groups;    // groups of dims of a head that are turned
    int groups;         // and of dims that stay, where they are copied
    int head_dim;
};

// cos and sin of (p times the table's entry) / 2^64 turns. The place in a turn is exact modulo 2^64; taken to the
// nearest quarter, at most an eighth of a turn is left, whose rounding to f32 is 2^-25 of it: 2e-8 of the result.
__device__ __forceinline__ float2 turn(int p, unsigned long long step, float amplitude) {
    const uint32_t place = (uint32_t)(((unsigned long long)(long long)p * step) >> 32);
    const uint32_t quarter = (place + (1u << 29)) >> 30;
    float s, c;
    sincospif((float)(int)(place - (quarter << 30)) * 0x1p-31f, &s, &c);
    const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
    return make_float2((quarter + 1) & 2 ? -a * amplitude : a * amplitude, quarter & 2 ? -b * amplitude : b * amplitude);
}

// A values by one access; two bf16 values make a word.
template <typename T, int A>
struct alignas(sizeof(T) * A) Vec {
    T v[A];
};
template <typename T, int A, int N>
struct Group {   // N values by accesses of A, the first `left` of them
    Vec<T, A> v[N / A];
    __device__ __forceinline__ void load(const T *p, int left) {
#pragma unroll
        for (int i = 0; i < N / A; ++i)
            if (i * A < left) v[i] = *reinterpret_cast<const Vec<T, A> *>(p + i * A);
    }
    __device__ __forceinline__ void store(T *p, int left) const {
#pragma unroll
        for (int i = 0; i < N / A; ++i)
            if (i * A < left) *reinterpret_cast<Vec<T, A> *>(p + i * A) = v[i];
    }
    __device__ __forceinline__ void get(float (&x)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = Elem<T>::load(v[i / A].v, i % A);
    }
    __device__ __forceinline__ void set(const float (&x)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (sizeof(T) == 2 && A % 2 == 0) {
                if (i % 2 == 0) *reinterpret_cast<__nv_bfloat162 *>(&v[i / A].v[i % A]) = __floats2bfloat162_rn(x[i], x[i + 1]);
            } else {
                Elem<T>::store(v[i / A].v, i % A, x[i]);
            }
        }
    }
};

// A CTA has `per` rows. A thread has one group of a head's dims of a row: A dims and those half a rotary_dim further, or N
// neighbours (with neighbours as pairs, and of dims that stay). It makes their cosines and sines once and turns the group in
// its heads. Bound by HBM where there are many rows: index arithmetic is kept out of the loop over heads (64-bit divisions a
// thread, and places made anew a head, took 59 and 97 us for 3 x 5001 rows of 40 heads).
template <typename T, int A, bool INTERLEAVED>
__global__ void __launch_bounds__(kMostThreads) k_rotate(const RotateArgs a) {
    constexpr int N = INTERLEAVED && A == 1 ? 2 : A, kPairs = INTERLEAVED ? N / 2 : A, kBatch = 4;
    const int id = threadIdx.x / (unsigned)a.groups, group = threadIdx.x - id * a.groups;
    const int in_cta = id / (unsigned)a.subs, row = blockIdx.x * a.per + in_cta;
    if (in_cta >= a.per || row >= a.all) return;
    const int stream = (unsigned)row / (unsigned)a.rows, t = row - stream * a.rows;
    const int stride = a.subs * gridDim.y;
    const bool turned = group < a.pair_groups;
    const int lo = turned ? group * N : a.rotary + (group - a.pair_groups) * N, left = a.head_dim - lo;
    float2 cs[kPairs];
    bool made = false;
    auto run = [&](const talker_heads &s, int h) {   // heads h, h + stride, ...
        const T *in = static_cast<const T *>(s.in) + stream * s.in_stream + t * s.in_row + h * s.in_head + lo;
        T *out = static_cast<T *>(s.out) + stream * s.out_stream + t * s.out_row + h * s.out_head + lo;
        const long long in_step = stride * s.in_head, out_step = stride * s.out_head;
        // in batches: all of a batch is on its way before the first is turned (what is written may be what is read)
        for (; h < s.heads; h += kBatch * stride) {
            Group<T, A, N> x[kBatch], y[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b, in += in_step)
                if (h + b * stride < s.heads) {
                    x[b].load(in, left);
                    if (!INTERLEAVED && turned) y[b].load(in + a.rotary / 2, left);
                }
            if (turned && !made) {   // (while the first are on their way)
                const int p = a.positions[row];
#pragma unroll
                for (int i = 0; i < kPairs; ++i) cs[i] = turn(p, a.turns[group * kPairs + i], a.amplitude);
                made = true;
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b, out += out_step) {
                if (h + b * stride >= s.heads) break;
                if (turned) {
                    float u[N], v[N];
                    x[b].get(u);
                    if (!INTERLEAVED) y[b].get(v);
#pragma unroll
                    for (int i = 0; i < kPairs; ++i) {
                        float &p = u[INTERLEAVED ? 2 * i : i], &q = INTERLEAVED ? u[2 * i + 1] : v[i];
                        const float p0 = p;
                        p = p0 * cs[i].x - q * cs[i].y;
                        q = p0 * cs[i].y + q * cs[i].x;
                    }
                    x[b].set(u);
                    if (!INTERLEAVED) y[b].set(v);
                }
                x[b].store(out, left);
                if (!INTERLEAVED && turned) y[b].store(out + a.rotary / 2, left);
            }
        }
    };
    const int first = blockIdx.y * a.subs + id - in_cta * a.subs;
    run(a.set[0], first);
    const int skip = a.set[0].heads % (unsigned)stride;   // (as if the sets were one)
    run(a.set[1], first < skip ? first - skip + stride : first - skip);
}

template <typename T, int A>
void launch(const RotateArgs &a, int slices, bool interleaved, cudaStream_t st) {
    const dim3 grid((unsigned)((a.all + a.per - 1) / a.per), slices);
    const int threads = (a.per * a.subs * a.groups + 31) / 32 * 32;
    if (interleaved) k_rotate<T, A, true><<<grid, threads, 0, st>>>(a);
    else k_rotate<T, A, false><<<grid, threads, 0, st>>>(a);
}

}  // namespace

namespace talker_k {

bool rope_frequencies(const talker_rope &r, double *freq, double *amplitude) {
    if (r.rotary_dim < 2 || r.rotary_dim % 2 || r.scaling < TALKER_ROPE_NONE || r.scaling > TALKER_ROPE_YARN) return false;
    const bool ranged = r.scaling == TALKER_ROPE_SMOOTH || r.scaling == TALKER_ROPE_YARN;
    if (!(r.theta > 1.0) || !std::isfinite(r.theta)) return false;
    if (r.scaling != TALKER_ROPE_NONE && (!(r.factor >= 1.0) || !std::isfinite(r.factor))) return false;
    if (r.scaling == TALKER_ROPE_NTK && r.rotary_dim < 4) return false;
    if (ranged && (!(r.original > 0.0) || !std::isfinite(r.original) || !std::isfinite(r.low) || !(r.high > r.low) || !std::isfinite(r.high))) return false;
    if (r.scaling == TALKER_ROPE_YARN && (!(r.low > 0.0) || !(r.amplitude >= 0.0) || !std::isfinite(r.amplitude))) return false;
    const double d = r.rotary_dim;
    double lo = 0.0, hi = 0.0, theta = r.theta;
    *amplitude = 1.0;
    if (r.scaling == TALKER_ROPE_NTK) theta *= std::pow(r.factor, d / (d - 2.0));
    if (r.scaling == TALKER_ROPE_YARN) {
        auto pair = [&](double beta) { return d * std::log(r.original / (2.0 * kPi * beta)) / (2.0 * std::log(r.theta)); };
        lo = std::max(0.0, std::floor(pair(r.high)));
        hi = std::min(d - 1.0, std::ceil(pair(r.low)));
        *amplitude = r.amplitude > 0.0 ? r.amplitude : 0.1 * std::log(r.factor) + 1.0;
    }
    for (int i = 0; i < r.rotary_dim / 2; ++i) {
        double f = std::pow(theta, -2.0 * i / d), keep = 1.0;
        if (r.scaling == TALKER_ROPE_LINEAR) keep = 0.0;
        if (r.scaling == TALKER_ROPE_SMOOTH) keep = std::min(1.0, std::max(0.0, (r.original * f / (2.0 * kPi) - r.low) / (r.high - r.low)));
        if (r.scaling == TALKER_ROPE_YARN) keep = 1.0 - std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 0.001)));
        freq[i] = keep < 1.0 ? f * keep + f / r.factor * (1.0 - keep) : f;
    }
    return true;
}

}  // namespace talker_k

extern "C" {

talker_status talker_rope_turns(const talker_rope *r, uint64_t *turns, float *amplitude) {
    if (!r || !turns || !amplitude || r->rotary_dim < 2 || r->rotary_dim > kMostDims) return TALKER_EINVAL;
    double freq[kMostDims / 2], amp;
    if (!talker_k::rope_frequencies(*r, freq, &amp)) return TALKER_EINVAL;
    for (int i = 0; i < r->rotary_dim / 2; ++i) turns[i] = (uint64_t)std::llround(std::ldexp(freq[i] / (2.0 * kPi), 64));   // (at most 1 radian)
    *amplitude = (float)amp;
    return TALKER_OK;
}

talker_status talker_rotate(const uint64_t *turns, float amplitude, int head_dim, int rotary_dim, int interleaved,
                            const int32_t *positions, int streams, int rows, const talker_heads *sets, int n_sets,
                            int dtype, void *cuda_stream) {
    if (!turns || !positions || !sets || n_sets < 1 || n_sets > 2 || streams < 0 || rows < 0) return TALKER_EINVAL;
    if (head_dim < 2 || head_dim > kMostDims || rotary_dim < 2 || rotary_dim % 2 || rotary_dim > head_dim) return TALKER_EINVAL;
    if (dtype != TALKER_DTYPE_F32 && dtype != TALKER_DTYPE_BF16) return TALKER_EINVAL;
    const int size = dtype == TALKER_DTYPE_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(turns) % 8 || reinterpret_cast<uintptr_t>(positions) % 4) return TALKER_EINVAL;
    RotateArgs a{};
    bool copy = false;
    for (int i = 0; i < n_sets; ++i) {
        const talker_heads &s = sets[i];
        if (!s.in || !s.out || s.heads < 0 || s.heads > 16384) return TALKER_EINVAL;
        if (reinterpret_cast<uintptr_t>(s.in) % size || reinterpret_cast<uintptr_t>(s.out) % size) return TALKER_EINVAL;
        a.set[i] = s;
        a.heads += s.heads;
        copy |= s.in != s.out;
    }
    if (streams == 0 || rows == 0 || a.heads == 0) return TALKER_OK;
    for (int i = 0; i < n_sets; ++i) {   // heads of a result lie in places of their own
        const talker_heads &s = sets[i];
        if (s.heads > 0 && ((streams > 1 && s.out_stream == 0) || (rows > 1 && s.out_row == 0) || (s.heads > 1 && s.out_head == 0))) return TALKER_EINVAL;
    }
    // the largest vector that fits the dims and every tensor's place and strides
    int vp = 16 / size;
    auto fits = [&](int n) {
        long long bits = (interleaved ? rotary_dim : rotary_dim / 2) | (head_dim - rotary_dim);
        uintptr_t at = 0;
        for (int i = 0; i < n_sets; ++i) {
            const talker_heads &s = sets[i];
            at |= reinterpret_cast<uintptr_t>(s.in) | reinterpret_cast<uintptr_t>(s.out);
            if (streams > 1) bits |= s.in_stream | s.out_stream;
            if (rows > 1) bits |= s.in_row | s.out_row;
            if (s.heads > 1) bits |= s.in_head | s.out_head;
        }
        return bits % n == 0 && at % (n * size) == 0;
    };
    while (vp > 1 && !fits(vp)) vp /= 2;
    a.turns = reinterpret_cast<const unsigned long long *>(turns);
    a.positions = positions;
    a.amplitude = amplitude;
    a.rows = rows;
    a.rotary = rotary_dim;
    a.head_dim = head_dim;
    const int dims = interleaved ? std::max(vp, 2) : vp;   // of a group: also of dims that stay
    a.pair_groups = (interleaved ? rotary_dim : rotary_dim / 2) / dims;
    a.groups = a.pair_groups + (copy ? (head_dim - rotary_dim + dims - 1) / dims : 0);
    if ((long long)streams * rows > 1 << 30) return TALKER_EINVAL;
    a.all = streams * rows;
    // about ten heads a thread, so that cosines are shared; with few rows fewer, down to one
    const int room = std::max(1, 256 / a.groups);   // threads for a group, of a CTA
    const long long want = (152ll * 2048 + (long long)a.all * a.groups - 1) / ((long long)a.all * a.groups);   // for a row, to fill the GPU
    const int threads = (int)std::min<long long>(a.heads, std::max<long long>(want, (a.heads + 9) / 10));
    a.subs = std::min(room, threads);
    a.per = room / a.subs;
    const int slices = (threads + a.subs - 1) / a.subs;
    const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    if (dtype == TALKER_DTYPE_F32) {
        if (vp == 4) launch<float, 4>(a, slices, interleaved, st);
        else if (vp == 2) launch<float, 2>(a, slices, interleaved, st);
        else launch<float, 1>(a, slices, interleaved, st);
    } else {
        if (vp == 8) launch<__nv_bfloat16, 8>(a, slices, interleaved, st);
        else if (vp == 4) launch<__nv_bfloat16, 4>(a, slices, interleaved, st);
        else if (vp == 2) launch<__nv_bfloat16, 2>(a, slices, interleaved, st);
        else launch<__nv_bfloat16, 1>(a, slices, interleaved, st);
    }
    return cudaGetLastError() == cudaSuccess ? TALKER_OK : TALKER_ECUDA;
}

}  // extern "C"
