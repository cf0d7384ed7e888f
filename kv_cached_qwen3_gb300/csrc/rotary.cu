// Rotary positions of heads (include/talker_layer.h).
#include <algorithm>
#include <cmath>

#include "rows.cuh"
#include "talker_layer.h"

using namespace talker_dev;

namespace {

struct RotateArgs {
    const unsigned long long *turns;
    const int32_t *positions;
    talker_heads set[2];
    long long units;    // threads with work: rows * slices * groups
    float amplitude;
    int rows;           // of a stream
    int heads;          // of both sets
    int slices;         // a row's heads h, h + slices, ... are one thread's
    int half;           // rotary_dim / 2
    int pair_groups;    // groups of VP pairs of a head
    int groups;         // and of 2 VP dims that stay, where they are copied
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

// VP values by one access.
template <typename T, int VP>
struct alignas(sizeof(T) * VP) Vec {
    T v[VP];
};

// A thread has one group of VP pairs of a row, makes their cosines and sines once, and turns the group in every
// `slices`th head of the row: two vectors of VP values read and written.
template <typename T, int VP, bool INTERLEAVED>
__global__ void __launch_bounds__(256) k_rotate(const RotateArgs a) {
    using V = Vec<T, VP>;
    const long long u = (long long)blockIdx.x * 256 + threadIdx.x;
    if (u >= a.units) return;
    const int group = (int)(u % a.groups);
    const long long rest = u / a.groups;
    const int slice = (int)(rest % a.slices);
    const long long row = rest / a.slices;
    const long long stream = row / a.rows;
    const int t = (int)(row - stream * a.rows);
    const bool turned = group < a.pair_groups;
    int lo, hi;   // the first dims of the two vectors
    if (turned) {
        lo = INTERLEAVED ? 2 * group * VP : group * VP;
        hi = INTERLEAVED ? lo + VP : lo + a.half;
    } else {
        lo = 2 * a.half + (group - a.pair_groups) * 2 * VP;
        hi = lo + VP;
    }
    const bool two = hi < a.head_dim;
    float2 cs[VP];
    if (turned) {
        const int p = a.positions[row];
#pragma unroll
        for (int i = 0; i < VP; ++i) cs[i] = turn(p, a.turns[group * VP + i], a.amplitude);
    }
#pragma unroll 4
    for (int h = slice; h < a.heads; h += a.slices) {
        const int k = h >= a.set[0].heads;
        const talker_heads &s = a.set[k];
        const int head = k ? h - a.set[0].heads : h;
        const T *in = static_cast<const T *>(s.in) + stream * s.in_stream + t * s.in_row + head * s.in_head;
        T *out = static_cast<T *>(s.out) + stream * s.out_stream + t * s.out_row + head * s.out_head;
        V x = *reinterpret_cast<const V *>(in + lo), y{};
        if (two) y = *reinterpret_cast<const V *>(in + hi);
        if (turned) {
            float e[2 * VP];
#pragma unroll
            for (int i = 0; i < VP; ++i) e[i] = Elem<T>::load(x.v, i), e[VP + i] = Elem<T>::load(y.v, i);
#pragma unroll
            for (int i = 0; i < VP; ++i) {
                float &p = e[INTERLEAVED ? 2 * i : i], &q = e[INTERLEAVED ? 2 * i + 1 : VP + i];
                const float c = cs[i].x, n = cs[i].y, p0 = p;
                p = p0 * c - q * n;
                q = p0 * n + q * c;
            }
#pragma unroll
            for (int i = 0; i < VP; ++i) Elem<T>::store(x.v, i, e[i]), Elem<T>::store(y.v, i, e[VP + i]);
        }
        *reinterpret_cast<V *>(out + lo) = x;
        if (two) *reinterpret_cast<V *>(out + hi) = y;
    }
}

template <typename T, int VP>
void launch(const RotateArgs &a, bool interleaved, cudaStream_t st) {
    const unsigned blocks = (unsigned)((a.units + 255) / 256);
    if (interleaved) k_rotate<T, VP, true><<<blocks, 256, 0, st>>>(a);
    else k_rotate<T, VP, false><<<blocks, 256, 0, st>>>(a);
}

}  // namespace

extern "C" {

talker_status talker_rope_turns(const talker_rope *r, uint64_t *turns, float *amplitude) {
    if (!r || !turns || !amplitude || r->rotary_dim < 2 || r->rotary_dim % 2 || r->rotary_dim > 1 << 20) return TALKER_EINVAL;
    if (!(r->theta > 1.0) || !std::isfinite(r->theta)) return TALKER_EINVAL;
    const double pi = 3.14159265358979323846, d = r->rotary_dim;
    const bool ranged = r->scaling == TALKER_ROPE_SMOOTH || r->scaling == TALKER_ROPE_YARN;
    if (r->scaling < TALKER_ROPE_NONE || r->scaling > TALKER_ROPE_YARN) return TALKER_EINVAL;
    if (r->scaling != TALKER_ROPE_NONE && (!(r->factor >= 1.0) || !std::isfinite(r->factor))) return TALKER_EINVAL;
    if (r->scaling == TALKER_ROPE_NTK && r->rotary_dim < 4) return TALKER_EINVAL;
    if (ranged && (!(r->original > 0.0) || !std::isfinite(r->original) || !(r->low > 0.0) || !(r->high > r->low) || !std::isfinite(r->high)))
        return TALKER_EINVAL;
    *amplitude = 1.0f;
    double lo = 0.0, hi = 0.0, theta = r->theta;
    if (r->scaling == TALKER_ROPE_NTK) theta *= std::pow(r->factor, d / (d - 2.0));
    if (r->scaling == TALKER_ROPE_YARN) {
        if (!(r->amplitude >= 0.0) || !std::isfinite(r->amplitude)) return TALKER_EINVAL;
        auto pair = [&](double beta) { return d * std::log(r->original / (2.0 * pi * beta)) / (2.0 * std::log(r->theta)); };
        lo = std::max(0.0, std::floor(pair(r->high)));
        hi = std::min(d - 1.0, std::ceil(pair(r->low)));
        *amplitude = (float)(r->amplitude > 0.0 ? r->amplitude : 0.1 * std::log(r->factor) + 1.0);
    }
    for (int i = 0; i < r->rotary_dim / 2; ++i) {
        double f = std::pow(theta, -2.0 * i / d), keep = 1.0;
        if (r->scaling == TALKER_ROPE_LINEAR) keep = 0.0;
        if (r->scaling == TALKER_ROPE_SMOOTH)
            keep = std::min(1.0, std::max(0.0, (r->original * f / (2.0 * pi) - r->low) / (r->high - r->low)));
        if (r->scaling == TALKER_ROPE_YARN) keep = 1.0 - std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 0.001)));
        if (keep < 1.0) f = f * keep + f / r->factor * (1.0 - keep);
        turns[i] = (uint64_t)std::llround(std::ldexp(f / (2.0 * pi), 64));   // (f is at most 1 radian)
    }
    return TALKER_OK;
}

talker_status talker_rotate(const uint64_t *turns, float amplitude, int head_dim, int rotary_dim, int interleaved,
                            const int32_t *positions, int streams, int rows, const talker_heads *sets, int n_sets,
                            int dtype, void *cuda_stream) {
    if (!turns || !positions || !sets || n_sets < 1 || n_sets > 2 || streams < 0 || rows < 0) return TALKER_EINVAL;
    if (head_dim < 2 || head_dim > 1024 || rotary_dim < 2 || rotary_dim % 2 || rotary_dim > head_dim) return TALKER_EINVAL;
    if (dtype != TALKER_DTYPE_F32 && dtype != TALKER_DTYPE_BF16) return TALKER_EINVAL;
    const int size = dtype == TALKER_DTYPE_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(turns) % 8 || reinterpret_cast<uintptr_t>(positions) % 4) return TALKER_EINVAL;
    RotateArgs a{};
    bool copy = false;
    for (int i = 0; i < n_sets; ++i) {
        const talker_heads &s = sets[i];
        if (!s.in || !s.out || s.heads < 0 || s.heads > 65536) return TALKER_EINVAL;
        if (reinterpret_cast<uintptr_t>(s.in) % size || reinterpret_cast<uintptr_t>(s.out) % size) return TALKER_EINVAL;
        a.set[i] = s;
        a.heads += s.heads;
        copy |= s.in != s.out;
    }
    if (streams == 0 || rows == 0 || a.heads == 0) return TALKER_OK;
    // the largest vector that fits the dims and every tensor's place and strides
    int vp = 16 / size;
    auto fits = [&](int n) {
        long long bits = rotary_dim / 2 | (head_dim - rotary_dim);
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
    a.half = rotary_dim / 2;
    a.head_dim = head_dim;
    a.pair_groups = a.half / vp;
    a.groups = a.pair_groups + (copy ? (head_dim - rotary_dim + 2 * vp - 1) / (2 * vp) : 0);
    const long long n = (long long)streams * rows;
    a.slices = (int)std::min<long long>(a.heads, std::max<long long>(1, 152ll * 2048 / (n * a.groups)));
    a.units = n * a.slices * a.groups;
    if ((a.units + 255) / 256 > 0x7fffffffll) return TALKER_EINVAL;
    const cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    if (dtype == TALKER_DTYPE_F32) {
        if (vp == 4) launch<float, 4>(a, interleaved, st);
        else if (vp == 2) launch<float, 2>(a, interleaved, st);
        else launch<float, 1>(a, interleaved, st);
    } else {
        if (vp == 8) launch<__nv_bfloat16, 8>(a, interleaved, st);
        else if (vp == 4) launch<__nv_bfloat16, 4>(a, interleaved, st);
        else if (vp == 2) launch<__nv_bfloat16, 2>(a, interleaved, st);
        else launch<__nv_bfloat16, 1>(a, interleaved, st);
    }
    return cudaGetLastError() == cudaSuccess ? TALKER_OK : TALKER_ECUDA;
}

}  // extern "C"
