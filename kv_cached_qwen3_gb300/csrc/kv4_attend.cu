// Decode attention over the 4-bit paged cache (talker_kv4_attend).
#include <algorithm>
#include <math.h>

#include "kv4.cuh"

using namespace talker_dev;

namespace talker_k {

namespace {

constexpr int kWarps = 4;
constexpr int kMaxG = 8;
constexpr float kLog2e = 1.4426950408889634f;

template <typename T>
__device__ __forceinline__ float to_f32(T v) { return (float)v; }

// Grid (splits, n_kv, B): CTA (s, g, b) walks a range of pages of stream b and KV head g, its warps
// one key at a time (lane = HD / 32 dims), with an online softmax per warp.
template <int HD, typename TI, typename TO>
__global__ void __launch_bounds__(kWarps * 32) k_kv4_attend(const Kv4Attend a) {
    using Tile = Kv4Tile<HD>;
    constexpr int NB = Tile::NB, PD = HD / 32;
    __shared__ float wm[kWarps][kMaxG], wl[kWarps][kMaxG], wo[kWarps][kMaxG][HD];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int s = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
    const int G = a.n_q / a.c.n_kv_heads;
    int len = a.lens[b];
    if (len < 0 || len > a.c.pages_per_stream * kPage) {
        if (threadIdx.x == 0 && s == 0 && a.c.status != nullptr) atomicOr(a.c.status, ST_BAD_POSITION);
        len = -1;
    }
    const int npages = len > 0 ? (len + kPage - 1) / kPage : 0;
    const int per = (npages + a.splits - 1) / a.splits;
    const int pb = s * per, pe = min(pb + per, npages);
    float q[kMaxG][PD], m[kMaxG], l[kMaxG], o[kMaxG][PD];
#pragma unroll
    for (int h = 0; h < kMaxG; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
#pragma unroll
        for (int d = 0; d < PD; ++d) {
            o[h][d] = 0.f;
            q[h][d] = h < G ? to_f32(static_cast<const TI *>(a.q)[b * a.q_row + (size_t)(g * G + h) * HD + lane * PD + d]) *
                                  (a.scale * kLog2e)
                            : 0.f;
        }
    }
    if (len >= 0 && a.k_new != nullptr && s == 0 && warp == 0) {
        const size_t at = b * a.new_row + (size_t)g * HD + lane * PD;
#pragma unroll
        for (int h = 0; h < kMaxG; ++h) {
            float t = 0.f;
#pragma unroll
            for (int d = 0; d < PD; ++d) t = fmaf(q[h][d], to_f32(static_cast<const TI *>(a.k_new)[at + d]), t);
            m[h] = warp_sum(t);
            l[h] = 1.f;
#pragma unroll
            for (int d = 0; d < PD; ++d) o[h][d] = to_f32(static_cast<const TI *>(a.v_new)[at + d]);
        }
    }
    // this lane's codes of a row: dims lane * PD ..
    const int blk = lane * PD / 32, in = lane * PD % 32;
    const int kat = (in / 8) * 4 * NB + 4 * blk + (in % 8) / 2, vat = (in / 4) * 2 * NB + 2 * blk + (in % 4) / 2;
    for (int pg = pb; pg < pe; ++pg) {
        const int page = a.c.page_table[(size_t)b * a.c.pages_per_stream + pg];
        if (page < 0 || page >= a.c.n_pages) {
            if (threadIdx.x == 0 && a.c.status != nullptr) atomicOr(a.c.status, ST_BAD_ARG);
            continue;
        }
        const size_t off = (((size_t)page * a.c.n_layers + a.layer) * a.c.n_kv_heads + g) * Tile::kBytes;
        const unsigned char *kt = static_cast<const unsigned char *>(a.c.k) + off;
        const unsigned char *vt = static_cast<const unsigned char *>(a.c.v) + off;
        const int valid = min(kPage, len - pg * kPage);
        for (int j = warp; j < valid; j += kWarps) {
            uint32_t kw, vw;
            if (PD == 4) {
                kw = *reinterpret_cast<const uint16_t *>(kt + j * Tile::kRow + kat);
                vw = *reinterpret_cast<const uint16_t *>(vt + j * Tile::kRow + vat);
            } else {
                kw = kt[j * Tile::kRow + kat];
                vw = vt[j * Tile::kRow + vat];
            }
            const float kd = __half2float(*reinterpret_cast<const __half *>(kt + Tile::kScales + (j * NB + blk) * 2));
            const float vd = __half2float(*reinterpret_cast<const __half *>(vt + Tile::kScales + (j * NB + blk) * 2));
#pragma unroll
            for (int h = 0; h < kMaxG; ++h) {
                float t = 0.f;
#pragma unroll
                for (int d = 0; d < PD; ++d) t = fmaf(q[h][d], (float)((int)(kw >> (4 * d) & 15u) - 8) * kd, t);
                t = warp_sum(t);
                const float mn = fmaxf(m[h], t);
                const float al = m[h] == -INFINITY ? 0.f : exp2f(m[h] - mn), p = exp2f(t - mn);
                m[h] = mn;
                l[h] = fmaf(l[h], al, p);
#pragma unroll
                for (int d = 0; d < PD; ++d) o[h][d] = fmaf(p, (float)((int)(vw >> (4 * d) & 15u) - 8) * vd, o[h][d] * al);
            }
        }
    }
#pragma unroll
    for (int h = 0; h < kMaxG; ++h) {
        if (lane == 0) {
            wm[warp][h] = m[h];
            wl[warp][h] = l[h];
        }
#pragma unroll
        for (int d = 0; d < PD; ++d) wo[warp][h][lane * PD + d] = o[h][d];
    }
    __syncthreads();
    for (int idx = threadIdx.x; idx < G * HD; idx += kWarps * 32) {
        const int h = idx / HD, d = idx % HD;
        float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w][h]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float e = wm[w][h] == -INFINITY ? 0.f : exp2f(wm[w][h] - M);
            L = fmaf(wl[w][h], e, L);
            O = fmaf(wo[w][h][d], e, O);
        }
        const size_t row = (size_t)b * a.n_q + g * G + h;
        if (a.splits == 1) {
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
    const size_t row = (size_t)blockIdx.y * a.n_q + blockIdx.x;
    const float *ws = a.scratch + row * a.splits * (HD + 4);
    float M = -INFINITY, L = 0.f, O = 0.f;
    for (int s = 0; s < a.splits; ++s) M = fmaxf(M, ws[s * (HD + 4)]);
    for (int s = 0; s < a.splits; ++s) {
        const float m = ws[s * (HD + 4)], e = m == -INFINITY ? 0.f : exp2f(m - M);
        L = fmaf(ws[s * (HD + 4) + 1], e, L);
        O = fmaf(ws[s * (HD + 4) + 4 + threadIdx.x], e, O);
    }
    static_cast<TO *>(a.out)[row * HD + threadIdx.x] = (TO)(L == 0.f ? 0.f : O / L);
}

template <int HD, typename TI, typename TO>
cudaError_t launch_t(const Kv4Attend &a, cudaStream_t s) {
    k_kv4_attend<HD, TI, TO><<<dim3(a.splits, a.c.n_kv_heads, a.B), kWarps * 32, 0, s>>>(a);
    if (a.splits > 1) k_kv4_combine<HD, TO><<<dim3(a.n_q, a.B), HD, 0, s>>>(a);
    return cudaGetLastError();
}

template <int HD>
cudaError_t launch_hd(const Kv4Attend &a, int in_bf16, int out_bf16, cudaStream_t s) {
    if (in_bf16) return out_bf16 ? launch_t<HD, __nv_bfloat16, __nv_bfloat16>(a, s) : launch_t<HD, __nv_bfloat16, float>(a, s);
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
