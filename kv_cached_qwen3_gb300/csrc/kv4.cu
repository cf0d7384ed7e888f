// Rows written to and read from the 4-bit paged cache, and streams reordered by sharing pages.
#include "kv4.cuh"

using namespace talker_dev;

namespace talker_k {

namespace {

constexpr int kRowThreads = 256;

// Eight dims by one access of 32 bytes (f32) or 16 (bf16), or dim by dim.
template <typename T>
__device__ __forceinline__ void load8(const T *p, bool vec, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float *p, bool vec, float (&x)[8]) {
    if (vec) {
        asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                     : "l"(p));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = p[i];
    }
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, bool vec, float (&x)[8]) {
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
__device__ __forceinline__ void store8(float *p, bool vec, const float (&x)[8]) {
    if (vec) {
        asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]),
                     "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                     : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = x[i];
    }
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, bool vec, const float (&x)[8]) {
    if (vec) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = __float2bfloat16_rn(x[i]);
    }
}

// A thread has 8 dims of a row; the 4 * NB threads of a head row are neighbours.
struct RowPlace {
    unsigned char *tile;   // null: nothing to do
    int prow;
};

__device__ __forceinline__ RowPlace place_of(const Kv4Rows &r, int tile_bytes, int s, int l, int h, bool is_v, long long pos,
                                             bool report) {
    if (pos < 0 || pos >= (long long)r.c.pages_per_stream * kPage) {
        if (report && r.c.status != nullptr) atomicOr(r.c.status, ST_BAD_POSITION);
        return {nullptr, 0};
    }
    const int page = r.c.page_table[(size_t)(r.stream0 + s) * r.c.pages_per_stream + (int)(pos / kPage)];
    if (page < 0 || page >= r.c.n_pages) {
        if (report && r.c.status != nullptr) atomicOr(r.c.status, ST_BAD_ARG);
        return {nullptr, 0};
    }
    return {static_cast<unsigned char *>(is_v ? r.c.v : r.c.k) +
                (((size_t)page * r.c.n_layers + r.layer0 + l) * r.c.n_kv_heads + h) * tile_bytes,
            (int)(pos % kPage)};
}

// A row's word and scale of a lane; where tile is null, none.
struct Codes {
    uint32_t w;
    unsigned short d;
};
template <int HD>
__device__ __forceinline__ Codes load_codes(const unsigned char *tile, int prow, bool is_v, int b, int c) {
    using Tile = Kv4Tile<HD>;
    if (tile == nullptr) return {0, 0};
    return {*reinterpret_cast<const uint32_t *>(tile + prow * Tile::kRow + q4_word_at<Tile::NB>(is_v, b, c)),
            *reinterpret_cast<const unsigned short *>(tile + Tile::kScales + (prow * Tile::NB + b) * 2)};
}
// The values they stand for; every lane of the warp takes part.
__device__ __forceinline__ void values_of(const Codes &k, bool is_v, int b, float (&x)[8]) {
    q4_values8(is_v ? v_word(k.w, b) : k.w, __half2float(__ushort_as_half(k.d)), x);
}
// A lane's eight dims quantized into the tile; every lane of the warp takes part.
template <int HD, typename T>
__device__ __forceinline__ void store_codes(unsigned char *tile, int prow, bool is_v, int b, int c, const float (&x)[8]) {
    using Tile = Kv4Tile<HD>;
    unsigned short d;
    uint32_t w = q4_codes8<sizeof(T) == 2>(x, d);
    if (is_v) w = v_word(w, b);
    if (tile == nullptr) return;
    *reinterpret_cast<uint32_t *>(tile + prow * Tile::kRow + q4_word_at<Tile::NB>(is_v, b, c)) = w;
    if (c == 0) *reinterpret_cast<unsigned short *>(tile + Tile::kScales + (prow * Tile::NB + b) * 2) = d;
}

// Few rows: grid (items, streams, layers * 2), a head row per 4 * NB threads, rows of a head behind
// one another. A row of 32 streams in 5 layers: 2.3 us, most of it a launch's own time.
template <int HD, typename T, bool READ>
__global__ void __launch_bounds__(kRowThreads) k_kv4_rows(const Kv4Rows r, const bool vec) {
    using Tile = Kv4Tile<HD>;
    constexpr int TPR = 4 * Tile::NB;
    const int s = blockIdx.y, l = blockIdx.z >> 1;
    const bool is_v = blockIdx.z & 1;
    const int sub = threadIdx.x % TPR, b = sub >> 2, c = sub & 3;
    const unsigned item = blockIdx.x * (kRowThreads / TPR) + threadIdx.x / TPR;
    const int h = (int)(item / (unsigned)r.T), i = (int)(item - (unsigned)h * r.T);
    const bool on = h < r.c.n_kv_heads && (r.count == nullptr || i < r.count[s]);
    T *dense = static_cast<T *>(is_v ? r.v : r.k) + (l * r.st.layer + s * r.st.stream + i * r.st.row + h * r.st.head) +
               b * 32 + c * 8;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (!READ && on) load8<T>(dense, vec, x);
    RowPlace p{nullptr, 0};
    if (on) p = place_of(r, Tile::kBytes, s, l, h, is_v, (r.start != nullptr ? (long long)r.start[s] : 0) + i, sub == 0);
    if (READ) {
        values_of(load_codes<HD>(p.tile, p.prow, is_v, b, c), is_v, b, x);
        if (p.tile != nullptr) store8(dense, vec, x);
    } else {
        store_codes<HD, T>(p.tile, p.prow, is_v, b, c, x);
    }
}

// The rows [lo, hi) of one page that a call has of a stream, and where they lie.
struct PageRows {
    long long first;   // position of the page's row 0, counted from the call's row 0
    int lo, hi;
};
__device__ __forceinline__ PageRows page_rows(const Kv4Rows &r, int s, int slot, long long &pos) {
    const long long start = r.start != nullptr ? (long long)r.start[s] : 0;
    const int n = r.count != nullptr ? min(r.count[s], r.T) : r.T;
    pos = (start >= 0 ? start / kPage : -((kPage - 1 - start) / kPage)) * kPage + (long long)slot * kPage;
    return {pos - start, (int)max(0ll, start - pos), (int)min((long long)kPage, start + n - pos)};
}

// Many rows: a CTA per (page, head), kRowThreads / (4 * NB) rows at a time: one look-up of the page, and
// all its loads in flight. 28 layers x 4096 rows of 8 heads of 128 dims: f32 written in 172 us (6.2 TB/s of
// dense rows and codes, 92% of the measured copy rate), read in 165 (96%); bf16 written in 141 (63%; bound by
// the quantization's instructions, nearly the same for half the bytes), read in 96 (92%).
// Grid (pages * heads, streams, layers * 2) to write and (pages * heads, streams, layers) to read, where a
// CTA takes K and V, whose loads are small.
template <int HD, typename T>
__global__ void __launch_bounds__(kRowThreads) k_kv4_write_pages(const Kv4Rows r, const bool vec) {
    using Tile = Kv4Tile<HD>;
    constexpr int TPR = 4 * Tile::NB, RP = kRowThreads / TPR, kPasses = kPage / RP;
    const int s = blockIdx.y, l = blockIdx.z >> 1;
    const bool is_v = blockIdx.z & 1;
    const int h = blockIdx.x % r.c.n_kv_heads, slot = blockIdx.x / r.c.n_kv_heads;
    const int sub = threadIdx.x % TPR, b = sub >> 2, c = sub & 3;
    long long pos;
    const PageRows at = page_rows(r, s, slot, pos);
    if (at.lo >= at.hi) return;
    const T *dense = static_cast<const T *>(is_v ? r.v : r.k) + (l * r.st.layer + s * r.st.stream + h * r.st.head) + b * 32 + c * 8;
    float x[kPasses][8];
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
        const int row = at.lo + u * RP + threadIdx.x / TPR;
        if (row < at.hi) {
            load8<T>(dense + (at.first + row) * r.st.row, vec, x[u]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[u][e] = 0.f;
        }
    }
    const RowPlace p = place_of(r, Tile::kBytes, s, l, h, is_v, pos, threadIdx.x == 0);
    if (p.tile == nullptr) return;
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
        const int row = at.lo + u * RP + threadIdx.x / TPR;
        if (at.lo + u * RP < at.hi) store_codes<HD, T>(row < at.hi ? p.tile : nullptr, row, is_v, b, c, x[u]);
    }
}
template <int HD, typename T>
__global__ void __launch_bounds__(kRowThreads) k_kv4_read_pages(const Kv4Rows r, const bool vec) {
    using Tile = Kv4Tile<HD>;
    constexpr int TPR = 4 * Tile::NB, RP = kRowThreads / TPR, kPasses = kPage / RP;
    const int s = blockIdx.y, l = blockIdx.z;
    const int h = blockIdx.x % r.c.n_kv_heads, slot = blockIdx.x / r.c.n_kv_heads;
    const int sub = threadIdx.x % TPR, b = sub >> 2, c = sub & 3;
    long long pos;
    const PageRows at = page_rows(r, s, slot, pos);
    if (at.lo >= at.hi) return;
    const RowPlace p = place_of(r, Tile::kBytes, s, l, h, false, pos, threadIdx.x == 0);
    if (p.tile == nullptr) return;
    unsigned char *tiles[2] = {p.tile, static_cast<unsigned char *>(r.c.v) + (p.tile - static_cast<unsigned char *>(r.c.k))};
    Codes k[2][kPasses];
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int u = 0; u < kPasses; ++u) {
            const int row = at.lo + u * RP + threadIdx.x / TPR;
            k[v][u] = load_codes<HD>(row < at.hi ? tiles[v] : nullptr, row, v, b, c);
        }
    const int64_t off = l * r.st.layer + s * r.st.stream + h * r.st.head + b * 32 + c * 8;
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
        for (int u = 0; u < kPasses; ++u) {
            const int row = at.lo + u * RP + threadIdx.x / TPR;
            if (at.lo + u * RP >= at.hi) continue;
            float x[8];
            values_of(k[v][u], v, b, x);
            if (row < at.hi) store8(static_cast<T *>(v ? r.v : r.k) + off + (at.first + row) * r.st.row, vec, x);
        }
}

// From this many rows a stream on, a CTA per page is faster: a page's loads are in flight at once, but a
// small part of a page leaves most of its CTA without work. 32 streams, 5 layers, 8 heads of 128 in f32,
// us by rows / by pages: written, 32 rows 11.9 / 17.9, 64 22.8 / 23.8, 128 43.6 / 40.4, 256 84.1 / 70.2;
// read, 16 rows 6.0 / 6.9, 32 9.8 / 9.5, 64 19.9 / 15.1, 256 72.4 / 61.7. (bf16: 128 rows written 42.3 / 35.0.)
constexpr int kWritePageRows = 96, kReadPageRows = 32;

template <int HD, typename T, bool READ>
cudaError_t launch_rows_t(const Kv4Rows &r, bool vec, cudaStream_t s) {
    if (r.T >= (READ ? kReadPageRows : kWritePageRows)) {
        const long long slots = ((long long)r.T + kPage - 2) / kPage + 1;   // pages that T rows can touch
        const dim3 grid((unsigned)(slots * r.c.n_kv_heads), r.n_streams, READ ? r.n_layers : 2 * r.n_layers);
        if (READ) k_kv4_read_pages<HD, T><<<grid, kRowThreads, 0, s>>>(r, vec);
        else k_kv4_write_pages<HD, T><<<grid, kRowThreads, 0, s>>>(r, vec);
    } else {
        const long long items = (long long)r.T * r.c.n_kv_heads;
        const int per = kRowThreads / (HD / 8);
        k_kv4_rows<HD, T, READ><<<dim3((unsigned)((items + per - 1) / per), r.n_streams, 2 * r.n_layers), kRowThreads, 0, s>>>(r, vec);
    }
    return cudaGetLastError();
}

// ---- reorder

struct ReorderScratch {   // one warp's sets of streams
    uint32_t used[32], need[32];
};

__device__ __forceinline__ int parent_of(const KvReorder &r, int i) {
    const int p = i < r.R ? r.parents[i] : i;
    return p >= 0 && p < r.n_streams && (r.group == 0 || p / r.group == i / r.group) ? p : i;
}
__device__ __forceinline__ int length_of(const KvReorder &r, int p) { return min(max(r.lens[p], 0), r.pps * kPage); }

// What stream p, whose tail page is in column `tail`, holds of column j: its page's r, plus kFull if the page
// is full (else it is the tail), or -1.
constexpr int kFull = 0x4000;
__device__ __forceinline__ int entry_of(const KvReorder &r, int j, int p, int tail, bool report) {
    const int entry = r.table[(size_t)p * r.pps + j], er = entry / r.pps;
    const bool ok = entry >= 0 && entry - er * r.pps == j && er < r.n_streams;
    if (report && !ok && j <= tail && r.status != nullptr) atomicOr(r.status, ST_BAD_ARG);
    return ok && j <= tail ? er | (j < tail ? kFull : 0) : -1;
}

// One warp finds column j of the new table from the entries of its rows' parents. Row i keeps its parent's page where that is full
// (shared), and takes it over at the parent's tail page, unless a row before it did (another child) or a
// stream shares the page (as one may after this one was cut shorter); every other row needs a page of
// its own, and gets the pages of the column's set {r * pps + j} that no kept entry uses, in order. A row
// refers to one page of a column, so there are always enough. Writes the column when `store`; returns
// row `ask`'s entry.
__device__ int reorder_column(const KvReorder &r, int j, int ask, bool store, const short *entries, ReorderScratch &w) {
    const int lane = threadIdx.x & 31;
    w.used[lane] = w.need[lane] = 0;
    __syncwarp();
    int answer = -1;
    for (int i = lane; i < r.n_streams; i += 32) {
        const int e = entries[i], er = e & ~kFull;
        if (e < 0 || !(e & kFull)) continue;
        atomicOr(&w.used[er >> 5], 1u << (er & 31));
        if (store) r.table_out[(size_t)i * r.pps + j] = er * r.pps + j;
        if (i == ask) answer = er * r.pps + j;
    }
    __syncwarp();
    for (int base = 0; base < r.n_streams; base += 32) {
        const int i = base + lane;
        const bool in = i < r.n_streams;
        const int e = in ? entries[i] : -1, er = e;
        const bool full = e >= 0 && (e & kFull), tail = e >= 0 && !full;
        const uint32_t same = __match_any_sync(0xffffffffu, tail ? er : -1 - lane);
        const bool takes = tail && (same & ((1u << lane) - 1)) == 0 && !(w.used[er >> 5] >> (er & 31) & 1u);
        __syncwarp();
        if (takes) {
            atomicOr(&w.used[er >> 5], 1u << (er & 31));
            if (store) r.table_out[(size_t)i * r.pps + j] = er * r.pps + j;
            if (i == ask) answer = er * r.pps + j;
        }
        const uint32_t wants = __ballot_sync(0xffffffffu, in && !takes && !full);
        if (lane == 0) w.need[base >> 5] = wants;
        __syncwarp();
    }
    // free pages of the column: lane holds word `lane` of their set and how many lie before it
    uint32_t fw = ~w.used[lane];
    const int left = r.n_streams - 32 * lane;
    fw &= left >= 32 ? 0xffffffffu : (left > 0 ? (1u << left) - 1 : 0u);
    int before = __popc(fw);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += t;
    }
    before -= __popc(fw);
    const int first = store ? 0 : ask & ~31, last = store ? r.n_streams : first + 1;   // (just the row that is asked for)
    int taken = __reduce_add_sync(0xffffffffu, 32 * lane < first ? __popc(w.need[lane]) : 0);
    for (int base = first; base < last; base += 32) {
        const uint32_t wants = w.need[base >> 5];
        int k = taken + __popc(wants & ((1u << lane) - 1));
        taken += __popc(wants);
        int word = 0;   // the last word with at most k free pages before it
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            if (__shfl_sync(0xffffffffu, before, word + o) <= k) word += o;
        uint32_t bits = __shfl_sync(0xffffffffu, fw, word);
        k -= __shfl_sync(0xffffffffu, before, word);
        if (wants >> lane & 1u) {
            while (k-- > 0) bits &= bits - 1;
            const int entry = (32 * word + __ffs(bits) - 1) * r.pps + j;
            if (store) r.table_out[(size_t)(base + lane) * r.pps + j] = entry;
            if (base + lane == ask) answer = entry;
        }
    }
    return __shfl_sync(0xffffffffu, answer, ask & 31);
}

// The first table_blocks CTAs write the table, a warp per column, and the lengths. The others copy
// the rows of a tail page that its stream did not take over from its parent: copy_blocks CTAs per
// stream, a warp per tile. Each finds its destination itself (the column is a few hundred bytes), so
// that one launch does it all. Sources are pages that stay in use, destinations pages that nothing
// in use refers to, so copies need no order. 32 streams of 700 rows in 5 layers 6.2 us, of 8192 rows in
// 28 layers (tails at a page's end: nothing to copy) 3.2, 512 streams of 1000 rows in 5 layers 36: bound by
// the chain parents -> lengths -> table -> column of a copying CTA, not by the copies.
__global__ void __launch_bounds__(256) k_reorder(const KvReorder r, int table_blocks, int copy_blocks) {
    __shared__ ReorderScratch scratch[8];
    __shared__ short entries[8][kReorderMaxStreams];
    __shared__ int to_s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x < table_blocks) {
        const int j = blockIdx.x * 8 + warp;
        if (blockIdx.x == 0)
            for (int i = threadIdx.x; i < r.n_streams; i += 256) {
                const int asked = i < r.R ? r.parents[i] : i, p = parent_of(r, i);
                r.lens_out[i] = length_of(r, p);
                if (r.status != nullptr && asked != p) atomicOr(r.status, ST_BAD_ARG);
                if (r.status != nullptr && r.lens[p] != length_of(r, p)) atomicOr(r.status, ST_BAD_POSITION);
            }
        if (j >= r.pps) return;
#pragma unroll 4
        for (int k = lane; k < r.n_streams; k += 32) {
            const int pk = parent_of(r, k);
            entries[warp][k] = (short)entry_of(r, j, pk, length_of(r, pk) / kPage, true);
        }
        __syncwarp();
        reorder_column(r, j, 0, true, entries[warp], scratch[warp]);
        return;
    }
    const int i = (blockIdx.x - table_blocks) / copy_blocks, part = (blockIdx.x - table_blocks) % copy_blocks;
    const int p = parent_of(r, i), len = length_of(r, p);
    int k = threadIdx.x, pk = k < r.n_streams ? parent_of(r, k) : 0, tail = length_of(r, pk) / kPage;
    const int col = len / kPage, rows = len % kPage;
    if (rows == 0) return;
    const int sr = entry_of(r, col, p, col, false);
    int other = 0;   // whether a row before i takes the page over, or a stream shares it
    while (k < r.n_streams) {
        const int e = entry_of(r, col, pk, tail, false);
        entries[0][k] = (short)e;
        other |= e >= 0 && (e & ~kFull) == sr && ((e & kFull) || k < i);
        if ((k += 256) < r.n_streams) pk = parent_of(r, k), tail = length_of(r, pk) / kPage;
    }
    if (!__syncthreads_or(other) || sr < 0) return;
    if (warp == 0) {
        const int dst = reorder_column(r, col, i, false, entries[0], scratch[0]);
        if (lane == 0) to_s = dst;
    }
    __syncthreads();
    const int src = sr * r.pps + col, dst = to_s, t = part * 8 + warp;
    if (t >= 2 * r.n_tiles) return;
    unsigned char *pool = t < r.n_tiles ? r.k : r.v;
    const size_t off = (size_t)(t < r.n_tiles ? t : t - r.n_tiles) * r.tile_bytes;
    const uint4 *from = reinterpret_cast<const uint4 *>(pool + src * r.page_bytes + off);
    uint4 *to = reinterpret_cast<uint4 *>(pool + dst * r.page_bytes + off);
    const int codes = rows * r.row_bytes / 16, scales = (rows * r.scale_bytes + 15) / 16, sc0 = kPage * r.row_bytes / 16;
#pragma unroll 4
    for (int e = lane; e < codes; e += 32) to[e] = from[e];
    for (int e = lane; e < scales; e += 32) to[sc0 + e] = from[sc0 + e];
}

}  // namespace

cudaError_t launch_kv4_rows(const Kv4Rows &r, int dtype, bool read, cudaStream_t s) {
    if (r.T == 0 || r.n_streams == 0 || r.n_layers == 0) return cudaSuccess;
    const int size = dtype == TALKER_DTYPE_BF16 ? 2 : 4, v = 8;
    // one access for eight dims where every head row starts on its boundary
    const bool vec = (reinterpret_cast<uintptr_t>(r.k) | reinterpret_cast<uintptr_t>(r.v)) % (v * size) == 0 &&
                     r.st.layer % v == 0 && r.st.stream % v == 0 && r.st.row % v == 0 && r.st.head % v == 0;
    const bool bf16 = dtype == TALKER_DTYPE_BF16;
    if (r.c.head_dim == 128) {
        if (read) return bf16 ? launch_rows_t<128, __nv_bfloat16, true>(r, vec, s) : launch_rows_t<128, float, true>(r, vec, s);
        return bf16 ? launch_rows_t<128, __nv_bfloat16, false>(r, vec, s) : launch_rows_t<128, float, false>(r, vec, s);
    }
    if (read) return bf16 ? launch_rows_t<64, __nv_bfloat16, true>(r, vec, s) : launch_rows_t<64, float, true>(r, vec, s);
    return bf16 ? launch_rows_t<64, __nv_bfloat16, false>(r, vec, s) : launch_rows_t<64, float, false>(r, vec, s);
}

cudaError_t launch_kv_reorder(const KvReorder &r, cudaStream_t s) {
    const int table_blocks = (r.pps + 7) / 8, copy_blocks = (2 * r.n_tiles + 7) / 8;
    const long long blocks = table_blocks + (long long)copy_blocks * r.n_streams;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    k_reorder<<<(unsigned)blocks, 256, 0, s>>>(r, table_blocks, copy_blocks);
    return cudaGetLastError();
}

}  // namespace talker_k

// ---- C-ABI

using namespace talker_k;

namespace {

bool sizes_ok(int n_layers, int n_kv, int hd) {
    return n_layers >= 1 && n_kv >= 1 && (hd == 64 || hd == 128) &&
           (long long)n_layers * n_kv <= 0x7fffffffll / kv4_tile_bytes(hd);
}

struct Span {
    const int32_t *p;
    size_t n;
};

talker_status status_of(cudaError_t e) {
    if (e == cudaSuccess) return TALKER_OK;
    cudaGetLastError();
    return TALKER_ECUDA;
}

talker_status rows_call(const talker_kv4 *c, int layer0, int n_layers, int stream0, int n_streams,
                        const int32_t *start, const int32_t *count, int T, void *k, void *v, int dtype,
                        const talker_kv4_strides *st, bool read, void *cuda_stream) {
    if (!kv4_cache_ok(c) || !k || !v || !st || T < 0 || n_layers < 0 || n_streams < 0) return TALKER_EINVAL;
    if (layer0 < 0 || layer0 > c->n_layers - n_layers || stream0 < 0 || stream0 > c->n_streams - n_streams)
        return TALKER_EINVAL;
    if (n_layers > 32767 || n_streams > 65535 || (long long)T * c->n_kv_heads > 0x7fffffffll) return TALKER_EINVAL;
    if (dtype != TALKER_DTYPE_F32 && dtype != TALKER_DTYPE_BF16) return TALKER_EINVAL;
    if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) % (dtype == TALKER_DTYPE_F32 ? 4 : 2))
        return TALKER_EINVAL;
    const Kv4Rows r{*c, layer0, n_layers, stream0, n_streams, start, count, T, k, v, *st};
    return status_of(launch_kv4_rows(r, dtype, read, static_cast<cudaStream_t>(cuda_stream)));
}

}  // namespace

namespace talker_k {

bool kv4_cache_ok(const talker_kv4 *c) {
    return c && c->k && c->v && c->page_table && sizes_ok(c->n_layers, c->n_kv_heads, c->head_dim) && c->n_pages >= 1 &&
           c->n_streams >= 1 && c->pages_per_stream >= 1 && c->pages_per_stream <= 0x7fffffff / talker_dev::kPage &&
           !((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) & 15u);
}

}  // namespace talker_k

extern "C" {

size_t talker_kv4_page_bytes(int n_layers, int n_kv_heads, int head_dim) {
    return sizes_ok(n_layers, n_kv_heads, head_dim) ? (size_t)n_layers * n_kv_heads * kv4_tile_bytes(head_dim) : 0;
}

talker_status talker_kv4_write(const talker_kv4 *c, int layer0, int n_layers, int stream0, int n_streams,
                               const int32_t *start, const int32_t *count, int T, const void *k, const void *v,
                               int dtype, const talker_kv4_strides *strides, void *cuda_stream) {
    return rows_call(c, layer0, n_layers, stream0, n_streams, start, count, T, const_cast<void *>(k),
                     const_cast<void *>(v), dtype, strides, false, cuda_stream);
}

talker_status talker_kv4_read(const talker_kv4 *c, int layer0, int n_layers, int stream0, int n_streams,
                              const int32_t *start, const int32_t *count, int T, void *k, void *v, int dtype,
                              const talker_kv4_strides *strides, void *cuda_stream) {
    return rows_call(c, layer0, n_layers, stream0, n_streams, start, count, T, k, v, dtype, strides, true, cuda_stream);
}

talker_status talker_kv4_reorder(const talker_kv4 *c, const int32_t *parents, int R, const int32_t *lens,
                                 int32_t *table_out, int32_t *lens_out, void *cuda_stream) {
    if (!kv4_cache_ok(c) || !lens || !table_out || !lens_out || R < 0 || R > c->n_streams || (R > 0 && !parents))
        return TALKER_EINVAL;
    if (c->n_streams > kReorderMaxStreams || (long long)c->n_streams * c->pages_per_stream > c->n_pages)
        return TALKER_EINVAL;
    const size_t nt = (size_t)c->n_streams * c->pages_per_stream, ns = c->n_streams;
    const Span in[3] = {{c->page_table, nt}, {lens, ns}, {parents, (size_t)R}}, out[2] = {{table_out, nt}, {lens_out, ns}};
    for (const Span &o : out)
        for (const Span &i : in)
            if (o.p < i.p + i.n && i.p < o.p + o.n) return TALKER_EINVAL;
    if (table_out < lens_out + ns && lens_out < table_out + nt) return TALKER_EINVAL;
    const int tile = kv4_tile_bytes(c->head_dim), tiles = c->n_layers * c->n_kv_heads;
    const KvReorder r{static_cast<unsigned char *>(c->k), static_cast<unsigned char *>(c->v), (size_t)tiles * tile,
                      tiles, c->head_dim / 2, c->head_dim / 16, tile, c->page_table, lens, parents, table_out, lens_out,
                      c->status, c->n_streams, c->pages_per_stream, R, 0};
    return status_of(launch_kv_reorder(r, static_cast<cudaStream_t>(cuda_stream)));
}

}  // extern "C"
