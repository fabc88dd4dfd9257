// Page copies inside an arena (forks, compaction) and the rewrite of page
// tables after a compaction.
//
// A copy of a page is pure traffic: its bytes read once and written once.
// The pages of a call are cut into pieces of kPiece 16-byte units; a CTA takes
// one piece, each of its threads kUnits units a CTA's width apart, all loaded
// before any is stored, so an SM holds its resident CTAs' pieces in flight.
// Measured: 96 pages of 7.9 MB (1,513 MB read and written) 225 us, 6.72 TB/s,
// 99 % of a plain copy's rate; four pages' first 77 positions (19 MB) 5.9 us,
// half of it the launch.
// A whole page is one run of bytes.  A page's first n positions are, for each
// layer, the first n rows of each K, V and indexer part, and the first n/4
// pooled rows: the piece's units are counted over those rows only, and each
// unit finds its part, head and row by division.
#include <algorithm>
#include <new>
#include <vector>

#include "pkv_dev.cuh"

namespace pkv {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kUnits = 8;                          // 16-byte units a thread holds
constexpr int kPiece = kCopyThreads * kUnits;      // units a CTA copies (32 KB)
constexpr int kMoves = 512;                        // pages of one launch (its parameters)

struct CopyArgs {
    uint8_t *base;
    int64_t page_bytes;
    int32_t n, n_layers, n_kv_heads, idx_dim, ptok, fp8;
    int32_t src[kMoves], dst[kMoves];
    int32_t n_pos[kMoves];   // positions copied (ptok: the whole page)
    int32_t first[kMoves];   // first piece of the copy
};

// 16-byte units of one layer's first n positions: K and V rows, e4m3 scales
// (a head's n scales are padded to whole units), indexer rows, pooled rows.
struct LayerUnits {
    int32_t kv, sc, ik, p;
    __host__ __device__ int32_t all() const { return kv + sc + ik + p; }
};
__host__ __device__ inline LayerUnits layer_units(bool fp8, int32_t h, int32_t idx_dim, int32_t n) {
    LayerUnits u;
    u.kv = 2 * h * n * (fp8 ? kHeadDim / 16 : kHeadDim / 8);
    u.sc = fp8 ? 2 * h * ((n + 3) / 4) : 0;
    u.ik = n * (idx_dim / 8);
    u.p = n / 4 * (idx_dim / 8);
    return u;
}

// Byte offset inside a layer's block of unit u of the first n positions, and
// how many of its 16 bytes are copied.
__device__ __forceinline__ int64_t unit_at(const CopyArgs &a, const LayerUnits &lu, int32_t n, int32_t u,
                                           int32_t *bytes) {
    const bool fp8 = a.fp8 != 0;
    const int32_t row = fp8 ? kHeadDim : 2 * kHeadDim;  // bytes of a K or V row
    const int64_t kv_bytes = 2 * (int64_t)a.n_kv_heads * a.ptok * row;
    *bytes = 16;
    if (u < lu.kv) {
        const int32_t per = n * (row / 16), head = u / per;  // K heads, then V heads
        return (int64_t)head * a.ptok * row + 16 * (int64_t)(u - head * per);
    }
    u -= lu.kv;
    if (u < lu.sc) {
        const int32_t per = (n + 3) / 4, head = u / per, at = u - head * per;
        *bytes = min(16, 4 * (n - 4 * at));
        return kv_bytes + 4 * (int64_t)head * a.ptok + 16 * at;
    }
    u -= lu.sc;
    const int64_t ik = kv_bytes + (fp8 ? 8 * (int64_t)a.n_kv_heads * a.ptok : 0);
    if (u < lu.ik) return ik + 16 * (int64_t)u;
    return ik + 2 * (int64_t)a.ptok * a.idx_dim + 16 * (int64_t)(u - lu.ik);
}

__global__ void __launch_bounds__(kCopyThreads)
    copy_kernel(const __grid_constant__ CopyArgs a) {
    // the copy of this piece: the last i with first[i] <= blockIdx.x
    int lo = 0, hi = a.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.first[mid] <= (int)blockIdx.x) lo = mid;
        else hi = mid - 1;
    }
    const int n = a.n_pos[lo];
    const int64_t u0 = (int64_t)(blockIdx.x - a.first[lo]) * kPiece + threadIdx.x;
    const uint8_t *src = a.base + a.src[lo] * a.page_bytes;
    uint8_t *dst = a.base + a.dst[lo] * a.page_bytes;
    int64_t at[kUnits];
    int32_t bytes[kUnits];
    if (n == a.ptok) {
        const int64_t all = a.page_bytes / 16;
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int64_t u = u0 + i * kCopyThreads;
            at[i] = 16 * u;
            bytes[i] = u < all ? 16 : 0;
        }
    } else {
        const LayerUnits lu = layer_units(a.fp8 != 0, a.n_kv_heads, a.idx_dim, n);
        const int32_t per = lu.all();
        const int64_t all = (int64_t)per * a.n_layers, layer_bytes = a.page_bytes / a.n_layers;
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int64_t u = u0 + i * kCopyThreads;
            bytes[i] = 0;
            at[i] = 0;
            if (u < all) {
                const int32_t layer = static_cast<int32_t>(u / per);
                at[i] = layer * layer_bytes + unit_at(a, lu, n, static_cast<int32_t>(u - (int64_t)layer * per), &bytes[i]);
            }
        }
    }
    pdl_wait();
    uint4 v[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
        if (bytes[i] > 0) v[i] = *reinterpret_cast<const uint4 *>(src + at[i]);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        if (bytes[i] == 16) {
            *reinterpret_cast<uint4 *>(dst + at[i]) = v[i];
        } else if (bytes[i] > 0) {  // a head's last scales
            const uint32_t w[3] = {v[i].x, v[i].y, v[i].z};
            for (int j = 0; j < bytes[i] / 4; ++j) reinterpret_cast<uint32_t *>(dst + at[i])[j] = w[j];
        }
    }
    pdl_trigger_after_writes();  // the next decode may read these rows early
}

constexpr int kTables = 64;         // tables of one launch
constexpr int kMapThreads = 256;

struct MapArgs {
    int32_t *table[kTables];
    int32_t n_table[kTables];
    int32_t first[kTables];          // first CTA of the table
    int32_t n_tables, n;
    int32_t src[kMoves], dst[kMoves];  // src ascending
};

// A thread an entry; the moves, sorted by src, are searched in shared memory.  A
// few thousand entries are one wave of CTAs, bound by the launch (5 us a call with
// its checks, four tables of 40 entries and 50 moves).
__global__ void __launch_bounds__(kMapThreads) remap_kernel(const __grid_constant__ MapArgs a) {
    __shared__ int32_t src[kMoves], dst[kMoves];
    for (int i = threadIdx.x; i < a.n; i += kMapThreads) {
        src[i] = a.src[i];
        dst[i] = a.dst[i];
    }
    int t = 0;
    for (int i = 1; i < a.n_tables; ++i)
        if (a.first[i] <= (int)blockIdx.x) t = i;
    int32_t *const table = a.table[t];
    const int64_t e = (int64_t)(blockIdx.x - a.first[t]) * kMapThreads + threadIdx.x;
    __syncthreads();
    pdl_wait();
    if (e < a.n_table[t]) {
        const int32_t id = table[e];
        int lo = 0, hi = a.n - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (src[mid] < id) lo = mid + 1;
            else hi = mid;
        }
        if (src[lo] == id) table[e] = dst[lo];
    }
    pdl_trigger_after_writes();  // the next decode reads the table before its wait
}

// Every id in [0, limit), the dst ids distinct and none of them a src; with
// distinct_src the src ids too.
bool moves_ok(const int32_t *src, const int32_t *dst, int32_t n, int64_t limit, bool distinct_src) {
    std::vector<int32_t> s(src, src + n), d(dst, dst + n);
    for (auto *v : {&s, &d}) {  // (a compaction plans its moves in order)
        if (v->front() > v->back()) std::reverse(v->begin(), v->end());
        if (!std::is_sorted(v->begin(), v->end())) std::sort(v->begin(), v->end());
    }
    if (s.front() < 0 || d.front() < 0 || s.back() >= limit || d.back() >= limit) return false;
    if (std::adjacent_find(d.begin(), d.end()) != d.end()) return false;
    if (distinct_src && std::adjacent_find(s.begin(), s.end()) != s.end()) return false;
    for (size_t i = 0, j = 0; i < s.size() && j < d.size();) {
        if (s[i] == d[j]) return false;
        if (s[i] < d[j]) ++i;
        else ++j;
    }
    return true;
}

int copy_pages(const pkv_layout *L, int32_t page_pos, void *base, int32_t n_pages, const int32_t *src,
               const int32_t *dst, const int32_t *n_pos, int32_t n, cudaStream_t stream) {
    if (!moves_ok(src, dst, n, n_pages, false)) return PKV_EINVAL;
    for (int32_t i = 0; n_pos && i < n; ++i)
        if (n_pos[i] < 0 || n_pos[i] > page_pos) return PKV_EINVAL;
    const bool fp8 = fp8_of(L);
    // a layer's units are counted in 32 bits
    if (layer_elems_f(fp8, L->n_kv_heads, L->idx_dim, page_pos) / 8 > INT32_MAX) return PKV_EINVAL;
    CopyArgs a;
    a.base = static_cast<uint8_t *>(base);
    a.page_bytes = 2 * L->n_layers * layer_elems_f(fp8, L->n_kv_heads, L->idx_dim, page_pos);
    a.n_layers = L->n_layers;
    a.n_kv_heads = L->n_kv_heads;
    a.idx_dim = L->idx_dim;
    a.ptok = page_pos;
    a.fp8 = fp8;
    for (int32_t i = 0; i < n;) {
        int64_t pieces = 0;
        a.n = 0;
        for (; i < n && a.n < kMoves; ++i) {
            const int32_t pos = n_pos ? n_pos[i] : page_pos;
            if (pos == 0) continue;
            const int64_t units = pos == page_pos
                                      ? a.page_bytes / 16
                                      : (int64_t)L->n_layers * layer_units(fp8, L->n_kv_heads, L->idx_dim, pos).all();
            const int64_t more = (units + kPiece - 1) / kPiece;
            if (pieces + more > INT32_MAX) break;
            a.src[a.n] = src[i];
            a.dst[a.n] = dst[i];
            a.n_pos[a.n] = pos;
            a.first[a.n++] = static_cast<int32_t>(pieces);
            pieces += more;
        }
        if (a.n == 0 && i < n) return PKV_EINVAL;  // a page of more pieces than a grid has
        if (a.n == 0) break;                       // nothing left but copies of no positions
        const cudaError_t e =
            launch_pdl(copy_kernel, static_cast<unsigned>(pieces), kCopyThreads, 0, stream, a);
        if (e != cudaSuccess) return PKV_ECUDA;
    }
    return PKV_OK;
}

int remap_tables(int32_t *const *tables, const int32_t *n_table, int32_t n_tables, const int32_t *src,
                 const int32_t *dst, int32_t n_moves, cudaStream_t stream) {
    if (!moves_ok(src, dst, n_moves, INT64_MAX, true)) return PKV_EINVAL;
    std::vector<int32_t> order(static_cast<size_t>(n_moves));
    const bool down = src[0] > src[n_moves - 1];
    for (int32_t i = 0; i < n_moves; ++i) order[i] = down ? n_moves - 1 - i : i;
    const auto before = [&](int32_t x, int32_t y) { return src[x] < src[y]; };
    if (!std::is_sorted(order.begin(), order.end(), before)) std::sort(order.begin(), order.end(), before);
    MapArgs a;
    // no dst is a src, so the groups of moves may follow each other in any order
    for (int32_t m0 = 0; m0 < n_moves; m0 += kMoves) {
        a.n = std::min(kMoves, n_moves - m0);
        for (int32_t i = 0; i < a.n; ++i) {
            a.src[i] = src[order[m0 + i]];
            a.dst[i] = dst[order[m0 + i]];
        }
        for (int32_t t = 0; t < n_tables;) {
            int64_t ctas = 0;
            a.n_tables = 0;
            for (; t < n_tables && a.n_tables < kTables; ++t) {
                if (n_table[t] == 0) continue;
                a.table[a.n_tables] = tables[t];
                a.n_table[a.n_tables] = n_table[t];
                a.first[a.n_tables++] = static_cast<int32_t>(ctas);
                ctas += ((int64_t)n_table[t] + kMapThreads - 1) / kMapThreads;
            }
            if (a.n_tables == 0) break;
            const cudaError_t e =
                launch_pdl(remap_kernel, static_cast<unsigned>(ctas), kMapThreads, 0, stream, a);
            if (e != cudaSuccess) return PKV_ECUDA;
        }
    }
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_pages_copy(const pkv_layout *L, int32_t page_pos, void *base, int32_t n_pages,
                              const int32_t *src, const int32_t *dst, const int32_t *n_pos, int32_t n,
                              cudaStream_t stream) {
    if (validate_layout(L) || !page_pos_ok(page_pos) || n_pages < 1 || n < 0) return PKV_EINVAL;
    if (!base || (reinterpret_cast<uintptr_t>(base) & 15u)) return PKV_EINVAL;
    if (n == 0) return PKV_OK;
    if (!src || !dst) return PKV_EINVAL;
    try {
        return copy_pages(L, page_pos, base, n_pages, src, dst, n_pos, n, stream);
    } catch (...) {  // no host memory for the checks' sorted lists
        return PKV_EINVAL;
    }
}

extern "C" int pkv_tables_remap(int32_t *const *tables, const int32_t *n_table, int32_t n_tables,
                                const int32_t *src, const int32_t *dst, int32_t n_moves,
                                cudaStream_t stream) {
    if (n_tables < 0 || n_moves < 0) return PKV_EINVAL;
    if ((n_tables > 0 && (!tables || !n_table)) || (n_moves > 0 && (!src || !dst))) return PKV_EINVAL;
    for (int32_t t = 0; t < n_tables; ++t) {
        if (n_table[t] < 0) return PKV_EINVAL;
        if (n_table[t] > 0 && (!tables[t] || (reinterpret_cast<uintptr_t>(tables[t]) & 3u))) return PKV_EINVAL;
    }
    if (n_moves == 0) return PKV_OK;
    try {
        return remap_tables(tables, n_table, n_tables, src, dst, n_moves, stream);
    } catch (...) {  // no host memory for the sorted moves
        return PKV_EINVAL;
    }
}
