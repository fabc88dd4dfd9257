// The page arena of the C ABI (host only): KV pages handed out lowest id
// first, runs of consecutive pages claimed from the top, both given back
// either at once or once the caller's stream has drained (an event polled,
// never waited on).  KV pages count their holders, so that forked streams
// share whole pages; a compaction moves the highest KV pages to the lowest
// free ids.
#include <algorithm>
#include <map>
#include <mutex>
#include <new>
#include <vector>

#include "pkv_internal.h"

using namespace pkv;

struct pkv_arena {
    pkv_layout layout;
    int32_t page_pos = 0;
    int64_t page_elems = 0;
    int32_t n_pages = 0;
    void *base = nullptr;
    std::vector<uint8_t> taken;  // 1 = a KV page, 2 = a run's page; held or pending release
    std::vector<int32_t> holders;  // of a KV page: streams that hold it, pending gives included
    std::vector<int32_t> going;    // of those, gives that wait for their stream
    std::vector<uint8_t> vacated;  // a compaction has moved the page; it waits for its last give
    std::map<int32_t, int32_t> runs;  // first id -> pages of each run held now
    int32_t n_free = 0;
    int32_t low = 0;  // no free page below this id
    struct Pending {
        void *ev;
        std::vector<int32_t> ids;
    };
    std::vector<Pending> pending;
    pkv_event_ops ops{};
    bool custom_ops = false;
    mutable std::mutex mu;
};

namespace {

int cuda_record(void *, cudaStream_t stream, void **ev) {
    cudaEvent_t e;
    if (cudaEventCreateWithFlags(&e, cudaEventDisableTiming) != cudaSuccess) return -1;
    if (cudaEventRecord(e, stream) != cudaSuccess) {
        cudaEventDestroy(e);
        return -1;
    }
    *ev = e;
    return 0;
}
int cuda_query(void *, void *ev) {
    cudaError_t r = cudaEventQuery(static_cast<cudaEvent_t>(ev));
    if (r == cudaSuccess) return 0;
    if (r == cudaErrorNotReady) {
        cudaGetLastError();  // not-ready is not sticky; clear it
        return 1;
    }
    return -1;
}
void cuda_destroy(void *, void *ev) { cudaEventDestroy(static_cast<cudaEvent_t>(ev)); }

const pkv_event_ops kCudaOps = {cuda_record, cuda_query, cuda_destroy, nullptr};

void free_page(pkv_arena *a, int32_t id) {
    a->taken[id] = a->vacated[id] = 0;
    a->n_free++;
    if (id < a->low) a->low = id;
}

// One holder of a page less: a KV page is free once it has none, a run's
// page at once.
void drop_holder(pkv_arena *a, int32_t id) {
    if (a->taken[id] == 1 && --a->holders[id] > 0) return;
    free_page(a, id);
}

// Holders whose give is not under way (0: free, a run's page, or going).
int32_t live_holders(const pkv_arena *a, int32_t id) {
    return a->taken[id] == 1 ? a->holders[id] - a->going[id] : 0;
}

bool held_once_each(const pkv_arena *a, const std::vector<int32_t> &sorted) {
    for (size_t i = 0; i < sorted.size(); ++i) {
        if (sorted[i] < 0 || sorted[i] >= a->n_pages || live_holders(a, sorted[i]) < 1) return false;
        if (i && sorted[i] == sorted[i - 1]) return false;
    }
    return true;
}

// The lowest free page (there is one: n_free > 0), taken by one holder.
int32_t take_lowest(pkv_arena *a) {
    int32_t id = a->low;
    while (a->taken[id]) ++id;
    a->taken[id] = 1;
    a->holders[id] = 1;
    a->n_free--;
    a->low = id + 1;
    return id;
}

// Move releases whose stream work has finished back to the free pages.
int poll_pending(pkv_arena *a) {
    int rc = PKV_OK;
    size_t keep = 0;
    for (size_t i = 0; i < a->pending.size(); ++i) {
        auto &p = a->pending[i];
        int q = a->ops.query(a->ops.ctx, p.ev);
        if (q == 0) {
            a->ops.destroy(a->ops.ctx, p.ev);
            for (int32_t id : p.ids) {
                if (a->taken[id] == 1) a->going[id]--;
                drop_holder(a, id);
            }
        } else {
            if (q < 0) rc = PKV_ECUDA;
            if (keep != i) a->pending[keep] = std::move(p);
            ++keep;
        }
    }
    a->pending.resize(keep);
    return rc;
}

}  // namespace

extern "C" int pkv_arena_create(const pkv_layout *layout, int32_t page_pos, void *dev_base,
                                size_t bytes, pkv_arena **out) {
    if (!out) return PKV_EINVAL;
    *out = nullptr;
    if (validate_layout(layout) || !page_pos_ok(page_pos) || !dev_base) return PKV_EINVAL;
    if (reinterpret_cast<uintptr_t>(dev_base) & 15u) return PKV_EINVAL;
    int64_t ps = (int64_t)layout->n_layers *
                 layer_elems_f(fp8_of(layout), layout->n_kv_heads, layout->idx_dim, page_pos);
    int64_t n = static_cast<int64_t>(bytes / 2) / ps;
    if (n < 1 || n > INT32_MAX) return PKV_EINVAL;
    pkv_arena *a = new (std::nothrow) pkv_arena;
    if (!a) return PKV_EINVAL;
    a->layout = *layout;
    a->page_pos = page_pos;
    a->page_elems = ps;
    a->n_pages = static_cast<int32_t>(n);
    a->base = dev_base;
    try {
        a->taken.assign(static_cast<size_t>(n), 0);
        a->holders.assign(static_cast<size_t>(n), 0);
        a->going.assign(static_cast<size_t>(n), 0);
        a->vacated.assign(static_cast<size_t>(n), 0);
    } catch (...) {  // no host memory for the books of so many pages
        delete a;
        return PKV_EINVAL;
    }
    a->n_free = a->n_pages;
    a->ops = kCudaOps;
    *out = a;
    return PKV_OK;
}

extern "C" int pkv_arena_destroy(pkv_arena *a) {
    if (!a) return PKV_EINVAL;
    for (auto &p : a->pending) a->ops.destroy(a->ops.ctx, p.ev);
    delete a;
    return PKV_OK;
}

extern "C" int pkv_arena_set_event_ops(pkv_arena *a, const pkv_event_ops *ops) {
    if (!a) return PKV_EINVAL;
    std::lock_guard<std::mutex> g(a->mu);
    if (!a->pending.empty()) return PKV_EINVAL;  // events of one kind at a time
    if (ops && (!ops->record || !ops->query || !ops->destroy)) return PKV_EINVAL;
    a->ops = ops ? *ops : kCudaOps;
    a->custom_ops = ops != nullptr;
    return PKV_OK;
}

extern "C" int pkv_arena_info(pkv_arena *a, int32_t *n_pages, int32_t *n_free,
                              int64_t *page_elems) {
    if (!a) return PKV_EINVAL;
    std::lock_guard<std::mutex> g(a->mu);
    int rc = poll_pending(a);
    if (n_pages) *n_pages = a->n_pages;
    if (n_free) *n_free = a->n_free;
    if (page_elems) *page_elems = a->page_elems;
    return rc;
}

extern "C" int pkv_pages_take(pkv_arena *a, int32_t n, int32_t *ids_out) {
    if (!a || n < 0 || (n > 0 && !ids_out)) return PKV_EINVAL;
    std::lock_guard<std::mutex> g(a->mu);
    int rc = poll_pending(a);
    if (rc) return rc;
    if (n > a->n_free) return PKV_EAGAIN;
    for (int32_t i = 0; i < n; ++i) ids_out[i] = take_lowest(a);
    return PKV_OK;
}

extern "C" int pkv_pages_give(pkv_arena *a, const int32_t *ids, int32_t n, cudaStream_t stream,
                              int32_t defer) {
    if (!a || n < 0 || (n > 0 && !ids)) return PKV_EINVAL;
    std::lock_guard<std::mutex> g(a->mu);
    // every id must be in range, held, and listed once
    std::vector<int32_t> v;
    try {
        v.assign(ids, ids + n);
        // room before anything changes; grown by doubling, as the list may be long
        if (defer && a->pending.size() == a->pending.capacity())
            a->pending.reserve(std::max<size_t>(16, 2 * a->pending.size()));
    } catch (...) {  // no host memory for the sorted list
        return PKV_EINVAL;
    }
    std::sort(v.begin(), v.end());
    if (!held_once_each(a, v)) return PKV_EINVAL;
    if (n == 0) return PKV_OK;
    if (!defer) {
        for (int32_t id : v) drop_holder(a, id);
        return PKV_OK;
    }
    void *ev = nullptr;
    if (a->ops.record(a->ops.ctx, stream, &ev) != 0) return PKV_ECUDA;
    for (int32_t id : v) a->going[id]++;
    a->pending.push_back({ev, std::move(v)});
    return PKV_OK;
}

// ---- sharing and compaction -----------------------------------------------------

extern "C" int pkv_pages_fork(pkv_arena *a, const int32_t *ids, int32_t n, int32_t len,
                              int32_t *ids_out, int32_t *copy_src, int32_t *copy_dst,
                              int32_t *copy_pos) {
    if (!a || n < 0 || len < 0 || !copy_src || !copy_dst || !copy_pos) return PKV_EINVAL;
    if (n > 0 && (!ids || !ids_out)) return PKV_EINVAL;
    if (n != len / a->page_pos + (len % a->page_pos ? 1 : 0)) return PKV_EINVAL;
    std::lock_guard<std::mutex> g(a->mu);
    int rc = poll_pending(a);
    if (rc) return rc;
    const int32_t tail = len % a->page_pos;
    try {
        std::vector<int32_t> v;
        for (int32_t i = 0; i < n; ++i)
            if (ids[i] != -1) v.push_back(ids[i]);
        std::sort(v.begin(), v.end());
        if (!held_once_each(a, v) || (tail && ids[n - 1] == -1)) return PKV_EINVAL;
    } catch (...) {  // no host memory for the sorted list
        return PKV_EINVAL;
    }
    if (tail && a->n_free < 1) return PKV_EAGAIN;
    const int32_t last = tail ? ids[n - 1] : -1;
    for (int32_t i = 0; i < n; ++i) {
        ids_out[i] = ids[i];
        if (ids[i] != -1 && !(tail && i == n - 1)) a->holders[ids[i]]++;
    }
    *copy_src = last;
    *copy_dst = -1;
    *copy_pos = tail;
    if (tail) *copy_dst = ids_out[n - 1] = take_lowest(a);
    return PKV_OK;
}

extern "C" int pkv_pages_holders(pkv_arena *a, const int32_t *ids, int32_t n, int32_t *holders_out) {
    if (!a || n < 0 || (n > 0 && (!ids || !holders_out))) return PKV_EINVAL;
    std::lock_guard<std::mutex> g(a->mu);
    int rc = poll_pending(a);
    if (rc) return rc;
    for (int32_t i = 0; i < n; ++i)
        if (ids[i] < 0 || ids[i] >= a->n_pages) return PKV_EINVAL;
    for (int32_t i = 0; i < n; ++i) holders_out[i] = live_holders(a, ids[i]);
    return PKV_OK;
}

extern "C" int pkv_arena_compact(pkv_arena *a, int32_t max_moves, int32_t *src_out,
                                 int32_t *dst_out, int32_t *n_out) {
    if (!a || max_moves < 0 || !n_out || (max_moves > 0 && (!src_out || !dst_out))) return PKV_EINVAL;
    std::lock_guard<std::mutex> g(a->mu);
    int rc = poll_pending(a);
    if (rc) return rc;
    int32_t moves = 0, dst = a->low;
    for (int32_t src = a->n_pages - 1; moves < max_moves; --src) {
        while (dst < src && a->taken[dst]) ++dst;
        if (dst >= src) break;  // no free page below the highest one left
        if (live_holders(a, src) < 1 || a->vacated[src]) continue;
        a->taken[dst] = 1;
        a->holders[dst] = live_holders(a, src);
        a->holders[src] = a->going[src] + 1;  // the caller's, beside the gives under way
        a->vacated[src] = 1;
        a->n_free--;
        src_out[moves] = src;
        dst_out[moves++] = dst;
    }
    *n_out = moves;
    return PKV_OK;
}

// ---- runs ---------------------------------------------------------------------

extern "C" int pkv_run_pages(const pkv_arena *a, uint64_t run_bytes, int32_t *k_out) {
    if (!a || !k_out) return PKV_EINVAL;
    const uint64_t page_bytes = 2 * static_cast<uint64_t>(a->page_elems);
    const uint64_t k = run_bytes / page_bytes + (run_bytes % page_bytes ? 1 : 0);
    if (k > static_cast<uint64_t>(INT32_MAX)) return PKV_EINVAL;
    *k_out = static_cast<int32_t>(k);
    return PKV_OK;
}

extern "C" int pkv_run_take(pkv_arena *a, int32_t k, int32_t *first_out) {
    if (!a || k < 1 || !first_out) return PKV_EINVAL;
    std::lock_guard<std::mutex> g(a->mu);
    int rc = poll_pending(a);
    if (rc) return rc;
    if (k > a->n_free) return PKV_EAGAIN;
    // scan down from the top; the first window of k free pages met is the
    // highest one
    int32_t streak = 0;
    for (int32_t id = a->n_pages - 1; id >= 0; --id) {
        streak = a->taken[id] ? 0 : streak + 1;
        if (streak == k) {
            for (int32_t j = id; j < id + k; ++j) a->taken[j] = 2;
            a->n_free -= k;
            a->runs[id] = k;
            *first_out = id;
            return PKV_OK;
        }
    }
    return PKV_EAGAIN;
}

namespace {
bool run_held(const pkv_arena *a, int32_t first, int32_t k) {
    auto it = a->runs.find(first);
    return it != a->runs.end() && it->second == k;
}
}  // namespace

extern "C" int pkv_run_give(pkv_arena *a, int32_t first, int32_t k, cudaStream_t stream,
                            int32_t defer) {
    if (!a) return PKV_EINVAL;
    std::lock_guard<std::mutex> g(a->mu);
    if (!run_held(a, first, k)) return PKV_EINVAL;
    std::vector<int32_t> ids(static_cast<size_t>(k));
    for (int32_t j = 0; j < k; ++j) ids[j] = first + j;
    if (defer) {
        void *ev = nullptr;
        if (a->ops.record(a->ops.ctx, stream, &ev) != 0) return PKV_ECUDA;
        a->pending.push_back({ev, std::move(ids)});
    } else {
        for (int32_t id : ids) free_page(a, id);
    }
    a->runs.erase(first);
    return PKV_OK;
}

extern "C" int pkv_run_map(const pkv_arena *a, int32_t first, int32_t k, const uint64_t *part_bytes,
                           int32_t n_parts, uint64_t align, void **ptrs_out) {
    if (!a || n_parts < 0 || (n_parts > 0 && (!part_bytes || !ptrs_out))) return PKV_EINVAL;
    if (align < 16 || align > 4096 || (align & (align - 1))) return PKV_EINVAL;
    std::lock_guard<std::mutex> g(a->mu);
    if (!run_held(a, first, k)) return PKV_EINVAL;
    const uint64_t page_bytes = 2 * static_cast<uint64_t>(a->page_elems);
    const uint64_t lo = reinterpret_cast<uintptr_t>(a->base) + static_cast<uint64_t>(first) * page_bytes;
    const uint64_t hi = lo + static_cast<uint64_t>(k) * page_bytes;
    std::vector<uint64_t> at(static_cast<size_t>(n_parts));
    uint64_t cur = lo;
    for (int32_t i = 0; i < n_parts; ++i) {
        cur = (cur + align - 1) & ~(align - 1);
        if (cur > hi || part_bytes[i] > hi - cur) return PKV_EINVAL;
        at[i] = cur;
        cur += part_bytes[i];
    }
    for (int32_t i = 0; i < n_parts; ++i) ptrs_out[i] = reinterpret_cast<void *>(at[i]);
    return PKV_OK;
}

extern "C" int pkv_arena_pg(const pkv_arena *a, const int32_t *dev_table, int32_t n_table,
                            pkv_pg *out) {
    if (!a || !dev_table || n_table < 1 || !out) return PKV_EINVAL;
    out->base = a->base;
    out->table = dev_table;
    out->page_elems = a->page_elems;
    out->page_pos = a->page_pos;
    out->n_pages = a->n_pages;
    out->n_table = n_table;
    out->reserved = 0;
    return PKV_OK;
}

