// Host side of the pages of the paged 8-bit cache (include/hk_gemm.h):
// hk_kv8_arrange, hk_kv8_compact and hk_kv8_copy_pages: argument checks,
// workspace and launches.
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/hk_gemm.h"
#include "host_internal.h"
#include "kv8_host.h"
#include "kv8_pages.cuh"

namespace {

using namespace hk::kv8;
using namespace hk_kv8;

constexpr int64_t kMaxPages = int64_t(1) << 30;         // (mask words and ranks stay within 31 bits)

bool pool_shape_ok(const hk_kv8_pool* p) {
    return p && p->num_pages >= 1 && p->num_pages <= kMaxPages && p->rows >= 1 && p->rows <= kLimit / 2 && p->max_pages >= 1 &&
           p->page_size >= 1 && p->max_pages <= (kLimit - 127) / p->page_size && int64_t(p->rows) * p->max_pages <= kLimit;
}

hk_status check_pool(const hk_kv8_pool* p) {
    if (!p) return fail(HK_ERR_INVALID_ARG, "null pool");
    if (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128)
        return fail(HK_ERR_INVALID_ARG, "page size %d (supported: 16, 32, 64, 128)", (int)p->page_size);
    if (!pool_shape_ok(p))
        return fail(HK_ERR_INVALID_ARG, "a pool of %lld pages, %d rows of %d", (long long)p->num_pages, (int)p->rows, (int)p->max_pages);
    if (p->rows > 1 && p->table_stride < p->max_pages) return fail(HK_ERR_INVALID_ARG, "block table rows overlap");
    if (!p->refs || !p->table || !p->held) return fail(HK_ERR_INVALID_ARG, "null pool pointer");
    if (!aligned(p->refs, 4) || !aligned(p->table, 4) || !aligned(p->held, 4))
        return fail(HK_ERR_MISALIGNED, "references, block table and held tokens must be 4-byte aligned");
    return HK_OK;
}

// Caches that pages are copied between: n of each, alike in all but their number of pages.
hk_status check_caches(const hk_kv8_cache* dst, const hk_kv8_cache* src, int32_t n) {
    if (n < 0) return fail(HK_ERR_INVALID_ARG, "%d caches", (int)n);
    if (n > 0 && (!dst || !src)) return fail(HK_ERR_INVALID_ARG, "null caches");
    for (int32_t i = 0; i < n; ++i) {
        hk_status s = check_cache(dst + i);
        if (s == HK_OK) s = check_cache(src + i);
        if (s != HK_OK) return s;
        const hk_kv8_cache &d = dst[i], &a = src[i];
        if (d.heads != a.heads || d.page_size != a.page_size || d.head_dim != a.head_dim)
            return fail(HK_ERR_INVALID_ARG, "cache %d: the pages of the two caches differ in shape", (int)i);
        if (d.num_pages != dst[0].num_pages || a.num_pages != src[0].num_pages)
            return fail(HK_ERR_INVALID_ARG, "cache %d has another number of pages than the first", (int)i);
    }
    return HK_OK;
}

// A pool's caches: pages of its size, as many.
hk_status check_pool_caches(const hk_kv8_pool* p, const hk_kv8_cache* c, int32_t n) {
    hk_status s = check_caches(c, c, n);
    if (s != HK_OK) return s;
    for (int32_t i = 0; i < n; ++i)
        if (c[i].page_size != p->page_size || c[i].num_pages != p->num_pages)
            return fail(HK_ERR_INVALID_ARG, "cache %d: %lld pages of %d tokens, the pool has %lld of %d", (int)i, (long long)c[i].num_pages,
                        (int)c[i].page_size, (long long)p->num_pages, (int)p->page_size);
    return HK_OK;
}

hk_status device_status(uint32_t** status) {
    int device = 0, sms = 0;
    const hk_status s = current_device(&device, &sms);
    return s == HK_OK ? hk_host::status_word(device, status) : s;
}

// Copies the listed pages of every cache; `count`: the list's length on the device, at most n.
hk_status copy_pages(const hk_kv8_cache* dst, const hk_kv8_cache* src, int32_t n_caches, const int32_t* dst_pages,
                     const int32_t* src_pages, const int32_t* count, int64_t n, uint32_t* status, cudaStream_t st) {
    CopyParams p = {};
    p.src = src_pages;
    p.dst = dst_pages;
    p.count = count;
    p.n = n;
    p.status = status;
    // caches of one shape go together
    for (int32_t first = 0; first < n_caches;) {
        const hk_kv8_cache& c = dst[first];
        p.caches = 0;
        p.heads = c.heads;
        p.src_pages = src[first].num_pages;
        p.dst_pages = c.num_pages;
        p.page_vecs = static_cast<int32_t>(int64_t(c.heads) * c.page_size * c.head_dim / 16);
        p.parts = static_cast<int32_t>(ceil_div(p.page_vecs, kCopyVecs));
        for (; first < n_caches && p.caches < kMaxCaches && dst[first].heads == c.heads && dst[first].head_dim == c.head_dim &&
               dst[first].page_size == c.page_size;
             ++first, ++p.caches) {
            CopyParams::Cache& to = p.cache[p.caches];
            const hk_kv8_cache &d = dst[first], &a = src[first];
            to.from[0] = static_cast<const uint4*>(a.k_codes);
            to.from[1] = static_cast<const uint4*>(a.v_codes);
            to.to[0] = static_cast<uint4*>(d.k_codes);
            to.to[1] = static_cast<uint4*>(d.v_codes);
            to.scale_from[0] = a.k_scale;
            to.scale_from[1] = a.v_scale;
            to.scale_to[0] = d.k_scale;
            to.scale_to[1] = d.v_scale;
        }
        // (a list whose length the host does not know: as many blocks as are resident at a time)
        const int64_t steps = int64_t(p.caches) * 2 * p.parts;
        const int64_t blocks = std::min<int64_t>(n > kLimit / steps ? kLimit : ceil_div(n * steps, 8), int64_t(kSms) * 8);
        const cudaError_t e = launch_early(&kv8_copy_pages_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, p);
        if (e != cudaSuccess) return cuda_fail(HK_ERR_LAUNCH, "launching the copy of pages", e);
    }
    return HK_OK;
}

// Places of the workspace's parts.
struct Workspace {
    size_t mask[2], chunk_count, rows[3], pages[3], copies, table, counts, total;
};

Workspace workspace(const hk_kv8_pool* p, bool compact) {
    Workspace w = {};
    size_t at = 0;
    auto take = [&](size_t ints) {
        const size_t here = at;
        at += (ints * 4 + 255) / 256 * 256;
        return here;
    };
    const size_t chunks = static_cast<size_t>(ceil_div(p->num_pages, kChunkPages)), rows = static_cast<size_t>(p->rows);
    const size_t pages = static_cast<size_t>(p->num_pages);
    w.mask[0] = take(chunks * kChunkWords);
    w.chunk_count = take(chunks);
    w.pages[0] = take(pages);
    if (compact) {
        w.pages[1] = take(pages);
        w.pages[2] = take(pages);
        w.counts = take(2);
    } else {
        w.mask[1] = take(chunks * kChunkWords);
        for (int i = 0; i < 3; ++i) w.rows[i] = take(rows);
        w.copies = take(2 * rows);
        w.table = take(rows * static_cast<size_t>(p->max_pages));
    }
    w.total = at;
    return w;
}

hk_status check_workspace(size_t need, const void* workspace, size_t bytes) {
    if (!workspace || bytes < need)
        return fail(HK_ERR_WORKSPACE, "%zu bytes of workspace needed, %zu given", need, workspace ? bytes : size_t(0));
    if (!aligned(workspace, 256)) return fail(HK_ERR_WORKSPACE, "the workspace must be 256-byte aligned");
    return HK_OK;
}

PoolParams pool_params(const hk_kv8_pool* pool, const Workspace& w, char* base, uint32_t* status) {
    PoolParams p = {};
    p.refs = pool->refs;
    p.table = pool->table;
    p.held = pool->held;
    p.num_pages = pool->num_pages;
    p.table_stride = pool->table_stride;
    p.rows = pool->rows;
    p.max_pages = pool->max_pages;
    p.page_shift = pool->page_size == 16 ? 4 : pool->page_size == 32 ? 5 : pool->page_size == 64 ? 6 : 7;
    p.chunks = static_cast<int32_t>(ceil_div(pool->num_pages, kChunkPages));
    p.free_mask = reinterpret_cast<uint32_t*>(base + w.mask[0]);
    p.chunk_count = reinterpret_cast<int32_t*>(base + w.chunk_count);
    p.status = status;
    return p;
}

}  // namespace

extern "C" size_t hk_kv8_arrange_workspace_size(const hk_kv8_pool* pool) { return pool_shape_ok(pool) ? workspace(pool, false).total : 0; }

extern "C" size_t hk_kv8_compact_workspace_size(const hk_kv8_pool* pool) { return pool_shape_ok(pool) ? workspace(pool, true).total : 0; }

extern "C" hk_status hk_kv8_arrange(const hk_kv8_pool* pool, const int32_t* keep, const int32_t* room, const int32_t* parents,
                                    const hk_kv8_cache* caches, int32_t n_caches, int32_t* copies, int32_t* missing,
                                    void* scratch, size_t workspace_bytes, void* stream) {
    hk_status s = check_pool(pool);
    if (s == HK_OK) s = check_pool_caches(pool, caches, n_caches);
    if (s != HK_OK) return s;
    if (!keep || !room || !missing) return fail(HK_ERR_INVALID_ARG, "null keep, room or missing");
    if (!aligned(keep, 4) || !aligned(room, 4) || !aligned(parents, 4) || !aligned(copies, 4) || !aligned(missing, 4))
        return fail(HK_ERR_MISALIGNED, "keep, room, parents, copies and missing must be 4-byte aligned");
    const Workspace w = workspace(pool, false);
    if ((s = check_workspace(w.total, scratch, workspace_bytes)) != HK_OK) return s;
    uint32_t* status = nullptr;
    if ((s = device_status(&status)) != HK_OK) return s;
    char* const base = static_cast<char*>(scratch);
    PoolParams p = pool_params(pool, w, base, status);
    p.once_mask = reinterpret_cast<uint32_t*>(base + w.mask[1]);
    p.keep = keep;
    p.room = room;
    p.parents = parents;
    p.need = reinterpret_cast<int32_t*>(base + w.rows[0]);
    p.old_held = reinterpret_cast<int32_t*>(base + w.rows[1]);
    p.bound = reinterpret_cast<int32_t*>(base + w.rows[2]);
    p.old_table = reinterpret_cast<int32_t*>(base + w.table);
    p.fresh = reinterpret_cast<int32_t*>(base + w.pages[0]);
    p.copy_src = copies ? copies : reinterpret_cast<int32_t*>(base + w.copies);
    p.copy_dst = p.copy_src + pool->rows;
    p.missing = missing;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = launch_early(&kv8_arrange_look_kernel, dim3(static_cast<unsigned>(int64_t(p.chunks) + p.rows)), dim3(256), 0, st, p);
    if (e == cudaSuccess) e = launch_early(&kv8_arrange_rows_kernel, dim3(static_cast<unsigned>(p.rows)), dim3(256), 0, st, p);
    if (e != cudaSuccess) return cuda_fail(HK_ERR_LAUNCH, "launching the arrangement of pages", e);
    return copy_pages(caches, caches, n_caches, p.copy_dst, p.copy_src, nullptr, pool->rows, status, st);
}

extern "C" hk_status hk_kv8_compact(const hk_kv8_pool* pool, const hk_kv8_cache* caches, int32_t n_caches, int32_t* moved,
                                    void* scratch, size_t workspace_bytes, void* stream) {
    hk_status s = check_pool(pool);
    if (s == HK_OK) s = check_pool_caches(pool, caches, n_caches);
    if (s != HK_OK) return s;
    if (!moved) return fail(HK_ERR_INVALID_ARG, "null moved");
    if (!aligned(moved, 4)) return fail(HK_ERR_MISALIGNED, "moved must be 4-byte aligned");
    const Workspace w = workspace(pool, true);
    if ((s = check_workspace(w.total, scratch, workspace_bytes)) != HK_OK) return s;
    uint32_t* status = nullptr;
    if ((s = device_status(&status)) != HK_OK) return s;
    char* const base = static_cast<char*>(scratch);
    CompactParams c = {};
    c.pool = pool_params(pool, w, base, status);
    c.rank = reinterpret_cast<int32_t*>(base + w.pages[0]);
    c.holes = reinterpret_cast<int32_t*>(base + w.pages[1]);
    c.movers = reinterpret_cast<int32_t*>(base + w.pages[2]);
    c.count = reinterpret_cast<int32_t*>(base + w.counts);
    c.moved = moved;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = launch_early(&kv8_compact_look_kernel, dim3(static_cast<unsigned>(c.pool.chunks)), dim3(256), 0, st, c);
    if (e == cudaSuccess) e = launch_early(&kv8_compact_rank_kernel, dim3(static_cast<unsigned>(c.pool.chunks)), dim3(256), 0, st, c);
    const int64_t movers = std::min<int64_t>(ceil_div(pool->num_pages / 2 + 1, 256), 4 * kSms);
    if (e == cudaSuccess) e = launch_early(&kv8_compact_rows_kernel, dim3(static_cast<unsigned>(pool->rows + movers)), dim3(256), 0, st, c);
    if (e != cudaSuccess) return cuda_fail(HK_ERR_LAUNCH, "launching the compaction of pages", e);
    return copy_pages(caches, caches, n_caches, c.holes, c.movers, c.count + 1, pool->num_pages, status, st);
}

extern "C" hk_status hk_kv8_copy_pages(const hk_kv8_cache* dst, const hk_kv8_cache* src, int32_t n_caches,
                                       const int32_t* dst_pages, const int32_t* src_pages, int64_t n, void* stream) {
    hk_status s = check_caches(dst, src, n_caches);
    if (s != HK_OK) return s;
    if (n < 0 || n > kLimit) return fail(HK_ERR_INVALID_ARG, "%lld pages to copy", (long long)n);
    if (n == 0 || n_caches == 0) return HK_OK;
    if (!dst_pages || !src_pages) return fail(HK_ERR_INVALID_ARG, "null pages");
    if (!aligned(dst_pages, 4) || !aligned(src_pages, 4)) return fail(HK_ERR_MISALIGNED, "pages must be 4-byte aligned");
    uint32_t* status = nullptr;
    if ((s = device_status(&status)) != HK_OK) return s;
    return copy_pages(dst, src, n_caches, dst_pages, src_pages, nullptr, n, status, static_cast<cudaStream_t>(stream));
}
