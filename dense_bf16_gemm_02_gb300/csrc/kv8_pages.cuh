// The pages of the paged 8-bit cache: which of them a sequence holds, and copying them.
//
// A pool is a count of the table entries that name each page (refs; 0: free), a
// block table of one row per sequence, and the tokens whose pages each row holds.
//
// Arranging. Row i becomes the first keep[i] tokens of what row p = parents[i] was,
// with pages for room[i] tokens. A page that is whole within keep[i] is shared (one
// more reference); the pages above it, which row i will write, are its own: p's
// page where row i goes on in p's place (i = p, or the lowest row with parent p
// where p itself goes elsewhere: p's heir), nobody else names the page and no other
// row keeps it whole; else a free one, with p's page to be copied into it where it holds tokens of
// keep[i]. Free is what was free before the call, so no page is copied from and
// into in one call, and the lowest free pages go to the lowest rows' lowest slots:
// nothing depends on timing.
//
// Two kernels. The first only reads: per 4096 pages two bit masks (free, named
// once) and the number of free ones; per row what it needs and a copy of its entries
// (other rows read them while the row itself is rewritten). The second has a
// block per row: the rows' needs are added up to its place among the free
// pages, the masks say which those are. Integers added with atomics: the order does not
// matter. The work is a few words per row and page of the pool, so latency bounds
// it: two launches, each a chain of a few loads. 256 rows of up to 8192 tokens: 9 us in a graph; one row of 257
// pages forked to 64, with 63 pages of 128 KB copied in each of 4 layers: 25 us, of which the copies are 10.
//
// Compacting. With U pages in use, the k-th used page at U or above moves to the k-th free
// page below U: masks and counts, ranks, then tables and references, then the copies (a pool of 6000 pages of which 1300 move
// 128 KB in each of two caches: 132 us, of which the copies are 108).
//
// Loads of what earlier kernels may have changed go past L1: a grid may have started before their writes.
//
// Copying is bound by memory: 4 KB of one page per step of a warp, from a list on the device. 1300 pages of 8 heads x 64
// tokens of 128 in two caches: 108 us, 6.3 TB/s read and written (four loads in flight: 112; steps of a block, 16 KB: 113), 2000
// pages of 2 heads x 16 tokens of 64: 6.1 us, 5.4 TB/s (15.4 in steps of a block, which such a page does not fill).
#pragma once

#include <cstdint>

#include "bounded_wait.cuh"

namespace hk {
namespace kv8 {

constexpr int kChunkPages = 4096;          // pages of a block of the first kernels: 128 mask words
constexpr int kChunkWords = kChunkPages / 32;
constexpr int kMaxCaches = 16;             // caches of one copying launch

struct PoolParams {
    int32_t* refs;
    int32_t* table;
    int32_t* held;
    int64_t num_pages, table_stride;
    int32_t rows, max_pages, page_shift;
    const int32_t* keep;
    const int32_t* room;
    const int32_t* parents;                // or null: every row its own
    int32_t chunks;
    uint32_t* free_mask;                   // [chunks · 128]; compacting: of used pages
    uint32_t* once_mask;
    int32_t* chunk_count;                  // [chunks] free (compacting: used) pages
    int32_t* need;                         // [rows] free pages that the row takes; -1: arguments out of range
    int32_t* old_held;                     // [rows]
    int32_t* bound;                        // [rows] the row goes on in its parent's pages that end above so many tokens
    int32_t* old_table;                    // [rows, max_pages], with parents only
    int32_t* fresh;                        // [num_pages] the free pages that are taken, in order
    int32_t* copy_src;                     // [rows] page to copy, or -1
    int32_t* copy_dst;
    int32_t* missing;
    uint32_t* status;
};

// Exclusive sums of `v` over the block's 256 threads; `total` of all.
__device__ __forceinline__ int block_sums(int v, int& total, int* shared8) {
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        if (static_cast<int>(lane) >= d) inc += o;
    }
    __syncthreads();                       // (the last call's readers are done)
    if (lane == 31) shared8[warp] = inc;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        const int n = shared8[w];
        if (w < static_cast<int>(warp)) before += n;
        total += n;
    }
    return before + inc - v;
}

// Bit masks of the pages of chunk `c` and their number: free and named once, or (kUsed) in use.
template <bool kUsed>
__device__ __forceinline__ void mask_chunk(const PoolParams& p, int c, int* shared8) {
    const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
    int count = 0;
#pragma unroll 4
    for (int i = 0; i < kChunkWords / 8; ++i) {
        const int word = c * kChunkWords + i * 8 + static_cast<int>(warp);
        const int64_t page = static_cast<int64_t>(word) * 32 + lane;
        const int32_t n = page < p.num_pages ? __ldcg(p.refs + page) : -1;
        const uint32_t first = __ballot_sync(0xffffffffu, kUsed ? n > 0 : n == 0);
        const uint32_t once = __ballot_sync(0xffffffffu, n == 1);
        count += __popc(first);
        if (lane == 0) {
            p.free_mask[word] = first;
            if (!kUsed) p.once_mask[word] = once;
        }
    }
    int total;
    block_sums(lane == 0 ? count : 0, total, shared8);
    if (threadIdx.x == 0) p.chunk_count[c] = total;
}

__device__ __forceinline__ bool bit_of(const uint32_t* mask, int page) { return __ldcg(mask + (page >> 5)) >> (page & 31) & 1u; }

// Slots of `tokens` tokens.
__device__ __forceinline__ int slots_of(int tokens, int shift) {
    return static_cast<int>((static_cast<uint32_t>(tokens) + (1u << shift) - 1) >> shift);
}

// Does the page of slot s end above `tokens` (is it not whole within them)?
__device__ __forceinline__ bool ends_above(int s, int shift, int tokens) { return (static_cast<int64_t>(s + 1) << shift) > tokens; }

static __global__ void __launch_bounds__(256)
kv8_arrange_look_kernel(const PoolParams p) {
    __shared__ int shared8[8];
    __shared__ int earlier, kept;          // is there a row before with the same parent; most tokens that another one keeps
    griddep_launch_dependents();
    griddep_wait();                        // launched early behind the kernel that may have written the tables
    if (static_cast<int>(blockIdx.x) < p.chunks) {
        mask_chunk<false>(p, static_cast<int>(blockIdx.x), shared8);
        return;
    }
    const int i = static_cast<int>(blockIdx.x) - p.chunks;
    if (threadIdx.x == 0) earlier = kept = 0;
    __syncthreads();
    const int64_t most = static_cast<int64_t>(p.max_pages) << p.page_shift;
    const int par = p.parents != nullptr ? __ldcg(p.parents + i) : i;
    const int held = __ldcg(p.held + i), keep = __ldcg(p.keep + i), room = __ldcg(p.room + i);
    bool bad = par < 0 || par >= p.rows || held < 0 || held > most || keep < 0 || room < keep || room > most;
    int par_held = bad ? 0 : __ldcg(p.held + par);
    bad = bad || par_held < 0 || par_held > most || keep > par_held;
    int need = 0;
    int bound = 0;
    if (!bad) {
        if (p.parents != nullptr) {
            for (int j = static_cast<int>(threadIdx.x); j < p.rows; j += 256) {
                if (j == i || __ldcg(p.parents + j) != par) continue;
                if (j < i) earlier = 1;
                atomicMax(&kept, __ldcg(p.keep + j));
            }
            __syncthreads();
            // (its parent's heir: itself, or the lowest row with this parent where the parent goes elsewhere)
            const bool heir = par == i || (earlier == 0 && __ldcg(p.parents + par) != par);
            bound = heir ? kept : 0x7FFFFFFF;
        }
        const int whole = keep >> p.page_shift, slots = slots_of(room, p.page_shift);
        const int had = slots_of(held, p.page_shift), par_had = slots_of(par_held, p.page_shift);
        const int32_t* const mine = p.table + i * p.table_stride;
        const int32_t* const theirs = p.table + par * p.table_stride;
        bool wrong = false;
        auto out_of_range = [&](int32_t e) { return e < 0 || e >= p.num_pages; };
        // (whole pages of a row that stays its own are not looked at: nothing is done with them)
        const int from = par == i ? whole : 0;
        for (int s = from + static_cast<int>(threadIdx.x); s < had; s += 256) {
            const int32_t e = __ldcg(mine + s);
            wrong = wrong || out_of_range(e);
            if (p.parents != nullptr) p.old_table[static_cast<int64_t>(i) * p.max_pages + s] = e;
        }
        if (p.parents != nullptr)
            for (int s = static_cast<int>(threadIdx.x); s < min(from, had); s += 256)
                p.old_table[static_cast<int64_t>(i) * p.max_pages + s] = __ldcg(mine + s);
        if (par != i)
            for (int s = static_cast<int>(threadIdx.x); s < min(max(whole, min(slots, par_had)), par_had); s += 256)
                wrong = wrong || out_of_range(__ldcg(theirs + s));
        bad = __syncthreads_or(wrong);
        if (!bad) {
            int n = 0;
            for (int s = whole + static_cast<int>(threadIdx.x); s < slots; s += 256) {
                const bool taken = ends_above(s, p.page_shift, bound) && s < par_had && __ldcg(p.refs + __ldcg(theirs + s)) == 1;
                n += taken ? 0 : 1;
            }
            block_sums(n, need, shared8);
        }
    }
    if (threadIdx.x == 0) {
        p.need[i] = bad ? -1 : need;
        p.old_held[i] = held;
        p.bound[i] = bound;
        if (bad) atomicOr(p.status, kErrPage);
    }
}

static __global__ void __launch_bounds__(256)
kv8_arrange_rows_kernel(const PoolParams p) {
    __shared__ int shared8[8];
    __shared__ int lo_chunk, hi_chunk;
    griddep_launch_dependents();
    griddep_wait();
    const int i = static_cast<int>(blockIdx.x);
    const int t = static_cast<int>(threadIdx.x);
    if (t == 0) {
        lo_chunk = 0x7FFFFFFF;
        hi_chunk = -1;
    }
    // ---- what all rows need, what those before this one do, and the pages that are free
    int64_t before = 0, wanted = 0, free_pages = 0;
    bool bad = false;
    for (int j = t; j < p.rows; j += 256) {
        const int n = __ldcg(p.need + j);
        bad = bad || n < 0;
        wanted += n;
        if (j < i) before += n;
    }
    for (int c = t; c < p.chunks; c += 256) free_pages += __ldcg(p.chunk_count + c);
    bad = __syncthreads_or(bad);
    __shared__ long long sums[8][3];
#pragma unroll
    for (int d = 16; d > 0; d /= 2) {
        before += __shfl_xor_sync(0xffffffffu, before, d);
        wanted += __shfl_xor_sync(0xffffffffu, wanted, d);
        free_pages += __shfl_xor_sync(0xffffffffu, free_pages, d);
    }
    if ((t & 31) == 0) {
        sums[t >> 5][0] = before;
        sums[t >> 5][1] = wanted;
        sums[t >> 5][2] = free_pages;
    }
    __syncthreads();
    before = wanted = free_pages = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        before += sums[w][0];
        wanted += sums[w][1];
        free_pages += sums[w][2];
    }
    const bool refused = bad || wanted > free_pages;
    if (t == 0) {
        p.copy_src[i] = p.copy_dst[i] = -1;
        if (i == 0) *p.missing = bad ? -1 : static_cast<int32_t>(max(0ll, static_cast<long long>(wanted - free_pages)));
    }
    if (refused) return;                   // (all rows stay as they were)

    const int par = p.parents != nullptr ? __ldcg(p.parents + i) : i;
    const int keep = __ldcg(p.keep + i), room = __ldcg(p.room + i);
    const int held = __ldcg(p.old_held + i), par_held = __ldcg(p.old_held + par);
    const int bound = __ldcg(p.bound + i);
    const int need = __ldcg(p.need + i);
    const int whole = keep >> p.page_shift, slots = slots_of(room, p.page_shift);
    const int had = slots_of(held, p.page_shift), par_had = slots_of(par_held, p.page_shift);
    // ---- the free pages [before, before + need), lowest first
    if (need > 0) {
        int64_t base = 0;
        for (int c0 = 0; c0 < p.chunks && base < before + need; c0 += 256) {
            const int n = c0 + t < p.chunks ? __ldcg(p.chunk_count + c0 + t) : 0;
            int total;
            const int64_t at = base + block_sums(n, total, shared8);
            if (n > 0 && at < before + need && at + n > before) {
                atomicMin(&lo_chunk, c0 + t);
                atomicMax(&hi_chunk, c0 + t);
                // (the sum of the chunks before the lowest one is what its thread knows)
            }
            __syncthreads();
            if (c0 + t == lo_chunk) sums[0][0] = at;
            base += total;
        }
        __syncthreads();
        base = sums[0][0];
        for (int w0 = lo_chunk * kChunkWords; w0 < (hi_chunk + 1) * kChunkWords; w0 += 256) {
            uint32_t bits = w0 + t < (hi_chunk + 1) * kChunkWords ? __ldcg(p.free_mask + w0 + t) : 0u;
            int total;
            int64_t rank = base + block_sums(__popc(bits), total, shared8);
            for (; bits != 0; bits &= bits - 1, ++rank)
                if (rank >= before && rank < before + need) p.fresh[rank] = (w0 + t) * 32 + __ffs(static_cast<int>(bits)) - 1;
            base += total;
        }
        __syncthreads();
    }
    // ---- the row's entries and the references
    int32_t* const row = p.table + i * p.table_stride;
    const int32_t* const was = p.parents != nullptr ? p.old_table + static_cast<int64_t>(i) * p.max_pages : row;
    const int32_t* const from = p.parents != nullptr ? p.old_table + static_cast<int64_t>(par) * p.max_pages : row;
    const int first = par == i ? whole : 0;          // (whole pages of its own stay)
    int64_t next = before;
    for (int s0 = first; s0 < max(slots, had); s0 += 256) {
        const int s = s0 + t;
        const bool wants = s < slots, there = s < par_had;
        const int32_t old = s < had ? __ldcg(was + s) : -1;
        const int32_t cand = there && wants ? __ldcg(from + s) : -1;
        const bool fresh = wants && s >= whole && !(there && ends_above(s, p.page_shift, bound) && bit_of(p.once_mask, cand));
        int total;
        const int place = block_sums(fresh ? 1 : 0, total, shared8);
        int32_t now = -1;
        if (wants) {
            now = fresh ? __ldcg(p.fresh + next + place) : cand;
            if (fresh && (static_cast<int64_t>(s) << p.page_shift) < keep) {
                p.copy_src[i] = cand;
                p.copy_dst[i] = now;
            }
            row[s] = now;
        }
        if (now != old) {
            if (now >= 0) atomicAdd(p.refs + now, 1);
            if (old >= 0) atomicSub(p.refs + old, 1);
        }
        next += total;
    }
    if (t == 0) p.held[i] = room;
}

// ------------------------------------------------------------------ compacting

struct CompactParams {
    PoolParams pool;
    int32_t* rank;                         // [num_pages] a moving page's number
    int32_t* holes;                        // [num_pages] where number k goes
    int32_t* movers;                       // [num_pages]
    int32_t* moved;                        // [num_pages] where each page is now; -1: it is free
    int32_t* count;                        // [2] pages in use (U), pages that move
};

static __global__ void __launch_bounds__(256)
kv8_compact_look_kernel(const CompactParams c) {
    __shared__ int shared8[8];
    griddep_launch_dependents();
    griddep_wait();
    mask_chunk<true>(c.pool, static_cast<int>(blockIdx.x), shared8);
}

static __global__ void __launch_bounds__(256)
kv8_compact_rank_kernel(const CompactParams c) {
    const PoolParams& p = c.pool;
    __shared__ int shared8[8];
    __shared__ int here_before, below;     // used pages before this block's chunk; before page U
    griddep_launch_dependents();
    griddep_wait();
    const int t = static_cast<int>(threadIdx.x), chunk = static_cast<int>(blockIdx.x);
    int used = 0;
    for (int c0 = 0; c0 < p.chunks; c0 += 256) {
        const int n = c0 + t < p.chunks ? __ldcg(p.chunk_count + c0 + t) : 0;
        int total;
        const int at = used + block_sums(n, total, shared8);
        if (c0 + t == chunk) here_before = at;
        used += total;
    }
    // used pages below page `used`: the chunks before its own, then words
    const int cut = used / kChunkPages;
    if (t == 0) below = 0;
    __syncthreads();
    int sum = 0;
    for (int j = t; j < min(cut, p.chunks); j += 256) sum += __ldcg(p.chunk_count + j);
    if (cut < p.chunks && t < kChunkWords) {
        const int word = cut * kChunkWords + t, at = word * 32;      // (its first page)
        uint32_t bits = __ldcg(p.free_mask + word);
        if (at + 32 > used) bits = at >= used ? 0u : bits & ((1u << (used - at)) - 1u);
        sum += __popc(bits);
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if ((t & 31) == 0) atomicAdd(&below, sum);
    __syncthreads();
    if (chunk == 0 && t == 0) {
        c.count[0] = used;
        c.count[1] = used - below;
    }
    const uint32_t bits = t < kChunkWords ? __ldcg(p.free_mask + chunk * kChunkWords + t) : 0u;
    int total;
    int before = here_before + block_sums(__popc(bits), total, shared8);
    if (t >= kChunkWords) return;
    for (int j = 0; j < 32; ++j) {
        const int64_t page = (static_cast<int64_t>(chunk) * kChunkWords + t) * 32 + j;
        if (page >= p.num_pages) break;
        if (bits >> j & 1u) {
            if (page >= used) {
                c.rank[page] = before - below;
                c.movers[before - below] = static_cast<int32_t>(page);
            } else {
                c.moved[page] = static_cast<int32_t>(page);
            }
            ++before;
        } else {
            c.moved[page] = -1;
            if (page < used) c.holes[page - before] = static_cast<int32_t>(page);
        }
    }
}

// Blocks [0, rows): the table's rows. The others: references and places of the moving pages.
static __global__ void __launch_bounds__(256)
kv8_compact_rows_kernel(const CompactParams c) {
    const PoolParams& p = c.pool;
    griddep_launch_dependents();
    griddep_wait();
    const int used = __ldcg(c.count), moving = __ldcg(c.count + 1);
    if (static_cast<int>(blockIdx.x) >= p.rows) {
        const int blocks = static_cast<int>(gridDim.x) - p.rows;
        for (int64_t k = (static_cast<int64_t>(blockIdx.x) - p.rows) * 256 + threadIdx.x; k < moving; k += int64_t(256) * blocks) {
            const int32_t from = __ldcg(c.movers + k), to = __ldcg(c.holes + k);
            c.moved[from] = to;
            p.refs[to] = __ldcg(p.refs + from);
            p.refs[from] = 0;
        }
        return;
    }
    const int i = static_cast<int>(blockIdx.x);
    const int64_t most = static_cast<int64_t>(p.max_pages) << p.page_shift;
    const int held = __ldcg(p.held + i);
    bool wrong = held < 0 || held > most;
    int32_t* const row = p.table + i * p.table_stride;
    const int had = wrong ? 0 : slots_of(held, p.page_shift);
    for (int s = static_cast<int>(threadIdx.x); s < had; s += 256) {
        const int32_t e = __ldcg(row + s);
        if (e < 0 || e >= p.num_pages) wrong = true;
        else if (e >= used && bit_of(p.free_mask, e)) row[s] = __ldcg(c.holes + __ldcg(c.rank + e));
    }
    if (wrong) atomicOr(p.status, kErrPage);
}

// -------------------------------------------------------------------- copying

struct CopyParams {
    struct Cache {
        const uint4* from[2];
        uint4* to[2];
        const float* scale_from[2];
        float* scale_to[2];
    } cache[kMaxCaches];
    const int32_t* src;                    // pages to copy; -1: none
    const int32_t* dst;
    const int32_t* count;                  // of the list, or null: n
    int64_t n, src_pages, dst_pages;
    int32_t caches, heads;
    int32_t page_vecs;                     // 16-byte pieces of a page's keys or values
    int32_t parts;                         // steps of a page
    uint32_t* status;
};

constexpr int kCopyVecs = 256;             // 16-byte pieces of a step of a warp: 4 KB, eight loads in flight per lane

static __global__ void __launch_bounds__(256)
kv8_copy_pages_kernel(const CopyParams p) {
    griddep_launch_dependents();
    griddep_wait();
    const int lane = static_cast<int>(threadIdx.x & 31u);
    const int64_t n = p.count != nullptr ? min(static_cast<int64_t>(__ldcg(p.count)), p.n) : p.n;
    const uint32_t per_entry = static_cast<uint32_t>(p.caches) * 2u * static_cast<uint32_t>(p.parts);
    const int64_t steps = n * per_entry;
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); item < steps; item += static_cast<int64_t>(gridDim.x) * 8) {
        const int64_t entry = steps <= 0xFFFFFFFFll ? static_cast<int64_t>(static_cast<uint32_t>(item) / per_entry) : item / per_entry;
        uint32_t rest = static_cast<uint32_t>(item - entry * per_entry);
        const int32_t src = __ldcg(p.src + entry), dst = __ldcg(p.dst + entry);
        if (src == -1 && dst == -1) continue;
        if (src < 0 || src >= p.src_pages || dst < 0 || dst >= p.dst_pages) {
            if (lane == 0) atomicOr(p.status, kErrPage);
            continue;
        }
        const int part = static_cast<int>(rest % static_cast<uint32_t>(p.parts));
        rest /= static_cast<uint32_t>(p.parts);
        const int kv = static_cast<int>(rest & 1u);
        const CopyParams::Cache& c = p.cache[rest >> 1];
        const uint4* const from = c.from[kv] + static_cast<int64_t>(src) * p.page_vecs;
        uint4* const to = c.to[kv] + static_cast<int64_t>(dst) * p.page_vecs;
        const int at = part * kCopyVecs + lane, end = min(p.page_vecs, (part + 1) * kCopyVecs);
        uint4 x[kCopyVecs / 32];
#pragma unroll
        for (int k = 0; k < kCopyVecs / 32; ++k)
            if (at + 32 * k < end) x[k] = from[at + 32 * k];
#pragma unroll
        for (int k = 0; k < kCopyVecs / 32; ++k)
            if (at + 32 * k < end) to[at + 32 * k] = x[k];
        if (part == 0)
            for (int h = lane; h < p.heads; h += 32)
                c.scale_to[kv][static_cast<int64_t>(dst) * p.heads + h] = c.scale_from[kv][static_cast<int64_t>(src) * p.heads + h];
    }
}

}  // namespace kv8
}  // namespace hk
