// Attention of a few query rows per sequence over the paged 8-bit cache, for
// sequences that begin with the same tokens in the same pages (answers to one prompt, requests
// behind one system prompt): the shared pages are read once for all of them.
//
// A group is consecutive sequences whose first `shared` tokens lie in the pages that the
// first one's table row names. Their query rows (sequences × tokens × the query heads of a KV
// head) are stacked into units over those pages, and every sequence has units of its
// own over its remaining tokens; with the running maxima m and sums l of both,
//
//   O = (O_1 2^(m_1 - m) + O_2 2^(m_2 - m)) / (l_1 2^(m_1 - m) + l_2 2^(m_2 - m)),  m = max(m_1, m_2)
//
// What is shared is rounded down to 128 tokens, so that it ends with a page and a tile; and
// a sequence takes part only if all its queries see all of it (else its own units begin
// at its first token, and its rows among the stacked ones are left unused): a shared unit
// needs no masks, and no value of a token that a query does not see meets that query.
//
// Both kinds of units run as in kv8_decode.cuh: tiles of 32 tokens of all units in
// one order, cut into equal runs, one per warp, whatever the lengths are; sums of units that
// are split, and of sequences with a shared part, go through memory and are added up by a second
// kernel, in order. Without a shared part a whole unit is finished at once. Tiles bound it: 16 rows by 32 tokens
// some 1 us of a warp whatever its rows hold, 45 sequences in 6 groups behind 5003 tokens (28/4 heads of 64, fp16) 33 to 39 us
// (255 registers a thread; at head dimension 128 the compiler spills 64 bytes).
// Where the shared units run on the tensor-core kernel (kv8_shared_mma.cuh), what sequences have of their own is
// mostly short, and a block to a unit is quicker: no plan over all lengths before the first load, and
// the unit's warps load at the same time; only units of more than `own_limit` tiles are spread.
#pragma once

#include "kv8_decode.cuh"

namespace hk {
namespace kv8 {

constexpr int kMaxShared = 512;        // sequences, and groups, of one launch
constexpr int kSharedStep = 128;       // tokens that what is shared is rounded down to
constexpr int kWideRows = 128;         // stacked rows of a unit on the tensor-core kernel

template <int kD>
struct SharedGeometry {
    using G = DecodeGeometry<kD>;
    static constexpr int kOffPrefix = kDecodeWarps * G::kWarpBytes;                   // tiles before each group's and sequence's
    static constexpr int kOffGroups = kOffPrefix + (2 * kMaxShared + 1) * 4;          // first sequence of each group
    static constexpr int kOffShared = kOffGroups + (kMaxShared + 1) * 4;              // shared tiles of each group
    static constexpr int kOffStart = kOffShared + kMaxShared * 4;                     // first own tile of each sequence
    static constexpr int kOffBars = (kOffStart + kMaxShared * 4 + 7) / 8 * 8;
    static constexpr int kSmemBytes = kOffBars + kDecodeWarps * G::kStages * 8 + 1024;
    static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two blocks per SM");
};

struct SharedParams : DecodeParams {
    const int32_t* groups;         // [G + 1] first sequence of each group, B at the end
    const int32_t* shared;         // [G] shared tokens
    int32_t G, b0, n, all;         // groups; this launch: sequences [b0, b0 + n) of all
    int64_t whole[2];              // rows of part_o and part_ml where the sums of whole units begin: shared, own
    int4* shared_info;             // as info, of the units of the groups: [KV head][shared_units]
    int32_t shared_units;
    int32_t own_limit;             // a sequence's own units of up to so many tiles are blocks of kv8_own_kernel
    int32_t wide_runs;             // CTAs that work on the shared units of 128 rows (kv8_shared_mma.cuh); 0: units of 16 rows here
    int64_t shared_slots;          // row of part_o and part_ml where the sums of split units of 128 rows begin
    int4* seqs;                    // [n]: shared tiles, place of the group, its first sequence of this launch, queries
};

// Group of a launch: its sequences in it, and its shared tiles.
struct Group {
    int first, n, tiles;           // first sequence of the launch, counted from b0
};

__device__ __forceinline__ int shared_rows(const SharedParams& p, int n) { return n * p.T * p.group; }

// Where the shared units of the group in place `j` (of the launch's groups; for units of 128 rows, of all) with first sequence
// `first` begin in shared_info.
__device__ __forceinline__ int shared_unit0(const SharedParams& p, int j, int first) { return shared_rows(p, first) / kRows + j; }

// Tokens that the first query of a sequence sees (the fewest of its queries).
__device__ __forceinline__ int least_seen(const SharedParams& p, const Sequence& s) {
    if (s.count == 0) return 0;
    return p.causal ? max(0, s.len - s.count + 1) : s.len;
}

// Are a group's sequences and its shared tokens what they may be? (Where one group's are not, none shares anything: groups that
// overlap would name more tiles than are counted.)
__device__ __forceinline__ bool group_in_order(const SharedParams& p, int j, int first, int next, int shared) {
    return first >= 0 && next > first && next <= p.all && shared >= 0 && (j > 0 || first == 0);
}

// Tiles of a group's shared part: what its first sequence, of `len` tokens, has of it, in whole steps.
__device__ __forceinline__ int shared_tiles(const SharedParams& p, int shared, int len) {
    const int64_t most = min(min(static_cast<int64_t>(shared), static_cast<int64_t>(len)), static_cast<int64_t>(p.max_pages) * p.page_size);
    return static_cast<int>(max(static_cast<int64_t>(0), most)) / kSharedStep * (kSharedStep / kTileKeys);
}

// The tile that a sequence's own part begins at, in a group of so many shared tiles: it takes part if all its queries see them.
__device__ __forceinline__ int own_start(const SharedParams& p, const Sequence& s, int tiles) {
    return tiles > 0 && least_seen(p, s) >= static_cast<int64_t>(tiles) * kTileKeys ? tiles : 0;
}

// 16 stacked rows of a group: KV head h, rows [16 rt, 16 rt + 16).
struct SharedRows {
    const SharedParams& p;
    int b, n, h, rt;               // first sequence of the group in this launch, and how many
    const int32_t* table;          // of the group's first sequence

    __device__ __forceinline__ const int32_t* pages() const { return table; }
    __device__ __forceinline__ bool several() const { return false; }
    template <typename T>
    __device__ __forceinline__ const T* row(int r, bool& live, int& limit) const {
        const int row = rt * kRows + r, per = p.T * p.group;
        const int seq = row / per, rest = row - seq * per, t = rest / p.group;
        live = seq < n;
        limit = 0x7FFFFFFF;
        return static_cast<const T*>(p.q) + (b + seq) * p.q_stride_b + t * p.q_stride_t +
               static_cast<int64_t>(h * p.group + rest - t * p.group) * p.q_stride_h;
    }
};

// Tiles of the unit of row tile rt of a sequence whose own part begins at tile `start`, of which there is one at least.
__device__ __forceinline__ int own_tiles(int end, int start) { return max(1, (end + kTileKeys - 1) / kTileKeys - start); }

// Those of them that the spreading kernel works on.
__device__ __forceinline__ int spread_tiles(const SharedParams& p, int end, int start) {
    const int tiles = own_tiles(end, start);
    return tiles > p.own_limit ? tiles : 0;
}

// Sequences of group `j` in this launch.
__device__ __forceinline__ Group group_of(const SharedParams& p, const int32_t* first_of, const int32_t* tiles_of_group, int j) {
    const int first = max(first_of[j], p.b0), end = min(first_of[j + 1], p.b0 + p.n);
    return Group{first - p.b0, max(0, end - first), tiles_of_group[j]};
}

// What the spreading kernel's blocks all work out first: groups, shared tiles, where the sequences' own parts begin, and (at
// i + 1) the tiles of each section i: the groups' shared units, then the sequences' own. Returns the number of groups.
template <int kThreads>
__device__ __forceinline__ int plan_sections(const SharedParams& p, int32_t* first_of, int32_t* tiles_of_group, int32_t* start, int32_t* prefix) {
    const int t = static_cast<int>(threadIdx.x);
    __shared__ int lowest;
    Sequence mine = {0, 0};                  // (asked for ahead of what the groups' loads are waited for)
    if (t < p.n) mine = sequence(p, p.b0 + t);
    int g0 = 0;
    if (p.b0 > 0) {                          // the group of sequence b0
        if (t == 0) {
            int lo = 0, hi = p.G - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (p.groups[mid] <= p.b0) lo = mid; else hi = mid - 1;
            }
            lowest = lo;
        }
        __syncthreads();
        g0 = lowest;
    }
    const int groups = min(p.G - g0, kMaxShared);
    bool bad = false;
    for (int j = t; j <= groups; j += kThreads) {
        const int first = p.groups[g0 + j];
        if (j < groups) {
            const int shared = p.shared[g0 + j];
            const bool in_order = group_in_order(p, g0 + j, first, p.groups[g0 + j + 1], shared);
            tiles_of_group[j] = in_order && first < p.b0 + p.n ? shared_tiles(p, shared, p.lengths[first]) : 0;
            bad = bad || !in_order;
        }
        bad = bad || (g0 + j == p.G && first != p.all);
        first_of[j] = first;
    }
    auto off = [&](int j) {                  // (of groups that this launch does not plan for)
        const int next = p.groups[j + 1];
        return !group_in_order(p, j, p.groups[j], next, p.shared[j]) || (j + 1 == p.G && next != p.all);
    };
    // The kernels for units of 128 rows and for own parts look at every group, and what is shared has to be the same to all three.
    // Groups that are too many for that are looked at once, a part by each block of the first launch, so as to be reported.
    if (p.wide_runs > 0)
        for (int j = t; j < g0; j += kThreads) bad = bad || off(j);
    if (bad) atomicOr(p.wait.status, kErrPage);
    if (p.b0 == 0)
        for (int64_t j = groups + static_cast<int64_t>(blockIdx.x) * kThreads + t; j < p.G; j += static_cast<int64_t>(gridDim.x) * kThreads)
            if (off(static_cast<int>(j))) atomicOr(p.wait.status, kErrPage);
    if (__syncthreads_or(bad)) {
        for (int j = t; j < groups; j += kThreads) tiles_of_group[j] = 0;
        __syncthreads();
    }
    for (int j = t; j < groups; j += kThreads) {
        const Group gr = group_of(p, first_of, tiles_of_group, j);
        prefix[j + 1] = p.wide_runs > 0 ? 0 : (shared_rows(p, gr.n) + kRows - 1) / kRows * gr.tiles * p.Hkv;
    }
    for (int i = t; i < p.n; i += kThreads) {
        const int b = p.b0 + i;
        int lo = 0, hi = groups - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (first_of[mid] <= b) lo = mid; else hi = mid - 1;
        }
        const Sequence s = i == t ? mine : sequence(p, b);
        const bool member = first_of[lo] >= 0 && first_of[lo] <= b && b < first_of[lo + 1];
        const int from = own_start(p, s, member ? tiles_of_group[lo] : 0);
        start[i] = from;
        if (blockIdx.x == 0) p.seqs[i] = make_int4(from, lo, max(first_of[lo], p.b0) - p.b0, s.count);
        int tiles = 0;
        for (int rt = 0; rt < p.row_tiles; ++rt) tiles += spread_tiles(p, row_tile_end(p, s, rt), from);
        prefix[groups + i + 1] = tiles * p.Hkv;
    }
    __syncthreads();
    return groups;
}

template <int kD, typename T>
__global__ void __launch_bounds__(32 * kDecodeWarps, 2)
kv8_shared_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v, const SharedParams p) {
    using G = DecodeGeometry<kD>;
    using S = SharedGeometry<kD>;
    constexpr int kNTiles = kD / 8;
    constexpr int kOwn = kD / 4;
    constexpr int kThreads = 32 * kDecodeWarps;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const smem = smem_raw + (base - raw);
    const uint32_t warp = threadIdx.x >> 5, lane = lane_id();
    const uint32_t g = lane >> 2, c = lane & 3u;
    const int self = static_cast<int>(blockIdx.x) * kDecodeWarps + static_cast<int>(warp);

    griddep_launch_dependents();             // the next kernel may be scheduled; it waits for this grid's end
    if (threadIdx.x == 0) {
        prefetch_tensor_map(&tmap_k);
        prefetch_tensor_map(&tmap_v);
    }
    const uint32_t ring = base + warp * G::kWarpBytes;
    const uint32_t bars = base + S::kOffBars + 8u * warp * G::kStages;
    if (lane == 0) {
        for (int s = 0; s < G::kStages; ++s) mbar_init(bars + 8u * s, s == 0 && (p.flags & kFlagDropArrive) ? 2 : 1);
        fence_mbar_init_cluster();
    }
    griddep_wait();                          // launched early behind the kernel that may have written the cache or q
    int32_t* const prefix = reinterpret_cast<int32_t*>(smem + S::kOffPrefix);
    int32_t* const first_of = reinterpret_cast<int32_t*>(smem + S::kOffGroups);
    int32_t* const tiles_of_group = reinterpret_cast<int32_t*>(smem + S::kOffShared);
    int32_t* const start = reinterpret_cast<int32_t*>(smem + S::kOffStart);
    const int groups = plan_sections<kThreads>(p, first_of, tiles_of_group, start, prefix);
    const int sections = groups + p.n;       // the groups' shared units, then the sequences' own
    if (warp == 0) {
        int sum = 0;
        for (int i0 = 0; i0 < sections; i0 += 32) {
            const int i = i0 + static_cast<int>(lane);
            int inc = i < sections ? prefix[i + 1] : 0;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int o = __shfl_up_sync(0xffffffffu, inc, d);
                if (static_cast<int>(lane) >= d) inc += o;
            }
            if (i < sections) prefix[i + 1] = sum + inc;
            sum += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) prefix[0] = 0;
    }
    __syncthreads();

    const int total = prefix[sections];
    const int per = (total + p.warps - 1) / p.warps;
    const int begin = static_cast<int>(min(static_cast<int64_t>(total), static_cast<int64_t>(self) * per));
    const int end = static_cast<int>(min(static_cast<int64_t>(total), static_cast<int64_t>(begin) + per));
    bool ok = true;
    int fills = 0, uses = 0;                 // ring stages filled and consumed so far

    int at = begin, section = 0;
    if (begin < end) {
        int lo = 0, hi = sections - 1;       // the last section that begins at or before this run (those without tiles end there)
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= begin) lo = mid; else hi = mid - 1;
        }
        section = lo;
    }
    while (at < end) {
        // ---- the unit of tile `at`
        while (prefix[section + 1] <= at) ++section;
        const bool is_shared = section < groups;
        int local = at - prefix[section];
        const int head_tiles = (prefix[section + 1] - prefix[section]) / p.Hkv;
        const int h = local / head_tiles;
        local -= h * head_tiles;
        const int i = section - groups, b = p.b0 + i;      // (of a sequence's own part)
        Group gr = {0, 0, 0};
        Sequence seq = {0, 0};
        int rt = 0, unit_tiles, first, key_end, tile0 = 0;
        if (is_shared) {
            gr = group_of(p, first_of, tiles_of_group, section);
            unit_tiles = gr.tiles;
            rt = local / unit_tiles;
            first = local - rt * unit_tiles;
            key_end = unit_tiles * kTileKeys;
        } else {
            seq = sequence(p, b);
            first = local;
            tile0 = start[i];
            while (first >= (unit_tiles = spread_tiles(p, key_end = row_tile_end(p, seq, rt), tile0)) && rt + 1 < p.row_tiles) {
                first -= unit_tiles;
                ++rt;
            }
        }
        const int last = min(unit_tiles, first + (end - at));   // tiles [first, last) of the unit

        float o[kNTiles][4], m[2], l[2];
        if (is_shared)
            ok = attend<kD, T, G::kStages>(p, &tmap_k, &tmap_v, ring, bars, fills, uses,
                                           SharedRows{p, p.b0 + gr.first, gr.n, h, rt, p.table + first_of[section] * p.table_stride}, h,
                                           key_end, first, last, o, m, l);
        else     // (a part that ends before it begins has one tile to see nothing in: no token is read)
            ok = attend<kD, T, G::kStages>(p, &tmap_k, &tmap_v, ring, bars, fills, uses, UnitRows{p, b, h, rt, seq}, h,
                                           key_end > tile0 * kTileKeys ? key_end : 0, tile0 + first, tile0 + last, o, m, l);
        if (!ok) break;

        // ---- finish the unit or leave its sums
        const bool whole = first == 0 && last == unit_tiles;
        const int slot = 2 * self + (at == begin ? 0 : 1);
        if (first == 0 && lane == 0) {       // this run holds the unit's first tile: it tells how the unit is made up
            const int parts = whole ? 0 : (at + unit_tiles - 1) / per - at / per + 1;
            const int4 record = make_int4(parts, slot, self, 0);
            if (is_shared) p.shared_info[static_cast<int64_t>(h) * p.shared_units + shared_unit0(p, section, gr.first) + rt] = record;
            else p.info[(static_cast<int64_t>(i) * p.Hkv + h) * p.row_tiles + rt] = record;
        }
        const bool finish = whole && !is_shared && tile0 == 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = static_cast<int>(g) + 8 * e, row = rt * kRows + r;
            int s = i, rest = row;                                // sequence of the launch, row of it
            if (is_shared) {
                s = row / (p.T * p.group);
                rest = row - s * (p.T * p.group);
                if (s >= gr.n) continue;
                s += gr.first;
            }
            const int t = rest / p.group, head = h * p.group + rest - t * p.group;
            if (t >= p.T) continue;
            float v[kOwn];
            const bool any = l[e] > 0.0f || l[e] != l[e];        // (a row that sees nothing may hold NaN sums)
            const float mul = !finish ? 1.0f : 1.0f / l[e];
#pragma unroll
            for (int j = 0; j < kNTiles; ++j) {
                v[j] = any ? o[j][2 * e] * mul : 0.0f;
                v[kNTiles + j] = any ? o[j][2 * e + 1] * mul : 0.0f;
            }
            const int64_t out_row = (static_cast<int64_t>(s) * p.T + t) * p.Hq + head;     // of the launch
            if (finish) {
                T* const dst = static_cast<T*>(p.o) + b * p.o_stride_b + t * p.o_stride_t + head * p.o_stride_h + c * kOwn;
                store_row<T, kOwn>(dst, v, p.vec_o != 0);
                if (p.lse != nullptr && c == 0)
                    p.lse[static_cast<int64_t>(p.b0) * p.T * p.Hq + out_row] = any ? (m[e] + log2f(l[e])) * 0.69314718055994531f : -INFINITY;
            } else {
                const int64_t at_row = whole ? p.whole[is_shared ? 0 : 1] + out_row : static_cast<int64_t>(slot) * kRows + r;
                float4* const dst = reinterpret_cast<float4*>(p.part_o + at_row * kD + c * kOwn);
#pragma unroll
                for (int k = 0; k < kOwn / 4; ++k) dst[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                if (c == 0) {
                    p.part_ml[2 * at_row] = any ? m[e] : -INFINITY;
                    p.part_ml[2 * at_row + 1] = any ? l[e] : 0.0f;
                }
            }
        }
        at += last - first;
    }
    // abort: the copies in flight land before the block ends
    if (!ok)
        for (; uses < fills; ++uses) wait_mbar_drain(bars + 8u * (uses % G::kStages), (uses / G::kStages) & 1);
}

// Sums in memory that make up 16 rows of a sequence and KV head: those of its own part, where the spreading kernel left it, and
// those of the stacked rows' units of 128, of which the 16 rows may lie in two.
struct RowParts {
    const SharedParams& p;
    int64_t out_row0;              // of the launch, of query token 0 and the KV head's first query head
    int row0;                      // rt * 16
    int4 own;                      // record of the own part; own_parts 0: it is in shared memory
    int own_parts;
    int4 shared0, shared1;         // records of the stacked rows' units, the second from row `cut` on
    int cut, stacked0;             // stacked row of row 0; -1: nothing shared

    __device__ __forceinline__ int4 unit(int r) const {
        const bool before = r < cut;
        return make_int4(before ? shared0.x : shared1.x, before ? shared0.y : shared1.y, before ? shared0.z : shared1.z, 0);
    }
    __device__ __forceinline__ int64_t out_row(int r) const {
        const int row = row0 + r, t = row / p.group;
        return out_row0 + static_cast<int64_t>(t) * p.Hq + (row - t * p.group);
    }
    __device__ __forceinline__ int parts(int r) const { return own_parts + (stacked0 >= 0 ? max(unit(r).x, 1) : 0); }
    // The row of part_o and part_ml of part k.
    __device__ __forceinline__ int64_t at(int r, int k) const {
        const bool mine = k < own_parts;
        const int4 u = unit(r);
        const int4 x = make_int4(mine ? own.x : u.x, mine ? own.y : u.y, mine ? own.z : u.z, 0);
        if (x.x == 0) return (mine ? p.whole[1] : p.whole[0]) + out_row(r);
        const int part = mine ? k : k - own_parts;
        const int64_t slot = part == 0 ? static_cast<int64_t>(x.y) : 2 * (static_cast<int64_t>(x.z) + part);
        return mine ? slot * kRows + r : p.shared_slots + slot * kWideRows + (stacked0 + r) % kWideRows;
    }
};

// Adds parts k = warp, warp + kWarps, ... of each of the first `rows` rows to what the warp holds of them: sums in
// shared memory at `part` (rows of four times kPitch), maxima and sums in `ml`. Four rows and four parts at a time, since
// each trip to memory takes longer than what is done with what it brings.
template <int kD, int kWarps, int kPitch>
__device__ __forceinline__ void add_parts(const RowParts& in, int rows, int warp, float* part, float (*ml)[2]) {
    constexpr int kVec = kD / 32, kAtATime = 4;
    const int lane = static_cast<int>(lane_id());
    const SharedParams& p = in.p;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += kAtATime) {
        float acc[kAtATime][kVec], m[kAtATime], l[kAtATime];
        int n[kAtATime], most = 0;
#pragma unroll
        for (int q = 0; q < kAtATime; ++q) {
            const int r = min(r0 + q, rows - 1);
            n[q] = in.parts(r);
            most = max(most, n[q]);
            m[q] = ml[r][0];
            l[q] = ml[r][1];
            const bool have = m[q] > -INFINITY || l[q] != 0.0f;      // (else nothing has been written at `part`)
            const float* const src = part + (r * 4 + lane / 8) * kPitch + lane % 8 * kVec;
#pragma unroll
            for (int v = 0; v < kVec; ++v) acc[q][v] = have ? src[v] : 0.0f;
        }
#pragma unroll 1
        for (int k0 = warp; k0 < most; k0 += kAtATime * kWarps) {
            float2 f[kAtATime][kAtATime];
            float x[kAtATime][kAtATime][kVec];
#pragma unroll
            for (int u = 0; u < kAtATime; ++u)
#pragma unroll
                for (int q = 0; q < kAtATime; ++q) {
                    if (k0 + u * kWarps >= most) continue;
                    const int64_t a = in.at(min(r0 + q, rows - 1), min(k0 + u * kWarps, n[q] - 1));
                    f[u][q] = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + a);
                    if constexpr (kVec == 4) {
                        const float4 o = __ldcg(reinterpret_cast<const float4*>(p.part_o + a * kD) + lane);
                        x[u][q][0] = o.x; x[u][q][1] = o.y; x[u][q][2] = o.z; x[u][q][3] = o.w;
                    } else {
                        const float2 o = __ldcg(reinterpret_cast<const float2*>(p.part_o + a * kD) + lane);
                        x[u][q][0] = o.x; x[u][q][1] = o.y;
                    }
                }
#pragma unroll
            for (int q = 0; q < kAtATime; ++q) {
                float top = m[q];
#pragma unroll
                for (int u = 0; u < kAtATime; ++u)
                    if (k0 + u * kWarps < n[q]) top = fmaxf(top, f[u][q].x);
                // (a maximum of -inf has a sum of 0, or of NaN, which stays one)
                const float before = m[q] == -INFINITY ? 1.0f : ex2_approx(m[q] - top);
                m[q] = top;
                l[q] *= before;
#pragma unroll
                for (int v = 0; v < kVec; ++v) acc[q][v] *= before;
#pragma unroll
                for (int u = 0; u < kAtATime; ++u) {
                    if (k0 + u * kWarps >= n[q]) continue;
                    const float weight = f[u][q].x == -INFINITY ? 0.0f : ex2_approx(f[u][q].x - top);
                    l[q] += f[u][q].x == -INFINITY ? f[u][q].y : f[u][q].y * weight;
#pragma unroll
                    for (int v = 0; v < kVec; ++v) acc[q][v] += x[u][q][v] * weight;
                }
            }
        }
        __syncwarp();                        // every lane has read the rows' sums
#pragma unroll
        for (int q = 0; q < kAtATime; ++q) {
            if (r0 + q >= rows) break;
            float* const dst = part + ((r0 + q) * 4 + lane / 8) * kPitch + lane % 8 * kVec;
#pragma unroll
            for (int v = 0; v < kVec; ++v) dst[v] = acc[q][v];
            if (lane == 0) {
                ml[r0 + q][0] = m[q];
                ml[r0 + q][1] = l[q];
            }
        }
    }
}

// What a sequence has of its own, and its output, a block to a unit, behind the tensor-core kernel and beside its last blocks (for
// up to 64 groups): the warps share out the tiles of an own part of up to own_limit, then the sums that the
// tensor-core kernel left of its rows (and those of a longer own part, which the first kernel has spread over the GPU), and
// join theirs in shared memory. 26 us for 64 sequences of 512 tokens (8 KV heads of 128, 34 MB: 20 of it the tiles, in a row of
// trips to memory, 6 the joining). A kernel for the joining alone, with the own parts' sums through memory, made a call for 16
// sequences of 4 queries behind 8192 tokens 53 us instead of 47.
template <int kD, typename T, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, kBlockWarps / kWarps)
kv8_own_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v, const SharedParams p) {
    using G = DecodeGeometry<kD>;
    using B = BlockGeometry<kD, kWarps>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ float warp_ml[kWarps][kRows][2];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const smem = smem_raw + (base - raw);
    const uint32_t warp = threadIdx.x >> 5, lane = lane_id();
    const uint32_t g = lane >> 2, c = lane & 3u;
    const uint32_t ring = base + warp * G::kWarpBytes, bars = base + B::kOffBars + 8u * warp * G::kStages;
    griddep_launch_dependents();
    if (threadIdx.x == 0) {
        prefetch_tensor_map(&tmap_k);
        prefetch_tensor_map(&tmap_v);
    }
    if (lane == 0) {
        for (int s = 0; s < G::kStages; ++s) mbar_init(bars + 8u * s, s == 0 && (p.flags & kFlagDropArrive) ? 2 : 1);
        fence_mbar_init_cluster();
    }
    __syncwarp();
    int unit = static_cast<int>(blockIdx.x);
    const int rt = unit % p.row_tiles;
    unit /= p.row_tiles;
    const int h = unit % p.Hkv, i = unit / p.Hkv, b = p.b0 + i;
    // ---- where the sequence's own part begins, and where its stacked rows lie: its group is one lane's
    int start = 0, place = 0, first_of = 0;
    const Sequence seq = sequence(p, b);
    {
        int shared = 0, of = -1;
        bool in_order = true;
        for (int j0 = 0; j0 < p.G; j0 += 32) {
            const int j = j0 + static_cast<int>(lane);
            if (j >= p.G) continue;
            const int first = p.groups[j], next = p.groups[j + 1], tokens = p.shared[j];
            in_order = in_order && group_in_order(p, j, first, next, tokens) && (j + 1 < p.G || next == p.all);
            if (first <= b && b < next) {
                shared = tokens;
                of = first;
                place = j;
            }
        }
        const uint32_t who = __ballot_sync(0xffffffffu, of >= 0);
        if (__all_sync(0xffffffffu, in_order) && who != 0) {
            const int from = __ffs(static_cast<int>(who)) - 1;
            of = __shfl_sync(0xffffffffu, of, from);
            shared = __shfl_sync(0xffffffffu, shared, from);
            place = __shfl_sync(0xffffffffu, place, from);
            first_of = max(of - p.b0, 0);
            start = own_start(p, seq, shared_tiles(p, shared, p.lengths[of]));
        }
    }
    const int key_end = row_tile_end(p, seq, rt);
    const int tiles = own_tiles(key_end, start);
    const bool mine = tiles <= p.own_limit;
    float* const part = reinterpret_cast<float*>(smem + warp * G::kWarpBytes);
    bool ok = true;
    {
        float o[kD / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
        const int first = start + static_cast<int>(warp) * tiles / kWarps, last = start + static_cast<int>(warp + 1) * tiles / kWarps;
        if (mine && first < last && key_end > start * kTileKeys) {
            int fills = 0, uses = 0;
            ok = attend<kD, T, G::kStages>(p, &tmap_k, &tmap_v, ring, bars, fills, uses, UnitRows{p, b, h, rt, seq}, h, key_end, first, last,
                                           o, m, l);
            if (ok) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float4* const dst = reinterpret_cast<float4*>(part + ((g + 8 * e) * 4 + c) * B::kPitch);
#pragma unroll
                    for (int k = 0; k < kD / 32; ++k) {
                        dst[k] = make_float4(o[4 * k][2 * e], o[4 * k + 1][2 * e], o[4 * k + 2][2 * e], o[4 * k + 3][2 * e]);
                        dst[kD / 32 + k] =
                            make_float4(o[4 * k][2 * e + 1], o[4 * k + 1][2 * e + 1], o[4 * k + 2][2 * e + 1], o[4 * k + 3][2 * e + 1]);
                    }
                }
            } else {                         // the copies in flight land before the block ends
                for (; uses < fills; ++uses) wait_mbar_drain(bars + 8u * (uses % G::kStages), (uses / G::kStages) & 1);
            }
        }
        if (c == 0) {                        // (a warp without tiles has a maximum of -inf)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                warp_ml[warp][g + 8 * e][0] = ok ? m[e] : -INFINITY;
                warp_ml[warp][g + 8 * e][1] = ok ? l[e] : 0.0f;
            }
        }
        __syncwarp();
    }
    // ---- what the kernels before left of these rows
    griddep_wait();                          // (this grid may have run beside those before it)
    const int live = min(max(seq.count * p.group - rt * kRows, 0), kRows);       // rows that are queries
    int4 own = make_int4(0, 0, 0, 0);
    if (!mine) own = __ldcg(p.info + (static_cast<int64_t>(i) * p.Hkv + h) * p.row_tiles + rt);      // (past L1: written meanwhile)
    const bool finished = !mine && start == 0 && own.x == 0;
    if (ok && live > 0 && (start > 0 || !mine) && !finished) {
        const int stacked0 = start > 0 ? shared_rows(p, i - first_of) + rt * kRows : -1;
        RowParts in = {p, static_cast<int64_t>(i) * p.T * p.Hq + h * p.group, rt * kRows, own, mine ? 0 : max(own.x, 1),
                       make_int4(0, 0, 0, 0), make_int4(0, 0, 0, 0), kRows, stacked0};
        if (start > 0) {
            const int4* const records = p.shared_info + static_cast<int64_t>(h) * p.shared_units + shared_unit0(p, place, first_of);
            in.shared0 = __ldcg(records + stacked0 / kWideRows);
            in.shared1 = __ldcg(records + (stacked0 + live - 1) / kWideRows);
            in.cut = kWideRows - stacked0 % kWideRows;
        }
        // (a launch whose waits gave up leaves records unwritten: what they hold is no place to read from)
        auto wrong = [&](const int4& x, int runs) { return x.x < 0 || (x.x > 0 && (x.y < 0 || x.y >= 2 * runs || x.z < 0 || x.x > runs - x.z)); };
        if (wrong(own, p.warps) || wrong(in.shared0, p.wide_runs) || wrong(in.shared1, p.wide_runs)) ok = false;
        else add_parts<kD, kWarps, B::kPitch>(in, live, static_cast<int>(warp), part, warp_ml[warp]);
    }
    ok = !__syncthreads_or(!ok);
    // 16 threads per row, kD / 16 columns each
    constexpr int kCols = kD / 16;
    const int col = static_cast<int>(threadIdx.x & 15u) * kCols;
#pragma unroll 1
    for (int r = static_cast<int>(threadIdx.x >> 4); !finished && ok && r < kRows; r += 2 * kWarps) {
        const int row = rt * kRows + r;
        const int t = row / p.group, head = h * p.group + row % p.group;
        if (t >= p.T) break;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, warp_ml[w][r][0]);
        float l = 0.0f, acc[kCols];
#pragma unroll
        for (int k = 0; k < kCols; ++k) acc[k] = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float mw = warp_ml[w][r][0], lw = warp_ml[w][r][1];
            if (mw > -INFINITY || lw != 0.0f) {  // (a row that a warp's tokens are all hidden from has left zeros)
                const float weight = ex2_approx(mw - m);
                l += lw * weight;
                const float* const src =
                    reinterpret_cast<const float*>(smem + w * G::kWarpBytes) + (r * 4 + col / B::kOwn) * B::kPitch + col % B::kOwn;
#pragma unroll
                for (int k = 0; k < kCols; ++k) acc[k] += src[k] * weight;
            }
        }
        const bool any = r < live && (l > 0.0f || l != l);
        const float mul = any ? 1.0f / l : 0.0f;
        T* const dst = static_cast<T*>(p.o) + b * p.o_stride_b + t * p.o_stride_t + head * p.o_stride_h + col;
#pragma unroll
        for (int k = 0; k < kCols; ++k) dst[k] = from_float<T>(any ? acc[k] * mul : 0.0f);
        if (p.lse != nullptr && col == 0)
            p.lse[(static_cast<int64_t>(b) * p.T + t) * p.Hq + head] = any ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
}

// Adds up what the kernels above left: kSplit warps of a block to a row (eight where there are few rows, of many parts each),
// of which each takes every kSplit-th part. A row's parts are those of its shared unit, then those of its own: the maximum over
// all of them first, then the weighted sums, joined through shared memory in order.
template <int kD, typename T, int kSplit>
__global__ void __launch_bounds__(256)
kv8_shared_combine_kernel(const SharedParams p) {
    constexpr int kVec = kD / 32;            // floats of a lane
    constexpr int kBatch = 4;                // parts whose loads are in flight at a time
    __shared__ float joined[8][kD + 1];
    griddep_launch_dependents();
    griddep_wait();
    const int warp = static_cast<int>(threadIdx.x >> 5), share = warp % kSplit;
    const int64_t out_row = static_cast<int64_t>(blockIdx.x) * (8 / kSplit) + warp / kSplit;
    const int lane = static_cast<int>(lane_id());
    // (with several warps to a row a block has one row or whole rows: they leave together)
    if (out_row >= static_cast<int64_t>(p.n) * p.T * p.Hq) return;
    const int head = static_cast<int>(out_row % p.Hq), t = static_cast<int>(out_row / p.Hq % p.T);
    const int i = static_cast<int>(out_row / p.Hq / p.T), h = head / p.group;
    const int row = t * p.group + head - h * p.group;
    const int4 seq = __ldcg(p.seqs + i);     // (past L1: this grid may have started before the writes)
    const int4 own = __ldcg(p.info + (static_cast<int64_t>(i) * p.Hkv + h) * p.row_tiles + row / kRows);
    int4 shared = make_int4(0, 0, 0, 0);
    int shared_row = 0;
    if (seq.x > 0) {
        shared_row = shared_rows(p, i - seq.z) + row;
        shared = __ldcg(p.shared_info + static_cast<int64_t>(h) * p.shared_units + shared_unit0(p, seq.y, seq.z) + shared_row / kRows);
    } else if (own.x == 0) {
        return;                              // finished
    }
    // (a launch whose waits gave up leaves records unwritten: what they hold is no place to read from)
    auto wrong = [&](const int4& x) { return x.x < 0 || (x.x > 0 && (x.y < 0 || x.y >= 2 * p.warps || x.z < 0 || x.x > p.warps - x.z)); };
    if (wrong(own) || wrong(shared)) return;
    const int first_parts = seq.x > 0 ? max(shared.x, 1) : 0, parts = first_parts + max(own.x, 1);
    auto row_of = [&](int k) {
        const bool of_shared = k < first_parts;
        const int4& x = of_shared ? shared : own;
        const int part = of_shared ? k : k - first_parts;
        if (x.x == 0) return p.whole[of_shared ? 0 : 1] + out_row;
        const int64_t slot = part == 0 ? static_cast<int64_t>(x.y) : 2 * (static_cast<int64_t>(x.z) + part);
        return slot * kRows + (of_shared ? shared_row : row) % kRows;
    };
    float m = -INFINITY, l = 0.0f, acc[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) acc[k] = 0.0f;
    for (int k = lane; k < parts; k += 32) m = fmaxf(m, __ldcg(p.part_ml + 2 * row_of(k)));
#pragma unroll
    for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    for (int k0 = share; k0 < parts; k0 += kBatch * kSplit) {
        float pm[kBatch], pl[kBatch], x[kBatch][kVec];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const int64_t a = row_of(min(k0 + q * kSplit, parts - 1));
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + a);
            pm[q] = ml.x;
            pl[q] = ml.y;
            if constexpr (kVec == 4) {
                const float4 f = __ldcg(reinterpret_cast<const float4*>(p.part_o + a * kD) + lane);
                x[q][0] = f.x; x[q][1] = f.y; x[q][2] = f.z; x[q][3] = f.w;
            } else {
                const float2 f = __ldcg(reinterpret_cast<const float2*>(p.part_o + a * kD) + lane);
                x[q][0] = f.x; x[q][1] = f.y;
            }
        }
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const bool counts = k0 + q * kSplit < parts;
            const float weight = !counts || pm[q] == -INFINITY ? 0.0f : ex2_approx(pm[q] - m);
            l += !counts ? 0.0f : pm[q] == -INFINITY ? pl[q] : pl[q] * weight;       // (a NaN sum stays one)
#pragma unroll
            for (int k = 0; k < kVec; ++k) acc[k] += x[q][k] * weight;
        }
    }
    if constexpr (kSplit > 1) {
#pragma unroll
        for (int k = 0; k < kVec; ++k) joined[warp][lane * kVec + k] = acc[k];
        if (lane == 0) joined[warp][kD] = l;
        named_barrier_sync(1 + warp / kSplit, 32 * kSplit);
        if (share != 0) return;
#pragma unroll
        for (int w = 1; w < kSplit; ++w) {
            l += joined[warp + w][kD];
#pragma unroll
            for (int k = 0; k < kVec; ++k) acc[k] += joined[warp + w][lane * kVec + k];
        }
    }
    const bool any = t < seq.w && (l > 0.0f || l != l);      // (a row past the queries has stacked sums of what lies there)
    const float mul = any ? 1.0f / l : 0.0f;
    T* const dst = static_cast<T*>(p.o) + (p.b0 + i) * p.o_stride_b + t * p.o_stride_t + head * p.o_stride_h + lane * kVec;
#pragma unroll
    for (int k = 0; k < kVec; ++k) dst[k] = from_float<T>(any ? acc[k] * mul : 0.0f);
    if (p.lse != nullptr && lane == 0)
        p.lse[static_cast<int64_t>(p.b0) * p.T * p.Hq + out_row] = any ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace kv8
}  // namespace hk
