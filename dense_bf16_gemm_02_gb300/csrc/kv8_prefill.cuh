// Attention of many query rows over the paged 8-bit cache: a prompt, or a chunk
// of one, against everything the cache holds.
//
// With hundreds of rows per KV head the tensor cores bound the work
// (4 · rows · tokens · D operations against 2 · D bytes per token), so the rows
// run on the attention-forward kernel (attn_kernel.cuh: tcgen05.mma, two
// 128-row query tiles per CTA) with a policy of their own, after one pass that
// brings the sequences' keys and values to bf16, page by page, in the
// workspace. E4M3 times a power of two is exact in bf16, and the pass reads 1
// and writes 2 bytes per element, once for all query heads and rows: at 2048
// rows x 8 heads per KV head under 3 % of the products' time (converting inside
// the kernel would repeat it for every pair of query tiles). 2048 tokens x 64 heads of
// 128 against 16384 tokens x 8 heads: 806 us, 1.28 PFLOP/s, 21 of them the pass.
//
// Rows of a tile are `pack` query heads of one KV head for each of 128 / pack
// tokens, so that the heads of a group share each K/V block that is loaded and a
// tile spans few tokens (its causal edge wastes less).
//
// A value that is NaN would reach every row of a block of 128 tokens through weights of 0,
// so the pass writes 0 in its place and counts the pages with one; a last kernel, which
// otherwise ends at once (1.0 to 1.4 us of a call), then puts NaN into the rows that see
// such a token and takes its pages off the count.
#pragma once

#include <cstdint>

#include "attn_kernel.cuh"
#include "bounded_wait.cuh"
#include "elements.cuh"

namespace hk {
namespace kv8 {

struct PrefillParams : attn::AttnParams {
    const int32_t* lengths;
    const int32_t* counts;         // or null (T)
    int32_t T, room;               // query tokens; most cached tokens of a sequence
    int32_t group;                 // Hq / Hkv
    int32_t pack_shift;            // log2 of the query heads in a tile's rows
    int64_t o_stride_b, o_stride_t, o_stride_h;
};

struct CachedItems {
    using Params = PrefillParams;
    static constexpr bool kEmptyRows = true;

    struct Seq {
        int len, count;
    };
    static __device__ __forceinline__ Seq seq(const Params& p, int b) {
        const int len = p.lengths[b], count = p.counts != nullptr ? p.counts[b] : p.T;
        return Seq{max(0, min(len, p.room)), max(0, min(count, p.T))};
    }

    // K/V blocks that the tokens [tok0, tok0 + 128 / pack) need
    static __device__ __forceinline__ int tile_blocks(const Params& p, const Seq& s, int tok0) {
        if (tok0 >= s.count) return 0;
        const int last = min(tok0 + (attn::kTileQ >> p.pack_shift), s.count) - 1;
        const int end = p.causal ? max(0, s.len - s.count + last + 1) : s.len;
        return (end + attn::kBlockKV - 1) / attn::kBlockKV;
    }

    static __device__ __forceinline__ attn::AttnItem item(const Params& p, int w) {
        attn::AttnItem it;
        const int heads = p.Hq >> p.pack_shift;          // groups of `pack` query heads
        const int bh_count = p.B * heads;
        const int slot_q = w / bh_count;
        it.bh = w - slot_q * bh_count;
        const int qp = p.causal ? p.q_pairs - 1 - slot_q : slot_q;
        const int b = it.bh / heads;
        const int head0 = (it.bh - b * heads) << p.pack_shift;
        it.kvh = b * p.Hkv + head0 / p.group;
        it.q0 = qp * (attn::kTiles * attn::kTileQ);
        const Seq s = seq(p, b);
        it.n_t0 = tile_blocks(p, s, it.q0 >> p.pack_shift);
        it.n_t1 = tile_blocks(p, s, (it.q0 + attn::kTileQ) >> p.pack_shift);
        it.n_all = max(it.n_t0, it.n_t1);
        return it;
    }

    static __device__ __forceinline__ void load_q(const Params& p, uint32_t dst, const void* tmap, const attn::AttnItem& it,
                                                  int t, int c, uint32_t bar) {
        const int heads = p.Hq >> p.pack_shift;
        const int b = it.bh / heads;
        tma_load_4d(dst, tmap, c * 64, (it.bh - b * heads) << p.pack_shift, (it.q0 + t * attn::kTileQ) >> p.pack_shift, b, bar);
    }

    static __device__ __forceinline__ int key_end(const Params& p, const attn::AttnItem& it, int t, int r) {
        const Seq s = seq(p, it.bh / (p.Hq >> p.pack_shift));
        const int tok = (it.q0 + t * attn::kTileQ + r) >> p.pack_shift;
        if (tok >= s.count) return 0;
        return p.causal ? max(0, s.len - s.count + tok + 1) : s.len;
    }

    template <int kD>
    static __device__ __forceinline__ attn::AttnRow row(const Params& p, const attn::AttnItem& it, int t, int r) {
        const int heads = p.Hq >> p.pack_shift;
        const int b = it.bh / heads;
        const int tok = (it.q0 + t * attn::kTileQ + r) >> p.pack_shift;
        const int head = ((it.bh - b * heads) << p.pack_shift) + (r & ((1 << p.pack_shift) - 1));
        return attn::AttnRow{tok < p.T, b * p.o_stride_b + tok * p.o_stride_t + head * p.o_stride_h,
                             (static_cast<int64_t>(b) * p.T + tok) * p.Hq + head};
    }
};

// The status word that counts widened pages (of a head and sequence) with NaN values, of all calls that are between
// the pass and the kernel that takes them off again, on whatever stream. While it is 0 there is nothing to look for.
constexpr int kNanPages = 2;

struct WidenParams {
    const uint8_t* codes[2];       // keys, values
    const float* scale[2];
    uint16_t* out[2];              // bf16 [B, Hkv, rows, D]
    const int32_t* table;
    int64_t table_stride;
    const int32_t* lengths;
    const int32_t* counts;
    int64_t rows;                  // max_pages * page_size
    int64_t num_pages;
    int32_t T, Hkv, D, page_size, max_pages;
    uint32_t* status;
};

// Keys and values of the sequences to bf16; block (page of a sequence, head,
// sequence). Tokens past a sequence's length up to the next multiple of 128
// become 0 (the attention kernel multiplies them by weights of 0).
static __global__ void __launch_bounds__(256)
kv8_widen_kernel(const WidenParams p) {
    const int slot = static_cast<int>(blockIdx.x), h = static_cast<int>(blockIdx.y), b = static_cast<int>(blockIdx.z);
    int len = p.lengths[b];
    if (slot == 0 && h == 0 && threadIdx.x == 0) {
        const int count = p.counts != nullptr ? p.counts[b] : p.T;
        if (len < 0 || len > p.rows || count < 0 || count > p.T) atomicOr(p.status, kErrPage);
    }
    len = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(len), p.rows)));
    const int first = slot * p.page_size;
    if (first >= (len + 127) / 128 * 128) return;
    int64_t page = -1;
    if (first < len) {
        page = p.table[b * p.table_stride + slot];
        if (page < 0 || page >= p.num_pages) {
            if (threadIdx.x == 0) atomicOr(p.status, kErrPage);
            page = -1;
        }
    }
    const int64_t src = (max(page, static_cast<int64_t>(0)) * p.Hkv + h);
    const int64_t dst = (static_cast<int64_t>(b) * p.Hkv + h) * p.rows + first;
    const int chunks = p.page_size * p.D / 16;
    const int chunk_shift = p.D == 128 ? 3 : 2;      // chunks of a token, as a shift
    bool any_nan = false;
    for (int i = static_cast<int>(threadIdx.x); i < 2 * chunks; i += 256) {
        const int kv = i >= chunks ? 1 : 0;
        const int at = i - kv * chunks;
        uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (page >= 0 && first + (at >> chunk_shift) < len) {
            const float s = (kv ? p.scale[1] : p.scale[0])[src];
            const uint4 x = __ldg(reinterpret_cast<const uint4*>((kv ? p.codes[1] : p.codes[0]) + src * p.page_size * p.D) + at);
            uint32_t w[4] = {x.x, x.y, x.z, x.w};
            if (kv == 1) {
                const uint32_t nan[4] = {nan_codes(w[0]), nan_codes(w[1]), nan_codes(w[2]), nan_codes(w[3])};
                if (((nan[0] | nan[1]) | (nan[2] | nan[3])) != 0) {
                    any_nan = true;
#pragma unroll
                    for (int k = 0; k < 4; ++k) w[k] &= ~nan[k];
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                uint32_t f;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)))));
                const __half2 v = *reinterpret_cast<const __half2*>(&f);
                o[k] = pack_bf16x2_rn(__float_as_uint(__low2float(v) * s), __float_as_uint(__high2float(v) * s));
            }
        }
        uint4* const out = reinterpret_cast<uint4*>((kv ? p.out[1] : p.out[0]) + dst * p.D) + 2 * at;
        out[0] = make_uint4(o[0], o[1], o[2], o[3]);
        out[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
    if (__syncthreads_or(any_nan) && threadIdx.x == 0) atomicAdd(p.status + kNanPages, 1u);
}

// After the attention kernel: NaN into every output that a NaN value belongs to; block (head, sequence). The first
// token that holds a NaN, for each dimension, says which rows see one.
static __global__ void __launch_bounds__(256)
kv8_nan_values_kernel(const WidenParams w, const PrefillParams p) {
    // (one thread looks: other blocks may take their pages off meanwhile, and a block goes or stays as a whole)
    if (!__syncthreads_or(threadIdx.x == 0 && *reinterpret_cast<volatile uint32_t*>(w.status + kNanPages) != 0u)) return;
    __shared__ int first[128];
    const int h = static_cast<int>(blockIdx.x), b = static_cast<int>(blockIdx.y);
    const uint32_t warp = threadIdx.x >> 5, lane = lane_id();
    const CachedItems::Seq s = CachedItems::seq(p, b);
    if (threadIdx.x < 128) first[threadIdx.x] = 0x7FFFFFFF;
    __syncthreads();
    const int slots = (s.len + w.page_size - 1) / w.page_size, row_chunks = w.D / 16;
    uint32_t pages = 0;                              // of this warp, with a NaN
    for (int slot = static_cast<int>(warp); slot < slots; slot += 8) {
        const int64_t page = w.table[b * w.table_stride + slot];
        if (page < 0 || page >= w.num_pages) continue;
        const uint4* const codes = reinterpret_cast<const uint4*>(w.codes[1] + (page * w.Hkv + h) * w.page_size * w.D);
        const int chunks = min(w.page_size, s.len - slot * w.page_size) * row_chunks;    // 16 codes each
        bool any = false;
#pragma unroll 4
        for (int i = static_cast<int>(lane); i < chunks; i += 32) {
            const uint4 x = codes[i];
            const uint32_t nan[4] = {nan_codes(x.x), nan_codes(x.y), nan_codes(x.z), nan_codes(x.w)};
            if (((nan[0] | nan[1]) | (nan[2] | nan[3])) == 0) continue;
            any = true;
            for (int k = 0; k < 16; ++k)
                if (nan[k >> 2] >> (8 * (k & 3)) & 1u) atomicMin(&first[i % row_chunks * 16 + k], slot * w.page_size + i / row_chunks);
        }
        pages += __any_sync(0xffffffffu, any) ? 1u : 0u;
    }
    if (lane == 0 && pages > 0) atomicSub(w.status + kNanPages, pages);
    if (!__syncthreads_or(pages > 0)) return;
    const int64_t outputs = static_cast<int64_t>(s.count) * p.group * w.D;
    for (int64_t i = threadIdx.x; i < outputs; i += 256) {
        const int d = static_cast<int>(i % w.D), row = static_cast<int>(i / w.D);
        const int t = row / p.group, head = h * p.group + row % p.group;
        const int end = p.causal ? max(0, s.len - s.count + t + 1) : s.len;
        if (first[d] < end) p.O[b * p.o_stride_b + t * p.o_stride_t + head * p.o_stride_h + d] = 0x7FFFu;
    }
}

}  // namespace kv8
}  // namespace hk
