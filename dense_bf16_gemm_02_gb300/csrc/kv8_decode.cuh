// Attention of a few query rows over a paged cache held in E4M3 (see
// kv8_append.cuh for the cache), for decoding: one or a few new tokens per
// sequence, every cached token read once.
//
//   O[r] = Σ_j P[r,j]·V[j] / Σ_j P[r,j],  P[r,j] = exp(scale · q_r·K[j] - m_r)
//
// What bounds it is reading the cache: 2·D bytes per token and KV head (64
// sequences of 32768 tokens, 8 heads of 128: 640 to 660 us, 6.5 to 6.7 TB/s of the 6.8 that a
// copy reaches; a tile takes a warp 1.36 us when the SM runs eight). A unit
// is 16 query rows (tokens × the query heads of one KV head, padded) of one
// sequence and KV head; a tile is 32 cached tokens of a unit. All tiles of all
// units, in order, are cut into equal runs, one per WARP of a grid that fills
// the GPU once, whatever the lengths of the sequences are. A warp streams its
// run through a ring of its own (TMA loads of code rows, swizzled so that the
// reads below meet no bank twice) and needs no other warp: no block-wide
// barrier, no imbalance between short and long sequences. A unit that lies
// inside one run is finished by its warp; the others leave unnormalised sums
// per run, which a second kernel adds up in order (no atomics: the result does
// not depend on timing).
//
// Arithmetic. mma.sync m16n8k16 with f16 operands and fp32 sums: the tensor
// work is a few per cent of its rate here, so the fragments' layout in
// registers (no staging through Tensor Memory) counts for more than the faster
// unit. Codes become f16 exactly, two per conversion. A query row is scaled by
// a power of two so that its largest magnitude lies in [2^10, 2^11): exact for
// every element down to 2^-24 of that, and the others err by at most 2^-35 of
// it. P is taken times 2^15 and rounded to f16: 11 bits down to 2^-29 of the
// row's largest weight, an absolute 2^-40 of it below (at P <= 1 f16's subnormal
// numbers began at 2^-14, and a tail of many small weights lost its mass while the
// sum counted it). The sum is kept unrounded in fp32. The page's scale multiplies
// the scores of its tokens and, for V and with the 2^-15, the sums of each tile's
// products before they join the running output, all in fp32.
//
// Column orders. A thread's fragment registers need pairs along K: the columns
// of an operand may be in any order as long as both operands agree, so a
// thread takes 16 consecutive codes of a row at a time (one 16-byte read).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <type_traits>

#include "bounded_wait.cuh"
#include "elements.cuh"
#include "ptx.cuh"

namespace hk {
namespace kv8 {

constexpr int kRows = 16;              // query rows of a unit
constexpr int kTileKeys = 32;
constexpr int kDecodeWarps = 4;        // warps of a block, each on its own
constexpr int kMaxBatch = 1024;        // sequences of one launch
constexpr uint32_t kFlagDropArrive = 0x1u; // test only: the first stage of no warp ever counts as filled
constexpr float kWeightShift = 15.0f;  // P is held times 2^15
constexpr float kWeightUnit = 0x1p-15f;

template <int kD>
struct DecodeGeometry {
    static_assert(kD == 64 || kD == 128, "head dimension 64 or 128");
    static constexpr int kHalfBytes = kTileKeys * kD;                 // K or V of a tile
    static constexpr int kStageBytes = 2 * kHalfBytes;
    static constexpr int kStages = kD == 128 ? 3 : 6;                 // 24 KB per warp
    static constexpr int kWarpBytes = kStages * kStageBytes;
    static constexpr int kOffPrefix = kDecodeWarps * kWarpBytes;      // tiles of the sequences up to each one
    static constexpr int kOffBars = kOffPrefix + (kMaxBatch + 1) * 8;
    static constexpr int kSmemBytes = kOffBars + kDecodeWarps * kStages * 8 + 1024;
    static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two blocks per SM");
};

struct DecodeParams {
    const void* q;
    int64_t q_stride_b, q_stride_t, q_stride_h;     // in elements
    void* o;
    int64_t o_stride_b, o_stride_t, o_stride_h;
    float* lse;                                     // [B, T, Hq] or null
    const float* k_scale;
    const float* v_scale;
    const int32_t* table;
    int64_t table_stride;
    const int32_t* lengths;
    const int32_t* counts;                          // query tokens of each sequence, or null (T)
    int32_t B, T, Hq, Hkv, group;                   // group = Hq / Hkv
    int32_t row_tiles;                              // ceil(T * group / 16)
    int32_t page_size, page_shift, max_pages;
    int64_t num_pages;
    int32_t causal, vec_q, vec_o;
    float scale_log2;                               // softmax scale · log2(e)
    int32_t warps;                                  // of kv8_decode_kernel's grid
    uint32_t flags;
    float* part_o;                                  // [2 · warps][16][D]
    float* part_ml;                                 // [2 · warps][16][2]
    int4* info;                                     // [units]: parts whose sums make up the unit (0: it is finished), first slot, first warp
    WaitCtx wait;
};

// Visible tokens of a sequence and its queries, with what is out of range clamped.
struct Sequence {
    int len, count;
};

__device__ __forceinline__ Sequence sequence(const DecodeParams& p, int b) {
    Sequence s;
    s.len = p.lengths[b];
    s.count = p.counts != nullptr ? p.counts[b] : p.T;
    const int64_t room = static_cast<int64_t>(p.max_pages) * p.page_size;
    if (s.len < 0 || s.len > room || s.count < 0 || s.count > p.T) {
        atomicOr(p.wait.status, kErrPage);
        s.len = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(s.len), room)));
        s.count = max(0, min(s.count, p.T));
    }
    return s;
}

// Tokens that the last row of row tile `rt` sees: the tile's runs end there.
__device__ __forceinline__ int row_tile_end(const DecodeParams& p, const Sequence& s, int rt) {
    const int t_first = rt * kRows / p.group;
    if (t_first >= s.count) return 0;
    if (!p.causal) return s.len;
    const int t_last = min((rt * kRows + kRows - 1) / p.group, s.count - 1);
    return max(0, s.len - s.count + t_last + 1);
}

__device__ __forceinline__ int tiles_of(int end) { return max(1, (end + kTileKeys - 1) / kTileKeys); }

__device__ __forceinline__ int sequence_tiles(const DecodeParams& p, const Sequence& s) {
    int n = 0;
    for (int rt = 0; rt < p.row_tiles; ++rt) n += tiles_of(row_tile_end(p, s, rt));
    return n;       // of one KV head
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t pair) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(pair)));
    return h;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

// Byte offset of 16-byte chunk `c` of row `r` in a tile that TMA wrote with
// 128-byte (D = 128) or 64-byte (D = 64) swizzling.
template <int kD>
__device__ __forceinline__ uint32_t chunk_offset(uint32_t r, uint32_t c) {
    return kD == 128 ? r * 128u + ((c ^ (r & 7u)) << 4) : r * 64u + ((c ^ ((r >> 1) & 3u)) << 4);
}

// kCols consecutive values of an output row, 16-byte stores where `vec`.
template <typename T, int kCols>
__device__ __forceinline__ void store_row(T* dst, const float (&v)[kCols], bool vec) {
    if (vec) {
#pragma unroll
        for (int i = 0; i < kCols / 8; ++i)
            reinterpret_cast<uint4*>(dst)[i] =
                make_uint4(pack_pair<T>(v[8 * i], v[8 * i + 1]), pack_pair<T>(v[8 * i + 2], v[8 * i + 3]),
                           pack_pair<T>(v[8 * i + 4], v[8 * i + 5]), pack_pair<T>(v[8 * i + 6], v[8 * i + 7]));
    } else {
#pragma unroll
        for (int i = 0; i < kCols; ++i) dst[i] = from_float<T>(v[i]);
    }
}

// V of a tile of 32 tokens from `key0` on, at `vb`, that not every row sees whole. A weight of 0 does not keep a NaN
// out of a product, so
// * rows past `key_end`, which hold whatever the page holds there, are cleared;
// * NaN codes, where some rows see tokens of the tile that others do not, are cleared, and bit 16 e + j is set in the
//   word of each of this thread's two rows that sees the token (they see `limit0` and `limit1` tokens), for output j
//   of half e of its columns. (Rows that see nothing at all need no care: what is stored for them does not come
//   from the sums. `several`: can rows differ in what they see?)
// Out of line and behind one branch: with a second branch in the loop that calls it every tile took longer (16
// sequences of 8000 tokens with 5 queries 90.7 us for 89.2, one query of 32768 tokens 24.9 for 24.5).
template <int kD>
__device__ __noinline__ uint2 edge_tile(uint32_t vb, int key0, int key_end, int limit0, int limit1, bool several) {
    const uint32_t lane = lane_id(), c = lane & 3u;
    const int from = key_end - key0;
    if (from < kTileKeys) {
        for (int i = static_cast<int>(lane); i < (kTileKeys - from) * (kD / 16); i += 32)
            st_shared_v4(vb + static_cast<uint32_t>(from * kD + 16 * i), 0, 0, 0, 0);   // (whole rows: any order inside)
        fence_proxy_async_smem();            // before a load into the stage may follow
        __syncwarp();
    }
    uint2 found = make_uint2(0, 0);
    const int some = min(limit0 > 0 ? limit0 : key_end, limit1 > 0 ? limit1 : key_end);
    if (!several || __reduce_min_sync(0xffffffffu, some) >= min(key0 + kTileKeys, key_end)) return found;
    // (a lane looks at every 32nd 16 bytes; whole rows, so their order inside does not matter here)
    constexpr int kRowChunks = kD / 16, kPasses = kTileKeys * kRowChunks / 32;
    uint32_t tokens = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const uint4 x = ld_shared_v4(vb + 16 * (lane + 32 * i));
        if (((nan_codes(x.x) | nan_codes(x.y)) | (nan_codes(x.z) | nan_codes(x.w))) != 0)
            tokens |= 1u << ((lane + 32 * i) / kRowChunks);
    }
    const bool nan = tokens != 0;
    tokens = __reduce_or_sync(0xffffffffu, tokens);
    for (; tokens != 0; tokens &= tokens - 1) {
        const int at = __ffs(static_cast<int>(tokens)) - 1;
        uint32_t bits = 0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            uint32_t w[kD / 32];
            if constexpr (kD == 128) {
                const uint4 x = ld_shared_v4(vb + chunk_offset<kD>(at, 2 * c + e));
                w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
            } else {
                const uint2 x = ld_shared_v2(vb + chunk_offset<kD>(at, c) + 8 * e);
                w[0] = x.x; w[1] = x.y;
            }
#pragma unroll
            for (int j = 0; j < kD / 8; ++j) bits |= (nan_codes(w[j >> 2]) >> (8 * (j & 3)) & 1u) << (16 * e + j);
        }
        if (key0 + at < limit0) found.x |= bits;
        if (key0 + at < limit1) found.y |= bits;
    }
    __syncwarp();
    if (nan) {
        for (int i = 0; i < kPasses; ++i) {
            const uint32_t at = vb + 16 * (lane + 32 * i);
            const uint4 x = ld_shared_v4(at);
            st_shared_v4(at, x.x & ~nan_codes(x.x), x.y & ~nan_codes(x.y), x.z & ~nan_codes(x.z), x.w & ~nan_codes(x.w));
        }
        fence_proxy_async_smem();            // before a load into the stage may follow
    }
    __syncwarp();
    return found;
}

// One warp over tiles [first, last) of a unit (16 query rows rt of sequence b,
// KV head h): the unnormalised output, maxima (log2 units) and this thread's
// share of the sums. `ring`, `bars`: the warp's own stages and their barriers.
// False when a wait gave up (the copies in flight are then still to be waited for).
template <int kD, typename T, int kStages>
__device__ __forceinline__ bool attend(const DecodeParams& p, const void* tmap_k, const void* tmap_v, uint32_t ring, uint32_t bars,
                                       int& fills, int& uses, int b, int h, int rt, const Sequence& seq, int key_end, int first,
                                       int last, float (&o)[kD / 8][4], float (&m)[2], float (&l)[2]) {
    constexpr int kWords = kD / 16;          // 4-code words of a row that a thread holds (one K step each)
    constexpr int kNTiles = kD / 8;          // 8-column tiles of the output
    constexpr int kOwn = kD / 4;             // output columns of a thread
    constexpr int kHalfBytes = kTileKeys * kD, kStageBytes = 2 * kHalfBytes;
    const uint32_t lane = lane_id();
    const uint32_t g = lane >> 2, c = lane & 3u;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    bool ok = true;

    // ---- pages and scales of 32 tiles, one tile per lane (two pages where a page is 16 tokens; -1: not a
    // page), for the tiles from `base` on and, once a load runs past them, for the 32 after those
    struct Window {
        int page0, page1;
        float ks0, ks1, vs0, vs1;
    };
    const bool two = p.page_size < kTileKeys;
    auto look_up = [&](Window& w, int tile0) {
        auto page_of = [&](int key) {
            if (key >= key_end) return -1;
            const int32_t pg = p.table[b * p.table_stride + (key >> p.page_shift)];
            if (pg < 0 || pg >= p.num_pages) {
                atomicOr(p.wait.status, kErrPage);
                return -1;
            }
            return static_cast<int>(pg);
        };
        const int key = (tile0 + static_cast<int>(lane)) * kTileKeys;
        w.page0 = page_of(key);
        w.page1 = two ? page_of(key + 16) : w.page0;
    };
    // (no page: scale 0, so that nothing of page 0, read in its place, comes through)
    auto look_up_scales = [&](Window& w) {
        auto scale_of = [&](const float* scale, int pg) {
            return pg >= 0 ? scale[static_cast<int64_t>(pg) * p.Hkv + h] : 0.0f;
        };
        w.ks0 = scale_of(p.k_scale, w.page0);
        w.vs0 = scale_of(p.v_scale, w.page0) * kWeightUnit;
        w.ks1 = two ? scale_of(p.k_scale, w.page1) : w.ks0;
        w.vs1 = two ? scale_of(p.v_scale, w.page1) * kWeightUnit : w.vs0;
    };
    const int seen = key_end > 0 ? last : first;      // a unit that sees nothing has no tile to read
    int base_tile = first, next = first;              // the current window's first tile, the next tile to load
    Window cur = {0, 0, 0.0f, 0.0f, 0.0f, 0.0f}, nxt = cur;
    auto feed = [&]() {
        const int at32 = next - base_tile;
        if (at32 == 32) {
            look_up(nxt, next);
            look_up_scales(nxt);
        }
        const int pg0 = __shfl_sync(0xffffffffu, at32 < 32 ? cur.page0 : nxt.page0, at32 & 31);
        const int pg1 = two ? __shfl_sync(0xffffffffu, at32 < 32 ? cur.page1 : nxt.page1, at32 & 31) : pg0;
        const int s = fills % kStages;
        if (lane == 0) {
            const uint32_t dst = ring + s * kStageBytes;
            mbar_arrive_expect_tx(full_bar(s), kStageBytes);
            const int row = (next * kTileKeys) & (p.page_size - 1);
            const int z0 = max(pg0, 0) * p.Hkv + h, z1 = max(pg1, 0) * p.Hkv + h;
            if (!two) {
                tma_load_3d(dst, tmap_k, 0, row, z0, full_bar(s));
                tma_load_3d(dst + kHalfBytes, tmap_v, 0, row, z0, full_bar(s));
            } else {
                tma_load_3d(dst, tmap_k, 0, 0, z0, full_bar(s));
                tma_load_3d(dst + kHalfBytes / 2, tmap_k, 0, 0, z1, full_bar(s));
                tma_load_3d(dst + kHalfBytes, tmap_v, 0, 0, z0, full_bar(s));
                tma_load_3d(dst + kHalfBytes * 3 / 2, tmap_v, 0, 0, z1, full_bar(s));
            }
        }
        ++fills;
        ++next;
    };
    // the first tiles' loads go out before anything else is waited for
    if (first < seen) {
        look_up(cur, first);
        for (int i = 0; i < kStages && next < seen; ++i) feed();
        look_up_scales(cur);
    }

    // ---- query rows g and g + 8 of the unit: f16 fragments and the factor of their scores
    uint32_t qf[kWords][4];
    float factor[2];
    int limit[2];                        // tokens the row sees
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = rt * kRows + static_cast<int>(g) + 8 * i;
        const int t = row / p.group;
        const bool live = t < seq.count;
        // (rows past T are never stored and need no mask)
        limit[i] = t >= p.T ? 0x7FFFFFFF : !live ? 0 : p.causal ? max(0, seq.len - seq.count + t + 1) : seq.len;
        const T* const src = static_cast<const T*>(p.q) + b * p.q_stride_b + t * p.q_stride_t +
                             static_cast<int64_t>(h * p.group + row % p.group) * p.q_stride_h;
        Raw8<T> rawq[kD / 32];
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < kD / 32; ++k) {
            rawq[k] = load8<T>(src, static_cast<int64_t>(c) * kOwn + 8 * k, live ? kD : 0, p.vec_q != 0);
            float v[8];
            widen8<T>(rawq[k], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7FFFFFFFu);
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^(10 - floor(log2 top)), kept a normal number; 1 for rows of zeros and rows with an infinity or NaN
        int field = 127 + 10 - (static_cast<int>(top >> 23) - 127);
        if (top == 0 || top >= 0x7F800000u) field = 127;
        field = min(max(field, 1), 253);
        const float mul = __uint_as_float(static_cast<uint32_t>(field) << 23);
        factor[i] = __uint_as_float(static_cast<uint32_t>(254 - field) << 23) * p.scale_log2;
#pragma unroll
        for (int k = 0; k < kD / 32; ++k) {
            float v[8];
            widen8<T>(rawq[k], v);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                qf[2 * k + w][i] = pack_f16x2(v[4 * w] * mul, v[4 * w + 1] * mul);
                qf[2 * k + w][2 + i] = pack_f16x2(v[4 * w + 2] * mul, v[4 * w + 3] * mul);
            }
        }
    }
    int all_see = min(limit[0], limit[1]);      // tokens that every row sees: no mask needed below
    all_see = __reduce_min_sync(0xffffffffu, all_see);

#pragma unroll
    for (int j = 0; j < kNTiles; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.0f;
    uint32_t nan_at[2] = {0, 0};             // NaN outputs of rows g and g + 8 (edge_tile)

    for (int tile = first; tile < seen; ++tile) {
        const int s = uses % kStages;
        if (!__all_sync(0xffffffffu, wait_mbar(p.wait, full_bar(s), (uses / kStages) & 1, kErrWaitData))) {
            ok = false;
            break;
        }
        ++uses;
        if (tile - base_tile == 32) {
            cur = nxt;
            base_tile = tile;
        }
        const float tks0 = __shfl_sync(0xffffffffu, cur.ks0, tile - base_tile);
        const float tvs0 = __shfl_sync(0xffffffffu, cur.vs0, tile - base_tile);
        const float tks1 = two ? __shfl_sync(0xffffffffu, cur.ks1, tile - base_tile) : tks0;
        const float tvs1 = two ? __shfl_sync(0xffffffffu, cur.vs1, tile - base_tile) : tvs0;
        const uint32_t kb = ring + s * kStageBytes, vb = kb + kHalfBytes;
        const int key0 = tile * kTileKeys;
        const bool masked = key0 + kTileKeys > all_see;      // (all_see is at most key_end)
        if (masked) {
            const uint2 found = edge_tile<kD>(vb, key0, key_end, limit[0], limit[1], p.T > 1);
            nan_at[0] |= found.x;
            nan_at[1] |= found.y;
        }

        // ---- scores of 32 tokens: key tiles of 8, column g of tile j is token 8 j + g
        // (the four tiles' sums are independent: they go round K step by K step)
        float sc[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.0f;
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
            uint4 x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = ld_shared_v4(kb + chunk_offset<kD>(8u * j + g, (kWords / 4) * c + i));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = 4 * i + e;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t w = e == 0 ? x[j].x : e == 1 ? x[j].y : e == 2 ? x[j].z : x[j].w;
                    mma_f16(sc[j], qf[k][0], qf[k][1], qf[k][2], qf[k][3], e4m3x2_to_f16x2(w & 0xFFFFu), e4m3x2_to_f16x2(w >> 16));
                }
            }
        }
        // ---- softmax of rows g (elements 0, 1) and g + 8 (2, 3); columns 2 c, 2 c + 1 of each tile
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float ks = j < 2 ? tks0 : tks1;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x = sc[j][e] * (factor[e >> 1] * ks);
                if (masked) {
                    const int key = key0 + 8 * j + static_cast<int>(2 * c) + (e & 1);
                    if (key >= limit[e >> 1]) x = -INFINITY;
                }
                sc[j][e] = x;
                mx[e >> 1] = fmaxf(mx[e >> 1], x);
            }
        }
        float alpha[2];
        bool moved = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
            const float now = fmaxf(m[i], mx[i]);
            alpha[i] = now > m[i] ? ex2_approx(m[i] - now) : 1.0f;
            moved = moved || now > m[i];
            m[i] = now;
            l[i] *= alpha[i];
        }
        const float sub0 = m[0] == -INFINITY ? 0.0f : m[0] - kWeightShift, sub1 = m[1] == -INFINITY ? 0.0f : m[1] - kWeightShift;
        uint32_t pf[4][2];               // P · 2^15 of tile j, rows g and g + 8, as f16 pairs
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float p0 = ex2_approx(sc[j][0] - sub0), p1 = ex2_approx(sc[j][1] - sub0);
            const float p2 = ex2_approx(sc[j][2] - sub1), p3 = ex2_approx(sc[j][3] - sub1);
            l[0] += p0 + p1;
            l[1] += p2 + p3;
            pf[j][0] = pack_f16x2(p0, p1);
            pf[j][1] = pack_f16x2(p2, p3);
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int j = 0; j < kNTiles; ++j) {
                o[j][0] *= alpha[0];
                o[j][1] *= alpha[0];
                o[j][2] *= alpha[1];
                o[j][3] *= alpha[1];
            }
        }
        // ---- O += (P·V) · scale: tokens in two steps of 16; column g of output tile j is
        // dimension g · (D / 8) + j, so a thread reads D / 8 consecutive codes of four rows
#pragma unroll
        for (int st = 0; st < 2; ++st) {
            const float vs = st == 0 ? tvs0 : tvs1;
            uint32_t r[4][kD / 32];      // rows 16 st + 2 c, + 1, + 8, + 9
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t row = 16u * st + 2u * c + (i & 1) + (i >> 1) * 8u;
                if constexpr (kD == 128) {
                    const uint4 x = ld_shared_v4(vb + chunk_offset<kD>(row, g));
                    r[i][0] = x.x;
                    r[i][1] = x.y;
                    r[i][2] = x.z;
                    r[i][3] = x.w;
                } else {
                    const uint2 x = ld_shared_v2(vb + chunk_offset<kD>(row, g >> 1) + (g & 1u) * 8u);
                    r[i][0] = x.x;
                    r[i][1] = x.y;
                }
            }
#pragma unroll
            for (int w = 0; w < kD / 32; ++w) {
                const uint32_t a0 = __byte_perm(r[0][w], r[1][w], 0x5140), a1 = __byte_perm(r[0][w], r[1][w], 0x7362);
                const uint32_t b0 = __byte_perm(r[2][w], r[3][w], 0x5140), b1 = __byte_perm(r[2][w], r[3][w], 0x7362);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t lo = e < 2 ? a0 : a1, hi = e < 2 ? b0 : b1;
                    const uint32_t v0 = e & 1 ? lo >> 16 : lo & 0xFFFFu, v1 = e & 1 ? hi >> 16 : hi & 0xFFFFu;
                    float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma_f16(t, pf[2 * st][0], pf[2 * st][1], pf[2 * st + 1][0], pf[2 * st + 1][1], e4m3x2_to_f16x2(v0),
                            e4m3x2_to_f16x2(v1));
                    const int j = 4 * w + e;
#pragma unroll
                    for (int q = 0; q < 4; ++q) o[j][q] = fmaf(t[q], vs, o[j][q]);
                }
            }
        }
        __syncwarp();                    // every lane has read the stage
        if (next < seen) feed();
    }
    if ((nan_at[0] | nan_at[1]) != 0) {
#pragma unroll
        for (int j = 0; j < kNTiles; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (nan_at[e >> 1] >> (16 * (e & 1) + j) & 1u) o[j][e] = NAN;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {            // the rows' sums over their four threads
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        l[i] *= kWeightUnit;
    }
    return ok;
}

template <int kD, typename T>
__global__ void __launch_bounds__(32 * kDecodeWarps, 2)
kv8_decode_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                  const DecodeParams p) {
    using G = DecodeGeometry<kD>;
    constexpr int kNTiles = kD / 8;          // 8-column tiles of the output
    constexpr int kOwn = kD / 4;             // output columns of a thread
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const smem = smem_raw + (base - raw);
    const uint32_t warp = threadIdx.x >> 5, lane = lane_id();
    const uint32_t g = lane >> 2, c = lane & 3u;
    const int self = static_cast<int>(blockIdx.x) * kDecodeWarps + static_cast<int>(warp);

    griddep_launch_dependents();             // the combining kernel may be scheduled; it waits for this grid's end
    if (threadIdx.x == 0) {
        prefetch_tensor_map(&tmap_k);
        prefetch_tensor_map(&tmap_v);
    }

    const uint32_t ring = base + warp * G::kWarpBytes;
    const uint32_t bars = base + G::kOffBars + 8u * warp * G::kStages;
    if (lane == 0) {
        for (int s = 0; s < G::kStages; ++s) mbar_init(bars + 8u * s, s == 0 && (p.flags & kFlagDropArrive) ? 2 : 1);
        fence_mbar_init_cluster();
    }
    griddep_wait();                          // launched early behind the kernel that may have written the cache or q
    // prefix[b]: tiles of the sequences before b, all KV heads
    int64_t* const prefix = reinterpret_cast<int64_t*>(smem + G::kOffPrefix);
    if (warp == 0) {
        int64_t sum = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int b = b0 + static_cast<int>(lane);
            int64_t n = 0;
            if (b < p.B) n = static_cast<int64_t>(sequence_tiles(p, sequence(p, b))) * p.Hkv;
            int64_t inc = n;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int64_t o = __shfl_up_sync(0xffffffffu, inc, d);
                if (static_cast<int>(lane) >= d) inc += o;
            }
            if (b < p.B) prefix[b] = sum + inc - n;
            sum += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) prefix[p.B] = sum;
    }
    __syncthreads();

    const int64_t total = prefix[p.B];
    const int64_t per = (total + p.warps - 1) / p.warps;
    const int64_t begin = min(total, self * per), end = min(total, begin + per);
    bool ok = true;
    int fills = 0, uses = 0;                 // ring stages filled and consumed so far

    // the unit of the run's first tile, and the tile's place in it
    int b = 0, h = 0, rt = 0, first = 0;
    Sequence seq = {0, 0};
    if (begin < end) {
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= begin) lo = mid; else hi = mid - 1;
        }
        b = lo;
        seq = sequence(p, b);
        const int head_tiles = sequence_tiles(p, seq);
        const int64_t local = begin - prefix[b];
        h = static_cast<int>(local / head_tiles);
        first = static_cast<int>(local - static_cast<int64_t>(h) * head_tiles);
        for (int n; first >= (n = tiles_of(row_tile_end(p, seq, rt))); ++rt) first -= n;
    }
    int64_t at = begin;
    while (at < end) {
        const int key_end = row_tile_end(p, seq, rt);
        const int unit_tiles = tiles_of(key_end);
        const int last = static_cast<int>(min(static_cast<int64_t>(unit_tiles), first + (end - at)));   // tiles [first, last)

        float o[kNTiles][4], m[2], l[2];
        ok = attend<kD, T, G::kStages>(p, &tmap_k, &tmap_v, ring, bars, fills, uses, b, h, rt, seq, key_end, first, last, o, m, l);
        if (!ok) break;

        // ---- finish the unit or leave its partial sums
        const bool whole = first == 0 && last == unit_tiles;
        const int slot = 2 * self + (at == begin ? 0 : 1);
        if (first == 0 && lane == 0) {       // this run holds the unit's first tile: it tells how the unit is made up
            const int parts = whole ? 0 : static_cast<int>((at + unit_tiles - 1) / per - at / per + 1);
            p.info[(static_cast<int64_t>(b) * p.Hkv + h) * p.row_tiles + rt] = make_int4(parts, slot, self, 0);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = rt * kRows + static_cast<int>(g) + 8 * i;
            const int t = row / p.group;
            const int head = h * p.group + row % p.group;
            float v[kOwn];
            // columns 2 c and 2 c + 1 of output tile j: dimensions 2 c (D / 8) + j and (2 c + 1)(D / 8) + j
            const bool any = l[i] > 0.0f || l[i] != l[i];        // (a row that sees nothing may hold NaN sums)
            const float mul = !whole ? 1.0f : 1.0f / l[i];
#pragma unroll
            for (int j = 0; j < kNTiles; ++j) {
                v[j] = any ? o[j][2 * i] * mul : 0.0f;
                v[kNTiles + j] = any ? o[j][2 * i + 1] * mul : 0.0f;
            }
            if (whole) {
                if (t < p.T) {
                    T* const dst = static_cast<T*>(p.o) + b * p.o_stride_b + t * p.o_stride_t + head * p.o_stride_h + c * kOwn;
                    store_row<T, kOwn>(dst, v, p.vec_o != 0);
                    if (p.lse != nullptr && c == 0)
                        p.lse[(static_cast<int64_t>(b) * p.T + t) * p.Hq + head] =
                            any ? (m[i] + log2f(l[i])) * 0.69314718055994531f : -INFINITY;
                }
            } else if (t < p.T) {
                const int64_t at_row = static_cast<int64_t>(slot) * kRows + g + 8 * i;
                float4* const dst = reinterpret_cast<float4*>(p.part_o + at_row * kD + c * kOwn);
#pragma unroll
                for (int k = 0; k < kOwn / 4; ++k) dst[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                if (c == 0) {
                    p.part_ml[2 * at_row] = m[i];
                    p.part_ml[2 * at_row + 1] = l[i];
                }
            }
        }
        // the next unit: row tiles innermost, then heads, then sequences (every sequence has tiles)
        at += last - first;
        first = 0;
        if (++rt == p.row_tiles) {
            rt = 0;
            if (++h == p.Hkv) {
                h = 0;
                if (++b < p.B) seq = sequence(p, b);
            }
        }
    }
    // abort: the copies in flight land before the block ends
    if (!ok)
        for (; uses < fills; ++uses) wait_mbar_drain(bars + 8u * (uses % G::kStages), (uses / G::kStages) & 1);
}

// One block, or cluster of blocks, per unit: its kWarps warps (1 to 8, so that an
// SM always holds 8) share the unit's tiles out among them, a block joins its
// warps' sums in shared memory and the blocks of a cluster then join theirs
// through distributed shared memory, each for its share of the rows. For
// sequences that are short, or few: one launch, no pass over lengths before the
// first load, no sums through memory.
constexpr int kBlockWarps = 8;         // warps of an SM; of a block in a cluster
constexpr int kMaxCluster = 16;        // blocks of a cluster

template <int kD, int kWarps>
struct BlockGeometry {
    using G = DecodeGeometry<kD>;
    static constexpr int kOffBars = kWarps * G::kWarpBytes;
    static constexpr int kSmemBytes = kOffBars + kWarps * G::kStages * 8 + 1024;
    // a warp's sums in its ring's place: the columns of a thread 16 bytes apart from the next thread's, so
    // that eight threads' 16-byte stores meet no bank twice
    static constexpr int kOwn = kD / 4;
    static constexpr int kPitch = kOwn + 4;                           // floats
    static constexpr int kSumBytes = kRows * 4 * kPitch * 4;
    // the block's joined sums: [row][D] after the first warp's
    static constexpr int kOffJoined = (kSumBytes + 15) / 16 * 16;
    static_assert(kOffJoined + kRows * kD * 4 <= G::kWarpBytes &&
                      (kSmemBytes + 3 * 1024) * (kBlockWarps / kWarps) <= 228 * 1024, "shared memory");
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

template <int kD, typename T, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, kBlockWarps / kWarps)
kv8_decode_block_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                        const DecodeParams p, const int blocks) {
    using G = DecodeGeometry<kD>;
    using B = BlockGeometry<kD, kWarps>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ float warp_ml[kWarps][kRows][2];
    __shared__ float block_ml[kRows][2];
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
    griddep_wait();                          // launched early behind the kernel that may have written the cache or q
    const int rank = static_cast<int>(blockIdx.x) % blocks;        // the block's place in its cluster
    int unit = static_cast<int>(blockIdx.x) / blocks;
    const int rt = unit % p.row_tiles;
    unit /= p.row_tiles;
    const int h = unit % p.Hkv, b = unit / p.Hkv;
    const Sequence seq = sequence(p, b);
    const int key_end = row_tile_end(p, seq, rt);
    const int tiles = (key_end + kTileKeys - 1) / kTileKeys;
    // tiles to warps, the blocks' first warps before the second ones, so that few tiles meet many SMs
    const int shares = blocks * kWarps, share = static_cast<int>(warp) * blocks + rank;
    const int first = static_cast<int>(static_cast<int64_t>(share) * tiles / shares);
    const int last = static_cast<int>(static_cast<int64_t>(share + 1) * tiles / shares);
    bool ok = true;
    {
        float o[kD / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
        if (first < last) {
            int fills = 0, uses = 0;
            ok = attend<kD, T, G::kStages>(p, &tmap_k, &tmap_v, ring, bars, fills, uses, b, h, rt, seq, key_end, first, last, o, m, l);
            if (ok) {
                float* const part = reinterpret_cast<float*>(smem + warp * G::kWarpBytes);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float4* const dst = reinterpret_cast<float4*>(part + ((g + 8 * i) * 4 + c) * B::kPitch);
#pragma unroll
                    for (int k = 0; k < kD / 32; ++k) {
                        dst[k] = make_float4(o[4 * k][2 * i], o[4 * k + 1][2 * i], o[4 * k + 2][2 * i], o[4 * k + 3][2 * i]);
                        dst[kD / 32 + k] =
                            make_float4(o[4 * k][2 * i + 1], o[4 * k + 1][2 * i + 1], o[4 * k + 2][2 * i + 1], o[4 * k + 3][2 * i + 1]);
                    }
                }
            } else {                         // the copies in flight land before the block ends
                for (; uses < fills; ++uses) wait_mbar_drain(bars + 8u * (uses % G::kStages), (uses / G::kStages) & 1);
            }
        }
        if (c == 0) {                        // (a warp without tiles has a maximum of -inf)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                warp_ml[warp][g + 8 * i][0] = ok ? m[i] : -INFINITY;
                warp_ml[warp][g + 8 * i][1] = ok ? l[i] : 0.0f;
            }
        }
    }
    ok = !__syncthreads_or(!ok);
    // 16 threads per row, kD / 16 columns each
    constexpr int kCols = kD / 16;
    const int col = static_cast<int>(threadIdx.x & 15u) * kCols;
    // (two rows to a warp: one pass with eight warps, as in a cluster)
#pragma unroll 1
    for (int r = static_cast<int>(threadIdx.x >> 4); r < kRows; r += 2 * kWarps) {
        const int row = rt * kRows + r;
        const int t = row / p.group, head = h * p.group + row % p.group;
        if (kWarps < kBlockWarps && t >= p.T) continue;
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
                const float* const part =
                    reinterpret_cast<const float*>(smem + w * G::kWarpBytes) + (r * 4 + col / B::kOwn) * B::kPitch + col % B::kOwn;
#pragma unroll
                for (int k = 0; k < kCols; ++k) acc[k] += part[k] * weight;
            }
        }
        bool mine = true;                        // does this block store this row
        if (kWarps == kBlockWarps && blocks > 1) {
            float* const joined = reinterpret_cast<float*>(smem + B::kOffJoined);
#pragma unroll
            for (int k = 0; k < kCols / 4; ++k)
                reinterpret_cast<float4*>(joined + r * kD + col)[k] = make_float4(acc[4 * k], acc[4 * k + 1], acc[4 * k + 2], acc[4 * k + 3]);
            if (col == 0) {
                block_ml[r][0] = ok ? m : -INFINITY;
                block_ml[r][1] = ok ? l : 0.0f;
            }
            cluster_sync();
            mine = r % blocks == rank;
            if (mine) {
                const uint32_t ml_at = smem_addr(&block_ml[r][0]);
                const uint32_t at = base + B::kOffJoined + static_cast<uint32_t>(r * kD + col) * 4u;
                float ms[kMaxCluster], ls[kMaxCluster];
                m = -INFINITY;
#pragma unroll
                for (int q = 0; q < kMaxCluster; ++q) {
                    ms[q] = -INFINITY;
                    ls[q] = 0.0f;
                    if (q < blocks) {
                        ms[q] = ld_cluster_f32(map_to_cta(ml_at, q));
                        ls[q] = ld_cluster_f32(map_to_cta(ml_at + 4, q));
                    }
                }
#pragma unroll
                for (int q = 0; q < kMaxCluster; ++q) m = fmaxf(m, ms[q]);
                l = 0.0f;
#pragma unroll
                for (int k = 0; k < kCols; ++k) acc[k] = 0.0f;
#pragma unroll
                for (int q0 = 0; q0 < kMaxCluster; q0 += 8) {      // eight blocks' sums in flight
                    float4 x[8][kCols / 4];
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (q0 + q < blocks)
#pragma unroll
                            for (int k = 0; k < kCols / 4; ++k) x[q][k] = ld_cluster_v4(map_to_cta(at + 16 * k, q0 + q));
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        if (q0 + q < blocks && (ms[q0 + q] > -INFINITY || ls[q0 + q] != 0.0f)) {
                            const float weight = ex2_approx(ms[q0 + q] - m);
                            l += ls[q0 + q] * weight;
#pragma unroll
                            for (int k = 0; k < kCols / 4; ++k) {
                                acc[4 * k] += x[q][k].x * weight;
                                acc[4 * k + 1] += x[q][k].y * weight;
                                acc[4 * k + 2] += x[q][k].z * weight;
                                acc[4 * k + 3] += x[q][k].w * weight;
                            }
                        }
                    }
                }
            }
            cluster_sync();                      // no block leaves while another reads its sums
        }
        if (!ok || !mine || t >= p.T) continue;  // (nothing is stored by a block whose wait gave up)
        const bool any = l > 0.0f || l != l;
        const float mul = any ? 1.0f / l : 0.0f;
        T* const dst = static_cast<T*>(p.o) + b * p.o_stride_b + t * p.o_stride_t + head * p.o_stride_h + col;
#pragma unroll
        for (int k = 0; k < kCols; ++k) acc[k] *= mul;
        if (p.vec_o) {
#pragma unroll
            for (int k = 0; k < kCols / 4; ++k)
                reinterpret_cast<uint2*>(dst)[k] =
                    make_uint2(pack_pair<T>(acc[4 * k], acc[4 * k + 1]), pack_pair<T>(acc[4 * k + 2], acc[4 * k + 3]));
        } else {
#pragma unroll
            for (int k = 0; k < kCols; ++k) dst[k] = from_float<T>(acc[k]);
        }
        if (p.lse != nullptr && col == 0)
            p.lse[(static_cast<int64_t>(b) * p.T + t) * p.Hq + head] = any ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
}

// Adds up the partial sums of the units that several warps' runs share: grid
// (unit, rows), kSplit warps to a row, of which each takes every kSplit-th part:
// the row's maximum over the parts first, then the weighted sums, joined through
// shared memory in order. Eight warps to a row where there are few units (of
// many parts each), one where there are many (of few).
template <int kD, typename T, int kSplit>
__global__ void __launch_bounds__(256)
kv8_combine_kernel(const DecodeParams p) {
    constexpr int kVec = kD / 32;            // floats of a lane
    constexpr int kBatch = kSplit > 1 ? 8 : 4;   // parts whose loads are in flight at a time
    __shared__ float joined[8][kD + 1];
    griddep_launch_dependents();
    griddep_wait();
    const int4 info = __ldcg(p.info + blockIdx.x);   // (past L1: this grid may have started before the writes)
    const int parts = info.x;
    if (parts == 0) return;
    // (a launch whose waits gave up leaves records unwritten: what they hold is no place to read from)
    if (parts < 0 || info.y < 0 || info.y >= 2 * p.warps || info.z < 0 || parts > p.warps - info.z) return;
    const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
    int unit = static_cast<int>(blockIdx.x);
    const int rt = unit % p.row_tiles;
    unit /= p.row_tiles;
    const int h = unit % p.Hkv, b = unit / p.Hkv;
    const int r = static_cast<int>(blockIdx.y) * (8 / kSplit) + warp / kSplit, row = rt * kRows + r;
    const int share = warp % kSplit;
    const int t = row / p.group, head = h * p.group + row % p.group;
    const bool live = t < p.T;
    // part i of the unit: the leader's slot, then the first slot of each warp that follows
    auto row_of = [&](int i) {
        const int64_t slot = i == 0 ? info.y : 2 * (static_cast<int64_t>(info.z) + i);
        return slot * kRows + r;
    };
    float m = -INFINITY, l = 0.0f, acc[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) acc[k] = 0.0f;
    if (live) {
        // (every warp of a row looks at all its maxima)
        for (int i0 = 0; i0 < parts; i0 += 256) {
            float x[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = __ldcg(p.part_ml + 2 * row_of(min(i0 + 32 * q + lane, parts - 1)));
#pragma unroll
            for (int q = 0; q < 8; ++q) m = fmaxf(m, x[q]);
        }
#pragma unroll
        for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        // up to kN parts, their loads in flight together: no test or branch between them, which would take them
        // one at a time (past the last part it is loaded again and not counted)
        auto batch = [&](int i0, auto size) {
            constexpr int kN = decltype(size)::value;
            float pm[kN], pl[kN], x[kN][kVec];
#pragma unroll
            for (int q = 0; q < kN; ++q) {
                const int64_t a = row_of(min(i0 + kSplit * q, parts - 1));
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
            for (int q = 0; q < kN; ++q) {
                const bool counts = i0 + kSplit * q < parts;
                const float weight = !counts || pm[q] == -INFINITY ? 0.0f : ex2_approx(pm[q] - m);
                l += !counts ? 0.0f : pm[q] == -INFINITY ? pl[q] : pl[q] * weight;       // (a NaN sum stays one)
#pragma unroll
                for (int k = 0; k < kVec; ++k) acc[k] += x[q][k] * weight;
            }
        };
        int i0 = share;
        for (; i0 + kSplit * 2 < parts; i0 += kSplit * kBatch) batch(i0, std::integral_constant<int, kBatch>{});
        if (i0 < parts) batch(i0, std::integral_constant<int, 2>{});
    }
    if constexpr (kSplit > 1) {
#pragma unroll
        for (int k = 0; k < kVec; ++k) joined[warp][lane * kVec + k] = acc[k];
        if (lane == 0) joined[warp][kD] = l;
        __syncthreads();
        if (share != 0) return;
#pragma unroll
        for (int w = 1; w < kSplit; ++w) {
            l += joined[warp + w][kD];
#pragma unroll
            for (int k = 0; k < kVec; ++k) acc[k] += joined[warp + w][lane * kVec + k];
        }
    }
    if (!live) return;
    const bool any = l > 0.0f || l != l;
    const float mul = any ? 1.0f / l : 0.0f;
    T* const dst = static_cast<T*>(p.o) + b * p.o_stride_b + t * p.o_stride_t + head * p.o_stride_h + lane * kVec;
#pragma unroll
    for (int k = 0; k < kVec; ++k) dst[k] = from_float<T>(acc[k] * mul);
    if (p.lse != nullptr && lane == 0)
        p.lse[(static_cast<int64_t>(b) * p.T + t) * p.Hq + head] = any ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace kv8
}  // namespace hk
