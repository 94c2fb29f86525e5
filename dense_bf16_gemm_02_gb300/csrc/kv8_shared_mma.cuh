// The shared part of kv8_shared.cuh for many query rows, on the fifth-generation tensor cores.
//
// With 64 sequences of 8 query heads per KV head a shared token meets 512 rows: 4 · 512 · D
// operations for 2 · D bytes, so the tensor cores bound the work and mma.sync with 16 rows
// to a unit (each of which converts every tile again) is the wrong tool. Here a unit is 128 stacked rows
// of a group and KV head: S = Q·Kᵀ (two buffers) and O += P·V in Tensor Memory on tcgen05.mma, P and
// Q in Tensor Memory too (shared memory is what MMAs and conversion wait for). All units' blocks of
// 128 tokens, in order, are cut into equal runs, one per CTA, since a prefix has few units and many blocks: each run
// leaves unnormalised rows, maxima and sums of its units in memory, which kv8_own_kernel adds up.
//
// A CTA: two producing warps stream the codes of K and V page by page (TMA) into a ring; eight
// converting warps write them, as the 128-byte-swizzled f16 rows that the MMAs read, into a second one; one thread
// issues the MMAs; a softmax warpgroup has a thread to a row, as in attn_kernel.cuh. Conversion competes
// with the softmax for the same pipes, so it is kept short: codes become f16, two per
// conversion instruction and exactly, and are met by queries in f16: a row is scaled by a power
// of two as in kv8_decode.cuh (exact down to 2^-24 of its largest element). The pages'
// scales do not touch the keys: a chain of the row's maximum is 16 columns, a page at least,
// and takes the scale as a whole, and the exponential's multiply-add has it as its factor. Those of the
// values, powers of two, become factors within a block: O is in units of the largest scale of values that the
// unit's run has seen, and a page's values are multiplied by what its scale is of it, down to 2^-14, exactly. Blocks with
// pages below that, or 2^7 above the first block's unit, have values and weights in bf16 (each code's bits
// moved to where bf16 has them, times 2^120, which E4M3's exponent bias is less): f16 weights hold down to 2^-31 of the largest, and
// values that are much larger than others would make what lies below count. They have their 11 bits down to 2^-21 of it (kv8_decode.cuh,
// whose maximum is never behind: 2^-29), since a maximum that may be 2^8 behind leaves 2^7 for the shift: with 2^4 and 2^11, which would
// hold 2^-25, 64 sequences behind 16384 tokens take 75 us (75) and 128 behind 32768 207 (205), with 2^2 and 2^13 77 and 210.
// At the launch's 128 registers a thread the compiler spills 46 bytes.
//
// Measured: 56 us for 64 sequences of 64 query heads (8 KV heads of 128) behind 16384 tokens, 153 us for 128 behind 32768
// (898 TFLOP/s, 0.47 of the 1917 measured for large GEMMs; tensor pipe 37 % busy, DRAM 6 %): some 2300 cycles for a
// block of 128 x 128, of which the MMAs take 1080, and some 20 us to start, fill and drain. With conversions, exponentials,
// packing and maxima all left out it is 1950, with the MMAs too 1800: what is left is the chain from S through the softmax's loads and
// stores of Tensor Memory to P·V. One producing warp, which waited for each look-up of pages, bound it at 2900. What was tried (us of a
// call, 64 behind 16384 and 128 behind 32768, with 77 and 208 as it is): two threads to a row, which tell
// each other their maxima 81 and 216; converting warps of K and V apart, with rings of their own 82 and 211; every
// code loaded before the first one is converted 80 and 214. Two tiles of 128 rows to a unit (so that a block is converted once for 256)
// took 10000 cycles a block: Q and P of two tiles leave shared memory for two blocks in each ring, too few to hide a
// load and a conversion.
#pragma once

#include <type_traits>

#include "attn_kernel.cuh"
#include "kv8_shared.cuh"

namespace hk {
namespace kv8 {

constexpr int kWideGroups = 64;        // groups of a call on this form
constexpr int kWideBlock = 128;        // tokens of a block
constexpr int kWideThreads = 512;
constexpr int kWideIssueWarp = 4, kWideLoadWarp = 5, kWideConvertWarp = 8;      // after four softmax warps; two load, eight convert
constexpr int kConvertThreads = 256;
constexpr int kSoftmaxRegs = 216, kConvertRegs = 96, kIssueRegs = 104;
constexpr int kWideRegisters = 128 * kSoftmaxRegs + 256 * kConvertRegs + 128 * kIssueRegs;
static_assert(kWideRegisters <= kWideThreads * 128, "registers of the launch");
constexpr float kWideShift = 7.0f;      // weights are 2^7 times what the running maximum makes them (2^15 at most): f16 holds them down to 2^-31
constexpr uint32_t kErrSoftmaxWait = 1u << 19;

template <int kD>
struct WideGeometry {
    static constexpr int kChunkBytes = 128 * 128;                             // 128 rows of 64 16-bit elements
    static constexpr int kTileBytes = kD / 64 * kChunkBytes;                  // a block of K or V
    static constexpr int kSlots = kD == 128 ? 4 : 6;                          // K and V blocks in 16 bits
    static constexpr int kRaw = kD == 128 ? 6 : 8;                            // and as codes
    static constexpr int kRawBytes = kWideBlock * kD;
    static constexpr int kOffKV = 0;
    static constexpr int kOffRaw = kOffKV + kSlots * kTileBytes;
    static constexpr int kOffBars = kOffRaw + kRaw * kRawBytes;
    // q_full, q_empty, p_full, o_done, s_full[2], s_free[2], kv_full and kv_empty of the slots, raw_full and raw_empty
    static constexpr int kNumBars = 8 + 2 * kSlots + 2 * kRaw;
    // factors of the values of 16 tokens each: [kRaw][8] pairs, and whether they are f16
    static constexpr int kFactorBytes = 9 * 4;
    static constexpr int kOffFactors = kOffBars + kNumBars * 8;
    // of the last kScales blocks (no role is so far ahead of the softmax): scales of the keys of 16 tokens each; whether the values
    // are f16, what O is multiplied by before the block, and the unit of O
    static constexpr int kScales = 16, kScaleBytes = 48;
    static constexpr int kOffScales = (kOffFactors + kRaw * kFactorBytes + 15) / 16 * 16;         // (read 16 bytes at a time)
    static_assert(3 + (kSlots + kRaw + 1) / 2 < kScales, "blocks ahead of the softmax");
    static constexpr int kOffTmemHolder = kOffScales + kScales * kScaleBytes;
    static constexpr int kOffPlan = kOffTmemHolder + 16;                      // blocks, first sequence, blocks of each group
    static constexpr int kSmemBytes = kOffPlan + (3 * kWideGroups + 2) * 4 + 1024;
    static_assert(kSmemBytes <= attn::kSmemLimit, "shared memory");
    static_assert(kOffRaw % 1024 == 0 && kOffKV % 1024 == 0 && kOffBars % 8 == 0 && kOffFactors % 4 == 0 && kOffScales % 16 == 0, "alignment");
    // TMEM columns: O (kD), S_0, S_1 (128 each), P (64: two bf16 per column), Q (kD / 2: two f16 per column)
    static constexpr int kColO = 0, kColS = 128, kColP = 384, kColQ = 448, kTmemCols = 512;
    static_assert(kColQ + kD / 2 <= kTmemCols, "TMEM");
    static constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128) & ~((7u << 7) | (7u << 10));     // A and B f16
    static constexpr uint32_t kIdescPVWide = idesc_bf16_f32(128, kD) | (1u << 16);                // B (V) MN-major
    static constexpr uint32_t kIdescPV = kIdescPVWide & ~((7u << 7) | (7u << 10));                // A and B f16
};

// A run's share of a unit: blocks [first, last) of `blocks` for rows from `row0` on.
struct WidePiece {
    int section, h, tile, first, last, blocks;
    Group group;
    bool valid;
};

// Walks a run of blocks [at, end) through the units.
struct WideWalk {
    const SharedParams& p;
    const int32_t* prefix;     // blocks before each group
    const int32_t* first_of;
    const int32_t* blocks_of;
    int at, end, section;

    __device__ __forceinline__ WidePiece next() {
        WidePiece w;
        w.valid = at < end;
        if (!w.valid) return w;
        while (prefix[section + 1] <= at) ++section;
        w.section = section;
        w.blocks = blocks_of[section];
        const int first = max(first_of[section], p.b0), last_seq = min(first_of[section + 1], p.b0 + p.n);
        w.group = Group{first - p.b0, max(0, last_seq - first), w.blocks * (kSharedStep / kTileKeys)};
        const int tiles = (shared_rows(p, w.group.n) + kWideRows - 1) / kWideRows;
        int local = at - prefix[section];
        const int unit = local / w.blocks;
        w.first = local - unit * w.blocks;
        w.h = unit / tiles;
        w.tile = unit - w.h * tiles;
        w.last = min(w.blocks, w.first + end - at);
        at += w.last - w.first;
        return w;
    }
};

// a · b, of two bf16 each.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Four codes to bf16 times `factor` / 2^120, in two words of two.
__device__ __forceinline__ uint2 codes_to_bf16(uint32_t w, uint32_t factor) {
    // each code in a low byte, four bits up (its exponent then ends at bit 10, where bf16's lowest four exponent bits do), and the
    // sign from bit 11 to bit 15: x + 15 (x & 0x800). Half of it multiply-adds, which leaves the logic pipe free
    const uint32_t l0 = __byte_perm(w, 0u, 0x4140) * 16u, l1 = __byte_perm(w, 0u, 0x4342) * 16u;
    const uint32_t a = (l0 & 0x08000800u) * 15u + l0, b = (l1 & 0x08000800u) * 15u + l1;
    return make_uint2(mul_bf16x2(a, factor), mul_bf16x2(b, factor));
}

// bf16 NaN (0x7FFF) in the places of two NaN codes, the low ones of `nan` (0xFF each).
__device__ __forceinline__ uint32_t nan_pair(uint32_t nan) { return __byte_perm(nan, 0u, 0x1100) & 0x7FFF7FFFu; }

// Bounded waits without a call: a kernel that splits its registers may make none. Those on the chain of S, softmax and P·V
// poll; the others let the hardware suspend them.
template <bool kSuspend>
__device__ __forceinline__ bool wide_wait(const WaitCtx& c, uint32_t bar, uint32_t parity, uint32_t code) {
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        if (kSuspend ? mbar_try_wait_suspend(bar, parity, 20000) : mbar_test_wait(bar, parity)) return true;
        if (kSuspend || (it & 4095u) == 0) {
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            if (wait_aborted(c)) return false;
            if (now - t0 > c.timeout_ns) {
                atomicOr(c.status, code);
                atomicExch(c.status + 1, c.launch_id);
                __threadfence();
                return false;
            }
        }
    }
}

template <int kD, typename T>
__global__ void __launch_bounds__(kWideThreads, 1)
kv8_shared_mma_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v, const SharedParams p) {
    using W = WideGeometry<kD>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const smem = smem_raw + (base - raw);
    const uint32_t warp = threadIdx.x >> 5;
    const uint32_t lane = lane_id();

    auto bar = [&](int i) { return base + W::kOffBars + 8u * static_cast<uint32_t>(i); };
    const uint32_t q_full = bar(0), q_empty = bar(1), p_full = bar(2), o_done = bar(3);
    auto s_full = [&](int i) { return bar(4 + i); };
    auto s_free = [&](int i) { return bar(6 + i); };
    auto kv_full = [&](int s) { return bar(8 + s); };
    auto kv_empty = [&](int s) { return bar(8 + W::kSlots + s); };
    auto raw_full = [&](int s) { return bar(8 + 2 * W::kSlots + s); };
    auto raw_empty = [&](int s) { return bar(8 + 2 * W::kSlots + W::kRaw + s); };
    auto slot_addr = [&](int s) { return base + W::kOffKV + static_cast<uint32_t>(s) * W::kTileBytes; };
    auto raw_addr = [&](int s) { return base + W::kOffRaw + static_cast<uint32_t>(s) * W::kRawBytes; };
    auto factor_addr = [&](int s) { return base + W::kOffFactors + static_cast<uint32_t>(s) * W::kFactorBytes; };
    auto scales_addr = [&](int block) { return base + W::kOffScales + static_cast<uint32_t>(block % W::kScales * W::kScaleBytes); };
    const uint32_t tmem_holder = base + W::kOffTmemHolder;
    int32_t* const prefix = reinterpret_cast<int32_t*>(smem + W::kOffPlan);
    int32_t* const first_of = prefix + kWideGroups + 1;
    int32_t* const blocks_of = first_of + kWideGroups + 1;

    if (threadIdx.x == 0) {
        mbar_init(q_full, 128);
        mbar_init(q_empty, 1);                 // the last S of the piece is done
        mbar_init(p_full, 128);
        mbar_init(o_done, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full(i), 1);
            mbar_init(s_free(i), 128);
        }
        for (int s = 0; s < W::kSlots; ++s) {
            mbar_init(kv_full(s), kConvertThreads / 32);
            mbar_init(kv_empty(s), 1);
        }
        for (int s = 0; s < W::kRaw; ++s) {
            mbar_init(raw_full(s), s == 0 && (p.flags & kFlagDropArrive) ? 2 : 1);
            mbar_init(raw_empty(s), kConvertThreads / 32);
        }
        fence_mbar_init_cluster();
    }
    if (threadIdx.x == 32) {
        prefetch_tensor_map(&tmap_k);
        prefetch_tensor_map(&tmap_v);
    }
    if (warp == kWideIssueWarp) {
        tmem_alloc_one(tmem_holder, W::kTmemCols);
        tmem_relinquish_one();
    }
    griddep_wait();                            // launched early behind the spreading kernel, which waits for what wrote the cache or q
    griddep_launch_dependents();               // (now: what follows on the stream may run beside this grid, see launch())
    // ---- the groups' blocks; the CTA's run
    {
        bool bad = false;        // (what is out of order the spreading kernel reports)
        static_assert(kWideGroups < kWideThreads, "a thread to a group");
        const int j = static_cast<int>(threadIdx.x);
        if (j <= p.G) {
            const int first = p.groups[j];
            first_of[j] = first;
            if (j < p.G) {
                const int shared = p.shared[j];
                bad = !group_in_order(p, j, first, p.groups[j + 1], shared);
                blocks_of[j] = bad ? 0 : shared_tiles(p, shared, p.lengths[first]) / (kSharedStep / kTileKeys);
            } else {
                bad = first != p.all;
            }
        }
        if (__syncthreads_or(bad)) {
            if (j < p.G) blocks_of[j] = 0;
            __syncthreads();
        }
        if (warp == 0) {
            int sum = 0;
            for (int j0 = 0; j0 < p.G; j0 += 32) {
                const int j = j0 + static_cast<int>(lane);
                int inc = 0;
                if (j < p.G && blocks_of[j] > 0) {
                    const int first = max(first_of[j], p.b0), last = min(first_of[j + 1], p.b0 + p.n);
                    inc = (shared_rows(p, max(0, last - first)) + kWideRows - 1) / kWideRows * blocks_of[j] * p.Hkv;
                }
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const int o = __shfl_up_sync(0xffffffffu, inc, d);
                    if (static_cast<int>(lane) >= d) inc += o;
                }
                if (j < p.G) prefix[j + 1] = sum + inc;
                sum += __shfl_sync(0xffffffffu, inc, 31);
            }
            if (lane == 0) prefix[0] = 0;
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(smem + W::kOffTmemHolder);
    const int ctas = static_cast<int>(gridDim.x), self = static_cast<int>(blockIdx.x);
    const int total = prefix[p.G], per = (total + ctas - 1) / ctas;
    WideWalk walk{p, prefix, first_of, blocks_of, 0, 0, 0};
    walk.at = static_cast<int>(min(static_cast<int64_t>(total), static_cast<int64_t>(self) * per));
    walk.end = static_cast<int>(min(static_cast<int64_t>(total), static_cast<int64_t>(walk.at) + per));
    const int begin = walk.at;
    bool abort_seen = false;
    // a warp's waits
    auto wait_warp = [&](uint32_t b, uint32_t parity, uint32_t code, auto suspend) {
        return __all_sync(0xffffffffu, wide_wait<decltype(suspend)::value>(p.wait, b, parity, code)) != 0;
    };
    constexpr std::integral_constant<bool, false> poll{};
    constexpr std::integral_constant<bool, true> suspend{};
    // position u of the order in which n blocks' K and V are used: K_0, (K_{j+1}, V_j)..., V_{n-1}
    auto block_at = [](int u, int n, bool& is_k) {
        is_k = u == 0 || ((u & 1) != 0 && u < 2 * n - 1);
        return u == 2 * n - 1 ? n - 1 : is_k ? (u + 1) / 2 : u / 2 - 1;
    };

    if (warp >= kWideConvertWarp) {
        // ------------------------------------------------ converting warps --
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvertRegs));
        constexpr int kTokenChunks = kD / 16;                          // 16-code pieces of a token
        constexpr int kPieces = kWideBlock * kTokenChunks / kConvertThreads;
        constexpr int kStepTokens = kConvertThreads / kTokenChunks;    // tokens between a thread's pieces
        const int ct = static_cast<int>(threadIdx.x) - kWideConvertWarp * 32;
        // eight threads whose 16-byte stores go together take 64 columns of two tokens, so that they meet no bank twice
        constexpr int kHalves = kD / 64;
        const uint32_t half = ct / 8 % kHalves, chunk = 4 * half + ct % 4, token = ct / (8 * kHalves) * 2 + ct / 4 % 2;
        int slot = 0, rs = 0;
        uint32_t ring_ph = 0, raw_ph = 0;
        // 16 columns of row `tok`: two 16-byte units of the 64-column half that they lie in
        auto put = [&](uint32_t tok, const uint32_t (&o)[8]) {
            const uint32_t row = slot_addr(slot) + half * W::kChunkBytes + tok * 128u, unit = 2u * (chunk & 3u), sw = tok & 7u;
            st_shared_v4(row + ((unit ^ sw) << 4), o[0], o[1], o[2], o[3]);
            st_shared_v4(row + (((unit + 1u) ^ sw) << 4), o[4], o[5], o[6], o[7]);
        };
        for (WidePiece w = walk.next(); w.valid && !abort_seen; w = walk.next()) {
            const int n = w.last - w.first;
            for (int u = 0; u < 2 * n; ++u) {
                bool is_k;
                block_at(u, n, is_k);
                if (!wait_warp(raw_full(rs), raw_ph, kErrWaitData, poll) || !wait_warp(kv_empty(slot), ring_ph ^ 1u, kErrWaitRing, poll)) {
                    abort_seen = true;
                    break;
                }
                if (is_k) {
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        const uint32_t tok = token + i * kStepTokens;
                        const uint4 x = ld_shared_v4(raw_addr(rs) + chunk_offset<kD>(tok, chunk));
                        const uint32_t words[4] = {x.x, x.y, x.z, x.w};
                        uint32_t o[8];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            o[2 * k] = e4m3x2_to_f16x2(words[k] & 0xFFFFu);
                            o[2 * k + 1] = e4m3x2_to_f16x2(words[k] >> 16);
                        }
                        put(tok, o);
                    }
                } else {
                    uint32_t half_values;
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(half_values) : "r"(factor_addr(rs) + 32u));
                    auto codes_of = [&](uint32_t tok) { return ld_shared_v4(raw_addr(rs) + chunk_offset<kD>(tok, chunk)); };
                    auto factor_of = [&](uint32_t tok) {
                        uint32_t factor;
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(factor) : "r"(factor_addr(rs) + 4u * (tok >> 4)));
                        return factor;
                    };
                    if (half_values != 0) {
#pragma unroll
                        for (int i = 0; i < kPieces; ++i) {
                            const uint32_t tok = token + i * kStepTokens, factor = factor_of(tok);
                            const uint4 x = codes_of(tok);
                            const uint32_t words[4] = {x.x, x.y, x.z, x.w};
                            uint32_t o[8];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                o[2 * k] = mul_f16x2(e4m3x2_to_f16x2(words[k] & 0xFFFFu), factor);
                                o[2 * k + 1] = mul_f16x2(e4m3x2_to_f16x2(words[k] >> 16), factor);
                            }
                            put(tok, o);
                        }
                    } else {
#pragma unroll 1
                        for (int i = 0; i < kPieces; ++i) {
                            const uint32_t tok = token + i * kStepTokens, factor = factor_of(tok);
                            const uint4 x = codes_of(tok);
                            const uint32_t words[4] = {x.x, x.y, x.z, x.w};
                            uint32_t o[8];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint2 v = codes_to_bf16(words[k], factor);
                                const uint32_t nan = nan_codes(words[k]);
                                o[2 * k] = v.x | nan_pair(nan);
                                o[2 * k + 1] = v.y | nan_pair(nan >> 16);
                            }
                            put(tok, o);
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(kv_full(slot));
                    mbar_arrive(raw_empty(rs));
                }
                if (++slot == W::kSlots) {
                    slot = 0;
                    ring_ph ^= 1u;
                }
                if (++rs == W::kRaw) {
                    rs = 0;
                    raw_ph ^= 1u;
                }
            }
        }
    } else if (warp >= kWideIssueWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == kWideLoadWarp || warp == kWideLoadWarp + 1) {
            // ------------------------------------- producing warps: one for K, one for V --
            const bool of_k = warp == kWideLoadWarp;
            int rs = 0, key_block = 0;
            uint32_t raw_ph = 0;
            const int boxes = kWideBlock >> p.page_shift;                // pages of a block
            for (WidePiece w = walk.next(); w.valid && !abort_seen; w = walk.next()) {
                const int32_t* const table = p.table + first_of[w.section] * p.table_stride;
                // pages (as rows of the tensor map) and scales of the 32 pieces of 16 tokens of blocks [window, window + 4), one
                // per lane; those of the next four blocks, whose loads are then under way, and the pages of the four after them
                struct Window {
                    int row;
                    float ks;
                    uint32_t vs;           // V's scale, a power of two
                };
                auto page_of = [&](int block) {
                    const int key = block * kWideBlock + static_cast<int>(lane) * 16;
                    return key < w.blocks * kWideBlock ? table[key >> p.page_shift] : 0;
                };
                auto look_up = [&](int pg) {
                    const bool good = pg >= 0 && pg < p.num_pages;
                    if (!good) atomicOr(p.wait.status, kErrPage);        // (scale 0: nothing of page 0, read in its place, comes through)
                    const int64_t ph = static_cast<int64_t>(good ? pg : 0) * p.Hkv + w.h;
                    return Window{static_cast<int>(ph), good && of_k ? p.k_scale[ph] : 0.0f, good ? __float_as_uint(p.v_scale[ph]) : 0u};
                };
                int window = w.first;
                int page = page_of(window), page_ahead = page_of(window + 4);
                Window cur = look_up(page), ahead = look_up(page_ahead);
                page = page_of(window + 8);
                // the unit of O from each block on, as an exponent field: the largest scale of values so far; and whether the block's
                // values are f16 in it
                uint32_t unit = 1, unit_first = 0;
                const int n = w.last - w.first;
                for (int u = 0; u < 2 * n; ++u) {
                    bool is_k;
                    const int block = w.first + block_at(u, n, is_k);
                    if (is_k == of_k) {
                        if (block >= window + 4) {
                            window += 4;
                            cur = ahead;
                            ahead = look_up(page);
                            page = page_of(window + 8);
                        }
                        const int at = (block - window) * 8;
                        if (!wait_warp(raw_empty(rs), raw_ph ^ 1u, kErrWaitRing, suspend)) {
                            abort_seen = true;
                            break;
                        }
                        // (the copies go out before the scales are waited for; the barrier's one arrival, which says what to expect, after)
                        const int row = __shfl_sync(0xffffffffu, cur.row, at + (static_cast<int>(lane) % boxes << p.page_shift >> 4));
                        if (static_cast<int>(lane) < boxes)
                            tma_load_3d(raw_addr(rs) + (lane << p.page_shift) * kD, is_k ? &tmap_k : &tmap_v, 0, 0, row, raw_full(rs));
                        const uint32_t vs = __shfl_sync(0xffffffffu, cur.vs, at + (lane & 7u)) >> 23 & 0xFFu;
                        const uint32_t unit_before = unit;
                        unit = max(unit, __reduce_max_sync(0xffffffffu, vs));
                        if (unit_first == 0) unit_first = unit;
                        // (2^-14 times the smallest code is two of f16's smallest steps; and weights that f16 does not
                        // hold are to matter nowhere, which much larger values than those before would make them)
                        const bool half_values = __all_sync(0xffffffffu, vs == 0 || vs + 14u >= unit) != 0 && unit <= unit_first + 7u;
                        if (is_k) {
                            const float ks = __shfl_sync(0xffffffffu, cur.ks, at + (lane & 7u));
                            if (lane < 8) asm volatile("st.shared.f32 [%0], %1;" ::"r"(scales_addr(key_block) + 4u * lane), "f"(ks) : "memory");
                            if (lane == 0)
                                st_shared_v4(scales_addr(key_block) + 32u, half_values ? 1u : 0u,
                                             unit - unit_before < 127u ? 127u - (unit - unit_before) << 23 : 0u, unit << 23, 0u);
                            ++key_block;
                        } else {
                            // 2^(scale - unit), in bf16 times 2^120 (no scale: 0)
                            const uint32_t below = unit - vs;
                            const uint32_t f = vs == 0 ? 0u : half_values ? (15u - below) << 10 : below < 247u ? (247u - below) << 7 : 0u;
                            if (lane < 8)
                                asm volatile("st.shared.b32 [%0], %1;" ::"r"(factor_addr(rs) + 4u * lane), "r"(f | f << 16) : "memory");
                            if (lane == 0) asm volatile("st.shared.b32 [%0], %1;" ::"r"(factor_addr(rs) + 32u), "r"(half_values ? 1u : 0u) : "memory");
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive_expect_tx(raw_full(rs), W::kRawBytes);
                    }
                    if (++rs == W::kRaw) {
                        rs = 0;
                        raw_ph ^= 1u;
                    }
                }
            }
        }
        // ------------------------------------------- MMA issue --
        // (the warp as a whole, one elected lane issuing: descriptors then stay in uniform registers)
        if (warp == kWideIssueWarp) {
            int slot = 0;
            uint32_t ring_ph = 0;
            // waits for the next position's block in 16 bits; its slot
            auto take = [&](int& at) {
                if (!wait_warp(kv_full(slot), ring_ph, kErrWaitData, poll)) return false;
                at = slot;
                if (++slot == W::kSlots) {
                    slot = 0;
                    ring_ph ^= 1u;
                }
                return true;
            };
            uint32_t nb = 0;             // blocks of S issued so far: buffer nb & 1, its phase nb / 2
            uint32_t pv = 0;             // of P·V
            int pieces = 0;
            for (WidePiece w = walk.next(); w.valid && !abort_seen; w = walk.next(), ++pieces) {
                const int n = w.last - w.first;
                if (!wait_warp(q_full, pieces & 1, kErrWaitData, poll)) {
                    abort_seen = true;
                    break;
                }
                auto issue_s = [&](bool last) {
                    int at;
                    if (nb >= 2 && !wait_warp(s_free(nb & 1u), (nb / 2 - 1) & 1u, kErrWaitAcc, poll)) return false;
                    if (!take(at)) return false;
                    tc_fence_after_sync();
                    if (elect_one()) {
                        const uint32_t s_tmem = tmem_base + W::kColS + (nb & 1u) * kWideBlock, ka = slot_addr(at);
#pragma unroll
                        for (int kk = 0; kk < kD / 16; ++kk)
                            mma_bf16_ts_one(s_tmem, tmem_base + W::kColQ + kk * 8,
                                            smem_desc_kmajor_sw128(ka + (kk >> 2) * W::kChunkBytes + (kk & 3) * 32), W::kIdescS, kk > 0 ? 1u : 0u);
                        mma_commit_one(s_full(nb & 1u));
                        mma_commit_one(kv_empty(at));
                        if (last) mma_commit_one(q_empty);
                    }
                    __syncwarp();
                    ++nb;
                    return true;
                };
                bool ok = issue_s(n == 1);
                for (int j = 0; ok && j < n; ++j, ++pv) {
                    int at;
                    ok = j + 1 == n || issue_s(j + 2 == n);
                    ok = ok && take(at);
                    // (read before what the next softmax waits for)
                    uint32_t half_values;
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(half_values) : "r"(scales_addr(static_cast<int>(pv)) + 32u));
                    half_values = __reduce_or_sync(0xffffffffu, half_values);
                    ok = ok && wait_warp(p_full, pv & 1u, kErrWaitAcc, poll);
                    if (!ok) break;
                    tc_fence_after_sync();
                    if (elect_one()) {
                        const uint32_t va = slot_addr(at);
                        auto issue_pv = [&](uint32_t idesc) {
#pragma unroll
                            for (int kk = 0; kk < kWideBlock / 16; ++kk)
                                mma_bf16_ts_one(tmem_base + W::kColO, tmem_base + W::kColP + kk * 8, smem_desc_mnmajor(va + kk * 2048, 128, W::kChunkBytes),
                                                idesc, (j == 0 && kk == 0) ? 0u : 1u);
                        };
                        if (half_values != 0) issue_pv(W::kIdescPV);
                        else issue_pv(W::kIdescPVWide);
                        mma_commit_one(o_done);
                        mma_commit_one(kv_empty(at));
                    }
                    __syncwarp();
                }
                if (!ok) abort_seen = true;
            }
        }
    } else {
        // ------------------------------------------ softmax warpgroup --
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int r = static_cast<int>(threadIdx.x);
        const uint32_t lane_off = (warp * 32u) << 16;
        const uint32_t o_addr = tmem_base + lane_off + W::kColO;
        const uint32_t p_addr = tmem_base + lane_off + W::kColP;
        float c = 0.0f;                // of this row: its scale's other factor times that of the softmax
        uint32_t nb = 0;               // blocks so far
        int pieces = 0;
        for (WidePiece w = walk.next(); w.valid && !abort_seen; w = walk.next()) {
            const int n = w.last - w.first, done = begin + static_cast<int>(nb);
            const bool whole = n == w.blocks;
            const int slot = 2 * self + (nb == 0 ? 0 : 1);
            if (w.first == 0 && threadIdx.x == 0) {     // this run holds the unit's first block: it tells how the unit is made up
                const int parts = whole ? 0 : (done + w.blocks - 1) / per - done / per + 1;
                p.shared_info[static_cast<int64_t>(w.h) * p.shared_units + shared_unit0(p, w.section, w.group.first) + w.tile] =
                    make_int4(parts, slot, self, 0);
            }
            // ---- this thread's row of Q, once the previous piece's S are done
            const int row = w.tile * kWideRows + r, per_seq = p.T * p.group;
            const bool live = row < shared_rows(p, w.group.n);
            const int seq = row / per_seq, rest = row - seq * per_seq, tok = rest / p.group;
            const int head = w.h * p.group + rest - tok * p.group;
            if (pieces > 0 && !wait_warp(q_empty, (pieces - 1) & 1, kErrSoftmaxWait, suspend)) {
                abort_seen = true;
                break;
            }
            tc_fence_after_sync();
            {
                const uint16_t* const src = static_cast<const uint16_t*>(p.q) + (p.b0 + w.group.first + seq) * p.q_stride_b +
                                            tok * p.q_stride_t + head * p.q_stride_h;
                Raw8<T> x[kD / 8];
                uint32_t top = 0;
#pragma unroll
                for (int k = 0; k < kD / 8; ++k) x[k].w[0] = live ? reinterpret_cast<const uint4*>(src)[k] : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < kD / 8; ++k) {
                    const uint32_t words[4] = {x[k].w[0].x, x[k].w[0].y, x[k].w[0].z, x[k].w[0].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = __vmaxu2(top, words[i] & 0x7FFF7FFFu);
                }
                top = max(top & 0xFFFFu, top >> 16);
                if constexpr (std::is_same<T, __half>::value)
                    top = __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(top))));
                else
                    top <<= 16;
                // 2^(10 - floor(log2 of the largest)), kept a normal number; 1 for rows of zeros and rows with an infinity or NaN
                int field = 127 + 10 - (static_cast<int>(top >> 23) - 127);
                if (top == 0 || top >= 0x7F800000u) field = 127;
                field = min(max(field, 1), 253);
                const float mul = __uint_as_float(static_cast<uint32_t>(field) << 23);
                c = __uint_as_float(static_cast<uint32_t>(254 - field) << 23) * p.scale_log2;
#pragma unroll
                for (int k = 0; k < kD / 64; ++k) {
                    uint32_t h[32];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float f[8];
                        widen8<T>(x[8 * k + e], f);
#pragma unroll
                        for (int i = 0; i < 4; ++i) h[4 * e + i] = pack_f16x2(f[2 * i] * mul, f[2 * i + 1] * mul);
                    }
                    tmem_store_32cols(tmem_base + lane_off + W::kColQ + 32 * k, h);
                }
                tmem_wait_st();
                tc_fence_before_sync();
            }
            mbar_arrive(q_full);
            ++pieces;
            float m = 0.0f, l = 0.0f;      // running maximum (log2 units) used for P, and sum of P
            float o_unit = 1.0f;           // of O
            for (int j = 0; j < n; ++j, ++nb) {
                const uint32_t s_addr = tmem_base + lane_off + W::kColS + (nb & 1u) * kWideBlock;
                if (!wait_warp(s_full(nb & 1u), nb / 2 & 1u, kErrSoftmaxWait, poll)) {
                    abort_seen = true;
                    break;
                }
                tc_fence_after_sync();
                uint32_t v[128];
                tmem_load_32cols_at<0>(s_addr + 0, v);
                tmem_load_32cols_at<32>(s_addr + 32, v);
                tmem_load_32cols_at<64>(s_addr + 64, v);
                tmem_load_32cols_at<96>(s_addr + 96, v);
                tmem_wait_ld();
                tc_fence_before_sync();
                mbar_arrive(s_free(nb & 1u));    // S is in registers: the block after the next may be computed
                float acc[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int e0 = 16 * k;
                    float a = fmax3(__uint_as_float(v[e0]), __uint_as_float(v[e0 + 1]), __uint_as_float(v[e0 + 2]));
#pragma unroll
                    for (int e = 3; e < 15; e += 2) a = fmax3(a, __uint_as_float(v[e0 + e]), __uint_as_float(v[e0 + e + 1]));
                    acc[k] = fmaxf(a, __uint_as_float(v[e0 + 15]));
                }
                // each chain's 16 columns lie in one page: their factor
                float cs[8], to_unit;
                bool half_values;
                {
                    const uint32_t at8 = scales_addr(static_cast<int>(nb));
                    const uint4 y = ld_shared_v4(at8 + 32u);
                    half_values = y.x != 0;
                    to_unit = j > 0 ? __uint_as_float(y.y) : 1.0f;
                    o_unit = __uint_as_float(y.z);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint4 x = ld_shared_v4(at8 + 16u * k);
                        cs[4 * k] = c * __uint_as_float(x.x);
                        cs[4 * k + 1] = c * __uint_as_float(x.y);
                        cs[4 * k + 2] = c * __uint_as_float(x.z);
                        cs[4 * k + 3] = c * __uint_as_float(x.w);
                    }
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[k] *= cs[k];
                float m_blk = fmax3(fmax3(acc[0], acc[1], acc[2]), fmax3(acc[3], acc[4], acc[5]), fmaxf(acc[6], acc[7]));
                // (scores of -inf alone: any finite maximum makes their weights 0)
                if (m_blk == -INFINITY) m_blk = j == 0 ? 0.0f : m;
                float alpha = 1.0f;
                if (j == 0) {
                    m = m_blk;
                } else if (m_blk > m + attn::kRescaleThreshold) {
                    alpha = ex2_approx(m - m_blk);
                    m = m_blk;
                    l *= alpha;
                }
                const uint64_t nm2 = f32x2(kWideShift - m, kWideShift - m);
                uint64_t sum2[4] = {0, 0, 0, 0};
                uint32_t pk[64];
                auto rescale_o = [&]() {
                    const float by = alpha * to_unit;
                    if (__any_sync(0xffffffffu, by != 1.0f)) {
#pragma unroll
                        for (int cc = 0; cc < kD / 32; ++cc) {
                            uint32_t o[32];
                            tmem_load_32cols(o_addr + 32 * cc, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
                            tmem_store_32cols(o_addr + 32 * cc, o);
                        }
                    }
                };
                auto exp_pair = [&](int e) {
                    const uint64_t x = ffma2(f32x2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), f32x2(cs[e >> 3], cs[e >> 3]), nm2);
                    float x0, x1;
                    f32x2_split(x, x0, x1);
                    const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                    sum2[e & 3] = fadd2(sum2[e & 3], f32x2(p0, p1));
                    v[2 * e] = __float_as_uint(p0);
                    v[2 * e + 1] = __float_as_uint(p1);
                };
                auto pack_half = [&](int e0) {
                    if (half_values) {
#pragma unroll
                        for (int e = e0; e < e0 + 32; ++e) pk[e] = pack_f16x2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
                    } else {
#pragma unroll
                        for (int e = e0; e < e0 + 32; ++e) pk[e] = pack_bf16x2_rn(v[2 * e], v[2 * e + 1]);
                    }
                };
#pragma unroll
                for (int e = 0; e < 32; ++e) exp_pair(e);
                pack_half(0);
                // P·V of the previous block must be done before its P is overwritten and O rescaled; the first half of P is
                // stored while the second is computed
                if (j > 0 && !wait_warp(o_done, (nb - 1) & 1u, kErrSoftmaxWait, poll)) {
                    abort_seen = true;
                    break;
                }
                tc_fence_after_sync();
                if (j > 0) rescale_o();
                tmem_store_32cols(p_addr, *reinterpret_cast<const uint32_t(*)[32]>(&pk[0]));
#pragma unroll
                for (int e = 32; e < 64; ++e) exp_pair(e);
                pack_half(32);
                {
                    const uint64_t s01 = fadd2(fadd2(sum2[0], sum2[1]), fadd2(sum2[2], sum2[3]));
                    float lo, hi;
                    f32x2_split(s01, lo, hi);
                    l += lo + hi;
                }
                tmem_store_32cols(p_addr + 32, *reinterpret_cast<const uint32_t(*)[32]>(&pk[32]));
                tmem_wait_st();
                tc_fence_before_sync();
                mbar_arrive(p_full);
            }
            // ---- the row's sums, unnormalised (reading O here, before this warp publishes the next piece's first P,
            // orders these reads before the P·V that overwrites O)
            if (!abort_seen) {
                if (!wait_warp(o_done, (nb - 1) & 1u, kErrSoftmaxWait, poll)) {
                    abort_seen = true;
                } else {
                    tc_fence_after_sync();
                    const int64_t out_row = (static_cast<int64_t>(w.group.first + seq) * p.T + tok) * p.Hq + head;
                    const int64_t at_row = whole ? p.whole[0] + out_row : p.shared_slots + static_cast<int64_t>(slot) * kWideRows + r;
                    const bool any = l > 0.0f || l != l;
                    // in units of the power of two in l, so that sums of values that fp32 holds are values that it holds
                    const int field = static_cast<int>(__float_as_uint(l) >> 23), exponent = l > 0.0f && field < 255 ? field - 127 : 0;
                    const float less = __uint_as_float(static_cast<uint32_t>(min(max(127 - exponent, 1), 254)) << 23), by = o_unit * less;
#pragma unroll
                    for (int cc = 0; cc < kD / 32; ++cc) {
                        uint32_t o[32];
                        tmem_load_32cols(o_addr + 32 * cc, o);
                        tmem_wait_ld();
                        if (live) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = any ? __float_as_uint(__uint_as_float(o[e]) * by) : 0u;
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                st_global_v4(p.part_o + at_row * kD + 32 * cc + 4 * e, o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        }
                    }
                    if (live) {
                        p.part_ml[2 * at_row] = any ? m - kWideShift + static_cast<float>(exponent) : -INFINITY;
                        p.part_ml[2 * at_row + 1] = any ? l * less : 0.0f;
                    }
                    tc_fence_before_sync();
                }
            }
        }
    }

    if (abort_seen || wait_aborted(p.wait)) {
        // let MMAs that were already issued land before teardown
        for (int i = 0; i < 200; ++i) __nanosleep(1000);
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kWideIssueWarp) {
        tc_fence_after_sync();
        tmem_dealloc_one(tmem_base, W::kTmemCols);
    }
}

}  // namespace kv8
}  // namespace hk
