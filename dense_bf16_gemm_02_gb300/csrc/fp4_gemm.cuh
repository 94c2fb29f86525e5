// Product of two microscaled 4-bit matrices, C = bf16(ga·gb · A·Bᵀ), for sm_103a.
//
//   C[i,j] = bf16_rne( ga·gb · Σ_b SA[i,b]·SB[j,b] · Σ_{k in block b} A[i,k]·B[j,k] )
//
// with E2M1 codes, two per byte, and a scale per 32 (UE8M0, MXFP4) or 16
// (E4M3, NVFP4) values of a row, laid out as fp4_quant.cuh describes. The
// tensor core multiplies codes and scales itself (tcgen05.mma kind::mxf4 with
// two scales, kind::mxf4nvf4 with four scales per row and 64 columns of K) and
// sums in fp32; products of two codes and their scales are exact.
//
// A K stage is one 128-byte swizzle atom of codes (256 columns): four MMAs of
// K = 64. Its scales are 2 (MXFP4) or 4 (NVFP4) tiles of 512 bytes per 128
// rows, contiguous in memory: one untiled bulk copy into shared memory, then
// tcgen05.cp into Tensor Memory, where tile q takes four columns.
//
// The MMA warp issues a stage's scale copies just before its MMAs, in one
// instruction stream (a copy is ordered before the MMAs that follow it). What
// that costs is the issuing: each of these instructions takes its operands from
// uniform registers. Measured per stage of 4 MMAs of a 256 × 256 tile, operands
// stepping through a ring: 517 cycles with 12 copies issued under elect.sync,
// 1049 to 1304 under a test of the lane id, where every operand is moved to a
// uniform register on its own; the MMAs alone take 515.
#pragma once

#include <cuda.h>
#include <cstdint>

#include "bounded_wait.cuh"
#include "fp4_quant.cuh"
#include "ptx.cuh"

namespace hk {
namespace fp4 {

constexpr int kStageCols = 256;        // K per stage
constexpr int kMmaCols = 64;           // K per MMA
constexpr int kMmasPerStage = kStageCols / kMmaCols;
constexpr int kStageRowBytes = 128;    // codes of a row and stage
constexpr int kSmemLimit = 232448;

constexpr uint32_t kFlagDropArrive = 0x1u;

// Scale tiles (512 bytes, 128 rows × 4 blocks) of 128 rows and one stage.
__host__ __device__ constexpr int scale_tiles(int fmt) { return kStageCols / block_cols(fmt) / 4; }

struct Fp4Params {
    int32_t M, N;                      // rows of A (tokens) and of B (features)
    int32_t k_stages;                  // ceil(K / 256)
    int32_t tiles_m, tiles_n;
    int32_t group_m;                   // pair kernel: tile rows that are swept together
    int32_t total_units, tail_start;   // pair kernel: work units; tiles from here on run as two halves
    const uint8_t* sfa;                // scale tiles of A and B
    const uint8_t* sfb;
    const float* ga;                   // global scales, or null (1)
    const float* gb;
    uint16_t* c;
    int64_t ldc;
    int32_t vec_c;                     // C's rows are 16-byte aligned
    uint32_t flags;
    WaitCtx wait;
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

// Instruction descriptor, kind::mxf4 and kind::mxf4nvf4: A and B in E2M1
// (format code 1 in bits 7-9 and 10-11), both K-major, N >> 3 in bits 17-22,
// scale type in bit 23 (1: UE8M0, 0: E4M3), M >> 7 in bits 27-28; the
// scale-factor ids (bits 4-5 for B, 29-30 for A) are or-ed in per MMA.
__host__ __device__ constexpr uint32_t idesc_fp4_f32(uint32_t m, uint32_t n, int fmt) {
    return (1u << 7) | (1u << 10) | ((n >> 3) << 17) | ((fmt == kMxfp4 ? 1u : 0u) << 23) | ((m >> 7) << 27);
}

// D[tmem] (+)= (A·sfa)[smem] · (B·sfb)[smem]ᵀ for one CTA or a CTA pair.
template <int kCG, int kFmt>
__device__ __forceinline__ void mma_fp4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t sfa_tmem, uint32_t sfb_tmem, uint32_t accumulate) {
    if constexpr (kCG == 1 && kFmt == kMxfp4)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
            : "memory");
    else if constexpr (kCG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
            : "memory");
    else if constexpr (kFmt == kMxfp4)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
            : "memory");
}

// Which scale tile MMA k of a stage reads, and the scale-factor id inside it:
// MXFP4 uses two of a tile's four blocks per MMA, NVFP4 all four.
template <int kFmt> __device__ __forceinline__ constexpr uint32_t mma_scale_tile(int k) {
    return kFmt == kMxfp4 ? static_cast<uint32_t>(k >> 1) : static_cast<uint32_t>(k);
}
template <int kFmt> __device__ __forceinline__ constexpr uint32_t mma_scale_id(int k) {
    return kFmt == kMxfp4 ? static_cast<uint32_t>(k & 1) * 2u : 0u;
}

__device__ __forceinline__ void tmem_load_16cols(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// The global scales' product as two factors: the product and 1, unless it comes near the ends of fp32's range (a sum
// times both may well be inside it); then its fraction with as much of its exponent as keeps a product with a sum
// inside, and the rest of the exponent, which the sums are lifted by first.
struct Alpha {
    float mul, lift;
    template <int kCount>
    __device__ __forceinline__ void lift_sums(uint32_t (&v)[kCount]) const {
        if (lift != 1.0f) {              // (the same in every thread)
#pragma unroll
            for (int i = 0; i < kCount; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * lift);
        }
    }
    __device__ __forceinline__ uint32_t of(uint32_t sum) const { return __float_as_uint(__uint_as_float(sum) * mul); }
};

__device__ __forceinline__ Alpha global_alpha(const Fp4Params& p) {
    const float a = p.ga != nullptr ? *p.ga : 1.0f, b = p.gb != nullptr ? *p.gb : 1.0f;
    const float product = a * b;
    if ((fabsf(product) >= 0x1p-80f && fabsf(product) <= 0x1p80f) || !isfinite(a) || !isfinite(b)) return Alpha{product, 1.0f};
    int ea, eb;
    const float fraction = frexpf(a, &ea) * frexpf(b, &eb);
    const int e = ea + eb, near = max(-80, min(80, e));
    return Alpha{ldexpf(fraction, near), ldexpf(1.0f, max(-149, min(127, e - near)))};
}

template <int kCols>
__device__ __forceinline__ void tmem_load_cols(uint32_t taddr, uint32_t (&v)[kCols]) {
    static_assert(kCols == 16 || kCols == 32, "16 or 32 columns");
    if constexpr (kCols == 16) tmem_load_16cols(taddr, v);
    else tmem_load_32cols(taddr, v);
}

// Sums of one feature and kStep tokens to their rows of C, as far as there are tokens.
template <int kStep>
__device__ __forceinline__ void store_tokens(uint16_t* dst, int64_t ldc, uint32_t (&v)[kStep], const Alpha alpha, int tokens) {
    alpha.lift_sums(v);
    uint32_t w[kStep / 2];
#pragma unroll
    for (int i = 0; i < kStep / 2; ++i)
        w[i] = pack_bf16x2_rn(alpha.of(v[2 * i]), alpha.of(v[2 * i + 1]));
    if (tokens >= kStep) {
#pragma unroll
        for (int e = 0; e < kStep; ++e) dst[e * ldc] = static_cast<uint16_t>(e & 1 ? w[e >> 1] >> 16 : w[e >> 1]);
    } else {
#pragma unroll
        for (int e = 0; e < kStep; ++e)
            if (e < tokens) dst[e * ldc] = static_cast<uint16_t>(e & 1 ? w[e >> 1] >> 16 : w[e >> 1]);
    }
}

// Tokens [t0, t1) of a tile whose K range kParts CTAs of a cluster shared: the
// sums of the parts, added in order. Four features of a token per thread (32
// threads a token, so a warp reads whole 512-byte rows); sixteen loads of each
// thread are in flight, since another CTA's shared memory is
// far away; none past t1, since its rate is low.
template <int kTok, int kParts>
__device__ __forceinline__ void join_tokens(const Fp4Params& p, uint32_t base, int tm, int tn, int t0, int t1, int warp, bool ok) {
    constexpr int kTokens = 16 / kParts;
    const int lane = static_cast<int>(lane_id());
    const int feature = tn * 128 + lane * 4;
    const Alpha alpha = global_alpha(p);
    uint32_t from[kParts];
#pragma unroll
    for (int r = 0; r < kParts; ++r) from[r] = map_to_cta(base + static_cast<uint32_t>(lane) * 16u, static_cast<uint32_t>(r));
#pragma unroll 1
    for (int t = t0 + warp; t < t1; t += 4 * kTokens) {
        float4 x[kTokens][kParts];
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
            if (t + 4 * i < t1) {
#pragma unroll
                for (int r = 0; r < kParts; ++r) x[i][r] = ld_cluster_v4(from[r] + static_cast<uint32_t>(t + 4 * i) * 512u);
            }
        }
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
            float4 sum = x[i][0];
#pragma unroll
            for (int r = 1; r < kParts; ++r) {
                sum.x += x[i][r].x;
                sum.y += x[i][r].y;
                sum.z += x[i][r].z;
                sum.w += x[i][r].w;
            }
            if (!ok || t + 4 * i >= t1) continue;
            uint16_t* const dst = p.c + static_cast<int64_t>(tm * kTok + t + 4 * i) * p.ldc + feature;
            uint32_t v[4] = {__float_as_uint(sum.x), __float_as_uint(sum.y), __float_as_uint(sum.z), __float_as_uint(sum.w)};
            alpha.lift_sums(v);
            const uint32_t w0 = pack_bf16x2_rn(alpha.of(v[0]), alpha.of(v[1]));
            const uint32_t w1 = pack_bf16x2_rn(alpha.of(v[2]), alpha.of(v[3]));
            if (p.vec_c && feature + 4 <= p.N) {
                *reinterpret_cast<uint2*>(dst) = make_uint2(w0, w1);
            } else {
                const uint32_t w[2] = {w0, w1};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (feature + e < p.N) dst[e] = static_cast<uint16_t>(e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xFFFFu);
            }
        }
    }
}

// ---------------------------------------------------- one-CTA tile kernel --
//
// For few tokens (rows of A) and for few tiles: a tile is 128 features × kTok
// tokens and the MMA's M side takes the features (rows of B), so that its N side
// need only be as wide as the tokens are many. The tile's K range may be cut over
// the CTAs of a cluster (one CTA per part); each leaves its fp32 sums in its
// shared memory, and the CTAs then each add up and store a share of the tile's
// tokens, in the order of the parts (the result does not depend on timing).
// Two CTAs fit on an SM, so a tile's start and end overlap another's stream.
//
// One token is bound by reading B: 28672 × 8192 MXFP4 in 20.8 us, 6.0 TB/s of the
// 6.8 that a copy reaches. Toward 128 tokens the tile's end counts: A's traffic
// from L2 comes to B's, and the sums go through one CTA's registers and, where K
// is cut, through other SMs' shared memory, whose rate is low (128 tokens in 4
// parts: 3 of 13 us at 8192 × 8192). 128 × 28672 × 8192 takes 24.3 us (26.2 when the
// epilogue took 16 columns at a time and tested each token).
template <int kTok, int kFmt>
struct SingleGeometry {
    static_assert(kTok == 16 || kTok == 32 || kTok == 64 || kTok == 128, "tokens per tile");
    static constexpr int kTileF = 128;                                      // features per tile
    static constexpr int kSfTiles = scale_tiles(kFmt);
    static constexpr int kSfBytes = 512 * kSfTiles;                         // scales of one operand and stage
    static constexpr int kWBytes = kTileF * kStageRowBytes;
    static constexpr int kTBytes = kTok * kStageRowBytes;
    static constexpr int kStageBytes = kWBytes + kTBytes + 2 * kSfBytes;
    static constexpr int kBudget = 113 * 1024 - 2048;                       // two CTAs per SM
    static constexpr int kSfCols = 8 * kSfTiles;                            // TMEM columns of a stage's scales
    static constexpr int kFitSmem = kBudget / kStageBytes;
    static constexpr int kFitTmem = (256 - kTok) / kSfCols;
    static constexpr int kStages = kFitSmem < kFitTmem ? kFitSmem : kFitTmem;
    static_assert(kStages >= 3, "pipeline too shallow");
    static constexpr int kOffW = 0;
    static constexpr int kOffT = kOffW + kStages * kWBytes;
    static constexpr int kOffSf = kOffT + kStages * kTBytes;
    static constexpr int kOffBars = kOffSf + kStages * 2 * kSfBytes;        // full[S], empty[S], acc
    static constexpr int kOffHolder = kOffBars + (2 * kStages + 1) * 8;
    static constexpr int kSmemBytes = kOffHolder + 16 + 1024;
    static constexpr int kSumBytes = kTok * kTileF * 4;                     // fp32 sums, in the ring's place
    static_assert(kSumBytes <= kOffBars, "the sums fit the ring");
    static constexpr int kColSf = kTok;
    static constexpr int kTmemCols = kColSf + kStages * kSfCols > 128 ? 256 : 128;
    static constexpr uint32_t kIdesc = idesc_fp4_f32(kTileF, kTok, kFmt);
    static constexpr int kThreads = 192;
};

template <int kTok, int kFmt>
__global__ void __launch_bounds__(192, 2)
gemm_fp4_single_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                       const Fp4Params p, const int splits) {
    using G = SingleGeometry<kTok, kFmt>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const smem = smem_raw + (base - raw);
    const uint32_t warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // known to be the same in every lane
    const uint32_t lane = lane_id();
    const int part = static_cast<int>(blockIdx.x) % splits;        // the CTA's rank in its cluster
    const int tile = static_cast<int>(blockIdx.x) / splits;
    const int tm = tile % p.tiles_m, tn = tile / p.tiles_m;
    const int ks_begin = static_cast<int>(static_cast<int64_t>(part) * p.k_stages / splits);
    const int ks_end = static_cast<int>(static_cast<int64_t>(part + 1) * p.k_stages / splits);

    auto full_bar = [&](int s) { return base + G::kOffBars + 8u * s; };
    auto empty_bar = [&](int s) { return base + G::kOffBars + 8u * (G::kStages + s); };
    const uint32_t acc_bar = base + G::kOffBars + 8u * (2 * G::kStages);

    griddep_launch_dependents();
    if (threadIdx.x == 0) {
        prefetch_tensor_map(&tmap_a);
        prefetch_tensor_map(&tmap_b);
        for (int s = 0; s < G::kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        mbar_init(acc_bar, 1);
        fence_mbar_init_cluster();
    }
    if (warp == 1) {
        tmem_alloc_one(base + G::kOffHolder, G::kTmemCols);
        tmem_relinquish_one();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(smem + G::kOffHolder);
    bool ok = true;

    if (warp == 0) {
        griddep_wait();                  // launched early behind the kernel that may have written the operands
        const uint8_t* const sft = p.sfa + (static_cast<int64_t>(tm) * kTok / 128) * p.k_stages * G::kSfBytes;
        const uint8_t* const sfw = p.sfb + static_cast<int64_t>(tn) * p.k_stages * G::kSfBytes;
        const bool drop = p.flags & kFlagDropArrive;       // test only: the first stage is never filled
        int fills = 0, stage = 0;
        uint32_t phase = 1;
        for (int ks = ks_begin; ks < ks_end; ++ks) {
            if (ok) ok = wait_mbar_poll(p.wait, empty_bar(stage), phase, kErrWaitRing);
            ok = __all_sync(0xffffffffu, ok);
            if (ok && !(drop && ks == ks_begin) && elect_one()) {
                const uint32_t sf = base + G::kOffSf + stage * 2 * G::kSfBytes;
                mbar_arrive_expect_tx(full_bar(stage), G::kStageBytes);
                tma_load_2d(base + G::kOffW + stage * G::kWBytes, &tmap_b, ks * kStageRowBytes, tn * G::kTileF, full_bar(stage));
                tma_load_2d(base + G::kOffT + stage * G::kTBytes, &tmap_a, ks * kStageRowBytes, tm * kTok, full_bar(stage));
                bulk_load(sf, sfw + static_cast<int64_t>(ks) * G::kSfBytes, G::kSfBytes, full_bar(stage));
                bulk_load(sf + G::kSfBytes, sft + static_cast<int64_t>(ks) * G::kSfBytes, G::kSfBytes, full_bar(stage));
            }
            __syncwarp();
            if (ok) ++fills;
            if (++stage == G::kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        // abort: the copies in flight land before the CTA ends
        if (lane == 0 && (!ok || wait_aborted(p.wait)))
            for (int f = fills > G::kStages ? fills - G::kStages : 0; f < fills; ++f)
                if (!drop || f > 0) wait_mbar_drain(full_bar(f % G::kStages), (f / G::kStages) & 1);
    } else if (warp == 1) {
        griddep_wait();                  // (its waits are for loads that begin then: the time limit is theirs alone)
        int stage = 0;
        uint32_t phase = 0;
        // (a column of a scale tile holds 32 rows: the second 64 tokens of 128 begin two columns on)
        const uint32_t t_shift = kTok == 64 ? 2u * (static_cast<uint32_t>(tm) & 1u) : 0u;
        // (after a wait that gave up the loop runs on without issuing: its exit depends on no wait, so that the
        // compiler sees every index as the same in all lanes)
        for (int ks = ks_begin; ks < ks_end; ++ks) {
            if (ok) ok = wait_mbar_poll(p.wait, full_bar(stage), phase, kErrWaitData);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after_sync();
            const uint32_t sf = desc_low(base + G::kOffSf + stage * 2 * G::kSfBytes, 16);
            const uint32_t sf_tmem = tmem_base + G::kColSf + stage * G::kSfCols;
            const uint32_t wd = desc_low(base + G::kOffW + stage * G::kWBytes, 16);
            const uint32_t td = desc_low(base + G::kOffT + stage * G::kTBytes, 16);
            if (ok && elect_one()) {
#pragma unroll
                for (int q = 0; q < 2 * G::kSfTiles; ++q)
                    tmem_cp_128x16b(sf_tmem + 4 * q, smem_desc(sf + ((512 * q) >> 4), desc_high_plain(128)));
#pragma unroll
                for (int k = 0; k < kMmasPerStage; ++k) {
                    const uint32_t id = mma_scale_id<kFmt>(k);
                    const uint32_t col = 4 * mma_scale_tile<kFmt>(k);
                    mma_fp4<1, kFmt>(tmem_base, smem_desc(wd + 2 * k, kDescHighKmajorSw128),
                                     smem_desc(td + 2 * k, kDescHighKmajorSw128), G::kIdesc | (id << 4) | (id << 29),
                                     sf_tmem + col, sf_tmem + 4 * G::kSfTiles + col + t_shift, (ks > ks_begin || k > 0) ? 1u : 0u);
                }
                mma_commit_one(empty_bar(stage));
            }
            __syncwarp();
            if (++stage == G::kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        // also on the abort path: everything issued completes before TMEM is freed. (A commit tracks what its own thread
        // issued, so it is the elected one's too: elect.sync picks the same lane every time, but not a known one.)
        if (elect_one()) mma_commit_one(acc_bar);
        __syncwarp();
        if (lane == 0 && !ok) wait_mbar_drain(acc_bar, 0);
        __syncwarp();
    } else {
        // ------------------------------------------------------ epilogue --
        griddep_wait();                  // before C is written or the global scales are read
        ok = __all_sync(0xffffffffu, wait_mbar(p.wait, acc_bar, 0, kErrWaitAcc) && !wait_aborted(p.wait));
        tc_fence_after_sync();
        const uint32_t q = warp & 3u;
        const int f_local = static_cast<int>(q * 32 + lane);
        const int feature = tn * G::kTileF + f_local;
        const uint32_t t_row = tmem_base + ((q * 32u) << 16);
        const Alpha alpha = global_alpha(p);
        // (columns of 32 tokens at a time, and no test or address of its own for each token where all of them are
        // inside C: one warp of a scheduler pays the latency of every instruction that depends on another)
        constexpr int kStep = kTok < 32 ? kTok : 32;
        if (splits == 1) {
#pragma unroll 1
            for (int c = 0; c < kTok; c += kStep) {
                const int left = p.M - (tm * kTok + c);
                if (left <= 0) break;
                uint32_t v[kStep];
                tmem_load_cols<kStep>(t_row + c, v);
                tmem_wait_ld();
                if (ok && feature < p.N)
                    store_tokens<kStep>(p.c + static_cast<int64_t>(tm * kTok + c) * p.ldc + feature, p.ldc, v, alpha, left);
            }
        } else {
            // this part's sums: [token][feature] fp32 in the ring's place (every MMA has
            // read its operands, and no copy is in flight)
            float* const sums = reinterpret_cast<float*>(smem);
#pragma unroll 1
            for (int c = 0; c < kTok; c += kStep) {
                uint32_t v[kStep];
                tmem_load_cols<kStep>(t_row + c, v);
                tmem_wait_ld();
                if (ok) {
#pragma unroll
                    for (int e = 0; e < kStep; ++e) sums[(c + e) * G::kTileF + f_local] = __uint_as_float(v[e]);
                }
            }
        }
        tc_fence_before_sync();
    }
    __syncwarp();
    if (splits > 1) {
        cluster_sync();
        // this CTA's share of the tokens
        if (warp >= 2) {
            const int each = (kTok + splits - 1) / splits;
            const int t0 = part * each, t1 = min(min(kTok, t0 + each), p.M - tm * kTok);
            if (splits == 2) join_tokens<kTok, 2>(p, base, tm, tn, t0, t1, static_cast<int>(warp) - 2, ok);
            else if (splits == 4) join_tokens<kTok, 4>(p, base, tm, tn, t0, t1, static_cast<int>(warp) - 2, ok);
            else join_tokens<kTok, 8>(p, base, tm, tn, t0, t1, static_cast<int>(warp) - 2, ok);
        }
        cluster_sync();    // no CTA leaves while another reads its sums
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_one(tmem_base, G::kTmemCols);
    }
}

// --------------------------------------------------- CTA-pair tile kernel --
//
// For many tokens: 256 × 256 tiles on a pair of CTAs (cta_group::2), a
// persistent grid, roles by warp: 0 loads, 1 issues the scale copies and the
// MMAs (leader CTA), 2-5 store.
//
// Tensor Memory holds two accumulators of 256 columns and a ring of scale
// slots, which together need more than its 512 columns: the accumulators
// OVERLAP by what is missing. The epilogue reads the overlapping columns of its
// tile first and then lets the next tile's MMAs begin, so that they wait for a
// few reads instead of a whole epilogue.
//
// 8192³ takes 153 us (MXFP4, 7.2 PFLOP/s) and 163 us (NVFP4). What bounds it is shared
// memory: a stage takes a CTA some 715 cycles, its MMAs alone 516 and its loads alone
// 541, and per stage the operands are written once and read (A's 16 KB, both halves of
// B), the scales too: 90 KB (NVFP4 96) at 128 bytes a cycle are 703 (750). Without the
// loads of the scales it took 141 us; scales loaded for two stages at a time, in rows of
// 1 or 2 KB, or with the loads issued under elect.sync, changed nothing or cost 3 to 9 %.
template <int kFmt>
struct PairGeometry {
    static constexpr int kTile = 256;                                       // rows of A and of B per tile
    static constexpr int kSfTiles = scale_tiles(kFmt);
    static constexpr int kSfBytes = 512 * kSfTiles;                         // scales of 128 rows and a stage
    static constexpr int kOpBytes = 128 * kStageRowBytes;                   // A or B rows of one CTA and stage
    static constexpr int kStageSf = 3 * kSfBytes;                           // own A rows, both halves of B
    static constexpr int kStageBytes = 2 * kOpBytes + kStageSf;
    static constexpr int kFit = (kSmemLimit - 2048 - 4 * 2048) / kStageBytes;
    static constexpr int kStages = kFit > 6 ? 6 : kFit;
    static_assert(kStages >= 4, "pipeline too shallow");
    static constexpr int kSfCols = 12 * kSfTiles;                           // TMEM columns of a stage's scales
    static constexpr int kSlots = kFmt == kMxfp4 ? 4 : 3;                   // scale slots
    static constexpr int kColSf = 512 - kSlots * kSfCols;
    static constexpr int kOverlap = 512 - kColSf;                           // columns that both accumulators use
    static constexpr int kCol1 = 256 - kOverlap;                            // where accumulator 1 begins
    static constexpr int kFirstChunks = (kOverlap + 31) / 32;               // 32-column chunks read before the hand-over
    static constexpr int kOffA = 0;
    static constexpr int kOffB = kStages * kOpBytes;
    static constexpr int kOffSf = 2 * kStages * kOpBytes;
    static constexpr int kStoreBytes = 32 * 64;                             // 32 × 32 outputs that a warp stores at a time
    static constexpr int kOffStore = kOffSf + kStages * kStageSf;
    // full[S], empty[S], acc_full[2], acc_free, drain
    static constexpr int kOffBars = kOffStore + 4 * kStoreBytes;
    static constexpr int kNumBars = 2 * kStages + 4;
    static constexpr int kOffHolder = kOffBars + kNumBars * 8;              // TMEM address, two flags
    static constexpr int kSmemBytes = kOffHolder + 16 + 1024;
    static_assert(kSmemBytes <= kSmemLimit, "shared memory");
    static constexpr uint32_t kIdesc = idesc_fp4_f32(256, 256, kFmt);
    static constexpr uint32_t kIdescHalf = idesc_fp4_f32(256, 128, kFmt);
    static constexpr int kThreads = 192;
};

// Work unit u -> tile and half (-1: the whole tile).
__device__ __forceinline__ void pair_unit(const Fp4Params& p, int u, int& tm, int& tn, int& half) {
    int t = u;
    half = -1;
    if (u >= p.tail_start) {
        t = p.tail_start + ((u - p.tail_start) >> 1);
        half = (u - p.tail_start) & 1;
    }
    const int per_group = p.group_m * p.tiles_n;
    const int g = t / per_group;
    const int first_m = g * p.group_m;
    const int rows = min(p.tiles_m - first_m, p.group_m);
    const int local = t - g * per_group;
    tm = first_m + local % rows;
    tn = local / rows;
}

// 32 rows × 32 columns of sums (lane: row) to bf16 and to C at (row0, col0),
// through the warp's buffer in shared memory (64-byte rows, swizzled) and a TMA store.
// Where TMA cannot write C (rows not 16-byte aligned; N not a multiple of 8 at
// the last columns, since it bounds a row to 16 bytes only) a warp writes a row's
// 32 columns at a time.
__device__ __forceinline__ void store_sums(const Fp4Params& p, const void* tmap_c, uint32_t buf, const uint8_t* buf_ptr,
                                           uint32_t (&v)[32], const Alpha alpha, int row0, int col0) {
    const uint32_t lane = lane_id();
    alpha.lift_sums(v);
    if (row0 >= p.M || col0 >= p.N) return;          // (the same in every lane)
    if (lane == 0) bulk_wait_group_read<0>();        // the store before has read the buffer
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = pack_bf16x2_rn(alpha.of(v[8 * j + 2 * i]), alpha.of(v[8 * j + 2 * i + 1]));
        st_shared_v4(buf + lane * 64u + ((static_cast<uint32_t>(j) ^ ((lane >> 1) & 3u)) << 4), w[0], w[1], w[2], w[3]);
    }
    if (p.vec_c && (col0 + 32 <= p.N || p.N % 8 == 0)) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d(tmap_c, buf, col0, row0);
            bulk_commit_group();
        }
    } else {
        __syncwarp();
        const int rows = min(32, p.M - row0);
        if (col0 + static_cast<int>(lane) < p.N) {
            uint16_t* dst = p.c + static_cast<int64_t>(row0) * p.ldc + col0 + lane;
            for (int r = 0; r < rows; ++r, dst += p.ldc)
                *dst = *reinterpret_cast<const uint16_t*>(buf_ptr + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + (lane & 7) * 2);
        }
        __syncwarp();                                // (before the buffer is written again)
    }
}

template <int kFmt>
__global__ void __launch_bounds__(192, 1)
gemm_fp4_pair_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                     const __grid_constant__ CUtensorMap tmap_b_half, const __grid_constant__ CUtensorMap tmap_sfa,
                     const __grid_constant__ CUtensorMap tmap_sfb, const __grid_constant__ CUtensorMap tmap_c,
                     const Fp4Params p) {
    using G = PairGeometry<kFmt>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const smem = smem_raw + (base - raw);
    const uint32_t warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // known to be the same in every lane
    const uint32_t lane = lane_id();
    const uint32_t rank = cluster_cta_rank();
    const int unit = blockIdx.x / 2, num_units = gridDim.x / 2;

    auto full_bar = [&](int s) { return base + G::kOffBars + 8u * s; };
    auto empty_bar = [&](int s) { return base + G::kOffBars + 8u * (G::kStages + s); };
    auto acc_full_bar = [&](int b) { return base + G::kOffBars + 8u * (2 * G::kStages + b); };
    const uint32_t acc_free_bar = base + G::kOffBars + 8u * (2 * G::kStages + 2);
    const uint32_t drain_bar = base + G::kOffBars + 8u * (2 * G::kStages + 3);

    if (threadIdx.x == 0) {
        for (int s = 0; s < G::kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) mbar_init(acc_full_bar(b), 1);
        mbar_init(drain_bar, 1);
        mbar_init(acc_free_bar, 8);            // four storing warps of each CTA
        fence_mbar_init_cluster();
    }
    griddep_launch_dependents();
    if (warp == 0 && lane == 0) {
        prefetch_tensor_map(&tmap_a);
        prefetch_tensor_map(&tmap_b);
        prefetch_tensor_map(&tmap_sfa);
        prefetch_tensor_map(&tmap_sfb);
        if (p.vec_c) prefetch_tensor_map(&tmap_c);
    }
    if (warp == 1) {
        tmem_alloc_pair(base + G::kOffHolder, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    cluster_sync();
    tc_fence_after_sync();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(smem + G::kOffHolder);
    bool ok = true;

    if (warp == 0) {
        // ------------------------------------------------------- loads --
        if (lane == 0) {
            griddep_wait();              // launched early behind the kernel that may have written the operands
            int stage = 0;
            uint32_t phase = 0;
            int64_t fills = 0, dropped = -1;
            for (int u = unit; u < p.total_units && ok; u += num_units) {
                int tm, tn, half;
                pair_unit(p, u, tm, tn, half);
                const int a_row = tm * 256 + static_cast<int>(rank) * 128;
                const int b_row = half < 0 ? tn * 256 + static_cast<int>(rank) * 128
                                           : tn * 256 + half * 128 + static_cast<int>(rank) * 64;
                const void* const b_map = half < 0 ? static_cast<const void*>(&tmap_b) : static_cast<const void*>(&tmap_b_half);
                // rows of 256 bytes of the scale tiles: kSfBytes per 128 rows and stage
                constexpr int kSfRows = G::kSfBytes / 256;
                const int sfa_group = tm * 2 + static_cast<int>(rank);
                // both groups of 128 rows of B in one load (of a half tile its own and the next; past the
                // matrix they read as 0)
                const int sfb_group = tn * 2 + (half > 0 ? 1 : 0);
                const uint32_t bytes = 2u * (G::kOpBytes + (half < 0 ? G::kOpBytes : G::kOpBytes / 2) + 3 * G::kSfBytes);
                for (int ks = 0; ks < p.k_stages; ++ks) {
                    if (!wait_mbar_poll(p.wait, empty_bar(stage), phase ^ 1u, kErrWaitRing)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) {
                        if ((p.flags & kFlagDropArrive) && dropped < 0) dropped = fills;   // test only: never armed
                        else mbar_arrive_expect_tx(full_bar(stage), bytes);
                    }
                    const uint32_t full = map_to_cta(full_bar(stage), 0);
                    const uint32_t sf = base + G::kOffSf + stage * G::kStageSf;
                    tma_load_3d_pair(sf, &tmap_sfa, 0, ks * kSfRows, sfa_group, full);
                    tma_load_3d_pair(sf + G::kSfBytes, &tmap_sfb, 0, ks * kSfRows, sfb_group, full);
                    tma_load_2d_pair(base + G::kOffA + stage * G::kOpBytes, &tmap_a, ks * kStageRowBytes, a_row, full);
                    tma_load_2d_pair(base + G::kOffB + stage * G::kOpBytes, b_map, ks * kStageRowBytes, b_row, full);
                    ++fills;
                    if (++stage == G::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (rank == 0 && (!ok || wait_aborted(p.wait)))     // the copies in flight land before the block ends
                for (int64_t f = fills > G::kStages ? fills - G::kStages : 0; f < fills; ++f)
                    if (f != dropped)
                        wait_mbar_drain(full_bar(static_cast<int>(f % G::kStages)), static_cast<uint32_t>((f / G::kStages) & 1));
        }
    } else if (warp == 1) {
        // -------------------------------------------------------- MMAs --
        griddep_wait();                  // (the time limit of its waits begins with the loads)
        if (rank == 0) {
            int stage = 0, slot = 0, local = 0;
            int old_stage = 0;                  // the stage whose MMAs used this slot last
            uint32_t phase = 0, old_phase = 0;
            int64_t it = 0;
            // (after a wait that gave up the loops run on without issuing: their exits depend on no wait, so
            // that the compiler sees every index as the same in all lanes)
            for (int u = unit; u < p.total_units; u += num_units, ++local) {
                int tm, tn, half;
                pair_unit(p, u, tm, tn, half);
                const uint32_t idesc = half < 0 ? G::kIdesc : G::kIdescHalf;
                const uint32_t d_tmem = tmem_base + (local & 1 ? G::kCol1 : 0);
                // the previous tile's epilogue has read the columns this accumulator shares with it
                if (ok && local > 0) ok = wait_mbar_cluster(p.wait, acc_free_bar, (local - 1) & 1, kErrWaitAcc);
                for (int ks = 0; ks < p.k_stages; ++ks, ++it) {
                    if (ok) ok = wait_mbar_poll(p.wait, full_bar(stage), phase, kErrWaitData);
                    // the slot's last scales have been used: those MMAs completed (the phase of their stage's
                    // empty barrier, which cannot run on past it before this stage's MMAs are issued)
                    if (it >= G::kSlots) {
                        if (ok) ok = wait_mbar_poll(p.wait, empty_bar(old_stage), old_phase, kErrWaitRing);
                        if (++old_stage == G::kStages) {
                            old_stage = 0;
                            old_phase ^= 1u;
                        }
                    }
                    ok = __all_sync(0xffffffffu, ok);
                    tc_fence_after_sync();
                    const uint32_t ad = desc_low(base + G::kOffA + stage * G::kOpBytes, 16);
                    const uint32_t bd = desc_low(base + G::kOffB + stage * G::kOpBytes, 16);
                    const uint32_t src = desc_low(base + G::kOffSf + stage * G::kStageSf, 16);
                    const uint32_t sf = tmem_base + G::kColSf + slot * G::kSfCols;
                    if (ok && elect_one()) {
                        // a slot holds a stage's scale tiles in order, of each first A's, then B's two groups of
                        // rows (a half tile has one group; what the other's place holds is copied and not used)
#pragma unroll
                        for (int q = 0; q < G::kSfTiles; ++q)
#pragma unroll
                            for (int j = 0; j < 3; ++j)
                                tmem_cp_128x16b_pair(sf + 12 * q + 4 * j,
                                                     smem_desc(src + ((j * G::kSfBytes + 512 * q) >> 4), desc_high_plain(128)));
#pragma unroll
                        for (int k = 0; k < kMmasPerStage; ++k) {
                            const uint32_t id = mma_scale_id<kFmt>(k);
                            const uint32_t at = sf + 12 * mma_scale_tile<kFmt>(k);
                            mma_fp4<2, kFmt>(d_tmem, smem_desc(ad + 2 * k, kDescHighKmajorSw128),
                                             smem_desc(bd + 2 * k, kDescHighKmajorSw128), idesc | (id << 4) | (id << 29), at,
                                             at + 4, (ks > 0 || k > 0) ? 1u : 0u);
                        }
                        mma_commit_pair_mask(empty_bar(stage), 0x3);
                    }
                    __syncwarp();
                    if (++stage == G::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++slot == G::kSlots) slot = 0;
                }
                if (ok && elect_one()) mma_commit_pair_mask(acc_full_bar(local & 1), 0x3);
                __syncwarp();
            }
            if (!ok || wait_aborted(p.wait)) {      // everything issued completes before TMEM is freed
                if (elect_one()) mma_commit_pair_mask(drain_bar, 0x1);
                __syncwarp();
                if (lane == 0) wait_mbar_drain(drain_bar, 0);
                __syncwarp();
            }
        }
    } else {
        // ----------------------------------------------------- epilogue --
        griddep_wait();                               // before C is written or the global scales are read
        const uint32_t q = warp & 3u;                 // TMEM lanes 32 q .. 32 q + 31
        const Alpha alpha = global_alpha(p);
        const uint32_t buf_addr = base + G::kOffStore + (warp - 2) * G::kStoreBytes;
        const uint8_t* const buf_ptr = smem + G::kOffStore + (warp - 2) * G::kStoreBytes;
        int local = 0;
        for (int u = unit; u < p.total_units; u += num_units, ++local) {
            int tm, tn, half;
            pair_unit(p, u, tm, tn, half);
            const int buf = local & 1;
            {
                // one thread waits, suspended; the four warps meet at a named barrier (a flag per parity)
                volatile uint32_t* const flag = reinterpret_cast<volatile uint32_t*>(smem + G::kOffHolder + 4) + buf;
                if (warp == 2 && lane == 0)
                    *flag = wait_mbar(p.wait, acc_full_bar(buf), (local >> 1) & 1, kErrWaitAcc) ? 1u : 0u;
                __syncwarp();
                named_barrier_sync(1, 128);
                if (*flag == 0u) {
                    ok = false;
                    break;
                }
            }
            tc_fence_after_sync();
            const int row0 = tm * 256 + static_cast<int>(rank * 128 + q * 32);
            const int col0 = tn * 256 + (half > 0 ? 128 : 0);
            const int chunks = half < 0 ? 8 : 4;
            const uint32_t t_row = tmem_base + ((q * 32u) << 16) + (buf ? G::kCol1 : 0);
            // accumulator 0 shares its last columns, accumulator 1 its first: those are read first
            auto chunk_of = [&](int i) { return buf ? i : chunks - 1 - i; };
            uint32_t v[G::kFirstChunks][32];
#pragma unroll
            for (int i = 0; i < G::kFirstChunks; ++i)
                if (i < chunks) tmem_load_32cols(t_row + 32 * chunk_of(i), v[i]);
            tmem_wait_ld();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(map_to_cta(acc_free_bar, 0));
#pragma unroll
            for (int i = 0; i < G::kFirstChunks; ++i)
                if (i < chunks) store_sums(p, &tmap_c, buf_addr, buf_ptr, v[i], alpha, row0, col0 + 32 * chunk_of(i));
#pragma unroll 1
            for (int i = G::kFirstChunks; i < chunks; ++i) {
                tmem_load_32cols(t_row + 32 * chunk_of(i), v[0]);
                tmem_wait_ld();
                store_sums(p, &tmap_c, buf_addr, buf_ptr, v[0], alpha, row0, col0 + 32 * chunk_of(i));
            }
            tc_fence_before_sync();
        }
        if (lane == 0) bulk_wait_group<0>();
    }
    __syncwarp();
    tc_fence_before_sync();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

}  // namespace fp4
}  // namespace hk
