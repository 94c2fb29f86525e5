// The shared part of kv8_shared.cuh for many query rows, on the fifth-generation tensor cores.
//
// With 64 sequences of 8 query heads per KV head a shared token meets 512 rows: 4 · 512 · D
// operations for 2 · D bytes, so the tensor cores bound the work and mma.sync with 16 rows
// to a unit (each of which converts every tile again) is the wrong tool. Here a unit is 256 stacked rows
// (two tiles of 128) of a group and KV head, and codes become bf16 once per unit: E4M3 times
// a power of two is exact in it.
//
// The schedule of a CTA is the attention-forward kernel's (attn_kernel.cuh): two softmax
// warpgroups of one tile each, a thread to a row; one MMA-issuing warp per tile; S = Q·Kᵀ
// and O += P·V in Tensor Memory; a ring of K and V blocks of 128 tokens. Two things differ. The
// ring is filled by a converting warpgroup: it loads 16 codes per thread (the next block's loads are in
// flight while this one's codes are converted), moves their bits to where bf16 has
// them, multiplies by 2^120 (E4M3's exponent bias is 120 less; exact, subnormal codes
// too) and by the page's scale, and writes the 128-byte-swizzled rows that
// the MMAs read. And all units' blocks, in order, are cut into equal runs, one per CTA, since a
// prefix has few units and many blocks: each run leaves unnormalised rows, maxima
// and sums of its units in memory for the combining kernel.
//
// Registers: 512 threads begin with 128 each; the softmax warpgroups take 184, the
// converting one 96, the MMA-issuing warps (a warpgroup, two of them idle) 48.
#pragma once

#include "attn_kernel.cuh"
#include "kv8_shared.cuh"

namespace hk {
namespace kv8 {

constexpr int kWideRows = 256;         // stacked rows of a unit
constexpr int kWideGroups = 64;        // groups of a call on this form
constexpr int kWideThreads = 512;
constexpr int kWideSoftmaxWarps = 8;
constexpr int kConvertThreads = 128;
constexpr int kSoftmaxRegs = 168, kConvertRegs = 120, kIssueRegs = 56;
constexpr int kWideRegisters = 256 * kSoftmaxRegs + 128 * kConvertRegs + 128 * kIssueRegs;
static_assert(kWideRegisters <= kWideThreads * 128, "registers of the launch");
constexpr uint32_t kErrSoftmaxWait = 1u << 19;

template <int kD>
struct WideGeometry {
    using A = attn::AttnGeometry<kD>;
    static_assert(A::kRowSplit == 1, "a thread to a row");
    static constexpr int kOffPlan = A::kOffXchg;                              // blocks, first sequence, blocks of each group
    static constexpr int kSmemBytes = kOffPlan + (3 * kWideGroups + 2) * 4 + 1024;
    static_assert(kSmemBytes <= attn::kSmemLimit, "shared memory");
};

// A run's share of a unit: blocks [first, last) of `blocks` for rows from `row0` on.
struct WidePiece {
    int section, h, pair, first, last, blocks;
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
        const int pairs = (shared_rows(p, w.group.n) + kWideRows - 1) / kWideRows;
        int local = at - prefix[section];
        const int unit = local / w.blocks;
        w.first = local - unit * w.blocks;
        w.h = unit / pairs;
        w.pair = unit - w.h * pairs;
        w.last = min(w.blocks, w.first + end - at);
        at += w.last - w.first;
        return w;
    }
};

template <int kD>
__device__ __forceinline__ bool wide_has_second_tile(const SharedParams& p, const WidePiece& w) {
    return shared_rows(p, w.group.n) > w.pair * kWideRows + kWideRows / 2;
}

// Four codes to bf16 times `unit` (2^120) times `scale`, in two words of two.
__device__ __forceinline__ uint2 codes_to_bf16(uint32_t w, uint32_t unit, uint32_t scale) {
    const uint32_t h0 = __byte_perm(w, 0u, 0x1404), h1 = __byte_perm(w, 0u, 0x3424);     // each code in a high byte
    uint32_t a = (h0 & 0x80008000u) | (h0 >> 4 & 0x07F007F0u), b = (h1 & 0x80008000u) | (h1 >> 4 & 0x07F007F0u);
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(unit));
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(b) : "r"(unit));
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(scale));
    asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(b) : "r"(scale));
    return make_uint2(a, b);
}

// bf16 NaN (0x7FFF) in the places of two NaN codes, the low ones of `nan` (0xFF each).
__device__ __forceinline__ uint32_t nan_pair(uint32_t nan) { return __byte_perm(nan, 0u, 0x1100) & 0x7FFF7FFFu; }

// wait_mbar_poll() without a call: a kernel that splits its registers may make none.
__device__ __forceinline__ bool wide_wait(const WaitCtx& c, uint32_t bar, uint32_t parity, uint32_t code) {
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        if (mbar_test_wait(bar, parity)) return true;
        if ((it & 4095u) == 0) {
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

template <int kD>
__global__ void __launch_bounds__(kWideThreads, 1)
kv8_shared_mma_kernel(const uint8_t* __restrict__ k_codes, const uint8_t* __restrict__ v_codes, const SharedParams p) {
    using G = attn::AttnGeometry<kD>;
    using W = WideGeometry<kD>;
    constexpr int kTileQ = attn::kTileQ, kTiles = attn::kTiles, kBlockKV = attn::kBlockKV;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const smem = smem_raw + (base - raw);
    const uint32_t warp = threadIdx.x >> 5;
    const uint32_t lane = lane_id();

    const uint32_t q_full = base + G::kOffBars;
    auto kv_full = [&](int s) { return base + G::kOffBars + 8u * (1 + s); };
    auto kv_empty = [&](int s) { return base + G::kOffBars + 8u * (1 + G::kSlots + s); };
    auto s_full = [&](int t) { return base + G::kOffBars + 8u * (1 + 2 * G::kSlots + t); };
    auto s_free = [&](int t) { return base + G::kOffBars + 8u * (3 + 2 * G::kSlots + t); };
    auto p_full = [&](int t) { return base + G::kOffBars + 8u * (5 + 2 * G::kSlots + t); };
    auto o_done = [&](int t) { return base + G::kOffBars + 8u * (7 + 2 * G::kSlots + t); };
    const uint32_t q_empty = base + G::kOffBars + 8u * (9 + 2 * G::kSlots);
    auto p_smem = [&](int t) { return base + G::kOffP + static_cast<uint32_t>(t) * G::kPBytes; };
    auto slot_addr = [&](int s) { return base + G::kOffKV + static_cast<uint32_t>(s) * G::kTileBytes; };
    const uint32_t tmem_holder = base + G::kOffTmemHolder;
    int32_t* const prefix = reinterpret_cast<int32_t*>(smem + W::kOffPlan);
    int32_t* const first_of = prefix + kWideGroups + 1;
    int32_t* const blocks_of = first_of + kWideGroups + 1;

    if (threadIdx.x == 0) {
        mbar_init(q_full, kConvertThreads / 32);
        mbar_init(q_empty, kTiles);            // each tile's MMA issuer, once its last S of the piece is done
        for (int s = 0; s < G::kSlots; ++s) {
            mbar_init(kv_full(s), kConvertThreads / 32 + (s == 0 && (p.flags & kFlagDropArrive) ? 1 : 0));
            mbar_init(kv_empty(s), kTiles);
        }
        for (int t = 0; t < kTiles; ++t) {
            mbar_init(s_full(t), 1);
            mbar_init(s_free(t), 4 * 32);
            mbar_init(p_full(t), 4 * 32);
            mbar_init(o_done(t), 1);
        }
        fence_mbar_init_cluster();
    }
    if (warp == kWideSoftmaxWarps) {
        tmem_alloc_one(tmem_holder, G::kTmemCols);
        tmem_relinquish_one();
    }
    griddep_wait();                            // launched early behind the kernel that may have written the cache or q
    griddep_launch_dependents();               // (now: what follows on the stream may run beside this grid, see launch())
    // ---- the groups' blocks; the CTA's run
    {
        const int64_t room = static_cast<int64_t>(p.max_pages) * p.page_size;
        for (int j = static_cast<int>(threadIdx.x); j <= p.G; j += kWideThreads) {
            const int first = p.groups[j];
            const bool in_order = first >= 0 && first <= p.all;
            int blocks = 0;
            if (j < p.G && in_order) {
                const int next = p.groups[j + 1], shared = p.shared[j];
                if (next > first && next <= p.all && shared >= 0) {      // (what is out of order the other kernel reports)
                    const int len = p.lengths[first];
                    const int64_t most = min(min(static_cast<int64_t>(shared), static_cast<int64_t>(len)), room);
                    blocks = static_cast<int>(max(static_cast<int64_t>(0), most)) / kSharedStep;
                }
            }
            first_of[j] = first;
            if (j < p.G) blocks_of[j] = blocks;
        }
        __syncthreads();
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
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(smem + G::kOffTmemHolder);
    const int ctas = static_cast<int>(gridDim.x), self = static_cast<int>(blockIdx.x);
    const int total = prefix[p.G], per = (total + ctas - 1) / ctas;
    WideWalk walk{p, prefix, first_of, blocks_of, 0, 0, 0};
    walk.at = static_cast<int>(min(static_cast<int64_t>(total), static_cast<int64_t>(self) * per));
    walk.end = static_cast<int>(min(static_cast<int64_t>(total), static_cast<int64_t>(walk.at) + per));
    const int begin = walk.at;
    bool abort_seen = false;
    auto wait_lane0 = [&](uint32_t bar, uint32_t parity, uint32_t code) {      // a warp's wait: lane 0 polls, all see it
        uint32_t ok = 0;
        if (lane == 0) ok = wide_wait(p.wait, bar, parity, code) ? 1u : 0u;
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (ok) (void)mbar_test_wait(bar, parity);
        __syncwarp();
        return ok != 0;
    };

    if (warp >= 12) {
        // ------------------------------------------------ converting warps --
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvertRegs));
        constexpr int kTokenChunks = kD / 16;                          // 16-code pieces of a token
        constexpr int kLoads = kBlockKV * kTokenChunks / kConvertThreads;
        constexpr int kStepTokens = kConvertThreads / kTokenChunks;    // tokens between a thread's loads
        const int ct = static_cast<int>(threadIdx.x) - 12 * 32;
        const int chunk = ct % kTokenChunks, token = ct / kTokenChunks;
        int slot = 0;
        uint32_t ring_ph = 0;
        int pieces = 0;
        // pages and scales of the 32 pieces of 16 tokens of blocks [window, window + 4), one per lane
        struct Window {
            int page;
            uint32_t ks, vs;       // scales as bf16 pairs
        };
        for (WidePiece w = walk.next(); w.valid && !abort_seen; w = walk.next(), ++pieces) {
            const int32_t* const table = p.table + first_of[w.section] * p.table_stride;
            auto look_up = [&](int block) {
                Window x = {0, 0u, 0u};
                const int key = block * kBlockKV + static_cast<int>(lane) * 16;
                if (key < w.blocks * kBlockKV) {
                    const int32_t pg = table[key >> p.page_shift];
                    if (pg < 0 || pg >= p.num_pages) {
                        atomicOr(p.wait.status, kErrPage);
                    } else {
                        x.page = pg;
                        const int64_t ph = static_cast<int64_t>(pg) * p.Hkv + w.h;
                        const uint32_t ks = __float_as_uint(p.k_scale[ph]) >> 16, vs = __float_as_uint(p.v_scale[ph]) >> 16;
                        x.ks = ks | ks << 16;
                        x.vs = vs | vs << 16;
                    }
                }
                return x;
            };
            int window = w.first;
            Window cur = look_up(window), ahead = look_up(window + 4);
            auto load = [&](uint4 (&x)[kLoads], bool is_k, int block) {
                const bool in_cur = block < window + 4;
                const uint8_t* const codes = is_k ? k_codes : v_codes;
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    const int tok = token + i * kStepTokens;
                    const int page = __shfl_sync(0xffffffffu, in_cur ? cur.page : ahead.page, (block - window & 3) * 8 + (tok >> 4));
                    const int place = (block * kBlockKV + tok) & (p.page_size - 1);
                    const int64_t row = ((static_cast<int64_t>(page) * p.Hkv + w.h) << p.page_shift) + place;
                    x[i] = *reinterpret_cast<const uint4*>(codes + row * kD + 16 * chunk);
                }
            };
            // position u of the consumption order: K_0, (K_{j+1}, V_j)..., V_{n-1}
            const int n = w.last - w.first;
            auto at_position = [&](int u, bool& is_k) {
                if (u == 0) { is_k = true; return w.first; }
                if (u == 2 * n - 1) { is_k = false; return w.last - 1; }
                is_k = (u & 1) != 0;
                return w.first + (is_k ? (u + 1) / 2 : u / 2 - 1);
            };
            auto convert = [&](const uint4 (&x)[kLoads], bool is_k, int block) {
                const bool in_cur = block < window + 4;
                const int s = slot;
                const uint32_t parity = ring_ph ^ 1u;
                if (++slot == G::kSlots) {
                    slot = 0;
                    ring_ph ^= 1u;
                }
                if (!wait_lane0(kv_empty(s), parity, kErrWaitRing)) return false;
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    const int tok = token + i * kStepTokens;
                    const uint32_t mine = is_k ? (in_cur ? cur.ks : ahead.ks) : (in_cur ? cur.vs : ahead.vs);
                    const uint32_t scale = __shfl_sync(0xffffffffu, mine, (block - window & 3) * 8 + (tok >> 4));
                    const uint32_t words[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                    uint32_t o[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint2 v = codes_to_bf16(words[k], 0x7B807B80u, scale);
                        o[2 * k] = v.x;
                        o[2 * k + 1] = v.y;
                    }
                    // a code 0x7F or 0xFF is the only one whose magnitude carries into its sign bit when 1 is added
                    uint32_t carry = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) carry |= (words[k] & 0x7F7F7F7Fu) + 0x01010101u;
                    if (carry & 0x80808080u) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t nan = nan_codes(words[k]);
                            o[2 * k] |= nan_pair(nan);
                            o[2 * k + 1] |= nan_pair(nan >> 16);
                        }
                    }
                    // 16 columns of row `tok`: two 16-byte units of the 64-column half that they lie in; the halves' threads
                    // (which meet the same banks) write them in opposite order
                    const uint32_t row = slot_addr(s) + (chunk >> 2) * G::kChunkBytes + static_cast<uint32_t>(tok) * 128u;
                    const uint32_t unit = 2u * (chunk & 3), sw = static_cast<uint32_t>(tok) & 7u, flip = chunk >> 2 & 1;
                    const uint32_t first = row + (((unit + flip) ^ sw) << 4), second = row + (((unit + 1 - flip) ^ sw) << 4);
                    if (flip) {
                        st_shared_v4(first, o[4], o[5], o[6], o[7]);
                        st_shared_v4(second, o[0], o[1], o[2], o[3]);
                    } else {
                        st_shared_v4(first, o[0], o[1], o[2], o[3]);
                        st_shared_v4(second, o[4], o[5], o[6], o[7]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(kv_full(s));
                return true;
            };
            uint4 a[kLoads], b[kLoads];
            load(a, true, w.first);
            // ---- Q of this piece once both issuers have finished the previous one's S
            if (pieces > 0 && !wait_lane0(q_empty, (pieces - 1) & 1, kErrWaitRing)) {
                abort_seen = true;
                break;
            }
            {
                constexpr int kRowUnits = kD / 8;
                const int rows = shared_rows(p, w.group.n), per_seq = p.T * p.group;
                const int tiles = wide_has_second_tile<kD>(p, w) ? 2 : 1;
#pragma unroll 4
                for (int i = ct; i < tiles * kTileQ * kRowUnits; i += kConvertThreads) {
                    const int r = i / kRowUnits, unit = i % kRowUnits;
                    const int row = w.pair * kWideRows + r;
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (row < rows) {
                        const int seq = row / per_seq, rest = row - seq * per_seq, t = rest / p.group;
                        const uint16_t* const src = static_cast<const uint16_t*>(p.q) + (p.b0 + w.group.first + seq) * p.q_stride_b +
                                                    t * p.q_stride_t + static_cast<int64_t>(w.h * p.group + rest - t * p.group) * p.q_stride_h;
                        x = *reinterpret_cast<const uint4*>(src + 8 * unit);
                    }
                    const uint32_t tile = r / kTileQ, tr = r % kTileQ;
                    st_shared_v4(base + G::kOffQ + tile * G::kTileBytes + (unit >> 3) * G::kChunkBytes + tr * 128u +
                                     (((unit & 7u) ^ (tr & 7u)) << 4), x.x, x.y, x.z, x.w);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }
            // two positions at a time: one's loads are in flight while the other is converted
            bool ok = true;
            for (int u = 0; u < 2 * n && ok; u += 2) {
                bool is_k0, is_k1, is_k2 = false;
                const int b0 = at_position(u, is_k0), b1 = at_position(u + 1, is_k1);
                load(b, is_k1, b1);
                ok = convert(a, is_k0, b0);
                if (!ok) break;
                if (u + 2 < 2 * n) {
                    const int b2 = at_position(u + 2, is_k2);
                    // (V of a block follows K of the next: the window moves when both are past its first four blocks)
                    if (min(b1, b2) >= window + 4) {
                        window += 4;
                        cur = ahead;
                        ahead = look_up(window + 4);
                    }
                    load(a, is_k2, b2);
                }
                ok = convert(b, is_k1, b1);
            }
            if (!ok) abort_seen = true;
        }
    } else if (warp >= kWideSoftmaxWarps) {
        // ------------------------------------------- MMA issue, one warp per tile --
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        const int t = static_cast<int>(warp) - kWideSoftmaxWarps;
        if (t < kTiles && lane == 0) {
            auto wait = [&](uint32_t bar, uint32_t parity, uint32_t code) {
                if (abort_seen) return false;
                if (!wide_wait(p.wait, bar, parity, code)) abort_seen = true;
                return !abort_seen;
            };
            int s0 = 0;              // ring slot of the piece's first position
            uint32_t ph0 = 0;        // and its phase
            auto kv_slot = [&](int u) { return (s0 + u) % G::kSlots; };
            auto kv_parity = [&](int u) { return ph0 ^ static_cast<uint32_t>(((s0 + u) / G::kSlots) & 1); };
            const uint32_t qa = base + G::kOffQ + t * G::kTileBytes;
            const uint32_t s_tmem = tmem_base + G::kColS + t * kBlockKV;
            const uint32_t o_tmem = tmem_base + G::kColO + t * kD;
            const uint32_t pa = p_smem(t);
            const uint32_t p_tmem = tmem_base + G::kColP + t * (kBlockKV / 2);
            uint32_t jp = 0;
            bool any_block = false;
            int pieces = 0;
            for (WidePiece w = walk.next(); w.valid && !abort_seen; w = walk.next(), ++pieces) {
                const int n_all = w.last - w.first;
                const int n = t == 0 || wide_has_second_tile<kD>(p, w) ? n_all : 0;
                if (!wait(q_full, pieces & 1, kErrWaitData)) break;
                auto issue_s = [&](int j, int u) {
                    if ((j > 0 || any_block) && !wait(s_free(t), jp ^ static_cast<uint32_t>((j - 1) & 1), kErrWaitAcc)) return false;
                    if (!wait(kv_full(kv_slot(u)), kv_parity(u), kErrWaitData)) return false;
                    tc_fence_after_sync();
                    const uint32_t ka = slot_addr(kv_slot(u));
#pragma unroll
                    for (int kk = 0; kk < kD / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * G::kChunkBytes + (kk & 3) * 32;
                        mma_bf16_one(s_tmem, smem_desc_kmajor_sw128(qa + off), smem_desc_kmajor_sw128(ka + off), G::kIdescS,
                                     kk > 0 ? 1u : 0u);
                    }
                    mma_commit_one(s_full(t));
                    mma_commit_one(kv_empty(kv_slot(u)));
                    if (j == n - 1) mma_commit_one(q_empty);
                    return true;
                };
                if (n == 0) {
                    mbar_arrive(q_empty);
                } else if (issue_s(0, 0)) {
                    for (int j = 0; j < n && !abort_seen; ++j) {
                        if (j + 1 < n && !issue_s(j + 1, attn::pos_k(j + 1))) break;
                        const int uv = attn::pos_v(j, n_all);
                        if (!wait(kv_full(kv_slot(uv)), kv_parity(uv), kErrWaitData)) break;
                        if (!wait(p_full(t), jp ^ static_cast<uint32_t>(j & 1), kErrWaitAcc)) break;
                        tc_fence_after_sync();
                        const uint32_t va = slot_addr(kv_slot(uv));
#pragma unroll
                        for (int kk = 0; kk < kBlockKV / 16; ++kk) {
                            const uint64_t vdesc = smem_desc_mnmajor(va + kk * 2048, 128, G::kChunkBytes);
                            const uint32_t acc = (j == 0 && kk == 0) ? 0u : 1u;
                            if constexpr (G::kPInTmem)
                                mma_bf16_ts_one(o_tmem, p_tmem + kk * 8, vdesc, G::kIdescPV, acc);
                            else
                                mma_bf16_one(o_tmem, smem_desc_kmajor_sw128(pa + (kk >> 2) * G::kChunkBytes + (kk & 3) * 32), vdesc,
                                             G::kIdescPV, acc);
                        }
                        mma_commit_one(o_done(t));
                        mma_commit_one(kv_empty(kv_slot(uv)));
                    }
                }
                // positions that this tile does not use: arrive once each has landed
                auto release = [&](int u) {
                    if (!wait(kv_full(kv_slot(u)), kv_parity(u), kErrWaitData)) return false;
                    mbar_arrive(kv_empty(kv_slot(u)));
                    return true;
                };
                for (int u = 0; n == 0 && u < 2 * n_all && !abort_seen; ++u)
                    if (!release(u)) break;
                ph0 ^= static_cast<uint32_t>(((s0 + 2 * n_all) / G::kSlots) & 1);
                s0 = (s0 + 2 * n_all) % G::kSlots;
                jp ^= static_cast<uint32_t>(n & 1);
                any_block = any_block || n > 0;
            }
        }
    } else {
        // ------------------------------------------ softmax warpgroups --
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int t = static_cast<int>(warp >> 2) & 1;
        const uint32_t quarter = warp & 3u;
        const int r = static_cast<int>(quarter * 32 + lane);
        const uint32_t lane_off = (quarter * 32u) << 16;
        const uint32_t s_addr = tmem_base + lane_off + G::kColS + t * kBlockKV;
        const uint32_t o_addr = tmem_base + lane_off + G::kColO + t * kD;
        const float c = p.scale_log2;
        uint32_t jp = 0;
        int done = begin;              // blocks of the run before this piece
        for (WidePiece w = walk.next(); w.valid && !abort_seen; w = walk.next()) {
            const int n_all = w.last - w.first;
            const int n = t == 0 || wide_has_second_tile<kD>(p, w) ? n_all : 0;
            const bool whole = n_all == w.blocks;
            const int slot = 2 * self + (done == begin ? 0 : 1);
            if (w.first == 0 && threadIdx.x == 0) {     // this run holds the unit's first block: it tells how the unit is made up
                const int parts = whole ? 0 : (done + w.blocks - 1) / per - done / per + 1;
                p.shared_info[static_cast<int64_t>(w.h) * p.shared_units + shared_unit0(p, w.section, w.group.first) + w.pair] =
                    make_int4(parts, slot, self, 0);
            }
            done += n_all;
            float m = 0.0f, l = 0.0f;      // running maximum (log2 units) used for P, and sum of P
            for (int j = 0; j < n; ++j) {
                const uint32_t par = jp ^ static_cast<uint32_t>(j & 1);
                if (!wait_lane0(s_full(t), par, kErrSoftmaxWait)) {
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
                mbar_arrive(s_free(t));    // S is in registers: the next block's may be computed
                float acc[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int e0 = 16 * k;
                    float a = fmax3(__uint_as_float(v[e0]), __uint_as_float(v[e0 + 1]), __uint_as_float(v[e0 + 2]));
#pragma unroll
                    for (int e = 3; e < 15; e += 2) a = fmax3(a, __uint_as_float(v[e0 + e]), __uint_as_float(v[e0 + e + 1]));
                    acc[k] = fmaxf(a, __uint_as_float(v[e0 + 15]));
                }
                const float mx = fmax3(fmax3(acc[0], acc[1], acc[2]), fmax3(acc[3], acc[4], acc[5]), fmaxf(acc[6], acc[7]));
                float m_blk = mx * c;
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
                const uint64_t c2 = f32x2(c, c);
                const uint64_t nm2 = f32x2(-m, -m);
                uint64_t sum2[4] = {0, 0, 0, 0};
                uint32_t pk[64];
                constexpr bool kEarlyP = G::kPInTmem;
                constexpr int kFirstPairs = kEarlyP ? 32 : 64;
                auto rescale_o = [&]() {
                    if (__any_sync(0xffffffffu, alpha != 1.0f)) {
#pragma unroll
                        for (int cc = 0; cc < kD / 32; ++cc) {
                            uint32_t o[32];
                            tmem_load_32cols(o_addr + 32 * cc, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_store_32cols(o_addr + 32 * cc, o);
                        }
                    }
                };
                auto exp_pair = [&](int e) {
                    const uint64_t x = ffma2(f32x2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), c2, nm2);
                    float x0, x1;
                    f32x2_split(x, x0, x1);
                    const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                    sum2[e & 3] = fadd2(sum2[e & 3], f32x2(p0, p1));
                    pk[e] = pack_bf16x2_rn(__float_as_uint(p0), __float_as_uint(p1));
                };
#pragma unroll
                for (int e = 0; e < kFirstPairs; ++e) exp_pair(e);
                const uint32_t p_addr = tmem_base + lane_off + G::kColP + t * (kBlockKV / 2);
                if constexpr (kEarlyP) {
                    if (j > 0 && !wait_lane0(o_done(t), par ^ 1u, kErrSoftmaxWait)) {
                        abort_seen = true;
                        break;
                    }
                    tc_fence_after_sync();
                    rescale_o();
                    tmem_store_32cols(p_addr, *reinterpret_cast<const uint32_t(*)[32]>(&pk[0]));
                }
#pragma unroll
                for (int e = kFirstPairs; e < 64; ++e) exp_pair(e);
                {
                    const uint64_t s01 = fadd2(fadd2(sum2[0], sum2[1]), fadd2(sum2[2], sum2[3]));
                    float lo, hi;
                    f32x2_split(s01, lo, hi);
                    l += lo + hi;
                }
                if constexpr (kEarlyP) {
                    tmem_store_32cols(p_addr + 32, *reinterpret_cast<const uint32_t(*)[32]>(&pk[32]));
                    tmem_wait_st();
                } else {
                    // P·V of the previous block must be done before its P is overwritten and O rescaled
                    if (j > 0 && !wait_lane0(o_done(t), par ^ 1u, kErrSoftmaxWait)) {
                        abort_seen = true;
                        break;
                    }
                    tc_fence_after_sync();
                    rescale_o();
                    tmem_wait_st();
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const uint32_t row = p_smem(t) + hh * G::kChunkBytes + static_cast<uint32_t>(r) * 128u;
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            st_shared_v4(row + ((static_cast<uint32_t>(x) ^ (static_cast<uint32_t>(r) & 7u)) << 4), pk[32 * hh + 4 * x],
                                         pk[32 * hh + 4 * x + 1], pk[32 * hh + 4 * x + 2], pk[32 * hh + 4 * x + 3]);
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before_sync();
                mbar_arrive(p_full(t));
            }
            // ---- the row's sums, unnormalised (reading O here, before this warp publishes the next piece's first P,
            // orders these reads before the P·V that overwrites O)
            if (!abort_seen && n > 0) {
                if (!wait_lane0(o_done(t), jp ^ static_cast<uint32_t>((n - 1) & 1), kErrSoftmaxWait)) {
                    abort_seen = true;
                } else {
                    tc_fence_after_sync();
                    const int in_unit = t * kTileQ + r, row = w.pair * kWideRows + in_unit;
                    const int per_seq = p.T * p.group;
                    const bool live = row < shared_rows(p, w.group.n);
                    const int seq = row / per_seq, rest = row - seq * per_seq, tok = rest / p.group;
                    const int64_t out_row = (static_cast<int64_t>(w.group.first + seq) * p.T + tok) * p.Hq + w.h * p.group + rest - tok * p.group;
                    const int64_t at_row = whole ? p.whole[0] + out_row : p.shared_slots + static_cast<int64_t>(slot) * kWideRows + in_unit;
                    const bool any = l > 0.0f || l != l;
#pragma unroll
                    for (int cc = 0; cc < kD / 32; ++cc) {
                        uint32_t o[32];
                        tmem_load_32cols(o_addr + 32 * cc, o);
                        tmem_wait_ld();
                        if (live) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                st_global_v4(p.part_o + at_row * kD + 32 * cc + 4 * e, any ? o[4 * e] : 0u, any ? o[4 * e + 1] : 0u,
                                             any ? o[4 * e + 2] : 0u, any ? o[4 * e + 3] : 0u);
                        }
                    }
                    if (live) {
                        p.part_ml[2 * at_row] = any ? m : -INFINITY;
                        p.part_ml[2 * at_row + 1] = any ? l : 0.0f;
                    }
                    tc_fence_before_sync();
                }
            }
            jp ^= static_cast<uint32_t>(n & 1);
        }
    }

    if (abort_seen || wait_aborted(p.wait)) {
        // let MMAs that were already issued land before teardown
        for (int i = 0; i < 200; ++i) __nanosleep(1000);
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kWideSoftmaxWarps) {
        tc_fence_after_sync();
        tmem_dealloc_one(tmem_base, G::kTmemCols);
    }
}

}  // namespace kv8
}  // namespace hk
