// Host side of hk_attention_kv8_shared (include/hk_gemm.h): argument checks,
// workspace and launches.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <mutex>

#include "../../include/hk_gemm.h"
#include "host_internal.h"
#include "kv8_host.h"
#include "kv8_shared.cuh"
#include "kv8_shared_mma.cuh"

namespace {

using namespace hk::kv8;
using namespace hk_kv8;

std::mutex g_setup_mutex;
bool g_setup[kMaxDevices] = {};

template <int kD, typename T, int kWarps>
cudaError_t setup_own() {
    return cudaFuncSetAttribute(kv8_own_kernel<kD, T, kWarps>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                BlockGeometry<kD, kWarps>::kSmemBytes);
}

template <int kD, typename T>
cudaError_t setup_one() {
    return cudaFuncSetAttribute(kv8_shared_kernel<kD, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, SharedGeometry<kD>::kSmemBytes);
}

// (a split of registers that adds up to more than the launch has would wait for ever)
template <int kD, typename T>
cudaError_t setup_wide() {
    cudaFuncAttributes a;
    cudaError_t e = cudaFuncGetAttributes(&a, kv8_shared_mma_kernel<kD, T>);
    if (e == cudaSuccess && a.numRegs * kWideThreads < kWideRegisters) e = cudaErrorLaunchOutOfResources;
    if (e == cudaSuccess) e = setup_own<kD, T, 1>();
    if (e == cudaSuccess) e = setup_own<kD, T, 2>();
    if (e == cudaSuccess) e = setup_own<kD, T, 4>();
    if (e == cudaSuccess) e = setup_own<kD, T, 8>();
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kv8_shared_mma_kernel<kD, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, WideGeometry<kD>::kSmemBytes);
    return e;
}

hk_status setup(int device) {
    std::lock_guard<std::mutex> lock(g_setup_mutex);
    if (g_setup[device]) return HK_OK;
    cudaError_t e = setup_one<64, __nv_bfloat16>();
    if (e == cudaSuccess) e = setup_one<64, __half>();
    if (e == cudaSuccess) e = setup_one<128, __nv_bfloat16>();
    if (e == cudaSuccess) e = setup_one<128, __half>();
    if (e == cudaSuccess) e = setup_wide<64, __nv_bfloat16>();
    if (e == cudaSuccess) e = setup_wide<64, __half>();
    if (e == cudaSuccess) e = setup_wide<128, __nv_bfloat16>();
    if (e == cudaSuccess) e = setup_wide<128, __half>();
    if (e != cudaSuccess) return cuda_fail(HK_ERR_CUDA, "configuring the shared attention kernels", e);
    g_setup[device] = true;
    return HK_OK;
}

// Tiles per warp up to which a sequence's own unit is a block's, beside the tensor-core kernel; beyond, it is spread over the
// GPU: long ones among few would leave SMs idle, one long one among many would be waited for. Both sides (a block's, spread), 8 KV
// heads, behind 8192 tokens, in microseconds: 64 sequences with 100 tokens of their own 53 and 59, with 1000 75 and 102, with
// 4000 132 and 160; 4 sequences with 2000 37 and 41, with 4000 47 and 43, with 16000 112 and 77.
constexpr int kOwnTiles = 32, kOwnTilesOfMany = 64;

// Sequences of one launch: what the kernel plans for, and as many as keep the sums of whole units at 2^17 rows (two of
// 64 MB at head dimension 128).
int64_t launch_batch(int64_t B, int64_t T, int64_t Hq) {
    return std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(B, kMaxShared), (int64_t(1) << 17) / (T * Hq)));
}

constexpr uint32_t kFormFlags = HK_KV8_FEW_ROWS | HK_KV8_MANY_ROWS;

// Can the tensor-core kernel take the shared units? It reads 16-byte aligned rows and holds so many groups.
bool wide_can(const void* Q, const int64_t q_strides[3], int64_t G) {
    return rows_aligned(Q, q_strides) && G <= kWideGroups;
}

// Who takes the call: attention_kv8 (every sequence reads all its tokens), the few-row kernels, or the tensor-core
// kernel with the few-row ones beside it.
enum Form { kOwn, kFew, kWide };

// Query rows of a sequence and KV head from which attention_kv8's own tiles are full and it takes the call. Both sides
// (tensor-core kernel here, attention_kv8), 8 KV heads of 128, in microseconds: 1024 rows, 8 sequences behind 2048, 8192 and
// 32768 tokens 260 and 108, 483 and 294, 1417 and 1523; 512 rows 141 and 69, 253 and 180, 714 and 1515. All in bf16: fp16 rows are then
// attention_kv8's few-row kernels', which take several times as long (include/hk_gemm.h), and were not measured against this form.
constexpr int64_t kOwnTileRows = 1024;

// By an estimate of the three times in microseconds, with the table's width for the lengths (which the host does not know) and
// all of it shared: a call of one token, every row that is joined, and every token of the table, of which attention_kv8 takes what
// attention_cost says (and a tenth for lengths that do not divide evenly), units of 16 stacked rows 48 millionths each (head
// dimension 64: 30), units of 128 rows 75 (55).
// Measured (attention_kv8, units of 16, of 128 rows; 8 KV heads of 128, 8 query heads each, one group of sequences with
// 300 tokens of their own): 8 behind 2048 tokens 14, 25, 30; 8 behind 8192 30, 32, 33; 16 behind 8192 52, 47, 36;
// 64 behind 2048 56, 67, 42; 64 behind 32768 548, 409, 107. 32 KV heads of a query head each: 16 behind 500 20, 22, 32;
// 16 behind 8192 153, 54, 54; 16 behind 32768 560, 87, 102. Head dimension 64: 16 behind 2048 14, 22, 26; 16 behind 8192 40, 34, 29;
// 64 of 16 query heads behind 4096 (their own tiles are full) 43, 54. It errs where two are near: 4 behind 32768 52, 50, 44 (it
// takes the second). All in bf16 with aligned rows and tables as wide as the sequences: fp16 and other rows go by the same figures, and where
// the table is much wider the estimates are of more tokens than there are (8 behind 2048 tokens in a table of 131072: the third, 30 for 14).
Form choose(const hk_kv8_cache* c, int64_t B, int64_t T, int64_t Hq, int64_t max_pages, int64_t G, bool wide, bool many) {
    const int64_t group = Hq / c->heads;
    if (T * group >= kOwnTileRows || launch_batch(B, T, Hq) < 2) return kOwn;
    const double room = 1e-6 * static_cast<double>(max_pages * c->page_size), stacked = static_cast<double>(B * T * group) / G;
    const double rows = static_cast<double>(B * T) * Hq, groups = static_cast<double>(G) * c->heads;
    const bool d64 = c->head_dim == 64;
    const double own_us = 8.0 + 1.1 * room * attention_cost(c, B, T, Hq, max_pages, many);
    const double few_us = (d64 ? 15.0 + 0.002 * rows : 18.0 + 0.006 * rows) + room * (d64 ? 30.0 : 48.0) * groups * std::ceil(stacked / kRows);
    const double wide_us = (d64 ? 25.0 : 30.0) + 0.001 * rows + room * (d64 ? 55.0 : 75.0) * groups * std::ceil(stacked / kWideRows);
    if (wide && wide_us < std::min(own_us, few_us)) return kWide;
    return few_us < own_us ? kFew : kOwn;
}

struct Workspace {
    int64_t whole[2], slots, rows;   // rows of sums: of split units of 16 rows, of whole ones, of split units of 128 rows
    int64_t shared_units;
    size_t ml, info, shared_info, seqs, total;
};

Workspace workspace(const hk_kv8_cache* c, int64_t B, int64_t T, int64_t Hq, int64_t G, bool wide) {
    const int64_t n = launch_batch(B, T, Hq), group = Hq / c->heads;
    const int64_t warps = 2 * kSms * kDecodeWarps;
    Workspace w;
    w.whole[0] = 2 * warps * kRows;
    w.whole[1] = w.whole[0] + n * T * Hq;
    w.slots = w.whole[1] + n * T * Hq;
    w.rows = w.slots + (wide ? int64_t(2) * kSms * kWideRows : 0);
    w.shared_units = n * T * group / kRows + std::min<int64_t>(G, kMaxShared) + 2;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    w.ml = up(static_cast<size_t>(w.rows * c->head_dim) * 4);
    w.info = w.ml + up(static_cast<size_t>(w.rows) * 8);
    w.shared_info = w.info + up(static_cast<size_t>(n * c->heads * ceil_div(T * group, kRows)) * sizeof(int4));
    w.seqs = w.shared_info + up(static_cast<size_t>(c->heads * w.shared_units) * sizeof(int4));
    w.total = w.seqs + up(static_cast<size_t>(n) * sizeof(int4));
    return w;
}

bool shape_ok(const hk_kv8_cache* c, int64_t B, int64_t T, int64_t Hq, int64_t max_pages, int64_t G) {
    return c && cache_shape_ok(c) && table_width_ok(max_pages, c->page_size) && B > 0 && B <= kLimit && T > 0 && Hq >= c->heads &&
           Hq <= kLimit && Hq % c->heads == 0 && T <= kLimit / 16 / (Hq / c->heads) && G > 0 && G <= B;
}

template <int kD, typename T, int kWarps>
cudaError_t launch_own(const CUtensorMap& tk, const CUtensorMap& tv, const SharedParams& p, cudaStream_t st) {
    return launch_early(&kv8_own_kernel<kD, T, kWarps>, dim3(static_cast<unsigned>(int64_t(p.n) * p.Hkv * p.row_tiles)),
                        dim3(32 * kWarps), BlockGeometry<kD, kWarps>::kSmemBytes, st, tk, tv, p);
}

template <int kD, typename T>
cudaError_t launch_spread(const CUtensorMap& tk, const CUtensorMap& tv, const SharedParams& p, cudaStream_t st) {
    return launch_early(&kv8_shared_kernel<kD, T>, dim3(static_cast<unsigned>(p.warps / kDecodeWarps)), dim3(32 * kDecodeWarps),
                        SharedGeometry<kD>::kSmemBytes, st, tk, tv, p);
}

// Long own parts over the GPU, the shared units on the tensor cores (a run of blocks to every SM), then the other own parts
// and the output: the last of them beside the last of the shared units, whose SMs do not all end at a time.
template <int kD, typename T>
cudaError_t launch_wide(const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& wide_k, const CUtensorMap& wide_v,
                        SharedParams& p, cudaStream_t st) {
    const int64_t units = int64_t(p.n) * p.Hkv * p.row_tiles;
    const int warps = block_warps(units, kBlockWarps);
    p.own_limit = warps * (units >= kSms ? kOwnTilesOfMany : kOwnTiles);
    cudaError_t e = launch_spread<kD, T>(tk, tv, p, st);
    if (e == cudaSuccess)
        e = launch_early(&kv8_shared_mma_kernel<kD, T>, dim3(static_cast<unsigned>(p.wide_runs)), dim3(kWideThreads),
                         WideGeometry<kD>::kSmemBytes, st, wide_k, wide_v, p);
    if (e != cudaSuccess) return e;
    switch (warps) {
        case 1: return launch_own<kD, T, 1>(tk, tv, p, st);
        case 2: return launch_own<kD, T, 2>(tk, tv, p, st);
        case 4: return launch_own<kD, T, 4>(tk, tv, p, st);
        default: return launch_own<kD, T, 8>(tk, tv, p, st);
    }
}

template <int kD, typename T>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& wide_k, const CUtensorMap& wide_v,
                   SharedParams p, cudaStream_t st) {
    if (p.wide_runs > 0) return launch_wide<kD, T>(tk, tv, wide_k, wide_v, p, st);
    const cudaError_t e = launch_spread<kD, T>(tk, tv, p, st);
    if (e != cudaSuccess) return e;
    const int64_t rows = int64_t(p.n) * p.T * p.Hq;
    // Warps to a row of the joining kernel, eight, two and one measured, calls in microseconds: 32 rows 20.1, 23.8, 29.8; 512 34.9,
    // 37.0, 38.6; 1176 43.5, 42.5, 45.0; 2048 93, 83, 85; 8192 180, 159, 153.
    const int split = rows <= 6 * kSms ? 8 : rows <= 24 * kSms ? 2 : 1;
    auto* fn = split == 8 ? &kv8_shared_combine_kernel<kD, T, 8> : split == 2 ? &kv8_shared_combine_kernel<kD, T, 2> : &kv8_shared_combine_kernel<kD, T, 1>;
    return launch_early(fn, dim3(static_cast<unsigned>(ceil_div(rows * split, 8))), dim3(256), 0, st, p);
}

// The form of a call.
Form form_of(uint32_t flags, const void* Q, int32_t type, const int64_t q_strides[3], const hk_kv8_cache* c, int64_t max_pages,
             const void* O, const int64_t o_strides[3], int64_t B, int64_t T, int64_t Hq, int64_t G) {
    if (flags & kFormFlags) return flags & HK_KV8_MANY_ROWS ? kWide : kFew;
    return choose(c, B, T, Hq, max_pages, G, wide_can(Q, q_strides, G), many_rows_can(Q, type, q_strides, O, o_strides, B, T, Hq));
}

}  // namespace

extern "C" size_t hk_attention_kv8_shared_workspace_size_ex(const void* Q, int32_t type, const int64_t q_strides[3],
                                                            const hk_kv8_cache* cache, int64_t max_pages, const void* O,
                                                            const int64_t o_strides[3], int64_t B, int64_t T, int64_t Hq, int64_t G,
                                                            uint32_t flags) {
    if (!shape_ok(cache, B, T, Hq, max_pages, G) || !q_strides || !o_strides) return 0;
    const Form form = form_of(flags, Q, type, q_strides, cache, max_pages, O, o_strides, B, T, Hq, G);
    return form == kOwn ? hk_attention_kv8_workspace_size_ex(Q, type, q_strides, cache, max_pages, O, o_strides, B, T, Hq, 0)
                        : workspace(cache, B, T, Hq, G, form == kWide).total;
}

extern "C" size_t hk_attention_kv8_shared_workspace_size(const hk_kv8_cache* cache, int64_t B, int64_t T, int64_t Hq,
                                                         int64_t max_pages, int64_t G) {
    if (!shape_ok(cache, B, T, Hq, max_pages, G)) return 0;
    // (whatever the queries' type and alignment, and for every form that the flags ask for)
    size_t own = 0;
    for (int i = 0; i < 4; ++i)
        if (choose(cache, B, T, Hq, max_pages, G, (i & 1) && G <= kWideGroups, i & 2) == kOwn)
            own = hk_attention_kv8_workspace_size(cache, B, T, Hq, max_pages);
    return std::max(own, T * (Hq / cache->heads) < kOwnTileRows ? workspace(cache, B, T, Hq, G, G <= kWideGroups).total : size_t(0));
}

extern "C" hk_status hk_attention_kv8_shared_ex(const void* Q, int32_t type, const int64_t q_strides[3], const hk_kv8_cache* cache,
                                                const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                                                const int32_t* lengths, const int32_t* counts, const int32_t* groups,
                                                const int32_t* shared, int64_t G, void* O, const int64_t o_strides[3], float* lse,
                                                int64_t B, int64_t T, int64_t Hq, int32_t causal, float scale, void* scratch,
                                                size_t workspace_bytes, uint32_t flags, uint64_t timeout_ns, void* stream) {
    hk_status s = check_cache(cache);
    if (s != HK_OK) return s;
    if ((flags & ~(kFormFlags | HK_KV8_FAULT_DROP_ARRIVE)) || (flags & kFormFlags) == kFormFlags) return fail(HK_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
    if (type != HK_TYPE_BF16 && type != HK_TYPE_FP16) return fail(HK_ERR_INVALID_ARG, "element type %d (bf16 or fp16)", (int)type);
    if (B < 0 || T < 0 || Hq < 0 || B > kLimit || T > kLimit || Hq > kLimit) return fail(HK_ERR_INVALID_ARG, "invalid size");
    if (Hq % cache->heads) return fail(HK_ERR_INVALID_ARG, "Hq=%lld is not a multiple of the cache's %d heads", (long long)Hq, (int)cache->heads);
    if (!std::isfinite(scale) || scale < 0.0f) return fail(HK_ERR_INVALID_ARG, "the scale must be finite and not negative");
    if (B == 0 || T == 0 || Hq == 0) return HK_OK;
    if (G < 1 || G > B) return fail(HK_ERR_INVALID_ARG, "%lld groups of %lld sequences", (long long)G, (long long)B);
    if ((s = check_table(block_table, table_stride, max_pages, B, lengths, counts, cache->page_size)) != HK_OK) return s;
    if (!groups || !shared) return fail(HK_ERR_INVALID_ARG, "null groups or shared tokens");
    if (!aligned(groups, 4) || !aligned(shared, 4)) return fail(HK_ERR_MISALIGNED, "groups and shared tokens must be 4-byte aligned");
    if (!Q || !O || !q_strides || !o_strides) return fail(HK_ERR_INVALID_ARG, "null queries, output or strides");
    if (!aligned(Q, 2) || !aligned(O, 2) || !aligned(lse, 4)) return fail(HK_ERR_MISALIGNED, "a pointer is not aligned to its elements");
    const int64_t sizes[3] = {B, T, Hq};
    for (int i = 0; i < 3; ++i)
        if (sizes[i] > 1 && std::llabs(o_strides[i]) < cache->head_dim) return fail(HK_ERR_INVALID_ARG, "the output's rows overlap");
    if (!shape_ok(cache, B, T, Hq, max_pages, G)) return fail(HK_ERR_INVALID_ARG, "problem too large");
    const int64_t group = Hq / cache->heads;
    const size_t need = hk_attention_kv8_shared_workspace_size_ex(Q, type, q_strides, cache, max_pages, O, o_strides, B, T, Hq, G, flags);
    if (need > 0 && (!scratch || workspace_bytes < need))
        return fail(HK_ERR_WORKSPACE, "%zu bytes of workspace needed, %zu given", need, scratch ? workspace_bytes : size_t(0));
    if (!aligned(scratch, 256)) return fail(HK_ERR_WORKSPACE, "the workspace must be 256-byte aligned");
    if ((flags & HK_KV8_MANY_ROWS) && !wide_can(Q, q_strides, G))
        return fail(HK_ERR_INVALID_ARG, "the tensor-core kernel takes queries with 16-byte aligned rows, and %d groups", kWideGroups);
    if ((flags & kFormFlags) && T * group >= kOwnTileRows)
        return fail(HK_ERR_INVALID_ARG, "%lld query rows of a sequence and KV head: attention_kv8's", (long long)(T * group));
    const Form form = form_of(flags, Q, type, q_strides, cache, max_pages, O, o_strides, B, T, Hq, G);
    if (form == kOwn)
        return hk_attention_kv8_ex(Q, type, q_strides, cache, block_table, table_stride, max_pages, lengths, counts, O, o_strides, lse,
                                   B, T, Hq, causal, scale, scratch, workspace_bytes, flags & ~kFormFlags, timeout_ns, stream);
    const bool wide = form == kWide;
    const int64_t batch = launch_batch(B, T, Hq), row_tiles = ceil_div(T * group, kRows);
    // (tiles of one launch, at most: every sequence's own and every group's shared ones)
    const int64_t unit_tiles = ceil_div(max_pages * cache->page_size, kTileKeys);
    if (unit_tiles > kLimit / (cache->heads * (batch * (2 * row_tiles + 1) + std::min<int64_t>(G, kMaxShared))))
        return fail(HK_ERR_INVALID_ARG, "problem too large");
    int device = 0, sms = 0;
    if ((s = current_device(&device, &sms)) != HK_OK) return s;
    if ((s = setup(device)) != HK_OK) return s;
    uint32_t* status = nullptr;
    if ((s = hk_host::status_word(device, &status)) != HK_OK) return s;
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    if ((s = hk_host::tensor_map_encoder(&enc)) != HK_OK) return s;
    CUtensorMap tk, tv;
    if ((s = encode_codes(enc, &tk, cache->k_codes, cache, kTileKeys)) != HK_OK) return s;
    if ((s = encode_codes(enc, &tv, cache->v_codes, cache, kTileKeys)) != HK_OK) return s;
    CUtensorMap wk = tk, wv = tv;                    // whole pages at a time
    if (wide && (s = encode_codes(enc, &wk, cache->k_codes, cache, cache->page_size)) != HK_OK) return s;
    if (wide && (s = encode_codes(enc, &wv, cache->v_codes, cache, cache->page_size)) != HK_OK) return s;

    const Workspace w = workspace(cache, B, T, Hq, G, wide);
    char* const base = static_cast<char*>(scratch);
    SharedParams p = {};
    p.q = Q;
    p.q_stride_b = q_strides[0];
    p.q_stride_t = q_strides[1];
    p.q_stride_h = q_strides[2];
    p.o = O;
    p.o_stride_b = o_strides[0];
    p.o_stride_t = o_strides[1];
    p.o_stride_h = o_strides[2];
    p.vec_q = rows_aligned(Q, q_strides);
    p.vec_o = rows_aligned(O, o_strides);
    p.lse = lse;
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    p.table = block_table;
    p.table_stride = table_stride;
    p.lengths = lengths;
    p.counts = counts;
    p.B = static_cast<int32_t>(B);
    p.T = static_cast<int32_t>(T);
    p.Hq = static_cast<int32_t>(Hq);
    p.Hkv = cache->heads;
    p.group = static_cast<int32_t>(group);
    p.row_tiles = static_cast<int32_t>(row_tiles);
    p.page_size = cache->page_size;
    p.page_shift = page_shift(cache->page_size);
    p.max_pages = static_cast<int32_t>(max_pages);
    p.num_pages = cache->num_pages;
    p.causal = causal ? 1 : 0;
    p.scale_log2 = static_cast<float>(
        1.4426950408889634 * (scale != 0.0f ? static_cast<double>(scale) : 1.0 / std::sqrt(static_cast<double>(cache->head_dim))));
    p.flags = flags & HK_KV8_FAULT_DROP_ARRIVE ? kFlagDropArrive : 0u;
    p.warps = 2 * std::min(sms, kSms) * kDecodeWarps;
    p.part_o = reinterpret_cast<float*>(base);
    p.part_ml = reinterpret_cast<float*>(base + w.ml);
    p.info = reinterpret_cast<int4*>(base + w.info);
    p.wait.status = status;
    p.wait.timeout_ns = timeout_ns ? timeout_ns : kDefaultTimeoutNs;
    p.groups = groups;
    p.shared = shared;
    p.G = static_cast<int32_t>(G);
    p.all = p.B;
    p.whole[0] = w.whole[0];
    p.whole[1] = w.whole[1];
    p.shared_info = reinterpret_cast<int4*>(base + w.shared_info);
    p.shared_units = static_cast<int32_t>(w.shared_units);
    p.wide_runs = wide ? std::min(sms, kSms) : 0;
    p.shared_slots = w.slots;
    p.seqs = reinterpret_cast<int4*>(base + w.seqs);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    for (int64_t b0 = 0; b0 < B; b0 += batch) {       // (launches of one stream: they may share the workspace)
        p.b0 = static_cast<int32_t>(b0);
        p.n = static_cast<int32_t>(std::min<int64_t>(B - b0, batch));
        p.wait.launch_id = hk_host::next_launch_id();
        const bool half = type == HK_TYPE_FP16;
        cudaError_t e;
        if (cache->head_dim == 64) e = half ? launch<64, __half>(tk, tv, wk, wv, p, st) : launch<64, __nv_bfloat16>(tk, tv, wk, wv, p, st);
        else e = half ? launch<128, __half>(tk, tv, wk, wv, p, st) : launch<128, __nv_bfloat16>(tk, tv, wk, wv, p, st);
        if (e != cudaSuccess) return cuda_fail(HK_ERR_LAUNCH, "launching the shared attention", e);
    }
    return HK_OK;
}

extern "C" hk_status hk_attention_kv8_shared(const void* Q, int32_t type, const int64_t q_strides[3], const hk_kv8_cache* cache,
                                             const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                                             const int32_t* lengths, const int32_t* counts, const int32_t* groups,
                                             const int32_t* shared, int64_t G, void* O, const int64_t o_strides[3], float* lse,
                                             int64_t B, int64_t T, int64_t Hq, int32_t causal, float scale, void* workspace,
                                             size_t workspace_bytes, void* stream) {
    return hk_attention_kv8_shared_ex(Q, type, q_strides, cache, block_table, table_stride, max_pages, lengths, counts, groups, shared,
                                      G, O, o_strides, lse, B, T, Hq, causal, scale, workspace, workspace_bytes, 0u, 0u, stream);
}
