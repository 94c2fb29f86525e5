// Host side of the paged 8-bit key/value cache (include/hk_gemm.h):
// hk_kv8_append and hk_attention_kv8: argument checks, tensor maps, workspace
// and launches.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <mutex>

#include "../../include/hk_gemm.h"
#include "host_internal.h"
#include "kv8_append.cuh"
#include "kv8_decode.cuh"
#include "kv8_host.h"
#include "kv8_prefill.cuh"

namespace {

using namespace hk::kv8;
using namespace hk_kv8;

template <typename T, int kD, int kWarps>
cudaError_t launch_append(const AppendParams& p, int steps, unsigned blocks, cudaStream_t st) {
    auto* fn = steps <= 1   ? &kv8_append_kernel<T, kD, kWarps, 1>
               : steps <= 2 ? &kv8_append_kernel<T, kD, kWarps, 2>
               : steps <= 4 ? &kv8_append_kernel<T, kD, kWarps, 4>
                            : &kv8_append_kernel<T, kD, kWarps, 8>;
    return launch_early(fn, dim3(blocks), dim3(256), 0, st, p);
}

template <typename T>
cudaError_t launch_append(const AppendParams& p, int D, bool one_warp, int steps, unsigned blocks, cudaStream_t st) {
    if (D == 64) return one_warp ? launch_append<T, 64, 1>(p, steps, blocks, st) : launch_append<T, 64, 8>(p, steps, blocks, st);
    return one_warp ? launch_append<T, 128, 1>(p, steps, blocks, st) : launch_append<T, 128, 8>(p, steps, blocks, st);
}

std::mutex g_setup_mutex;
bool g_setup[kMaxDevices] = {};
int g_clusters[kMaxDevices][kMaxCluster + 1] = {};     // clusters of each size that run at a time

template <int kD, typename T, int kWarps>
cudaError_t setup_block() {
    cudaError_t e = cudaFuncSetAttribute(kv8_decode_block_kernel<kD, T, kWarps>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         BlockGeometry<kD, kWarps>::kSmemBytes);
    if (e == cudaSuccess && kWarps == kBlockWarps)       // (clusters of 16 are more than every device has to run)
        e = cudaFuncSetAttribute(kv8_decode_block_kernel<kD, T, kWarps>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e;
}

template <int kD, typename T>
cudaError_t setup_decode() {
    cudaError_t e = cudaFuncSetAttribute(kv8_decode_kernel<kD, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, DecodeGeometry<kD>::kSmemBytes);
    if (e == cudaSuccess) e = setup_block<kD, T, 1>();
    if (e == cudaSuccess) e = setup_block<kD, T, 2>();
    if (e == cudaSuccess) e = setup_block<kD, T, 4>();
    if (e == cudaSuccess) e = setup_block<kD, T, 8>();
    return e;
}

template <int kD>
cudaError_t setup_prefill() {
    return cudaFuncSetAttribute(hk::attn::attn_fwd_kernel<kD, CachedItems>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                hk::attn::AttnGeometry<kD>::kSmemBytes);
}

hk_status setup(int device) {
    std::lock_guard<std::mutex> lock(g_setup_mutex);
    if (g_setup[device]) return HK_OK;
    cudaError_t e = setup_decode<64, __nv_bfloat16>();
    if (e == cudaSuccess) e = setup_decode<64, __half>();
    if (e == cudaSuccess) e = setup_decode<128, __nv_bfloat16>();
    if (e == cudaSuccess) e = setup_decode<128, __half>();
    if (e == cudaSuccess) e = setup_prefill<64>();
    if (e == cudaSuccess) e = setup_prefill<128>();
    // (a cluster needs its SMs in one part of the GPU: fewer blocks run at a time than there are SMs)
    for (int size = 1; size <= kMaxCluster && e == cudaSuccess; ++size) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        cfg.gridDim = dim3(static_cast<unsigned>(size * kSms));
        cfg.blockDim = dim3(32 * kBlockWarps);
        cfg.dynamicSmemBytes = BlockGeometry<128, kBlockWarps>::kSmemBytes;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(size);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        e = cudaOccupancyMaxActiveClusters(&clusters, kv8_decode_block_kernel<128, __nv_bfloat16, kBlockWarps>, &cfg);
        g_clusters[device][size] = clusters;
    }
    if (e != cudaSuccess) return cuda_fail(HK_ERR_CUDA, "configuring the cache attention kernels", e);
    g_setup[device] = true;
    return HK_OK;
}

// Sequences of one launch of the few-row kernels: units stay below 2^20 (or are one sequence's).
int64_t decode_batch(int64_t B, int64_t heads, int64_t row_tiles) {
    return std::min(B, std::min<int64_t>(kMaxBatch, std::max<int64_t>(1, (int64_t(1) << 20) / (heads * row_tiles))));
}

// Workspace of the kernel that spreads tiles over the GPU: partial sums and their
// maxima and sums for two units per warp, and a record per unit.
struct DecodeWorkspace {
    size_t ml, info, total;
};
DecodeWorkspace decode_workspace(const hk_kv8_cache* c, int64_t B, int64_t T, int64_t Hq) {
    const size_t warps = static_cast<size_t>(2 * kSms) * kDecodeWarps;
    const int64_t row_tiles = ceil_div(T * (Hq / c->heads), kRows);
    DecodeWorkspace w;
    w.ml = 2 * warps * kRows * static_cast<size_t>(c->head_dim) * 4;
    w.info = w.ml + 2 * warps * kRows * 2 * 4;
    w.total = w.info + static_cast<size_t>(decode_batch(B, c->heads, row_tiles) * c->heads * row_tiles) * sizeof(int4);
    return w;
}

// Query heads of a KV head that share a 128-row tile of the tensor-core kernel, as a power of two: all, where
// they divide it evenly.
int pack_shift_of(int64_t group) {
    int shift = 0;
    while (shift < 7 && group % (int64_t(2) << shift) == 0) ++shift;
    return shift;
}

// Tiles per warp up to which a unit is one block's or cluster's; beyond, all tiles are spread over the whole GPU and
// a second kernel adds up. By the table's width, which the host knows. Both sides, D 128, 8 KV heads, in microseconds
// by block or cluster and spread: 1 x 500 tokens 7.8 and 10.8, 1 x 32768 24.5 and 32.6, 8 x 4000 20.9 and 25.8,
// 64 x 1000 29 and 40, 64 x 2000 49 and 61; of every length up to 2000 46.5 and 46.4: lengths that differ cost blocks
// more, and longer tables leave more room for that, while what spreading costs (lengths are summed up before the
// first load, sums go through memory: some 10) stays the same.
constexpr int kBlockTiles = 32;

// Sequences that are brought to bf16 at a time: as many as fit 512 MB, one at least.
constexpr int64_t kWidenBytes = int64_t(512) << 20;

struct PrefillWorkspace {
    int64_t rows, seqs;      // rows of a head, sequences at a time
    size_t half, total;      // bytes of the keys (the values follow), of both
};

PrefillWorkspace prefill_workspace(const hk_kv8_cache* c, int64_t B, int64_t max_pages) {
    PrefillWorkspace w;
    w.rows = max_pages * c->page_size;
    const int64_t one = 2 * w.rows * c->heads * c->head_dim * 2;
    w.seqs = std::max<int64_t>(1, std::min<int64_t>(B, kWidenBytes / one));
    w.seqs = std::min<int64_t>(w.seqs, 65535);
    w.half = static_cast<size_t>(w.seqs * one / 2);
    w.total = 2 * w.half;
    return w;
}

// Millionths of a microsecond per cached token of each form (figures at many_rows).
double unit_cost(const hk_kv8_cache* c, int64_t B, int64_t T, int64_t Hq) {
    return 35.0 * static_cast<double>(B) * c->heads * ceil_div(T * (Hq / c->heads), kRows);
}

double item_cost(const hk_kv8_cache* c, int64_t B, int64_t T, int64_t Hq, int64_t max_pages) {
    const int pack = pack_shift_of(Hq / c->heads);
    const double seq_items = static_cast<double>(Hq >> pack) * ceil_div(T, (hk::attn::kTiles * hk::attn::kTileQ) >> pack);
    const int64_t seqs = prefill_workspace(c, B, max_pages).seqs;
    const double rounds = static_cast<double>(B / seqs) * std::ceil(static_cast<double>(seqs) * seq_items / kSms) +
                          std::ceil(static_cast<double>(B % seqs) * seq_items / kSms);
    return 13000.0 * rounds + 120.0 * static_cast<double>(B) * c->heads;
}

// Do the rows go to the tensor-core kernel? Both forms' time grows with the cached tokens; per token, in
// millionths of a microsecond, measured (D 64 and 128, 2000 to 16000 tokens): 35 for each unit of 16 rows and KV
// head, whatever their number, against 13000 for each round of 256-row items over the SMs and 120 for bringing
// one KV head's token to bf16. So 4 sequences x 8 heads x 8 queries run at 96 us by units and 236 us by items
// (16000 tokens), 32 queries at 300 and 269 us. Sequences that are not widened together (a wide table) do not
// share a round: 64 sequences of up to 2048 tokens, 32 queries of 32 heads, take 230 us by units and 2112 us by
// items with a table of 131072 tokens, 180 us by items with one of 2048.
bool many_rows(const hk_kv8_cache* c, int64_t B, int64_t T, int64_t Hq, int64_t max_pages) {
    return unit_cost(c, B, T, Hq) > item_cost(c, B, T, Hq, max_pages);
}

// Queries as [B, T, heads, D] in boxes of 64 columns × `pack` heads × 128 / pack tokens.
hk_status encode_queries(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, const void* q, const int64_t strides[3],
                         int64_t B, int64_t T, int64_t Hq, int64_t D, int pack) {
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hq), static_cast<cuuint64_t>(T),
                          static_cast<cuuint64_t>(B)};
    // (the stride of a dimension of one is never used, but has to be a valid one)
    cuuint64_t st[3] = {static_cast<cuuint64_t>(Hq > 1 ? strides[2] * 2 : 16), static_cast<cuuint64_t>(T > 1 ? strides[1] * 2 : 16),
                        static_cast<cuuint64_t>(B > 1 ? strides[0] * 2 : 16)};
    cuuint32_t box[4] = {64, static_cast<cuuint32_t>(pack), static_cast<cuuint32_t>(hk::attn::kTileQ / pack), 1};
    cuuint32_t elem_strides[4] = {1, 1, 1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, st, box, elem_strides,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(HK_ERR_INVALID_ARG, "encoding the tensor map of the queries failed (CUresult %d)", (int)r);
    return HK_OK;
}

// bf16 keys or values as [heads, rows, D] in boxes of 64 columns × 128 rows.
hk_status encode_wide(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, const void* ptr, int64_t heads, int64_t rows,
                      int64_t D) {
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(heads)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(rows * D) * 2};
    cuuint32_t box[3] = {64, 128, 1};
    cuuint32_t elem_strides[3] = {1, 1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, elem_strides,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(HK_ERR_INVALID_ARG, "encoding the tensor map of the workspace failed (CUresult %d)", (int)r);
    return HK_OK;
}

template <int kD>
void launch_prefill(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PrefillParams& p, int sms,
                    cudaStream_t st) {
    using G = hk::attn::AttnGeometry<kD>;
    hk::attn::attn_fwd_kernel<kD, CachedItems>
        <<<static_cast<unsigned>(std::min(p.n_items, sms)), G::kThreads, G::kSmemBytes, st>>>(tq, tk, tv, p);
}

template <int kD, typename T, int kWarps>
cudaError_t launch_block(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeParams& p, int cluster, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(static_cast<unsigned>(p.B * p.Hkv * p.row_tiles * cluster));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = BlockGeometry<kD, kWarps>::kSmemBytes;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, &kv8_decode_block_kernel<kD, T, kWarps>, tk, tv, p, cluster);
}

// How the few-row kernels share a call out: warps per unit in a block of its
// own (times the blocks of a cluster), or 0: all tiles over all warps of the GPU.
struct DecodePlan {
    int warps, cluster, blocks;
};

template <int kD, typename T>
cudaError_t launch_decode(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeParams& p, const DecodePlan& plan, cudaStream_t st) {
    switch (plan.warps) {
        case 1: return launch_block<kD, T, 1>(tk, tv, p, 1, st);
        case 2: return launch_block<kD, T, 2>(tk, tv, p, 1, st);
        case 4: return launch_block<kD, T, 4>(tk, tv, p, 1, st);
        case 8: return launch_block<kD, T, 8>(tk, tv, p, plan.cluster, st);
        default: break;
    }
    const int blocks = plan.blocks;
    cudaError_t e = launch_early(&kv8_decode_kernel<kD, T>, dim3(static_cast<unsigned>(blocks)), dim3(32 * kDecodeWarps),
                                 DecodeGeometry<kD>::kSmemBytes, st, tk, tv, p);
    if (e != cudaSuccess) return e;
    const int64_t units = int64_t(p.B) * p.Hkv * p.row_tiles;
    const int rows = std::min(kRows, p.T * p.group);
    const unsigned x = static_cast<unsigned>(units);
    if (units * rows <= 8 * kSms)
        return launch_early(&kv8_combine_kernel<kD, T, 8>, dim3(x, static_cast<unsigned>(rows)), dim3(256), 0, st, p);
    return launch_early(&kv8_combine_kernel<kD, T, 1>, dim3(x, static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0, st, p);
}

// Many query rows per KV head: the sequences' keys and values to bf16, then the
// attention-forward kernel, for as many sequences at a time as the workspace holds.
hk_status prefill(const void* Q, const int64_t q_strides[3], const hk_kv8_cache* c, const int32_t* table, int64_t table_stride,
                  int64_t max_pages, const int32_t* lengths, const int32_t* counts, void* O, const int64_t o_strides[3],
                  float* lse, int64_t B, int64_t T, int64_t Hq, int32_t causal, float scale_log2, void* workspace,
                  uint32_t* status, uint32_t flags, uint64_t timeout_ns, PFN_cuTensorMapEncodeTiled_v12000 enc, int sms, cudaStream_t st) {
    const PrefillWorkspace ws = prefill_workspace(c, B, max_pages);
    char* const wide[2] = {static_cast<char*>(workspace), static_cast<char*>(workspace) + ws.half};
    const int64_t group = Hq / c->heads;
    const int pack_shift = pack_shift_of(group);
    hk_status s;
    for (int64_t b0 = 0; b0 < B; b0 += ws.seqs) {
        const int64_t n = std::min(ws.seqs, B - b0);
        WidenParams w = {};
        w.codes[0] = static_cast<const uint8_t*>(c->k_codes);
        w.codes[1] = static_cast<const uint8_t*>(c->v_codes);
        w.scale[0] = c->k_scale;
        w.scale[1] = c->v_scale;
        w.out[0] = reinterpret_cast<uint16_t*>(wide[0]);
        w.out[1] = reinterpret_cast<uint16_t*>(wide[1]);
        w.table = table + b0 * table_stride;
        w.table_stride = table_stride;
        w.lengths = lengths + b0;
        w.counts = counts ? counts + b0 : nullptr;
        w.rows = ws.rows;
        w.num_pages = c->num_pages;
        w.T = static_cast<int32_t>(T);
        w.Hkv = c->heads;
        w.D = c->head_dim;
        w.page_size = c->page_size;
        w.max_pages = static_cast<int32_t>(max_pages);
        w.status = status;

        const int64_t tokens_per_pair = (hk::attn::kTiles * hk::attn::kTileQ) >> pack_shift;
        const int64_t q_pairs = ceil_div(T, tokens_per_pair);
        const int64_t items = n * (Hq >> pack_shift) * q_pairs;
        if (items > kLimit || n * c->heads > kLimit) return fail(HK_ERR_INVALID_ARG, "problem too large");
        PrefillParams p = {};
        p.B = static_cast<int32_t>(n);
        p.Hq = static_cast<int32_t>(Hq);
        p.Hkv = c->heads;
        p.causal = causal ? 1 : 0;
        p.q_pairs = static_cast<int32_t>(q_pairs);
        p.n_items = static_cast<int32_t>(items);
        p.scale_log2 = scale_log2;
        p.O = static_cast<uint16_t*>(O) + b0 * o_strides[0];
        p.lse = lse ? lse + b0 * T * Hq : nullptr;
        p.status = status;
        p.launch_id = hk_host::next_launch_id();
        p.flags = flags & HK_KV8_FAULT_DROP_ARRIVE ? hk::attn::kFlagDropArrive : 0u;
        p.timeout_ns = timeout_ns ? timeout_ns : kDefaultTimeoutNs;
        p.lengths = w.lengths;
        p.counts = w.counts;
        p.T = static_cast<int32_t>(T);
        p.room = static_cast<int32_t>(ws.rows);
        p.group = static_cast<int32_t>(group);
        p.pack_shift = pack_shift;
        p.o_stride_b = o_strides[0];
        p.o_stride_t = o_strides[1];
        p.o_stride_h = o_strides[2];
        CUtensorMap tq, tk, tv;
        if ((s = encode_queries(enc, &tq, static_cast<const uint16_t*>(Q) + b0 * q_strides[0], q_strides, n, T, Hq, c->head_dim,
                                1 << pack_shift)) != HK_OK) return s;
        if ((s = encode_wide(enc, &tk, wide[0], n * c->heads, ws.rows, c->head_dim)) != HK_OK) return s;
        if ((s = encode_wide(enc, &tv, wide[1], n * c->heads, ws.rows, c->head_dim)) != HK_OK) return s;
        const dim3 grid(static_cast<unsigned>(max_pages), static_cast<unsigned>(c->heads), static_cast<unsigned>(n));
        kv8_widen_kernel<<<grid, 256, 0, st>>>(w);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_fail(HK_ERR_LAUNCH, "launching the cache's conversion", e);
        if (c->head_dim == 64) launch_prefill<64>(tq, tk, tv, p, sms, st);
        else launch_prefill<128>(tq, tk, tv, p, sms, st);
        kv8_nan_values_kernel<<<dim3(static_cast<unsigned>(c->heads), static_cast<unsigned>(n)), 256, 0, st>>>(w, p);
        e = cudaGetLastError();
        if (e != cudaSuccess) return cuda_fail(HK_ERR_LAUNCH, "launching the cache attention", e);
    }
    return HK_OK;
}

}  // namespace

extern "C" hk_status hk_kv8_append(const hk_kv8_cache* cache, const void* K, const void* V, int32_t type, int64_t B,
                                   int64_t T, const int64_t k_strides[3], const int64_t v_strides[3],
                                   const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                                   const int32_t* starts, const int32_t* counts, void* stream) {
    hk_status s = check_cache(cache);
    if (s != HK_OK) return s;
    if (type < HK_TYPE_BF16 || type > HK_TYPE_FP32) return fail(HK_ERR_INVALID_ARG, "unknown element type %d", (int)type);
    if (B < 0 || T < 0 || B > kLimit || T > kLimit) return fail(HK_ERR_INVALID_ARG, "invalid size");
    if (B == 0 || T == 0) return HK_OK;
    if ((s = check_table(block_table, table_stride, max_pages, B, starts, counts, cache->page_size)) != HK_OK) return s;
    if (!K || !V || !k_strides || !v_strides) return fail(HK_ERR_INVALID_ARG, "null keys, values or strides");
    const int size = type == HK_TYPE_FP32 ? 4 : 2;
    if (!aligned(K, size) || !aligned(V, size)) return fail(HK_ERR_MISALIGNED, "keys or values not aligned to their elements");
    int device = 0, sms = 0;
    if ((s = current_device(&device, &sms)) != HK_OK) return s;
    uint32_t* status = nullptr;
    if ((s = hk_host::status_word(device, &status)) != HK_OK) return s;

    AppendParams p = {};
    const void* src[2] = {K, V};
    const int64_t* strides[2] = {k_strides, v_strides};
    for (int i = 0; i < 2; ++i) {
        p.src[i] = src[i];
        p.stride_b[i] = strides[i][0];
        p.stride_t[i] = strides[i][1];
        p.stride_h[i] = strides[i][2];
        p.vec[i] = aligned(src[i], 16);
        for (int k = 0; k < 3; ++k) p.vec[i] = p.vec[i] && (strides[i][k] * size) % 16 == 0;
    }
    p.codes[0] = static_cast<uint8_t*>(cache->k_codes);
    p.codes[1] = static_cast<uint8_t*>(cache->v_codes);
    p.scale[0] = cache->k_scale;
    p.scale[1] = cache->v_scale;
    p.table = block_table;
    p.table_stride = table_stride;
    p.starts = starts;
    p.counts = counts;
    p.B = static_cast<int32_t>(B);
    p.T = static_cast<int32_t>(T);
    p.Hkv = static_cast<uint32_t>(cache->heads);
    p.page_shift = page_shift(cache->page_size);
    p.max_pages = static_cast<int32_t>(max_pages);
    p.num_pages = cache->num_pages;
    p.slots = static_cast<uint32_t>((T + cache->page_size - 2) / cache->page_size + 1);
    p.status = status;
    if (B > (int64_t(1) << 40) / p.slots / p.Hkv) return fail(HK_ERR_INVALID_ARG, "problem too large");
    p.items = B * p.slots * p.Hkv;
    // one warp holds the new tokens of a page as long as they fit its registers (8 steps of 256 elements)
    const int64_t elements = std::min<int64_t>(T, cache->page_size) * cache->head_dim;
    const bool one_warp = elements <= kAppendSteps * 256;
    const int steps = static_cast<int>(ceil_div(elements, one_warp ? 256 : 8 * 256));
    const int64_t blocks = one_warp ? ceil_div(p.items, 8) : p.items;
    if (p.items > kLimit) return fail(HK_ERR_INVALID_ARG, "problem too large");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (type) {
        case HK_TYPE_BF16: e = launch_append<__nv_bfloat16>(p, cache->head_dim, one_warp, steps, static_cast<unsigned>(blocks), st); break;
        case HK_TYPE_FP16: e = launch_append<__half>(p, cache->head_dim, one_warp, steps, static_cast<unsigned>(blocks), st); break;
        default: e = launch_append<float>(p, cache->head_dim, one_warp, steps, static_cast<unsigned>(blocks), st); break;
    }
    return e == cudaSuccess ? HK_OK : cuda_fail(HK_ERR_LAUNCH, "launching the cache append", e);
}

namespace {

bool attention_shape_ok(const hk_kv8_cache* c, int64_t B, int64_t T, int64_t Hq, int64_t max_pages) {
    return c && cache_shape_ok(c) && table_width_ok(max_pages, c->page_size) && B > 0 && B <= kLimit && T > 0 && Hq >= c->heads &&
           Hq <= kLimit && T <= kLimit / 16 / (Hq / c->heads);
}

// Bytes for the few-row kernels: none where every unit is a block's or a cluster's.
size_t few_rows_bytes(const hk_kv8_cache* c, int64_t B, int64_t T, int64_t Hq, int64_t max_pages) {
    const int64_t row_tiles = ceil_div(T * (Hq / c->heads), kRows);
    const int64_t units = decode_batch(B, c->heads, row_tiles) * c->heads * row_tiles;
    if (ceil_div(max_pages * c->page_size, kTileKeys) <= block_warps(units, kBlockWarps) * kBlockTiles) return 0;
    return decode_workspace(c, B, T, Hq).total;
}

}  // namespace

namespace hk_kv8 {

// Can the tensor-core kernel run the call? It takes bf16 rows that TMA can read (aligned, and not one row for
// several places) and writes 16 bytes at a time.
bool many_rows_can(const void* Q, int32_t type, const int64_t q_strides[3], const void* O, const int64_t o_strides[3], int64_t B,
                   int64_t T, int64_t Hq) {
    return type == HK_TYPE_BF16 && rows_aligned(Q, q_strides) && rows_aligned(O, o_strides) && (B == 1 || q_strides[0] > 0) &&
           (T == 1 || q_strides[1] > 0) && (Hq == 1 || q_strides[2] > 0);
}

// (units at 25 millionths of a microsecond per cached token at head dimension 64, where both forms' order stays as it is)
double attention_cost(const hk_kv8_cache* c, int64_t B, int64_t T, int64_t Hq, int64_t max_pages, bool many_can) {
    if (many_can && many_rows(c, B, T, Hq, max_pages)) return item_cost(c, B, T, Hq, max_pages);
    return unit_cost(c, B, T, Hq) * (c->head_dim == 64 ? 25.0 / 35.0 : 1.0);
}

}  // namespace hk_kv8

namespace {

constexpr uint32_t kFormFlags = HK_KV8_FEW_ROWS | HK_KV8_MANY_ROWS;

// Does the call run on the tensor-core kernel?
bool takes_many_rows(uint32_t flags, const void* Q, int32_t type, const int64_t q_strides[3], const hk_kv8_cache* c, int64_t max_pages,
                     const void* O, const int64_t o_strides[3], int64_t B, int64_t T, int64_t Hq) {
    if (flags & kFormFlags) return flags & HK_KV8_MANY_ROWS;
    return many_rows(c, B, T, Hq, max_pages) && many_rows_can(Q, type, q_strides, O, o_strides, B, T, Hq);
}

}  // namespace

extern "C" size_t hk_attention_kv8_workspace_size(const hk_kv8_cache* cache, int64_t B, int64_t T, int64_t Hq,
                                                  int64_t max_pages) {
    if (!attention_shape_ok(cache, B, T, Hq, max_pages)) return 0;
    const size_t few = few_rows_bytes(cache, B, T, Hq, max_pages);
    return many_rows(cache, B, T, Hq, max_pages) ? std::max(few, prefill_workspace(cache, B, max_pages).total) : few;
}

extern "C" size_t hk_attention_kv8_workspace_size_ex(const void* Q, int32_t type, const int64_t q_strides[3],
                                                     const hk_kv8_cache* cache, int64_t max_pages, const void* O,
                                                     const int64_t o_strides[3], int64_t B, int64_t T, int64_t Hq,
                                                     uint32_t flags) {
    if (!attention_shape_ok(cache, B, T, Hq, max_pages) || !q_strides || !o_strides) return 0;
    return takes_many_rows(flags, Q, type, q_strides, cache, max_pages, O, o_strides, B, T, Hq)
               ? prefill_workspace(cache, B, max_pages).total
               : few_rows_bytes(cache, B, T, Hq, max_pages);
}

extern "C" hk_status hk_attention_kv8_ex(const void* Q, int32_t type, const int64_t q_strides[3], const hk_kv8_cache* cache,
                                         const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                                         const int32_t* lengths, const int32_t* counts, void* O,
                                         const int64_t o_strides[3], float* lse, int64_t B, int64_t T, int64_t Hq,
                                         int32_t causal, float scale, void* workspace, size_t workspace_bytes,
                                         uint32_t flags, uint64_t timeout_ns, void* stream) {
    hk_status s = check_cache(cache);
    if (s != HK_OK) return s;
    if ((flags & ~(kFormFlags | HK_KV8_FAULT_DROP_ARRIVE)) || (flags & kFormFlags) == kFormFlags) return fail(HK_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
    if (type != HK_TYPE_BF16 && type != HK_TYPE_FP16) return fail(HK_ERR_INVALID_ARG, "element type %d (bf16 or fp16)", (int)type);
    if (B < 0 || T < 0 || Hq < 0 || B > kLimit || T > kLimit || Hq > kLimit) return fail(HK_ERR_INVALID_ARG, "invalid size");
    if (Hq % cache->heads) return fail(HK_ERR_INVALID_ARG, "Hq=%lld is not a multiple of the cache's %d heads", (long long)Hq, (int)cache->heads);
    if (!std::isfinite(scale) || scale < 0.0f) return fail(HK_ERR_INVALID_ARG, "the scale must be finite and not negative");
    if (B == 0 || T == 0 || Hq == 0) return HK_OK;
    if ((s = check_table(block_table, table_stride, max_pages, B, lengths, counts, cache->page_size)) != HK_OK) return s;
    if (!Q || !O || !q_strides || !o_strides) return fail(HK_ERR_INVALID_ARG, "null queries, output or strides");
    if (!aligned(Q, 2) || !aligned(O, 2) || !aligned(lse, 4)) return fail(HK_ERR_MISALIGNED, "a pointer is not aligned to its elements");
    const int64_t sizes[3] = {B, T, Hq};
    for (int i = 0; i < 3; ++i)
        if (sizes[i] > 1 && std::llabs(o_strides[i]) < cache->head_dim) return fail(HK_ERR_INVALID_ARG, "the output's rows overlap");
    const int64_t group = Hq / cache->heads;
    if (T > kLimit / 16 / group || ceil_div(T * group, kRows) * (ceil_div(max_pages * cache->page_size, kTileKeys) + 1) > kLimit)
        return fail(HK_ERR_INVALID_ARG, "problem too large");
    if ((flags & HK_KV8_MANY_ROWS) && !many_rows_can(Q, type, q_strides, O, o_strides, B, T, Hq))
        return fail(HK_ERR_INVALID_ARG, "the many-row kernel takes bf16 queries and an output with 16-byte aligned rows");
    const DecodeWorkspace ws = decode_workspace(cache, B, T, Hq);
    const bool many = takes_many_rows(flags, Q, type, q_strides, cache, max_pages, O, o_strides, B, T, Hq);
    const size_t need = hk_attention_kv8_workspace_size_ex(Q, type, q_strides, cache, max_pages, O, o_strides, B, T, Hq, flags);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(HK_ERR_WORKSPACE, "%zu bytes of workspace needed, %zu given", need, workspace ? workspace_bytes : size_t(0));
    if (!aligned(workspace, 256)) return fail(HK_ERR_WORKSPACE, "the workspace must be 256-byte aligned");
    int device = 0, sms = 0;
    if ((s = current_device(&device, &sms)) != HK_OK) return s;
    if ((s = setup(device)) != HK_OK) return s;
    uint32_t* status = nullptr;
    if ((s = hk_host::status_word(device, &status)) != HK_OK) return s;
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    if ((s = hk_host::tensor_map_encoder(&enc)) != HK_OK) return s;
    const float scale_log2 = static_cast<float>(
        1.4426950408889634 * (scale != 0.0f ? static_cast<double>(scale) : 1.0 / std::sqrt(static_cast<double>(cache->head_dim))));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (many)
        return prefill(Q, q_strides, cache, block_table, table_stride, max_pages, lengths, counts, O, o_strides, lse, B, T, Hq,
                       causal, scale_log2, workspace, status, flags, timeout_ns, enc, sms, st);
    CUtensorMap tk, tv;
    if ((s = encode_codes(enc, &tk, cache->k_codes, cache, kTileKeys)) != HK_OK) return s;
    if ((s = encode_codes(enc, &tv, cache->v_codes, cache, kTileKeys)) != HK_OK) return s;

    DecodeParams p = {};
    p.q_stride_b = q_strides[0];
    p.q_stride_t = q_strides[1];
    p.q_stride_h = q_strides[2];
    p.o_stride_b = o_strides[0];
    p.o_stride_t = o_strides[1];
    p.o_stride_h = o_strides[2];
    p.vec_q = rows_aligned(Q, q_strides);
    p.vec_o = rows_aligned(O, o_strides);
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    p.table_stride = table_stride;
    p.T = static_cast<int32_t>(T);
    p.Hq = static_cast<int32_t>(Hq);
    p.Hkv = cache->heads;
    p.group = static_cast<int32_t>(group);
    p.row_tiles = static_cast<int32_t>(ceil_div(T * group, kRows));
    p.page_size = cache->page_size;
    p.page_shift = page_shift(cache->page_size);
    p.max_pages = static_cast<int32_t>(max_pages);
    p.num_pages = cache->num_pages;
    p.causal = causal ? 1 : 0;
    p.scale_log2 = scale_log2;
    p.flags = flags & HK_KV8_FAULT_DROP_ARRIVE ? kFlagDropArrive : 0u;
    char* const w = static_cast<char*>(workspace);
    p.part_o = reinterpret_cast<float*>(w);
    p.part_ml = reinterpret_cast<float*>(w + ws.ml);
    p.info = reinterpret_cast<int4*>(w + ws.info);
    p.wait.status = status;
    p.wait.timeout_ns = timeout_ns ? timeout_ns : kDefaultTimeoutNs;
    // one round of blocks, and no more than the table has room for tiles
    const int64_t batch = decode_batch(B, p.Hkv, p.row_tiles);
    const int64_t units = batch * p.Hkv * p.row_tiles;
    if (units > kLimit) return fail(HK_ERR_INVALID_ARG, "problem too large");
    const int64_t unit_room = ceil_div(max_pages * p.page_size, kTileKeys);
    DecodePlan plan = {0, 1, static_cast<int>(std::min<int64_t>(2 * std::min(sms, kSms), ceil_div(units * unit_room, kDecodeWarps)))};
    const int warps = block_warps(units, kBlockWarps);
    // a cluster of blocks where one block to a unit leaves SMs idle, as long as its warps have half a tile each (8
    // units: 12 blocks, 32768 tokens 24.5 us; 8 blocks 30)
    if (warps == kBlockWarps)
        for (int size = 2; size <= kMaxCluster && units <= g_clusters[device][size] && kBlockWarps / 2 * size <= unit_room; ++size)
            plan.cluster = size;
    if (unit_room <= int64_t(plan.cluster) * warps * kBlockTiles) plan.warps = warps;
    p.warps = plan.blocks * kDecodeWarps;

    for (int64_t b0 = 0; b0 < B; b0 += batch) {       // (launches of one stream: they may share the workspace)
        p.B = static_cast<int32_t>(std::min<int64_t>(B - b0, batch));
        p.q = static_cast<const uint16_t*>(Q) + b0 * p.q_stride_b;
        p.o = static_cast<uint16_t*>(O) + b0 * p.o_stride_b;
        p.lse = lse ? lse + b0 * T * Hq : nullptr;
        p.table = block_table + b0 * table_stride;
        p.lengths = lengths + b0;
        p.counts = counts ? counts + b0 : nullptr;
        p.wait.launch_id = hk_host::next_launch_id();
        cudaError_t e;
        const bool half = type == HK_TYPE_FP16;
        if (cache->head_dim == 64)
            e = half ? launch_decode<64, __half>(tk, tv, p, plan, st)
                     : launch_decode<64, __nv_bfloat16>(tk, tv, p, plan, st);
        else
            e = half ? launch_decode<128, __half>(tk, tv, p, plan, st)
                     : launch_decode<128, __nv_bfloat16>(tk, tv, p, plan, st);
        if (e != cudaSuccess) return cuda_fail(HK_ERR_LAUNCH, "launching the cache attention", e);
    }
    return HK_OK;
}

extern "C" hk_status hk_attention_kv8(const void* Q, int32_t type, const int64_t q_strides[3], const hk_kv8_cache* cache,
                                      const int32_t* block_table, int64_t table_stride, int64_t max_pages,
                                      const int32_t* lengths, const int32_t* counts, void* O, const int64_t o_strides[3],
                                      float* lse, int64_t B, int64_t T, int64_t Hq, int32_t causal, float scale,
                                      void* workspace, size_t workspace_bytes, void* stream) {
    return hk_attention_kv8_ex(Q, type, q_strides, cache, block_table, table_stride, max_pages, lengths, counts, O, o_strides,
                               lse, B, T, Hq, causal, scale, workspace, workspace_bytes, 0u, 0u, stream);
}
