// Host helpers of the paged 8-bit cache's entry points (hk_kv8.cu, hk_kv8_pages.cu,
// hk_kv8_shared.cu): errors, checks of caches and tables, launches, tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/hk_gemm.h"
#include "host_internal.h"

namespace hk_kv8 {

inline hk_status fail(hk_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline hk_status fail(hk_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return hk_host::set_error(s, buf);
}

inline hk_status cuda_fail(hk_status s, const char* what, cudaError_t e) {
    return fail(s, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

constexpr uint64_t kDefaultTimeoutNs = 1000000000ull;   // 1 s per bounded wait
constexpr int kMaxDevices = 64;
constexpr int64_t kLimit = (int64_t(1) << 31) - 1;
constexpr int kSms = 152;                               // the device's SMs: the workspace is sized without a device

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

constexpr int kMaxHeads = 65535;

// (the sizes below stay within 64 bits for what passes; the tokens of a sequence, rounded up to a tile, within 31)
inline bool cache_shape_ok(const hk_kv8_cache* c) {
    return (c->head_dim == 64 || c->head_dim == 128) &&
           (c->page_size == 16 || c->page_size == 32 || c->page_size == 64 || c->page_size == 128) && c->heads >= 1 &&
           c->heads <= kMaxHeads && c->num_pages >= 1 && c->num_pages <= kLimit / c->heads;
}
inline bool table_width_ok(int64_t max_pages, int32_t page_size) { return max_pages >= 1 && max_pages <= (kLimit - 127) / page_size; }

inline hk_status check_cache(const hk_kv8_cache* c) {
    if (!c) return fail(HK_ERR_INVALID_ARG, "null cache");
    if (c->head_dim != 64 && c->head_dim != 128)
        return fail(HK_ERR_INVALID_ARG, "head dimension %d (supported: 64, 128)", (int)c->head_dim);
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return fail(HK_ERR_INVALID_ARG, "page size %d (supported: 16, 32, 64, 128)", (int)c->page_size);
    if (!cache_shape_ok(c))
        return fail(HK_ERR_INVALID_ARG, "%lld pages of %d heads", (long long)c->num_pages, (int)c->heads);
    if (!c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale) return fail(HK_ERR_INVALID_ARG, "null cache pointer");
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return fail(HK_ERR_MISALIGNED, "cache codes must be 16-byte aligned, scales 4-byte aligned");
    return HK_OK;
}

inline hk_status check_table(const int32_t* table, int64_t stride, int64_t max_pages, int64_t B, const int32_t* lengths,
                      const int32_t* counts, int32_t page_size) {
    if (!table_width_ok(max_pages, page_size))
        return fail(HK_ERR_INVALID_ARG, "a block table of %lld pages per sequence", (long long)max_pages);
    if (stride < max_pages && B > 1) return fail(HK_ERR_INVALID_ARG, "block table rows overlap");
    if (!table || !lengths) return fail(HK_ERR_INVALID_ARG, "null block table or lengths");
    if (!aligned(table, 4) || !aligned(lengths, 4) || !aligned(counts, 4))
        return fail(HK_ERR_MISALIGNED, "block table, lengths and counts must be 4-byte aligned");
    return HK_OK;
}

inline hk_status current_device(int* device, int* sm_count) {
    cudaError_t e = cudaGetDevice(device);
    if (e != cudaSuccess) return cuda_fail(HK_ERR_CUDA, "cudaGetDevice", e);
    if (*device < 0 || *device >= kMaxDevices) return fail(HK_ERR_INVALID_ARG, "device %d out of range", *device);
    return hk_host::check_device(*device, sm_count);
}

// A launch that may begin while the kernel before it on the stream ends (the kernel waits for that end itself).
template <typename... Params, typename... Args>
inline cudaError_t launch_early(void (*fn)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

inline int page_shift(int32_t page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7; }

// Codes of keys or values as [pages · heads, page_size, D] in boxes of up to `tokens` tokens of one head.
inline hk_status encode_codes(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, const void* ptr, const hk_kv8_cache* c,
                              int32_t tokens) {
    const cuuint64_t D = static_cast<cuuint64_t>(c->head_dim);
    cuuint64_t dims[3] = {D, static_cast<cuuint64_t>(c->page_size), static_cast<cuuint64_t>(c->num_pages) * c->heads};
    cuuint64_t strides[2] = {D, D * c->page_size};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(D), static_cast<cuuint32_t>(std::min(c->page_size, tokens)), 1};
    cuuint32_t elem_strides[3] = {1, 1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box, elem_strides,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(HK_ERR_INVALID_ARG, "encoding the tensor map of the cache failed (CUresult %d)", (int)r);
    return HK_OK;
}

inline bool rows_aligned(const void* ptr, const int64_t strides[3]) {
    return aligned(ptr, 16) && strides[0] % 8 == 0 && strides[1] % 8 == 0 && strides[2] % 8 == 0;
}

// Warps of a block that has a unit to itself, of at most `most`, which fill an SM: as many as let one round of blocks hold all
// units.
inline int block_warps(int64_t units, int most) {
    int warps = most;
    while (warps > 1 && units > int64_t(kSms) * (most / warps)) warps /= 2;
    return warps;
}

// hk_attention_kv8's form for many rows: can it run the call? And what that entry point takes per token of a sequence's
// table, in millionths of a microsecond (hk_kv8.cu).
bool many_rows_can(const void* Q, int32_t type, const int64_t q_strides[3], const void* O, const int64_t o_strides[3], int64_t B,
                   int64_t T, int64_t Hq);
double attention_cost(const hk_kv8_cache* c, int64_t B, int64_t T, int64_t Hq, int64_t max_pages, bool many_can);

}  // namespace hk_kv8
