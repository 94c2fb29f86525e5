// Host side of the microscaled 4-bit entry points (include/hk_gemm.h):
// hk_fp4_quantize, hk_fp4_dequantize and hk_gemm_fp4: argument checks, tensor
// maps, the choice of tile and K split, and the launches.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>

#include "../../include/hk_gemm.h"
#include "fp4_gemm.cuh"
#include "fp4_quant.cuh"
#include "host_internal.h"

namespace {

using namespace hk::fp4;

hk_status fail(hk_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
hk_status fail(hk_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return hk_host::set_error(s, buf);
}

hk_status cuda_fail(hk_status s, const char* what, cudaError_t e) {
    return fail(s, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

constexpr uint64_t kDefaultTimeoutNs = 1000000000ull;   // 1 s per bounded wait
constexpr int kMaxDevices = 64;
constexpr int64_t kLimit = (int64_t(1) << 31) - 1;
constexpr int64_t kQuantBlocks = 152 * 16;               // blocks of a (de)quantisation, several rounds of what fits

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
int type_bytes(int32_t t) { return t == HK_TYPE_FP32 ? 4 : 2; }

hk_status check_format(int32_t format) {
    if (format != HK_FP4_MXFP4 && format != HK_FP4_NVFP4) return fail(HK_ERR_INVALID_ARG, "unknown 4-bit format %d", (int)format);
    return HK_OK;
}

// Sizes, codes and scales of one quantised matrix (pointers only when it has elements).
hk_status check_matrix(const char* name, const void* codes, int64_t ld, const void* scales, int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return fail(HK_ERR_INVALID_ARG, "negative size");
    if (rows > kLimit || cols > kLimit) return fail(HK_ERR_INVALID_ARG, "size of 2^31 or more");
    if (rows == 0 || cols == 0) return HK_OK;
    if (ld < ceil_div(cols, 32) * 16)
        return fail(HK_ERR_INVALID_ARG, "%s: leading dimension %lld below the %lld bytes of a row's codes", name,
                    (long long)ld, (long long)(ceil_div(cols, 32) * 16));
    if (!codes || !scales) return fail(HK_ERR_INVALID_ARG, "%s: null pointer", name);
    if (ld % 16 || !aligned(codes, 16) || !aligned(scales, 16))
        return fail(HK_ERR_MISALIGNED, "%s: codes and scales must be 16-byte aligned, the leading dimension a multiple of 16", name);
    return HK_OK;
}

hk_status current_device(int* device, int* sm_count) {
    cudaError_t e = cudaGetDevice(device);
    if (e != cudaSuccess) return cuda_fail(HK_ERR_CUDA, "cudaGetDevice", e);
    if (*device < 0 || *device >= kMaxDevices) return fail(HK_ERR_INVALID_ARG, "device %d out of range", *device);
    return hk_host::check_device(*device, sm_count);
}

// ------------------------------------------------ quantise and dequantise --

uint32_t spans_of(int64_t cols) { return static_cast<uint32_t>(ceil_div(cols, kChunkCols * kSpanChunks)); }

// Blocks of a (de)quantisation: a warp to a span of a row, up to several rounds of what fits the SMs (what a
// block of threads sets up is then paid for once).
unsigned quant_blocks(int64_t rows, int64_t cols) {
    return static_cast<unsigned>(std::min<int64_t>(ceil_div(rows * spans_of(cols), kQuantWarps), kQuantBlocks));
}

// A launch that may begin while the kernel before it on the stream ends (the kernel waits for that end itself).
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*fn)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args... args) {
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

template <typename T, int kFmt>
cudaError_t launch_quantize(const void* x, int64_t rows, int64_t cols, int64_t ldx, void* codes, int64_t ld, void* scales,
                            const float* g, cudaStream_t st) {
    const int vec = aligned(x, 16) && (ldx * sizeof(T)) % 16 == 0;
    return launch_early(&quantize_kernel<T, kFmt>, dim3(quant_blocks(ceil_div(rows, 128) * 128, cols)), dim3(32, kQuantWarps), 0, st,
                        static_cast<const T*>(x), rows, cols, ldx, static_cast<uint8_t*>(codes), ld, static_cast<uint8_t*>(scales), g,
                        spans_of(cols), vec);
}

template <typename T, int kFmt>
cudaError_t launch_dequantize(const void* codes, int64_t ld, const void* scales, const float* g, int64_t rows, int64_t cols,
                              void* y, int64_t ldy, cudaStream_t st) {
    const int vec = aligned(y, 16) && (ldy * sizeof(T)) % 16 == 0;
    return launch_early(&dequantize_kernel<T, kFmt>, dim3(quant_blocks(rows, cols)), dim3(32, kQuantWarps), 0, st,
                        static_cast<const uint8_t*>(codes), ld, static_cast<const uint8_t*>(scales), g, rows, cols,
                        static_cast<T*>(y), ldy, spans_of(cols), vec);
}

// ------------------------------------------------------------- the product --

using SingleFn = void (*)(CUtensorMap, CUtensorMap, Fp4Params, int);

struct SingleVariant {
    int tok;
    SingleFn fn;
    int smem, threads;
};

template <int kTok, int kFmt>
constexpr SingleVariant single_variant() {
    using G = SingleGeometry<kTok, kFmt>;
    return {kTok, &gemm_fp4_single_kernel<kTok, kFmt>, G::kSmemBytes, G::kThreads};
}

const SingleVariant kSingle[2][4] = {
    {single_variant<16, kMxfp4>(), single_variant<32, kMxfp4>(), single_variant<64, kMxfp4>(), single_variant<128, kMxfp4>()},
    {single_variant<16, kNvfp4>(), single_variant<32, kNvfp4>(), single_variant<64, kNvfp4>(), single_variant<128, kNvfp4>()},
};

using PairFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, Fp4Params);

struct PairVariant {
    PairFn fn;
    int smem, threads;
};

const PairVariant kPair[2] = {
    {&gemm_fp4_pair_kernel<kMxfp4>, PairGeometry<kMxfp4>::kSmemBytes, PairGeometry<kMxfp4>::kThreads},
    {&gemm_fp4_pair_kernel<kNvfp4>, PairGeometry<kNvfp4>::kSmemBytes, PairGeometry<kNvfp4>::kThreads},
};

std::mutex g_setup_mutex;
bool g_setup[kMaxDevices] = {};

hk_status setup(int device) {
    std::lock_guard<std::mutex> lock(g_setup_mutex);
    if (g_setup[device]) return HK_OK;
    for (const auto& row : kSingle)
        for (const SingleVariant& v : row) {
            cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(v.fn),
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem);
            if (e != cudaSuccess) return cuda_fail(HK_ERR_CUDA, "configuring a 4-bit product kernel", e);
        }
    for (const PairVariant& v : kPair) {
        cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(v.fn), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             v.smem);
        if (e != cudaSuccess) return cuda_fail(HK_ERR_CUDA, "configuring a 4-bit product kernel", e);
    }
    g_setup[device] = true;
    return HK_OK;
}

// Codes as rows of bytes in boxes of 128 bytes × box_rows, 128-byte swizzled;
// rows and bytes past the matrix read as 0.
hk_status encode_codes(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, const void* ptr, int64_t rows,
                       int64_t cols, int64_t ld, uint32_t box_rows, const char* name) {
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(ceil_div(cols, 32) * 16), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld)};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(kStageRowBytes), box_rows};
    cuuint32_t elem_strides[2] = {1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, elem_strides,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(HK_ERR_INVALID_ARG, "encoding the tensor map of %s failed (CUresult %d)", name, (int)r);
    return HK_OK;
}

// Scale tiles as [groups of 128 matrix rows][rows of 256 bytes], in boxes of one stage's tiles of `groups` groups.
hk_status encode_scales(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, const void* ptr, int64_t rows, int64_t cols,
                        int32_t format, uint32_t groups, const char* name) {
    const int64_t group_bytes = padded_blocks(cols, format) * 128;
    cuuint64_t dims[3] = {256, static_cast<cuuint64_t>(group_bytes / 256), static_cast<cuuint64_t>(ceil_div(rows, 128))};
    cuuint64_t strides[2] = {256, static_cast<cuuint64_t>(group_bytes)};
    cuuint32_t box[3] = {256, static_cast<cuuint32_t>(2 * scale_tiles(format)), groups};
    cuuint32_t elem_strides[3] = {1, 1, 1};
    CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box, elem_strides,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(HK_ERR_INVALID_ARG, "encoding the tensor map of %s failed (CUresult %d)", name, (int)r);
    return HK_OK;
}

// Many tokens: 256 × 256 tiles on CTA pairs.
hk_status launch_pair(PFN_cuTensorMapEncodeTiled_v12000 enc, Fp4Params p, const void* A, const void* B, int64_t K, int64_t lda,
                      int64_t ldb, int32_t format, int sm_count, cudaStream_t st) {
    hk_status s;
    p.tiles_m = static_cast<int32_t>(ceil_div(p.M, 256));
    p.tiles_n = static_cast<int32_t>(ceil_div(p.N, 256));
    p.group_m = 8;      // (4 and 16: the same at 4096^3 and 8192^3; 3 % slower at 2048 x 28672 x 8192, 3 % slower and 4 % faster at 4096)
    const int64_t tiles = int64_t(p.tiles_m) * p.tiles_n;
    const int64_t units = sm_count / 2;
    // the last round's tiles, when they fill at most half of the pairs, run as two halves each
    const int64_t last = tiles - (ceil_div(tiles, units) - 1) * units;
    const bool halves = 2 * last <= units;
    p.tail_start = static_cast<int32_t>(halves ? tiles - last : tiles);
    p.total_units = static_cast<int32_t>(halves ? tiles + last : tiles);
    CUtensorMap ta, tb, tbh, tsa, tsb;
    if ((s = encode_codes(enc, &ta, A, p.M, K, lda, 128, "A")) != HK_OK) return s;
    if ((s = encode_codes(enc, &tb, B, p.N, K, ldb, 128, "B")) != HK_OK) return s;
    if ((s = encode_codes(enc, &tbh, B, p.N, K, ldb, 64, "B")) != HK_OK) return s;
    if ((s = encode_scales(enc, &tsa, p.sfa, p.M, K, format, 1, "A's scales")) != HK_OK) return s;
    if ((s = encode_scales(enc, &tsb, p.sfb, p.N, K, format, 2, "B's scales")) != HK_OK) return s;
    CUtensorMap tc = ta;                 // (not used where C's rows are not 16-byte aligned)
    if (p.vec_c) {
        cuuint64_t dims[2] = {static_cast<cuuint64_t>(p.N), static_cast<cuuint64_t>(p.M)};
        cuuint64_t strides[1] = {static_cast<cuuint64_t>(p.ldc) * 2};
        cuuint32_t box[2] = {32, 32};
        cuuint32_t elem_strides[2] = {1, 1};
        CUresult r = enc(&tc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.c, dims, strides, box, elem_strides,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) return fail(HK_ERR_INVALID_ARG, "encoding the tensor map of C failed (CUresult %d)", (int)r);
    }
    const PairVariant& v = kPair[format == HK_FP4_NVFP4];
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<int64_t>(units, p.total_units)));
    cfg.blockDim = dim3(static_cast<unsigned>(v.threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(v.smem);
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, v.fn, ta, tb, tbh, tsa, tsb, tc, p);
    return e == cudaSuccess ? HK_OK : cuda_fail(HK_ERR_LAUNCH, "launching the 4-bit product", e);
}

// The one-CTA kernel's tile width and K parts. Estimated time in microseconds, fitted to 600 timings (M 1 to 128, 11
// shapes from 1000 x 3000 to 28672 x 8192, both formats): what memory (6.6 TB/s), the traffic from L2 (27 TB/s;
// rows that do not start on 128 bytes cost two lines for one) and the chain of stages (0.23 each) take, joined as a
// root of squares, and per round of CTAs the tile's epilogue (0.033 per token) and the join of K parts (1.0, of
// eight 1.4). The choice is 0.3 % off the best of what is allowed on average, 8 % at worst; the narrowest tile that
// holds all tokens with K cut until the GPU is full was 7 % and 47 % off (128 x 2048 x 8192: 64 tokens in 4 parts
// 7.8 us, 128 tokens in 8 parts 9.7; 100 x 6144 x 2048: 64 tokens unsplit 5.5, 128 tokens in 2 parts 7.9).
struct SinglePlan {
    const SingleVariant* v;
    int splits;
    double us;
};

SinglePlan plan_single(int64_t M, int64_t N, int64_t K, bool aligned_rows, int32_t format, int forced_splits, int sm_count) {
    SinglePlan best = {nullptr, 1, 0.0};
    const double k_stages = static_cast<double>(ceil_div(K, kStageCols));
    const double dram = static_cast<double>(M + N) * static_cast<double>(K) * (0.5 + 1.0 / block_cols(format)) * 1e-6;
    for (const SingleVariant& v : kSingle[format == HK_FP4_NVFP4]) {
        // 16 and 32 tokens only as the one tile (the scales of 128 rows come in columns of 32, and a tile may
        // begin at every second one); nothing wider than holds every token
        if (v.tok < 64 && M > v.tok) continue;
        if (v.tok > 16 && v.tok / 2 >= M) break;
        const double tiles = static_cast<double>(ceil_div(M, v.tok)) * static_cast<double>(ceil_div(N, 128));
        const double stage = (aligned_rows ? 1.0 : 2.0) * (128 + v.tok) * kStageRowBytes + 2.0 * 512 * scale_tiles(format);
        for (int splits = 1; splits <= 8; splits *= 2) {
            if (forced_splits ? splits != forced_splits : splits > 1 && (splits > k_stages || tiles * splits > 4 * sm_count)) continue;
            const double rounds = std::ceil(tiles * splits / (2 * sm_count));
            const double join = splits == 1 ? 0.0 : splits == 8 ? 1.4 : 1.0;
            const double memory = dram / 6.6, l2 = tiles * k_stages * stage * 1e-6 / 27.0;
            const double chain = 0.23 * std::ceil(k_stages / splits) * rounds;
            const double us = rounds * (0.033 * v.tok + join) + std::sqrt(memory * memory + l2 * l2 + chain * chain);
            if (best.v == nullptr || us < best.us) best = {&v, splits, us};
        }
    }
    best.us += 1.5;
    return best;
}

// The CTA-pair kernel's time, fitted likewise (M 130 to 2048, 8 shapes): memory and the chain of its 256 x 256 tiles'
// stages. Taking the kernel with the lower estimate is 0.2 % off the better of the two on average, 5 % at worst.
// (512 x 1024 x 4096: one CTA 7.0 us, pair 9.1; 512 x 8192 x 8192: 16.9 and 16.1; 1024 x 1024 x 28672: 19.4 and 38.8;
// 256 x 28672 x 8192: 35.8 and 30.9; 2048 x 4096 x 4096: 19.5 and 16.4.)
double pair_us(int64_t M, int64_t N, int64_t K, int32_t format, int sm_count) {
    const int64_t tiles = ceil_div(M, 256) * ceil_div(N, 256), units = sm_count / 2, rounds = ceil_div(tiles, units);
    const bool halves = 2 * (tiles - (rounds - 1) * units) <= units;          // the last round's tiles run as halves
    const double bytes = static_cast<double>(M + N) * static_cast<double>(K) * (0.5 + 1.0 / block_cols(format)) +
                         2.0 * static_cast<double>(M) * static_cast<double>(N);
    const double memory = bytes * 1e-6 / 5.8;
    const double chain = 0.46 * static_cast<double>(ceil_div(K, kStageCols)) * (static_cast<double>(rounds) - (halves ? 0.5 : 0.0));
    return 5.3 + std::sqrt(memory * memory + chain * chain);
}

}  // namespace

extern "C" size_t hk_fp4_scales_size(int64_t rows, int64_t cols, int32_t format) {
    if (rows <= 0 || cols <= 0 || rows > kLimit || cols > kLimit ||
        (format != HK_FP4_MXFP4 && format != HK_FP4_NVFP4))
        return 0;
    return static_cast<size_t>(ceil_div(rows, 128) * 128 * padded_blocks(cols, format));
}

extern "C" hk_status hk_fp4_quantize(const void* X, int32_t x_type, int64_t rows, int64_t cols, int64_t ldx, void* codes,
                                     int64_t ld_codes, void* scales, int32_t format, const float* global_scale,
                                     void* stream) {
    hk_status s = check_format(format);
    if (s != HK_OK) return s;
    if (x_type < HK_TYPE_BF16 || x_type > HK_TYPE_FP32) return fail(HK_ERR_INVALID_ARG, "unknown element type %d", (int)x_type);
    if ((s = check_matrix("quantised matrix", codes, ld_codes, scales, rows, cols)) != HK_OK) return s;
    if (ldx < cols) return fail(HK_ERR_INVALID_ARG, "leading dimension %lld below the %lld columns", (long long)ldx, (long long)cols);
    if (format == HK_FP4_MXFP4 && global_scale) return fail(HK_ERR_INVALID_ARG, "MXFP4 has no global scale");
    if (rows == 0 || cols == 0) return HK_OK;
    if (!X) return fail(HK_ERR_INVALID_ARG, "null input pointer");
    if (!aligned(X, type_bytes(x_type)) || !aligned(global_scale, 4)) return fail(HK_ERR_MISALIGNED, "a pointer is not aligned to its elements");
    int device = 0, sms = 0;
    if ((s = current_device(&device, &sms)) != HK_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool nv = format == HK_FP4_NVFP4;
    auto go = [&](auto mx_fn, auto nv_fn) { return (nv ? nv_fn : mx_fn)(X, rows, cols, ldx, codes, ld_codes, scales, global_scale, st); };
    cudaError_t e;
    switch (x_type) {
        case HK_TYPE_BF16: e = go(&launch_quantize<__nv_bfloat16, kMxfp4>, &launch_quantize<__nv_bfloat16, kNvfp4>); break;
        case HK_TYPE_FP16: e = go(&launch_quantize<__half, kMxfp4>, &launch_quantize<__half, kNvfp4>); break;
        default: e = go(&launch_quantize<float, kMxfp4>, &launch_quantize<float, kNvfp4>); break;
    }
    return e == cudaSuccess ? HK_OK : cuda_fail(HK_ERR_LAUNCH, "launching the quantisation", e);
}

extern "C" hk_status hk_fp4_dequantize(const void* codes, int64_t ld_codes, const void* scales, int32_t format,
                                       const float* global_scale, int64_t rows, int64_t cols, void* Y, int32_t y_type,
                                       int64_t ldy, void* stream) {
    hk_status s = check_format(format);
    if (s != HK_OK) return s;
    if (y_type < HK_TYPE_BF16 || y_type > HK_TYPE_FP32) return fail(HK_ERR_INVALID_ARG, "unknown element type %d", (int)y_type);
    if ((s = check_matrix("quantised matrix", codes, ld_codes, scales, rows, cols)) != HK_OK) return s;
    if (ldy < cols) return fail(HK_ERR_INVALID_ARG, "leading dimension %lld below the %lld columns", (long long)ldy, (long long)cols);
    if (format == HK_FP4_MXFP4 && global_scale) return fail(HK_ERR_INVALID_ARG, "MXFP4 has no global scale");
    if (rows == 0 || cols == 0) return HK_OK;
    if (!Y) return fail(HK_ERR_INVALID_ARG, "null output pointer");
    if (!aligned(Y, type_bytes(y_type)) || !aligned(global_scale, 4)) return fail(HK_ERR_MISALIGNED, "a pointer is not aligned to its elements");
    int device = 0, sms = 0;
    if ((s = current_device(&device, &sms)) != HK_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool nv = format == HK_FP4_NVFP4;
    auto go = [&](auto mx_fn, auto nv_fn) { return (nv ? nv_fn : mx_fn)(codes, ld_codes, scales, global_scale, rows, cols, Y, ldy, st); };
    cudaError_t e;
    switch (y_type) {
        case HK_TYPE_BF16: e = go(&launch_dequantize<__nv_bfloat16, kMxfp4>, &launch_dequantize<__nv_bfloat16, kNvfp4>); break;
        case HK_TYPE_FP16: e = go(&launch_dequantize<__half, kMxfp4>, &launch_dequantize<__half, kNvfp4>); break;
        default: e = go(&launch_dequantize<float, kMxfp4>, &launch_dequantize<float, kNvfp4>); break;
    }
    return e == cudaSuccess ? HK_OK : cuda_fail(HK_ERR_LAUNCH, "launching the dequantisation", e);
}

extern "C" hk_status hk_gemm_fp4_ex(const void* A, const void* SFA, const void* B, const void* SFB, void* C, int64_t M,
                                    int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldc, int32_t format,
                                    const float* global_a, const float* global_b, int32_t kernel, int32_t split_k,
                                    uint32_t flags, uint64_t timeout_ns, void* stream) {
    hk_status s = check_format(format);
    if (s != HK_OK) return s;
    if (flags & ~HK_FLAG_FAULT_DROP_ARRIVE) return fail(HK_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
    if (kernel != HK_KERNEL_AUTO && kernel != HK_KERNEL_PAIR_256x256 && kernel != HK_KERNEL_SINGLE_128x128)
        return fail(HK_ERR_INVALID_ARG, "unknown kernel id %d", (int)kernel);
    if (split_k != 0 && split_k != 1 && split_k != 2 && split_k != 4 && split_k != 8)
        return fail(HK_ERR_INVALID_ARG, "split_k %d (0, 1, 2, 4 or 8)", (int)split_k);
    if (M < 0 || N < 0 || K < 0) return fail(HK_ERR_INVALID_ARG, "negative size");
    if (ldc < N) return fail(HK_ERR_INVALID_ARG, "leading dimension of C below N");
    if (M == 0 || N == 0) return HK_OK;
    if ((s = check_matrix("A", A, lda, SFA, M, K)) != HK_OK) return s;
    if ((s = check_matrix("B", B, ldb, SFB, N, K)) != HK_OK) return s;
    if (format == HK_FP4_MXFP4 && (global_a || global_b)) return fail(HK_ERR_INVALID_ARG, "MXFP4 has no global scale");
    if (!C) return fail(HK_ERR_INVALID_ARG, "null output pointer");
    if (!aligned(C, 2) || !aligned(global_a, 4) || !aligned(global_b, 4))
        return fail(HK_ERR_MISALIGNED, "a pointer is not aligned to its elements");
    if (ceil_div(M, 16) * ceil_div(N, 128) > (int64_t(1) << 26)) return fail(HK_ERR_INVALID_ARG, "too many output tiles");
    if ((std::max(M, N) + 512) * (K + 256) > (int64_t(1) << 42)) return fail(HK_ERR_INVALID_ARG, "matrix of 2^42 elements or more");
    int device = 0, sms = 0;
    if ((s = current_device(&device, &sms)) != HK_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (K == 0) {
        e = cudaMemset2DAsync(C, static_cast<size_t>(ldc) * 2, 0, static_cast<size_t>(N) * 2, static_cast<size_t>(M), st);
        return e == cudaSuccess ? HK_OK : cuda_fail(HK_ERR_LAUNCH, "clearing C", e);
    }
    if ((s = setup(device)) != HK_OK) return s;
    uint32_t* status = nullptr;
    if ((s = hk_host::status_word(device, &status)) != HK_OK) return s;
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    if ((s = hk_host::tensor_map_encoder(&enc)) != HK_OK) return s;

    Fp4Params p = {};
    p.M = static_cast<int32_t>(M);
    p.N = static_cast<int32_t>(N);
    p.k_stages = static_cast<int32_t>(ceil_div(K, kStageCols));
    p.sfa = static_cast<const uint8_t*>(SFA);
    p.sfb = static_cast<const uint8_t*>(SFB);
    p.ga = global_a;
    p.gb = global_b;
    p.c = static_cast<uint16_t*>(C);
    p.ldc = ldc;
    p.vec_c = aligned(C, 16) && ldc % 8 == 0;
    p.flags = flags;
    p.wait.status = status;
    p.wait.launch_id = hk_host::next_launch_id();
    p.wait.timeout_ns = timeout_ns ? timeout_ns : kDefaultTimeoutNs;

    const SinglePlan plan = plan_single(M, N, K, lda % 128 == 0 && ldb % 128 == 0, format, split_k, sms);
    if (kernel == HK_KERNEL_PAIR_256x256 || (kernel == HK_KERNEL_AUTO && M > 128 && pair_us(M, N, K, format, sms) < plan.us))
        return launch_pair(enc, p, A, B, K, lda, ldb, format, sms, st);
    const SingleVariant* const v = plan.v;
    p.tiles_m = static_cast<int32_t>(ceil_div(M, v->tok));
    p.tiles_n = static_cast<int32_t>(ceil_div(N, 128));
    const int64_t tiles = int64_t(p.tiles_m) * p.tiles_n;
    int splits = plan.splits;
    while (splits > p.k_stages) splits /= 2;     // every part owns at least one stage
    CUtensorMap ta, tb;
    if ((s = encode_codes(enc, &ta, A, M, K, lda, static_cast<uint32_t>(v->tok), "A")) != HK_OK) return s;
    if ((s = encode_codes(enc, &tb, B, N, K, ldb, 128, "B")) != HK_OK) return s;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * splits));
    cfg.blockDim = dim3(static_cast<unsigned>(v->threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(v->smem);
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, v->fn, ta, tb, p, splits);
    return e == cudaSuccess ? HK_OK : cuda_fail(HK_ERR_LAUNCH, "launching the 4-bit product", e);
}

extern "C" hk_status hk_gemm_fp4(const void* A, const void* SFA, const void* B, const void* SFB, void* C, int64_t M,
                                 int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldc, int32_t format,
                                 const float* global_a, const float* global_b, void* stream) {
    return hk_gemm_fp4_ex(A, SFA, B, SFB, C, M, N, K, lda, ldb, ldc, format, global_a, global_b, HK_KERNEL_AUTO, 0, 0u, 0u,
                          stream);
}
