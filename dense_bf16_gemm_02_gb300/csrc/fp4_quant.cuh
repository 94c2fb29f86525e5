// Microscaled 4-bit floating point: quantisation of a matrix and its way back.
//
// A row of K values is cut into blocks along K. Each block keeps one scale and
// each value a 4-bit E2M1 code (1 sign, 2 exponent, 1 fraction bit; magnitudes
// 0, 0.5, 1, 1.5, 2, 3, 4, 6):
//
//   MXFP4: blocks of 32, scale 2^E with E = floor(log2 amax) - 2, kept as the
//          UE8M0 byte E + 127; code = e2m1_rne(x · 2^-E), magnitudes above 6
//          (at most 8 occur) to 6;
//   NVFP4: blocks of 16, scale s = e4m3_rne(amax / (6·g)), at most 448, for a
//          global scale g of the whole matrix; code = e2m1_rne(x · (1 / (s·g))).
//
// Multiplying by the reciprocal (one division per block) rounds once more than
// dividing each value would: at most 2^-23 relative, against E2M1's steps of
// 2^-2. A block that holds a NaN or an infinity gets a NaN scale and codes 0,
// so everything computed from it is NaN.
//
// Layout: two codes per byte, the even column in the low half; rows padded with
// code 0 to a multiple of 32 columns. Scales go to the tiles that the tensor
// core's scale copies read (128 rows × 4 blocks = 512 bytes, see
// scale_offset), with blocks padded (scale 0) to whole 256-column chunks and
// rows to whole tiles.
//
// What bounds both kernels is memory (per value 2 or 4 bytes are read and 0.53 or
// 0.56 written, or the other way round) as long as their instructions stay under
// some 60 per eight values: at 141 (a first form) issuing them took 79 us for
// 16384 x 8192 bf16 values; now 53 us, 6.4 TB/s read and written (MXFP4; the way
// back the same). A warp takes 1024 columns of a row, four chunks of 256
// whose loads (eight values per lane and chunk, 16 bytes of a 16-bit type) are all
// issued before the first is used; a block's maximum is a two- or one-step
// butterfly over the 4 or 2 lanes that hold it; the scale bytes of the four chunks
// are gathered into words together. Rows that are not 16-byte aligned, and a row's
// last columns, go through shared memory, so that memory is still read and written
// in consecutive elements.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "elements.cuh"
#include "ptx.cuh"

namespace hk {
namespace fp4 {

constexpr int kMxfp4 = 0;
constexpr int kNvfp4 = 1;
constexpr int kChunkCols = 256;    // columns of a chunk: 128 bytes of codes, whole scale tiles
constexpr int kSpanChunks = 4;     // chunks a warp loads at once
constexpr int kQuantWarps = 8;

__host__ __device__ constexpr int block_cols(int fmt) { return fmt == kNvfp4 ? 16 : 32; }

// Scale blocks of a row after padding: whole chunks.
__host__ __device__ constexpr int64_t padded_blocks(int64_t cols, int fmt) {
    return (cols + kChunkCols - 1) / kChunkCols * (kChunkCols / block_cols(fmt));
}

// Byte offset of the scale of block `b` of row `row` (nb: padded_blocks): tiles
// of 128 rows × 4 blocks, row groups outermost; inside a tile byte
// (row % 32)·16 + (row % 128 / 32)·4 + b % 4.
__host__ __device__ __forceinline__ int64_t scale_offset(int64_t row, int64_t b, int64_t nb) {
    return ((row >> 7) * (nb >> 2) + (b >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (b & 3);
}

// Eight floats to eight E2M1 codes (round to nearest even, magnitudes above 6
// to 6), value 0 in the lowest four bits.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// The values of eight E2M1 codes.
__device__ __forceinline__ void unpack_e2m1x8(uint32_t codes, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 p = *reinterpret_cast<const __half2*>(&h[i]);
        v[2 * i] = __low2float(p);
        v[2 * i + 1] = __high2float(p);
    }
}

// 2^(byte - 127); 255 is NaN.
__device__ __forceinline__ float ue8m0_value(uint32_t byte) {
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23);
}

template <int kFmt>
__device__ __forceinline__ float scale_value(uint32_t byte) {
    return kFmt == kNvfp4 ? e4m3_value(byte) : ue8m0_value(byte);
}

// The largest magnitude of three values; NaN if one of them is.
__device__ __forceinline__ float amax3(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A chunk's elements lane, lane + 32, ... (0 past the row's end) as they are
// read and written when a row cannot be taken 16 bytes at a time.
template <typename T>
struct Spread8 {
    T e[8];
};

template <typename T>
__device__ __forceinline__ Spread8<T> load_spread(const T* row, int64_t col, int64_t cols, uint32_t lane) {
    Spread8<T> r;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t c = col + lane + 32 * j;
        r.e[j] = c < cols ? row[c] : from_float<T>(0.0f);
    }
    return r;
}

// A global scale below 2^-60 is taken times 2^64 (kLift), and so is what meets it, so that s·g and its reciprocal
// stay within fp32's normal numbers (for s·g < 2^-128 the reciprocal alone would be infinite). Powers of two:
// every code and scale is the one that fp32 without a least exponent would give. The kernels' loops are compiled
// for both (one choice in the loop cost 18 % more instructions: 61.7 us for 57.6 at 16384 x 8192).
constexpr float kSmallScale = 0x1p-60f;
constexpr float kLift = 0x1p64f;

// ------------------------------------------------------------- quantise --

// NVFP4: what the scale bytes of a matrix with global scale g mean to the
// quantisation, 1 / (e4m3 · g), once per block of threads (two divisions per
// block of values would cost more than everything else).
__device__ __forceinline__ void fill_reciprocals(float (&table)[128], float g) {
    for (int i = static_cast<int>(threadIdx.y * 32 + threadIdx.x); i < 128; i += 32 * kQuantWarps) {
        const float d = __fmul_rn(e4m3_value(static_cast<uint32_t>(i)), g);
        table[i] = d > 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
    }
    __syncthreads();
}

// Eight values of a block to codes; the block's scale byte. `six_g`, `per_six_g`:
// 6·g and its reciprocal, both rounded to nearest; kLifted: g was taken times kLift.
template <int kFmt, bool kLifted>
__device__ __forceinline__ uint32_t quantize8(float (&v)[8], float six_g, float per_six_g, const float* reciprocals,
                                              uint32_t& byte) {
    float m = amax3(v[0], v[1], v[2]);
    m = amax3(m, v[3], v[4]);
    m = amax3(m, v[5], v[6]);
    m = amax3(m, v[7], 0.0f);
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
    if constexpr (kFmt == kMxfp4) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t top = __float_as_uint(m);
    float mul;
    if constexpr (kFmt == kMxfp4) {
        byte = max(top >> 23, 2u) - 2u;
        mul = __uint_as_float((254u - byte) << 23);        // 2^-(byte - 127), exact
    } else {
        // m / (6·g) to nearest by one correction of m · (1 / (6·g)) with its exact remainder (P. Markstein,
        // IBM J. Res. Dev. 34, 1990); where that leaves fp32's range the quotient is 0 or above 448 either way
        if constexpr (kLifted) {
            m = __fmul_rn(m, kLift);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], kLift);
        }
        const float q0 = __fmul_rn(m, per_six_g);
        const float q = __fmaf_rn(__fmaf_rn(-q0, six_g, m), per_six_g, q0);
        byte = e4m3_of(isfinite(q) ? q : q0);
        mul = reciprocals[byte & 0x7Fu];
    }
    const uint64_t mul2 = f32x2(mul, mul);
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f32x2_split(fmul2(f32x2(v[2 * i], v[2 * i + 1]), mul2), y[2 * i], y[2 * i + 1]);
    const uint32_t codes = pack_e2m1x8(y);
    const bool finite = top < 0x7F800000u;
    byte = finite ? byte : kFmt == kMxfp4 ? 255u : 0x7Fu;
    return finite ? codes : 0u;
}

// The scale bytes of four consecutive chunks, byte[i] of chunk i in all lanes of
// its block, to words of four blocks in the scale tiles: `at` is the address of
// the first chunk's first word (tiles are 512 bytes apart). Lanes of one block
// each take another chunk's byte, so that one exchange serves several chunks.
template <int kFmt>
__device__ __forceinline__ void store_scales(const uint32_t (&byte)[kSpanChunks], uint8_t* at, int chunks, uint32_t lane) {
    constexpr uint32_t kLanes = block_cols(kFmt) / 8;      // lanes of a block: 4 or 2
    constexpr int kWords = kChunkCols / block_cols(kFmt) / 4;   // words of a chunk: 2 or 4
    const uint32_t sub = lane % kLanes;
#pragma unroll
    for (int i0 = 0; i0 < kSpanChunks; i0 += static_cast<int>(kLanes)) {
        uint32_t b = byte[i0];
#pragma unroll
        for (uint32_t k = 1; k < kLanes; ++k) b = sub == k ? byte[i0 + k] : b;
        uint32_t word = b << (8 * ((lane / kLanes) & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, kLanes);
        word |= __shfl_xor_sync(0xffffffffu, word, 2 * kLanes);
        const int chunk = i0 + static_cast<int>(sub);
        if (((lane / kLanes) & 3) == 0 && chunk < chunks)
            *reinterpret_cast<uint32_t*>(at + (chunk * kWords + static_cast<int>(lane / (4 * kLanes))) * 512) = word;
    }
}

// What a warp works on: item i of rows × spans, a span being the 1024 columns
// that it loads at once. (A 64-bit division would cost a quarter of the item.)
struct Item {
    int64_t row, chunk;        // the span's first chunk
};

__device__ __forceinline__ Item item_of(uint64_t i, uint64_t items, uint32_t spans) {
    const uint64_t row = items <= 0xFFFFFFFFull ? static_cast<uint32_t>(i) / spans : i / spans;
    return Item{static_cast<int64_t>(row), static_cast<int64_t>(i - row * spans) * kSpanChunks};
}

// Every warp on items of its own: spans of the rows, padding rows of the last scale tile included (their scales are 0).
template <typename T, int kFmt, bool kLifted>
__device__ __forceinline__ void quantize_items(const T* x, int64_t rows, int64_t cols, int64_t ldx, uint8_t* codes, int64_t ld_codes,
                                               uint8_t* scales, uint32_t spans, int vec, float* staged, const float* reciprocals,
                                               float six_g, float per_six_g) {
    const uint32_t lane = threadIdx.x;
    const int64_t chunks = (cols + kChunkCols - 1) / kChunkCols;
    const int64_t whole = vec ? cols / kChunkCols : 0;     // chunks that are read 16 bytes at a time
    const int64_t code_cols = (cols + 31) / 32 * 32;
    constexpr int kScaleStep = kChunkCols / block_cols(kFmt) / 4 * 512;    // bytes of a chunk's scale tiles
    const uint64_t items = static_cast<uint64_t>((rows + 127) / 128 * 128) * spans;
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * kQuantWarps + threadIdx.y; i < items;
         i += static_cast<uint64_t>(gridDim.x) * kQuantWarps) {
        const Item item = item_of(i, items, spans);
        const int64_t row = item.row, c0 = item.chunk;
        const T* const src = x + row * ldx;
        uint8_t* const dst = codes + row * ld_codes + lane * 4;
        uint8_t* const scale_row = scales + (row >> 7) * chunks * kScaleStep + (row & 31) * 16 + ((row >> 5) & 3) * 4;
        uint32_t byte[kSpanChunks];
        const int n = static_cast<int>(min(chunks - c0, static_cast<int64_t>(kSpanChunks)));
        if (row >= rows) {
#pragma unroll
            for (int i = 0; i < kSpanChunks; ++i) byte[i] = 0;
        } else if (c0 + kSpanChunks <= whole) {
            Raw8<T> raw[kSpanChunks];
            const T* const at = src + c0 * kChunkCols + lane * 8;
#pragma unroll
            for (int i = 0; i < kSpanChunks; ++i) raw[i] = load8<T>(at + i * kChunkCols, 0, 8, true);
            uint8_t* const out = dst + c0 * (kChunkCols / 2);
#pragma unroll
            for (int i = 0; i < kSpanChunks; ++i) {
                float v[8];
                widen8<T>(raw[i], v);
                *reinterpret_cast<uint32_t*>(out + i * (kChunkCols / 2)) = quantize8<kFmt, kLifted>(v, six_g, per_six_g, reciprocals, byte[i]);
            }
        } else {
            Spread8<T> raw[kSpanChunks];
#pragma unroll
            for (int i = 0; i < kSpanChunks; ++i) raw[i] = load_spread<T>(src, (c0 + i) * kChunkCols, cols, lane);
            float* const buf = staged;
#pragma unroll
            for (int i = 0; i < kSpanChunks; ++i) {
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j) buf[lane + 32 * j] = to_float(raw[i].e[j]);
                __syncwarp();
                float v[8];
                memcpy(v, buf + lane * 8, sizeof v);
                const uint32_t packed = quantize8<kFmt, kLifted>(v, six_g, per_six_g, reciprocals, byte[i]);
                if ((c0 + i) * kChunkCols + lane * 8 < code_cols)
                    *reinterpret_cast<uint32_t*>(dst + (c0 + i) * (kChunkCols / 2)) = packed;
            }
        }
        store_scales<kFmt>(byte, scale_row + c0 * kScaleStep, n, lane);
    }
}

// Block (32, kQuantWarps).
template <typename T, int kFmt>
__global__ void __launch_bounds__(32 * kQuantWarps, 4)
quantize_kernel(const T* x, int64_t rows, int64_t cols, int64_t ldx, uint8_t* codes, int64_t ld_codes, uint8_t* scales,
                const float* global_scale, uint32_t spans, int vec) {
    __shared__ float staged[kQuantWarps][kChunkCols];
    __shared__ float reciprocals[kFmt == kNvfp4 ? 128 : 1];
    griddep_launch_dependents();
    griddep_wait();                  // launched early behind the kernel that may have written x
    if constexpr (kFmt == kNvfp4) {
        float g = global_scale != nullptr ? *global_scale : 1.0f;
        const bool small = g < kSmallScale;
        if (small) g = __fmul_rn(g, kLift);
        const float six_g = __fmul_rn(6.0f, g);
        const float per_six_g = fminf(__fdiv_rn(1.0f, six_g), 3.4028235e38f);   // (finite: 0 times it is 0)
        fill_reciprocals(reciprocals, g);
        if (small)
            quantize_items<T, kFmt, true>(x, rows, cols, ldx, codes, ld_codes, scales, spans, vec, staged[threadIdx.y], reciprocals,
                                          six_g, per_six_g);
        else
            quantize_items<T, kFmt, false>(x, rows, cols, ldx, codes, ld_codes, scales, spans, vec, staged[threadIdx.y], reciprocals,
                                           six_g, per_six_g);
    } else {
        quantize_items<T, kFmt, false>(x, rows, cols, ldx, codes, ld_codes, scales, spans, vec, staged[threadIdx.y], reciprocals, 6.0f,
                                       0.0f);
    }
}

// ----------------------------------------------------------- dequantise --

// Eight codes times their scale, rounded once to T; kLifted: the scale was taken times kLift.
template <typename T, bool kLifted>
__device__ __forceinline__ void dequantize8(uint32_t codes, float scale, T (&e)[8]) {
    float v[8];
    unpack_e2m1x8(codes, v);
    if constexpr (kLifted) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(__fmul_rn(v[i], scale), 1.0f / kLift);
        scale = 1.0f;
    }
    const uint64_t s2 = f32x2(scale, scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        f32x2_split(fmul2(f32x2(v[2 * i], v[2 * i + 1]), s2), a, b);
        if constexpr (sizeof(T) == 4) {
            e[2 * i] = a;
            e[2 * i + 1] = b;
        } else {
            const uint32_t pair = pack_pair<T>(a, b);
            memcpy(&e[2 * i], &pair, 4);
        }
    }
}

// y = code · (scale · g), rounded once to T.
template <typename T, int kFmt, bool kLifted>
__device__ __forceinline__ void dequantize_items(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, float g, int64_t rows,
                                                 int64_t cols, T* y, int64_t ldy, uint32_t spans, int vec, T* staged) {
    const uint32_t lane = threadIdx.x;
    const int64_t chunks = (cols + kChunkCols - 1) / kChunkCols;
    const int64_t whole = vec ? cols / kChunkCols : 0;
    const int64_t code_cols = (cols + 31) / 32 * 32;
    constexpr int kLanes = block_cols(kFmt) / 8;
    constexpr int kScaleStep = kChunkCols / block_cols(kFmt) / 4 * 512;
    const int block = static_cast<int>(lane) / kLanes;     // of this lane's values in a chunk
    const uint64_t items = static_cast<uint64_t>(rows) * spans;
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * kQuantWarps + threadIdx.y; i < items;
         i += static_cast<uint64_t>(gridDim.x) * kQuantWarps) {
        const Item item = item_of(i, items, spans);
        const int64_t row = item.row, c0 = item.chunk;
        const uint8_t* const src = codes + row * ld_codes + lane * 4;
        const uint8_t* const scale_row = scales + (row >> 7) * chunks * kScaleStep + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
                                         (block >> 2) * 512 + (block & 3);
        T* const dst = y + row * ldy;
        uint32_t packed[kSpanChunks], byte[kSpanChunks];
        const uint8_t* const at = src + c0 * (kChunkCols / 2);
        const uint8_t* const scale_at = scale_row + c0 * kScaleStep;
        if (c0 + kSpanChunks <= whole) {
#pragma unroll
            for (int i = 0; i < kSpanChunks; ++i) {
                packed[i] = *reinterpret_cast<const uint32_t*>(at + i * (kChunkCols / 2));
                byte[i] = scale_at[i * kScaleStep];
            }
            T* const out = dst + c0 * kChunkCols + lane * 8;
#pragma unroll
            for (int i = 0; i < kSpanChunks; ++i) {
                T e[8];
                dequantize8<T, kLifted>(packed[i], kFmt == kNvfp4 ? scale_value<kFmt>(byte[i]) * g : scale_value<kFmt>(byte[i]), e);
                uint4 o[sizeof(T) / 2];
                memcpy(o, e, sizeof o);
#pragma unroll
                for (int k = 0; k < static_cast<int>(sizeof(T) / 2); ++k) reinterpret_cast<uint4*>(out + i * kChunkCols)[k] = o[k];
            }
        } else {
            const int n = static_cast<int>(min(chunks - c0, static_cast<int64_t>(kSpanChunks)));
#pragma unroll
            for (int i = 0; i < kSpanChunks; ++i) {
                packed[i] = byte[i] = 0;
                if (i < n && (c0 + i) * kChunkCols + lane * 8 < code_cols) {
                    packed[i] = *reinterpret_cast<const uint32_t*>(at + i * (kChunkCols / 2));
                    byte[i] = scale_at[i * kScaleStep];
                }
            }
            T* const buf = staged;
#pragma unroll
            for (int i = 0; i < kSpanChunks; ++i) {
                if (i >= n) break;
                T e[8];
                dequantize8<T, kLifted>(packed[i], kFmt == kNvfp4 ? scale_value<kFmt>(byte[i]) * g : scale_value<kFmt>(byte[i]), e);
                __syncwarp();
                memcpy(buf + lane * 8, e, sizeof e);
                __syncwarp();
                const int64_t col = (c0 + i) * kChunkCols + lane;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col + 32 * j < cols) dst[col + 32 * j] = buf[lane + 32 * j];
            }
        }
    }
}

template <typename T, int kFmt>
__global__ void __launch_bounds__(32 * kQuantWarps, 6)
dequantize_kernel(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, const float* global_scale, int64_t rows,
                  int64_t cols, T* y, int64_t ldy, uint32_t spans, int vec) {
    __shared__ T staged[kQuantWarps][kChunkCols];
    griddep_launch_dependents();
    griddep_wait();                  // launched early behind the kernel that may have written the codes
    const float g = kFmt == kNvfp4 && global_scale != nullptr ? *global_scale : 1.0f;
    if (kFmt == kNvfp4 && g < kSmallScale)
        dequantize_items<T, kFmt, kFmt == kNvfp4>(codes, ld_codes, scales, __fmul_rn(g, kLift), rows, cols, y, ldy, spans, vec,
                                                  staged[threadIdx.y]);
    else
        dequantize_items<T, kFmt, false>(codes, ld_codes, scales, g, rows, cols, y, ldy, spans, vec, staged[threadIdx.y]);
}

}  // namespace fp4
}  // namespace hk
