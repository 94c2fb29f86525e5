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
// Both kernels are bound by memory: per value 2 (or 4) bytes are read and
// 0.53 or 0.56 written. A warp takes 1024 columns of a row, four chunks of 256
// whose loads (16 bytes per lane and chunk, contiguous over the warp) are all
// issued before the first is used; a block's maximum is a two- or one-step
// butterfly over the 4 or 2 lanes that hold it.
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

// ------------------------------------------------------------- quantise --

// One chunk of a row: this lane's 8 values to codes, the block's scale, and
// the scale words of the chunk (4 blocks each), which the first lane of each
// word's lanes stores.
template <int kFmt>
__device__ __forceinline__ void quantize_chunk(const float (&v)[8], float g, uint32_t lane, uint32_t& codes,
                                               uint32_t& scale_word) {
    uint32_t top = 0;   // the largest magnitude, as bits: NaN above infinity above numbers
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    if constexpr (kFmt == kMxfp4) top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    uint32_t byte;
    float mul;
    if constexpr (kFmt == kMxfp4) {
        const uint32_t exp_field = top >> 23;
        byte = exp_field > 2 ? exp_field - 2 : 0;
        mul = __uint_as_float((254u - byte) << 23);        // 2^-(byte - 127), exact
    } else {
        byte = e4m3_of(__fdiv_rn(__uint_as_float(top), __fmul_rn(6.0f, g)));
        const float d = __fmul_rn(e4m3_value(byte), g);
        mul = d > 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
    }
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = v[i] * mul;
    codes = pack_e2m1x8(y);
    if (top >= 0x7F800000u) {
        byte = kFmt == kMxfp4 ? 255u : 0x7Fu;
        codes = 0;
    }
    constexpr int kLanes = block_cols(kFmt) / 8;           // lanes of a block
    scale_word = byte << (8 * ((lane / kLanes) & 3));
    scale_word |= __shfl_xor_sync(0xffffffffu, scale_word, kLanes);
    scale_word |= __shfl_xor_sync(0xffffffffu, scale_word, 2 * kLanes);
}

// Block (32, kQuantWarps): `warps_per_row` (a power of two) warps of the block
// share a row; row groups of the block walk the rows (padding rows of the last
// scale tile included: their scales are 0).
template <typename T, int kFmt>
__global__ void __launch_bounds__(32 * kQuantWarps)
quantize_kernel(const T* __restrict__ x, int64_t rows, int64_t cols, int64_t ldx, uint8_t* __restrict__ codes,
                int64_t ld_codes, uint8_t* __restrict__ scales, const float* __restrict__ global_scale,
                int warps_per_row, int vec) {
    const uint32_t lane = threadIdx.x;
    const int rows_per_block = kQuantWarps / warps_per_row;
    const int w = static_cast<int>(threadIdx.y) & (warps_per_row - 1);
    const int sub = static_cast<int>(threadIdx.y) / warps_per_row;
    const float g = kFmt == kNvfp4 && global_scale != nullptr ? *global_scale : 1.0f;
    const int64_t nb = padded_blocks(cols, kFmt);
    const int64_t chunks = (cols + kChunkCols - 1) / kChunkCols;
    const int64_t code_cols = (cols + 31) / 32 * 32;
    const int64_t rows_pad = (rows + 127) / 128 * 128;
    constexpr int kLanesPerWord = 4 * block_cols(kFmt) / 8;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_block + sub; row < rows_pad;
         row += static_cast<int64_t>(gridDim.x) * rows_per_block) {
        const T* const src = x + row * ldx;
        for (int64_t c0 = (static_cast<int64_t>(blockIdx.y) * warps_per_row + w) * kSpanChunks; c0 < chunks;
             c0 += static_cast<int64_t>(gridDim.y) * warps_per_row * kSpanChunks) {
            Raw8<T> raw[kSpanChunks];
            if (row < rows) {
#pragma unroll
                for (int i = 0; i < kSpanChunks; ++i)
                    raw[i] = load8<T>(src, (c0 + i) * kChunkCols + lane * 8, cols, vec != 0);
            } else {
                memset(raw, 0, sizeof raw);
            }
#pragma unroll
            for (int i = 0; i < kSpanChunks; ++i) {
                const int64_t chunk = c0 + i;
                if (chunk >= chunks) break;
                float v[8];
                widen8<T>(raw[i], v);
                uint32_t packed, word;
                quantize_chunk<kFmt>(v, g, lane, packed, word);
                const int64_t col = chunk * kChunkCols + lane * 8;
                if (row < rows && col < code_cols)
                    *reinterpret_cast<uint32_t*>(codes + row * ld_codes + col / 2) = packed;
                if (lane % kLanesPerWord == 0)
                    *reinterpret_cast<uint32_t*>(scales + scale_offset(row, col / block_cols(kFmt), nb)) = word;
            }
        }
    }
}

// ----------------------------------------------------------- dequantise --

// y = code · (scale · g), rounded once to T.
template <typename T, int kFmt>
__global__ void __launch_bounds__(32 * kQuantWarps)
dequantize_kernel(const uint8_t* __restrict__ codes, int64_t ld_codes, const uint8_t* __restrict__ scales,
                  const float* __restrict__ global_scale, int64_t rows, int64_t cols, T* __restrict__ y, int64_t ldy,
                  int warps_per_row, int vec) {
    const uint32_t lane = threadIdx.x;
    const int rows_per_block = kQuantWarps / warps_per_row;
    const int w = static_cast<int>(threadIdx.y) & (warps_per_row - 1);
    const int sub = static_cast<int>(threadIdx.y) / warps_per_row;
    const float g = kFmt == kNvfp4 && global_scale != nullptr ? *global_scale : 1.0f;
    const int64_t nb = padded_blocks(cols, kFmt);
    const int64_t chunks = (cols + kChunkCols - 1) / kChunkCols;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_block + sub; row < rows;
         row += static_cast<int64_t>(gridDim.x) * rows_per_block) {
        const uint8_t* const src = codes + row * ld_codes;
        T* const dst = y + row * ldy;
        for (int64_t c0 = (static_cast<int64_t>(blockIdx.y) * warps_per_row + w) * kSpanChunks; c0 < chunks;
             c0 += static_cast<int64_t>(gridDim.y) * warps_per_row * kSpanChunks) {
            uint32_t packed[kSpanChunks], byte[kSpanChunks];
#pragma unroll
            for (int i = 0; i < kSpanChunks; ++i) {
                const int64_t col = (c0 + i) * kChunkCols + lane * 8;
                packed[i] = byte[i] = 0;
                if (col < cols) {
                    packed[i] = __ldg(reinterpret_cast<const uint32_t*>(src + col / 2));
                    byte[i] = __ldg(scales + scale_offset(row, col / block_cols(kFmt), nb));
                }
            }
#pragma unroll
            for (int i = 0; i < kSpanChunks; ++i) {
                const int64_t col = (c0 + i) * kChunkCols + lane * 8;
                if (col >= cols) break;
                float v[8];
                unpack_e2m1x8(packed[i], v);
                float s = scale_value<kFmt>(byte[i]);
                if constexpr (kFmt == kNvfp4) s *= g;
                T e[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) e[k] = from_float<T>(v[k] * s);
                if (vec && col + 8 <= cols) {
                    uint4* p = reinterpret_cast<uint4*>(dst + col);
                    uint4 o[sizeof(T) / 2];
                    memcpy(o, e, sizeof o);
#pragma unroll
                    for (int k = 0; k < static_cast<int>(sizeof(T) / 2); ++k) p[k] = o[k];
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (col + k < cols) dst[col + k] = e[k];
                }
            }
        }
    }
}

}  // namespace fp4
}  // namespace hk
