// Eight consecutive elements of bf16, fp16 or fp32 at a time, and single E4M3
// values: what the quantising kernels share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <cstring>

namespace hk {

// Eight consecutive elements as they lie in memory.
template <typename T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];
};

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }

template <typename T> __device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ float from_float<float>(float x) { return x; }

// Two floats rounded to T, `a` in the low half.
template <typename T> __device__ __forceinline__ uint32_t pack_pair(float a, float b);
template <> __device__ __forceinline__ uint32_t pack_pair<__nv_bfloat16>(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
template <> __device__ __forceinline__ uint32_t pack_pair<__half>(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Elements [col, col + 8) of a row of `cols`, 0 past its end. `vec`: the row
// is 16-byte aligned (16-byte loads). (Ordinary loads, not the read-only path:
// the kernels that use them may have started before the data was written.)
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* row, int64_t col, int64_t cols, bool vec) {
    Raw8<T> r;
    if (vec && col + 8 <= cols) {
        const uint4* p = reinterpret_cast<const uint4*>(row + col);
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.w[i] = p[i];
    } else {
        T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = col + i < cols ? row[col + i] : from_float<T>(0.0f);
        memcpy(&r, e, sizeof r);
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void widen8(const Raw8<T>& r, float (&v)[8]) {
    T e[8];
    memcpy(e, &r, sizeof r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_float(e[i]);
}

// x to E4M3 (round to nearest even, magnitudes above 448 to 448; NaN 0x7F).
__device__ __forceinline__ uint32_t e4m3_of(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(x));
    return r & 0xFFu;
}

__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(byte & 0xFFu)));
    return __low2float(*reinterpret_cast<const __half2*>(&h));
}

// 0xFF in the place of each of four E4M3 codes that is a NaN, 0 elsewhere.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu); }

}  // namespace hk
