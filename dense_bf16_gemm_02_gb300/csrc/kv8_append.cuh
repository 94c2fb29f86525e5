// Appending keys and values to a paged cache held in E4M3 with one scale per
// page and head.
//
// A page holds `page_size` tokens of every KV head: codes [page, head, token,
// D], one fp32 scale per (page, head), always a power of two, so that a value
// is code · scale and changing the scale moves only the exponent. The tokens
// that arrive in a page need the scale 2^e with the smallest e for which their
// largest finite magnitude is at most 448 · 2^e (E4M3's largest number); a page
// that holds earlier tokens keeps its scale if that is larger, else its codes
// are rounded once more to the new scale (exact unless they fall below E4M3's
// smallest normal number).
//
// One item is a (sequence, touched page, head), keys and values: one warp when
// few tokens arrive per page, else eight warps. The new tokens of an item
// stay in registers between the maximum and the rounding, so that they are read
// once. A block does one item, so latency and the number of blocks on an SM
// bound the kernel, and the issue of its instructions (54 % of the slots): the
// registers hold no more steps than a page needs, keys and values are in flight
// together, both are asked for before the page's index is looked at, and what does
// not depend on the data is known when it is compiled. 8 x 2048 tokens of 8 heads of
// 128, bf16: 17.9 us, 5.6 TB/s read and written (19.1 with head dimension and page
// size as arguments); 64 single tokens 2.4 us, a launch.
#pragma once

#include <cstdint>

#include "bounded_wait.cuh"
#include "elements.cuh"

namespace hk {
namespace kv8 {

struct AppendParams {
    const void* src[2];            // new keys, new values
    int64_t stride_b[2], stride_t[2], stride_h[2];   // in elements
    uint8_t* codes[2];             // [pages, Hkv, page_size, D]
    float* scale[2];               // [pages, Hkv]
    const int32_t* table;          // [B, max_pages]
    int64_t table_stride;
    const int32_t* starts;         // tokens of each sequence before the append
    const int32_t* counts;         // new tokens of each sequence, or null (T)
    int64_t items;                 // B * slots * Hkv, below 2^32
    int32_t B, T;
    uint32_t Hkv, slots;           // heads; pages a sequence can touch
    int32_t page_shift, max_pages; // log2 of the page's tokens
    int64_t num_pages;
    int32_t vec[2];                // 16-byte loads
    uint32_t* status;
};

constexpr int kAppendSteps = 8;    // most steps of a group of warps: 8 elements per lane and step

// The exponent field of the page scale for a largest magnitude (its bits).
__device__ __forceinline__ uint32_t scale_field(uint32_t amax_bits) {
    const int field = static_cast<int>(amax_bits >> 23);                   // 127 + floor(log2 amax)
    const int e = field - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u);       // 448 = 1.75 · 2^8
    return static_cast<uint32_t>(e < 1 ? 1 : e);
}

// Sixteen codes times a power of two, rounded to E4M3 again.
__device__ __forceinline__ uint32_t rescale_codes(uint32_t w, float ratio) {
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = (w >> (8 * i)) & 0xFFu;
        out |= e4m3_of(e4m3_value(b) * ratio) << (8 * i);
    }
    return out;
}

// The largest of the magnitude bits of eight elements, as they are held (16-bit
// types two to a word), and what a word of them means as fp32 bits. Kept apart
// from the conversion to fp32, so that no more than the elements themselves
// lives in registers between the loads and the stores.
template <typename T>
struct Magnitude;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

template <>
struct Magnitude<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t of(const Raw8<__nv_bfloat16>& r, uint32_t m) {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max_u16x2(m, w[i] & 0x7FFF7FFFu);
        return m;
    }
    static __device__ __forceinline__ uint32_t bits(uint32_t m) { return max(m & 0xFFFFu, m >> 16) << 16; }
};

template <>
struct Magnitude<__half> {
    static __device__ __forceinline__ uint32_t of(const Raw8<__half>& r, uint32_t m) {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max_u16x2(m, w[i] & 0x7FFF7FFFu);
        return m;
    }
    static __device__ __forceinline__ uint32_t bits(uint32_t m) {
        return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(max(m & 0xFFFFu, m >> 16)))));
    }
};

template <>
struct Magnitude<float> {
    static __device__ __forceinline__ uint32_t of(const Raw8<float>& r, uint32_t m) {
        const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
        return m;
    }
    static __device__ __forceinline__ uint32_t bits(uint32_t m) { return m; }
};

template <typename T, int kD, int kWarps, int kSteps>
__global__ void __launch_bounds__(256, 2 * kSteps * sizeof(Raw8<T>) <= 128 ? 4 : 2)
kv8_append_kernel(const AppendParams p) {
    constexpr int kLanes = kD / 8;                   // of a token: 8 elements each
    constexpr int kStepTokens = kWarps * 32 / kLanes;
    __shared__ uint32_t warp_top[2][8];
    griddep_launch_dependents();
    griddep_wait();                  // launched early behind the kernel that may have written the tokens
    const uint32_t lane = threadIdx.x & 31u;
    const uint32_t warp = threadIdx.x >> 5;
    const uint32_t member = kWarps == 1 ? 0 : warp;          // this warp's place in its item
    const int64_t item = kWarps == 1 ? static_cast<int64_t>(blockIdx.x) * 8 + warp : static_cast<int64_t>(blockIdx.x);
    if (item >= p.items) return;
    uint32_t rest = static_cast<uint32_t>(item);
    const uint32_t h = rest % p.Hkv;
    rest /= p.Hkv;
    const int b = static_cast<int>(rest / p.slots);
    const uint32_t nth = rest % p.slots;

    const int32_t start = p.starts[b];
    const int32_t count = p.counts != nullptr ? p.counts[b] : p.T;
    const int64_t room = static_cast<int64_t>(p.max_pages) << p.page_shift;
    const bool bad = start < 0 || count < 0 || count > p.T || start + static_cast<int64_t>(count) > room;
    if (bad) {
        if (lane == 0 && nth == 0) atomicOr(p.status, kErrPage);
        return;
    }
    // (below 2^32: the room is below 2^31, and so are the pages that T tokens can touch)
    const uint32_t slot = (static_cast<uint32_t>(start) >> p.page_shift) + nth;
    const uint32_t first = slot << p.page_shift;
    const uint32_t lo = max(static_cast<uint32_t>(start), first);                         // new tokens of this page
    const uint32_t hi = min(static_cast<uint32_t>(start) + static_cast<uint32_t>(count), first + (1u << p.page_shift));
    if (lo >= hi) return;
    const int old_tokens = static_cast<int>(lo - first);
    const int n = static_cast<int>(hi - lo);

    const int sub = static_cast<int>((member * 32 + lane) / kLanes);      // this lane's token of each step
    const int d = static_cast<int>(lane) % kLanes * 8;
    Raw8<T> raw[2][kSteps];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const T* const src = static_cast<const T*>(p.src[kv]) + b * p.stride_b[kv] +
                             static_cast<int64_t>(lo - static_cast<uint32_t>(start)) * p.stride_t[kv] + h * p.stride_h[kv] + d;
        // (one choice for all steps: with a choice at each load the next one waited for it; past the last token
        // it is taken again, which moves no maximum and needs no test)
        if (p.vec[kv]) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
                raw[kv][i] = load8<T>(src + min(i * kStepTokens + sub, n - 1) * p.stride_t[kv], 0, 8, true);
        } else {
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
                raw[kv][i] = load8<T>(src + min(i * kStepTokens + sub, n - 1) * p.stride_t[kv], 0, 8, false);
        }
    }
    const int64_t page = p.table[b * p.table_stride + slot];
    if (page < 0 || page >= p.num_pages) {
        if (lane == 0) atomicOr(p.status, kErrPage);
        return;
    }
    const int64_t ph = page * p.Hkv + h;
    float had[2] = {0.0f, 0.0f};
    if (old_tokens > 0) {
        had[0] = p.scale[0][ph];
        had[1] = p.scale[1][ph];
    }
    uint32_t top[2];                // largest finite magnitude, as bits
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) m = Magnitude<T>::of(raw[kv][i], m);
        top[kv] = __reduce_max_sync(0xffffffffu, Magnitude<T>::bits(m));
        if (top[kv] >= 0x7F800000u) {           // an infinity or NaN among this warp's values: without them
            m = 0;
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                float v[8];
                widen8<T>(raw[kv][i], v);
#pragma unroll
                for (int k = 0; k < 8; ++k) m = max(m, isfinite(v[k]) ? __float_as_uint(v[k]) & 0x7FFFFFFFu : 0u);
            }
            top[kv] = __reduce_max_sync(0xffffffffu, m);
        }
    }
    if constexpr (kWarps > 1) {
        if (lane < 2) warp_top[lane][warp] = lane == 0 ? top[0] : top[1];
        __syncthreads();
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) top[kv] = __reduce_max_sync(0xffffffffu, warp_top[kv][lane & 7u]);
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const float need = __uint_as_float(scale_field(top[kv]) << 23);
        const float scale = old_tokens > 0 ? fmaxf(need, had[kv]) : need;
        uint8_t* const dst = p.codes[kv] + (ph << p.page_shift) * kD;
        if (old_tokens > 0 && scale > had[kv]) {
            const float ratio = had[kv] / scale;
            uint4* const old = reinterpret_cast<uint4*>(dst);
            for (int i = static_cast<int>(member * 32 + lane); i < old_tokens * (kD / 16); i += 32 * kWarps) {
                uint4 w = old[i];
                w.x = rescale_codes(w.x, ratio);
                w.y = rescale_codes(w.y, ratio);
                w.z = rescale_codes(w.z, ratio);
                w.w = rescale_codes(w.w, ratio);
                old[i] = w;
            }
        }
        const float inv = 1.0f / scale;      // exact: a power of two
        const uint64_t inv2 = f32x2(inv, inv);
        uint8_t* const at = dst + (old_tokens + sub) * kD + d;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            if (i * kStepTokens + sub < n) {
                float v[8];
                widen8<T>(raw[kv][i], v);
                uint32_t w[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float y[4];
                    f32x2_split(fmul2(f32x2(v[4 * k], v[4 * k + 1]), inv2), y[0], y[1]);
                    f32x2_split(fmul2(f32x2(v[4 * k + 2], v[4 * k + 3]), inv2), y[2], y[3]);
                    asm("{\n\t.reg .b16 lo, hi;\n\t"
                        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
                        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
                        "mov.b32 %0, {lo, hi};\n\t}"
                        : "=r"(w[k])
                        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]));
                }
                *reinterpret_cast<uint2*>(at + i * (kStepTokens * kD)) = make_uint2(w[0], w[1]);
            }
        }
        if (member == 0 && lane == 0) p.scale[kv][ph] = scale;
    }
}

}  // namespace kv8
}  // namespace hk
