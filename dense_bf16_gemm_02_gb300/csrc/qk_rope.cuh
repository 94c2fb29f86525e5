// The norm of each head's query and key and the rotation by the token's position, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w          (per head; left out without eps)
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t),   t_i = position[axis(i)] * inv_freq[i]
//
// over the pairs (a, b) = (y_i, y_{i + R/2}) or (y_{2i}, y_{2i+1}) of the first R of D elements.
//
// Every element is read once and written once: what bounds it is memory. A row
// (one head of one token) is 8 elements each of 8, 16 or 32 lanes, so that a
// warp's load is whole lines; a warp keeps to one token and takes `steps` times
// 32 / lanes rows of its queries or keys, so that the angles are worked out once for all of them:
// as few as leave every SM full of warps (a decoding step), up to all heads (a
// prompt).
//
// Angles. A position times a frequency loses its fraction of a turn in 32 bits
// (position 10^6: an error of 0.06 radians). Here the frequency is taken as the
// turns per position, inv_freq / 2 pi, in fixed point with 64 bits behind the
// point: 24 bits of mantissa times a 64-bit 1 / 2 pi, shifted. Times the
// position modulo 2^64 that is the fraction of a turn to within 2^-33 whatever
// the position is (whole turns fall out at the top), for a handful of integer
// multiplications; its top 32 bits, signed, go to fp32 and to sincospi.
#pragma once

#include <cstdint>

#include "elements.cuh"
#include "ptx.cuh"

namespace hk {
namespace rope {

constexpr int kMaxAxes = 4;

struct RopeParams {
    const void* in[2];             // queries, keys
    void* out[2];
    const void* weight[2];         // [D] each, or null (1)
    int64_t in_b[2], in_t[2], in_h[2];       // strides in elements
    int64_t out_b[2], out_t[2], out_h[2];
    const int32_t* positions;
    int64_t pos_axis, pos_b, pos_t;          // strides of the positions
    const float* inv_freq;         // [half]
    int32_t section_end[kMaxAxes]; // pairs [.., section_end[a]) turn by axis a
    int32_t B, T, heads[2];        // heads of queries and keys
    int32_t D, half;               // R / 2
    int32_t op_steps[2];           // row steps of a token's queries, of its keys
    int32_t steps, shares;         // row steps of a warp; warps of a token
    int64_t warps;
    float eps;
    int32_t norm, weight_f32;
};

// inv_freq / 2 pi as a fraction of 2^64 (whole turns dropped). The largest frequencies lose bits: 2^e costs e of them.
__device__ __forceinline__ uint64_t turns_per_position(float f) {
    const uint32_t bits = __float_as_uint(f);
    const int field = static_cast<int>(bits >> 23 & 255u);
    const uint32_t m = (bits & 0x7FFFFFu) | (field ? 0x800000u : 0u);
    const int shift = 150 - max(field, 1);                  // f = m 2^-shift
    const uint64_t inv_2pi = 0x28BE60DB9391054Aull;         // 2^64 / 2 pi, from the digits of pi
    const uint64_t lo = inv_2pi * m, hi = __umul64hi(inv_2pi, static_cast<uint64_t>(m));
    uint64_t t;
    if (shift <= 0) t = lo << min(-shift, 63);
    else if (shift < 64) t = lo >> shift | hi << (64 - shift);
    else t = shift < 128 ? hi >> (shift - 64) : 0;
    return bits >> 31 ? 0 - t : t;
}

__device__ __forceinline__ void angle(const RopeParams& p, int pair, int64_t at, float& c, float& s) {
    const float f = p.inv_freq[pair];
    int axis = 0;
#pragma unroll
    for (int a = 0; a < kMaxAxes - 1; ++a) axis += pair >= p.section_end[a];
    const int64_t pos = p.positions[axis * p.pos_axis + at];
    const uint64_t turn = turns_per_position(f) * static_cast<uint64_t>(pos);
    const int32_t top = static_cast<int32_t>(turn + 0x80000000ull >> 32);
    sincospif(static_cast<float>(top) * 0x1p-31f, &s, &c);
    if (!isfinite(f)) c = s = NAN;
}

template <typename T>
__device__ __forceinline__ void weights8(const RopeParams& p, int op, int d, float (&w)[8]) {
    if (p.weight[op] == nullptr) {
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = 1.0f;
    } else if (p.weight_f32) {
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = static_cast<const float*>(p.weight[op])[d + k];
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = to_float(static_cast<const T*>(p.weight[op])[d + k]);
    }
}

// Eight elements of a row. kVec: 16 bytes at a time. No test around a load: the next one would wait for it.
template <typename T, bool kVec>
__device__ __forceinline__ Raw8<T> row8(const T* src) {
    Raw8<T> r;
    if constexpr (kVec) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.w[i] = reinterpret_cast<const uint4*>(src)[i];
    } else {
        T e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = src[i];
        memcpy(&r, e, sizeof r);
    }
    return r;
}

template <typename T, bool kVec>
__device__ __forceinline__ void store8(T* dst, const float (&v)[8]) {
    if constexpr (!kVec) {
#pragma unroll
        for (int k = 0; k < 8; ++k) dst[k] = from_float<T>(v[k]);
    } else if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(dst) =
            make_uint4(pack_pair<T>(v[0], v[1]), pack_pair<T>(v[2], v[3]), pack_pair<T>(v[4], v[5]), pack_pair<T>(v[6], v[7]));
    } else {
        reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

// The words of eight elements that another lane holds.
template <typename T>
__device__ __forceinline__ Raw8<T> shuffle8(const Raw8<T>& r, int from) {
    Raw8<T> o;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
        o.w[i] = make_uint4(__shfl_sync(0xffffffffu, r.w[i].x, from), __shfl_sync(0xffffffffu, r.w[i].y, from),
                            __shfl_sync(0xffffffffu, r.w[i].z, from), __shfl_sync(0xffffffffu, r.w[i].w, from));
    return o;
}

template <typename T, int kLanes, bool kInterleaved, bool kVec>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2)
qk_norm_rope_kernel(const RopeParams p) {
    constexpr int kRowsStep = 32 / kLanes;           // rows of a warp at a time
    griddep_launch_dependents();
    griddep_wait();                  // launched early behind the kernel that may have written the queries and keys
    const int64_t warp = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (warp >= p.warps) return;
    const int64_t token = warp / p.shares;
    const int share = static_cast<int>(warp - token * p.shares);
    const int64_t b = token / p.T, t = token - b * p.T;
    const int lane = static_cast<int>(lane_id());
    const int sub = lane % kLanes, d = 8 * sub;
    const bool live = d < p.D;

    // cos and sin of this lane's elements: of its 4 pairs (interleaved), or of the 8 pairs that it is one half of, four
    // of them worked out here and four by the lane that holds the other half
    constexpr int kAngles = kInterleaved ? 4 : 8;
    float c[kAngles], s[kAngles];
    const int64_t at = b * p.pos_b + t * p.pos_t;
    const bool turns = d < 2 * p.half;
    const bool second = !kInterleaved && d >= p.half;
    const int partner = kInterleaved || !turns ? lane : second ? lane - p.half / 8 : lane + p.half / 8;
    {
        const int pair0 = !turns ? 0 : kInterleaved ? d / 2 : second ? d - p.half : d;
        float mc[4], ms[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            mc[k] = 1.0f;
            ms[k] = 0.0f;
            if (turns) angle(p, pair0 + (second ? 4 : 0) + k, at, mc[k], ms[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (kInterleaved) {
                c[k] = mc[k];
                s[k] = ms[k];
            } else {
                const float oc = __shfl_sync(0xffffffffu, mc[k], partner), os = __shfl_sync(0xffffffffu, ms[k], partner);
                c[k] = second ? oc : mc[k];
                c[4 + k] = second ? mc[k] : oc;
                s[k] = second ? os : -ms[k];                 // (the first half's sin with its sign)
                s[4 + k] = second ? ms[k] : -os;
            }
        }
    }
    const float inv_d = 1.0f / static_cast<float>(p.D);
    constexpr int kFlight = sizeof(T) == 2 ? 4 : 2;  // steps whose loads are in flight together
    // steps [first, last) of the token's: its queries', then its keys'
    int first = share * p.steps;
    const int last = min(p.op_steps[0] + p.op_steps[1], first + p.steps);
    while (first < last) {
        const int op = first >= p.op_steps[0];
        const int base = op ? p.op_steps[0] : 0, end = min(last, op ? last : p.op_steps[0]);
        // an output is (x a + o b) / root: x the element, o the one that it is turned with, a and b weight times cos and sin
        uint64_t a2[4], b2[4];
        {
            float w[8];
            weights8<T>(p, op, live ? d : 0, w);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (kInterleaved) {
                    a2[k] = f32x2(w[2 * k] * c[k], w[2 * k + 1] * c[k]);
                    b2[k] = f32x2(-w[2 * k + 1] * s[k], w[2 * k] * s[k]);
                } else {
                    a2[k] = f32x2(w[2 * k] * c[2 * k], w[2 * k + 1] * c[2 * k + 1]);
                    const float o0 = __shfl_sync(0xffffffffu, w[2 * k], partner), o1 = __shfl_sync(0xffffffffu, w[2 * k + 1], partner);
                    b2[k] = f32x2(o0 * s[2 * k], o1 * s[2 * k + 1]);
                }
            }
        }
        const T* const src = static_cast<const T*>(p.in[op]) + b * p.in_b[op] + t * p.in_t[op] + (live ? d : 0);
        T* const dst = static_cast<T*>(p.out[op]) + b * p.out_b[op] + t * p.out_t[op] + d;
        const int64_t in_h = p.in_h[op], out_h = p.out_h[op];
        const int heads = p.heads[op];
        for (int s0 = first; s0 < end; s0 += kFlight) {
            const int r0 = (s0 - base) * kRowsStep + lane / kLanes;
            Raw8<T> raw[kFlight];
#pragma unroll
            for (int i = 0; i < kFlight; ++i)    // (past the end the last row is taken again and not stored)
                raw[i] = row8<T, kVec>(src + min(r0 + min(i, end - 1 - s0) * kRowsStep, heads - 1) * in_h);
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                if (s0 + i >= end) break;
                const int r = r0 + i * kRowsStep;
                float y[8], o[8];
                widen8<T>(raw[i], y);
                uint64_t y2[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) y2[k] = f32x2(y[2 * k], y[2 * k + 1]);
                float mul = 1.0f;
                if (p.norm) {
                    const uint64_t q = ffma2(y2[3], y2[3], ffma2(y2[2], y2[2], ffma2(y2[1], y2[1], fmul2(y2[0], y2[0]))));
                    float lo, hi;
                    f32x2_split(q, lo, hi);
                    float sum = live ? lo + hi : 0.0f;
#pragma unroll
                    for (int m = kLanes / 2; m > 0; m /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, m);
                    mul = rsqrtf(fmaf(sum, inv_d, p.eps));
                }
                if constexpr (kInterleaved) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) o[k] = y[k ^ 1];
                } else {
                    widen8<T>(shuffle8<T>(raw[i], partner), o);
                }
                float z[8];
                const uint64_t mul2 = f32x2(mul, mul);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint64_t x = fmul2(y2[k], a2[k]), turned = ffma2(f32x2(o[2 * k], o[2 * k + 1]), b2[k], x);
                    f32x2_split(fmul2(turns ? turned : x, mul2), z[2 * k], z[2 * k + 1]);      // (not plus 0 times an infinity)
                }
                if (r < heads && live) store8<T, kVec>(dst + r * out_h, z);
            }
        }
        first = end;
    }
}

}  // namespace rope
}  // namespace hk
