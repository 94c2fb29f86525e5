// The norm of each head's query and key and the rotation by the token's position, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w          (per head; left out without eps)
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t),   t_i = position[axis(i)] * inv_freq[i]
//
// over the pairs (a, b) = (y_i, y_{i + R/2}) or (y_{2i}, y_{2i+1}) of the first R of D elements.
//
// Every element is read once and written once: what bounds it is memory. A row
// (one head of one token) is 8 elements each of 8, 16 or 32 lanes, four of each half of
// the pairs, so that a pair is one lane's and a warp's load is whole lines; a warp keeps to one token and takes `steps` times
// 32 / lanes rows of its queries or keys, so that the angles are worked out once for all of them:
// as few as leave every SM full of warps (a decoding step), up to all heads (a
// prompt).
//
// Angles. A position times a frequency loses its fraction of a turn in 32 bits
// (position 10^6: an error of 0.06 radians). Here the frequency is taken as the
// turns per position, inv_freq / 2 pi, in fixed point with 64 bits behind the
// point: 24 bits of mantissa times a 64-bit 1 / 2 pi, shifted. Times the
// position modulo 2^64 that is the fraction of a turn to within 2^-32.4 whatever
// the position is (for frequencies up to 1; whole turns fall out at the top), for a handful of integer
// multiplications; its top 32 bits, signed, go to fp32, which rounds them by up to 2^-26 of a turn, and to sincospi.
//
// Measured: 16384 tokens of 72 heads of 128 in bf16 106 us, 5.7 TB/s read and written, 0.84 of a copy's rate (half the issue slots
// are taken; a test at each load, which made the loads wait for one another, took 256 us, 64-bit divisions to find rows 135, clamped
// row numbers instead of whole steps first and a rest 122); 5003 of 48 heads in fp16 28 us; 64 of 72 heads 5 us, a launch and
// two trips to memory.
#pragma once

#include <cstdint>
#include <type_traits>

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
    int32_t steps;                 // row steps of a warp
    uint32_t shares, warps;        // warps of a token, of all
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

// Four consecutive elements of bf16, fp16 or fp32.
template <typename T>
struct Raw4 {
    uint32_t w[sizeof(T)];
};

// kVec: in one access. No test around a load: the next one would wait for it.
template <typename T, bool kVec>
__device__ __forceinline__ Raw4<T> load4(const T* src) {
    Raw4<T> r;
    if constexpr (!kVec) {
        T e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = src[i];
        memcpy(&r, e, sizeof r);
    } else if constexpr (sizeof(T) == 2) {
        const uint2 x = *reinterpret_cast<const uint2*>(src);
        r.w[0] = x.x; r.w[1] = x.y;
    } else {
        const uint4 x = *reinterpret_cast<const uint4*>(src);
        r.w[0] = x.x; r.w[1] = x.y; r.w[2] = x.z; r.w[3] = x.w;
    }
    return r;
}

template <typename T, bool kVec>
__device__ __forceinline__ void store4(T* dst, const float (&v)[4]) {
    if constexpr (!kVec) {
#pragma unroll
        for (int k = 0; k < 4; ++k) dst[k] = from_float<T>(v[k]);
    } else if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_pair<T>(v[0], v[1]), pack_pair<T>(v[2], v[3]));
    } else {
        *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
    }
}

// As two pairs.
template <typename T>
__device__ __forceinline__ void pairs_of(const Raw4<T>& r, uint64_t (&v)[2]) {
    T e[4];
    memcpy(e, &r, sizeof r);
    v[0] = f32x2(to_float(e[0]), to_float(e[1]));
    v[1] = f32x2(to_float(e[2]), to_float(e[3]));
}

template <typename T>
__device__ __forceinline__ void weights4(const RopeParams& p, int op, int e, float* w) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
        w[k] = p.weight[op] == nullptr ? 1.0f
               : p.weight_f32          ? static_cast<const float*>(p.weight[op])[e + k]
                                       : to_float(static_cast<const T*>(p.weight[op])[e + k]);
}

__device__ __forceinline__ uint64_t swap_pair(uint64_t x) {
    float lo, hi;
    f32x2_split(x, lo, hi);
    return f32x2(hi, lo);
}

template <typename T, int kLanes, bool kInterleaved, bool kVec>
__global__ void __launch_bounds__(256, 3)
qk_norm_rope_kernel(const RopeParams p) {
    constexpr int kRowsStep = 32 / kLanes;           // rows of a warp at a time
    constexpr int kFlight = sizeof(T) == 2 ? 4 : 2;  // steps whose loads are in flight together
    griddep_launch_dependents();
    griddep_wait();                  // launched early behind the kernel that may have written the queries and keys
    const uint32_t warp = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (warp >= p.warps) return;
    const uint32_t token = warp / p.shares;
    const int share = static_cast<int>(warp - token * p.shares);
    const int64_t b = token / static_cast<uint32_t>(p.T), t = token - static_cast<uint32_t>(b) * p.T;
    const int lane = static_cast<int>(lane_id());
    const int sub = lane % kLanes, my_row = lane / kLanes;
    // This lane's elements: four from e0 and four from e1 on. Those of both halves of four pairs (or four whole pairs), for the
    // pairs that turn; then what does not turn, eight in a row.
    const int turning = p.half / 4;                  // lanes that turn pairs
    const bool turns = sub < turning, live = 8 * sub < p.D;
    const int e0 = !live ? 0 : kInterleaved || !turns ? 8 * sub : 4 * sub;
    const int e1 = !live ? 0 : kInterleaved || !turns ? 8 * sub + 4 : 4 * sub + p.half;
    // steps [first, last) of the token's: its queries', then its keys'
    int first = share * p.steps;
    const int last = min(p.op_steps[0] + p.op_steps[1], first + p.steps);

    float c[4], s[4];                // cos and sin of the four pairs
    {
        const int64_t at = b * p.pos_b + t * p.pos_t;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            c[k] = 1.0f;
            s[k] = 0.0f;
            if (turns) angle(p, 4 * sub + k, at, c[k], s[k]);
        }
    }
    const float inv_d = 1.0f / static_cast<float>(p.D);
    while (first < last) {
        const int op = first >= p.op_steps[0];
        const int base = op ? p.op_steps[0] : 0, end = min(last, op ? last : p.op_steps[0]);
        // an output is (x a + o b) / root: x the element, o the one that it is turned with, a and b weight times cos and sin
        uint64_t a2[4], b2[4];       // of e0's two pairs of elements, of e1's
        {
            float w[8];
            weights4<T>(p, op, e0, w);
            weights4<T>(p, op, e1, w + 4);
            if constexpr (kInterleaved) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    a2[k] = f32x2(w[2 * k] * c[k], w[2 * k + 1] * c[k]);
                    b2[k] = f32x2(-w[2 * k + 1] * s[k], w[2 * k] * s[k]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int i = 2 * k, j = 2 * k + 1;
                    a2[k] = f32x2(w[i] * c[i], w[j] * c[j]);
                    a2[2 + k] = f32x2(w[4 + i] * c[i], w[4 + j] * c[j]);
                    b2[k] = f32x2(-w[4 + i] * s[i], -w[4 + j] * s[j]);
                    b2[2 + k] = f32x2(w[i] * s[i], w[j] * s[j]);
                }
            }
        }
        const int heads = p.heads[op];
        const int64_t in_step = kRowsStep * p.in_h[op], out_step = kRowsStep * p.out_h[op];
        int row = (first - base) * kRowsStep + my_row;
        const T* const rows = static_cast<const T*>(p.in[op]) + b * p.in_b[op] + t * p.in_t[op];
        const T* src = rows + row * p.in_h[op];          // (not read where it is none of the rows)
        T* dst = static_cast<T*>(p.out[op]) + b * p.out_b[op] + t * p.out_t[op] + row * p.out_h[op];
        // kFlight steps from s0 on; `whole`: all of them are there, and their rows
        auto steps = [&](int s0, auto whole) {
            constexpr bool kWhole = decltype(whole)::value;
            Raw4<T> raw[kFlight][2];
            const T* at = kWhole ? src : rows + min(row, heads - 1) * p.in_h[op];
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {      // (past the end a row is taken again and not stored)
                raw[i][0] = load4<T, kVec>(at + e0);
                raw[i][1] = load4<T, kVec>(at + e1);
                if (kWhole || row + (i + 1) * kRowsStep < heads) at += in_step;
            }
            src += kFlight * in_step;
#pragma unroll
            for (int i = 0; i < kFlight; ++i) {
                if (!kWhole && s0 + i >= end) break;
                uint64_t y[4];
                pairs_of<T>(raw[i][0], *reinterpret_cast<uint64_t(*)[2]>(&y[0]));
                pairs_of<T>(raw[i][1], *reinterpret_cast<uint64_t(*)[2]>(&y[2]));
                uint64_t mul2 = f32x2(1.0f, 1.0f);
                if (p.norm) {
                    const uint64_t q = ffma2(y[3], y[3], ffma2(y[2], y[2], ffma2(y[1], y[1], fmul2(y[0], y[0]))));
                    float lo, hi;
                    f32x2_split(q, lo, hi);
                    float sum = live ? lo + hi : 0.0f;
#pragma unroll
                    for (int m = kLanes / 2; m > 0; m /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, m);
                    const float mul = rsqrtf(fmaf(sum, inv_d, p.eps));
                    mul2 = f32x2(mul, mul);
                }
                uint64_t z[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) z[k] = fmul2(y[k], a2[k]);
                if (turns) {                     // (not plus 0 times an infinity)
#pragma unroll
                    for (int k = 0; k < 4; ++k) z[k] = ffma2(kInterleaved ? swap_pair(y[k]) : y[k ^ 2], b2[k], z[k]);
                }
                float out[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) f32x2_split(fmul2(z[k], mul2), out[2 * k], out[2 * k + 1]);
                if (live && (kWhole || row < heads)) {
                    store4<T, kVec>(dst + e0, *reinterpret_cast<const float(*)[4]>(&out[0]));
                    store4<T, kVec>(dst + e1, *reinterpret_cast<const float(*)[4]>(&out[4]));
                }
                row += kRowsStep;
                dst += out_step;
            }
        };
        const int whole = base + heads / kRowsStep;      // steps up to there have all their rows
        int s0 = first;
        for (; s0 + kFlight <= min(end, whole); s0 += kFlight) steps(s0, std::integral_constant<bool, true>{});
        for (; s0 < end; s0 += kFlight) steps(s0, std::integral_constant<bool, false>{});
        first = end;
    }
}

}  // namespace rope
}  // namespace hk
