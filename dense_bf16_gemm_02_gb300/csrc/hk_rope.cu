// Host side of hk_qk_norm_rope (include/hk_gemm.h): argument checks and the launch.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>

#include "../../include/hk_gemm.h"
#include "host_internal.h"
#include "qk_rope.cuh"

namespace {

using namespace hk::rope;

hk_status fail(hk_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
hk_status fail(hk_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return hk_host::set_error(s, buf);
}

constexpr int64_t kLimit = (int64_t(1) << 31) - 1;
constexpr int kSms = 152;
constexpr int64_t kMaxHeads = 65535;
constexpr int64_t kWarpsPerSm = 24;      // warps that an SM holds
// A warp's angles, in steps of its rows. Counted as nothing, as 8 steps, as more than anything (a warp to a token): 500 tokens
// of 72 heads of 128 in bf16 take 19.0, 7.6, 7.7 us, 2000 tokens 24.5, 19.4, 21.6, 5003 of 48 heads 40.3, 29.6, 30.0.
constexpr int kAngleSteps = 8;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// One operand's rows, in and out: pointers, strides, alignment.
hk_status check_operand(const void* in, const int64_t in_s[3], const void* out, const int64_t out_s[3], int64_t B, int64_t T,
                        int64_t H, int64_t D, int size, bool* vec) {
    if (H == 0) return HK_OK;
    if (!in || !out || !in_s || !out_s) return fail(HK_ERR_INVALID_ARG, "null queries, keys, outputs or strides");
    if (!aligned(in, size) || !aligned(out, size)) return fail(HK_ERR_MISALIGNED, "a pointer is not aligned to its elements");
    const int64_t sizes[3] = {B, T, H};
    bool same = in == out;
    for (int i = 0; i < 3; ++i) {
        if (sizes[i] > 1 && std::llabs(out_s[i]) < D) return fail(HK_ERR_INVALID_ARG, "the output's rows overlap");
        if (sizes[i] > 1 && in_s[i] != out_s[i]) same = false;
        if (sizes[i] > 1 && ((in_s[i] * size) % 16 || (out_s[i] * size) % 16)) *vec = false;
    }
    if (in == out && !same) return fail(HK_ERR_INVALID_ARG, "an output over its input must have the input's strides");
    if (!aligned(in, 16) || !aligned(out, 16)) *vec = false;
    return HK_OK;
}

template <typename T, int kLanes>
cudaError_t launch(const RopeParams& p, bool interleaved, bool vec, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>((p.warps + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto* fn = interleaved ? (vec ? &qk_norm_rope_kernel<T, kLanes, true, true> : &qk_norm_rope_kernel<T, kLanes, true, false>)
                           : (vec ? &qk_norm_rope_kernel<T, kLanes, false, true> : &qk_norm_rope_kernel<T, kLanes, false, false>);
    return cudaLaunchKernelEx(&cfg, fn, p);
}

template <typename T>
cudaError_t launch(const RopeParams& p, int lanes, bool interleaved, bool vec, cudaStream_t st) {
    return lanes == 8    ? launch<T, 8>(p, interleaved, vec, st)
           : lanes == 16 ? launch<T, 16>(p, interleaved, vec, st)
                         : launch<T, 32>(p, interleaved, vec, st);
}

}  // namespace

extern "C" hk_status hk_qk_norm_rope(const void* Q, const int64_t q_strides[3], const void* K, const int64_t k_strides[3],
                                     void* QO, const int64_t qo_strides[3], void* KO, const int64_t ko_strides[3], int32_t type,
                                     int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t D, const void* q_weight,
                                     const void* k_weight, int32_t weight_type, float eps, const int32_t* positions,
                                     const int64_t pos_strides[3], const int32_t* sections, int32_t axes, const float* inv_freq,
                                     int64_t pairs, int32_t interleaved, void* stream) {
    if (type < HK_TYPE_BF16 || type > HK_TYPE_FP32) return fail(HK_ERR_INVALID_ARG, "unknown element type %d", (int)type);
    if (weight_type != type && weight_type != HK_TYPE_FP32)
        return fail(HK_ERR_INVALID_ARG, "weights of type %d (the elements' type or fp32)", (int)weight_type);
    if (B < 0 || T < 0 || Hq < 0 || Hk < 0 || B > kLimit || T > kLimit || Hq > kMaxHeads || Hk > kMaxHeads)
        return fail(HK_ERR_INVALID_ARG, "invalid size");
    if (D < 8 || D > 256 || D % 8) return fail(HK_ERR_INVALID_ARG, "head dimension %lld (multiples of 8 up to 256)", (long long)D);
    if (pairs < 0 || 2 * pairs > D || pairs % 8)
        return fail(HK_ERR_INVALID_ARG, "%lld pairs to turn (multiples of 8, at most half the head dimension)", (long long)pairs);
    if (std::isnan(eps) || std::isinf(eps)) return fail(HK_ERR_INVALID_ARG, "eps must be finite");
    if (axes < 1 || axes > kMaxAxes) return fail(HK_ERR_INVALID_ARG, "%d position axes (1 to %d)", (int)axes, kMaxAxes);
    RopeParams p = {};
    int64_t sum = 0;             // (a section is below 2^31 and there are four)
    for (int a = 0; a < kMaxAxes; ++a) {
        if (a < axes && sections) {
            if (sections[a] < 0) return fail(HK_ERR_INVALID_ARG, "a section of %d pairs", (int)sections[a]);
            sum += sections[a];
        } else if (a < axes) {
            if (axes > 1) return fail(HK_ERR_INVALID_ARG, "several axes need their sections");
            sum = pairs;
        }
        p.section_end[a] = static_cast<int32_t>(a < axes - 1 ? std::min(sum, pairs) : pairs);       // (the last axis has the rest)
    }
    if (sum != pairs) return fail(HK_ERR_INVALID_ARG, "the sections do not add up to the %lld pairs", (long long)pairs);
    if (B == 0 || T == 0 || Hq + Hk == 0) return HK_OK;
    if (B > (int64_t(1) << 40) / T) return fail(HK_ERR_INVALID_ARG, "problem too large");
    const int size = type == HK_TYPE_FP32 ? 4 : 2, wsize = weight_type == HK_TYPE_FP32 ? 4 : 2;
    bool vec = true;
    hk_status s = check_operand(Q, q_strides, QO, qo_strides, B, T, Hq, D, size, &vec);
    if (s == HK_OK) s = check_operand(K, k_strides, KO, ko_strides, B, T, Hk, D, size, &vec);
    if (s != HK_OK) return s;
    if (pairs > 0) {
        if (!positions || !pos_strides || !inv_freq) return fail(HK_ERR_INVALID_ARG, "null positions, strides or frequencies");
        if (!aligned(positions, 4) || !aligned(inv_freq, 4)) return fail(HK_ERR_MISALIGNED, "positions and frequencies must be 4-byte aligned");
    }
    if (!aligned(q_weight, wsize) || !aligned(k_weight, wsize)) return fail(HK_ERR_MISALIGNED, "a weight is not aligned to its elements");

    p.in[0] = Hq ? Q : K;            // (an operand without heads is never read)
    p.in[1] = K;
    p.out[0] = QO;
    p.out[1] = KO;
    p.norm = eps >= 0.0f;
    p.weight[0] = p.norm ? q_weight : nullptr;       // (the weights are the norm's)
    p.weight[1] = p.norm ? k_weight : nullptr;
    const int64_t* strides[4] = {q_strides, k_strides, qo_strides, ko_strides};
    for (int op = 0; op < 2; ++op) {
        if ((op ? Hk : Hq) == 0) continue;
        p.in_b[op] = strides[op][0];
        p.in_t[op] = strides[op][1];
        p.in_h[op] = strides[op][2];
        p.out_b[op] = strides[2 + op][0];
        p.out_t[op] = strides[2 + op][1];
        p.out_h[op] = strides[2 + op][2];
    }
    p.positions = positions;
    if (pairs > 0) {
        p.pos_axis = pos_strides[0];
        p.pos_b = pos_strides[1];
        p.pos_t = pos_strides[2];
    }
    p.inv_freq = inv_freq;
    p.B = static_cast<int32_t>(B);
    p.T = static_cast<int32_t>(T);
    p.heads[0] = static_cast<int32_t>(Hq);
    p.heads[1] = static_cast<int32_t>(Hk);
    p.D = static_cast<int32_t>(D);
    p.half = static_cast<int32_t>(pairs);
    p.eps = eps;
    p.weight_f32 = weight_type == HK_TYPE_FP32;
    const int lanes = D <= 64 ? 8 : D <= 128 ? 16 : 32;
    for (int op = 0; op < 2; ++op) p.op_steps[op] = (p.heads[op] + 32 / lanes - 1) / (32 / lanes);
    const int64_t token_steps = int64_t(p.op_steps[0]) + p.op_steps[1];
    // warps to a token: those whose rounds over the GPU take the least time, a warp's being its row steps and its angles
    int64_t shares = 1, least = INT64_MAX;
    for (int64_t rounds = 1; rounds <= 8; ++rounds) {
        const int64_t s = std::max<int64_t>(1, std::min(token_steps, rounds * kSms * kWarpsPerSm / (B * T)));
        const int64_t steps = (token_steps + s - 1) / s, warps = B * T * ((token_steps + steps - 1) / steps);
        const int64_t time = (warps + kSms * kWarpsPerSm - 1) / (kSms * kWarpsPerSm) * (steps + kAngleSteps);
        if (time < least) {
            least = time;
            shares = (token_steps + steps - 1) / steps;
        }
    }
    p.steps = static_cast<int32_t>((token_steps + shares - 1) / shares);
    if (B * T > kLimit / shares) return fail(HK_ERR_INVALID_ARG, "problem too large");
    p.shares = static_cast<uint32_t>(shares);
    p.warps = static_cast<uint32_t>(B * T * shares);
    int device = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return fail(HK_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
    if ((s = hk_host::check_device(device, &sms)) != HK_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (type) {
        case HK_TYPE_BF16: e = launch<__nv_bfloat16>(p, lanes, interleaved != 0, vec, st); break;
        case HK_TYPE_FP16: e = launch<__half>(p, lanes, interleaved != 0, vec, st); break;
        default: e = launch<float>(p, lanes, interleaved != 0, vec, st); break;
    }
    return e == cudaSuccess ? HK_OK : fail(HK_ERR_LAUNCH, "launching the head norm and rotation: %s", cudaGetErrorString(e));
}
