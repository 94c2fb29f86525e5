// Bounded mbarrier waits of the kernels that are not the bf16 / FP8 GEMM or
// the attention forward over contiguous K and V (those keep their own, tuned
// to their loops). A wait that runs out records an error in the device status
// word and aborts the launch: every other role sees that and gives up too.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace hk {

constexpr uint32_t kErrWaitRing = 1u << 16;      // a producer waited for a free ring slot
constexpr uint32_t kErrWaitData = 1u << 17;      // a consumer waited for loaded data
constexpr uint32_t kErrWaitAcc = 1u << 18;       // an accumulator's hand-over
constexpr uint32_t kErrPage = 1u << 24;          // a page index or length of a paged cache is out of range

struct WaitCtx {
    uint32_t* status;       // [0]: error bits (sticky), [1]: launch id that aborted
    uint32_t launch_id;
    uint64_t timeout_ns;
};

__device__ __forceinline__ bool wait_aborted(WaitCtx c) {
    return *reinterpret_cast<volatile uint32_t*>(c.status + 1) == c.launch_id;
}

static __device__ __noinline__ bool wait_mbar_slow(WaitCtx c, uint32_t bar, uint32_t parity, uint32_t code) {
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        if (mbar_try_wait_suspend(bar, parity, 20000)) return true;
        if (wait_aborted(c)) return false;
        if (global_timer_ns() - t0 > c.timeout_ns) {
            atomicOr(c.status, code);
            atomicExch(c.status + 1, c.launch_id);
            __threadfence();
            return false;
        }
    }
}

// Waits for phase `parity` of `bar`; false when the wait gave up.
__device__ __forceinline__ bool wait_mbar(WaitCtx c, uint32_t bar, uint32_t parity, uint32_t code) {
    for (int i = 0; i < 4; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return wait_mbar_slow(c, bar, parity, code);
}

// The same for a wait on a pipeline's critical path: polls without suspending
// (a suspended wait was measured to resume several hundred cycles after its
// phase completed). The clock is read every 4096 probes.
__device__ __forceinline__ bool wait_mbar_poll(WaitCtx c, uint32_t bar, uint32_t parity, uint32_t code) {
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
        if (mbar_test_wait(bar, parity)) return true;
        if ((it & 4095u) == 0) {
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            else if (now - t0 >= 20000) return wait_mbar_slow(c, bar, parity, code);
        }
    }
}

// For barriers that the peer CTA's threads arrive on with
// mbar_arrive_cluster_relaxed (they order tcgen05 operations only).
static __device__ __noinline__ bool wait_mbar_cluster_slow(WaitCtx c, uint32_t bar, uint32_t parity, uint32_t code) {
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait_cluster_relaxed(bar, parity)) return true;
        if ((it & 63u) == 0) {
            if (wait_aborted(c)) return false;
            if (global_timer_ns() - t0 > c.timeout_ns) {
                atomicOr(c.status, code);
                atomicExch(c.status + 1, c.launch_id);
                __threadfence();
                return false;
            }
        }
    }
}

__device__ __forceinline__ bool wait_mbar_cluster(WaitCtx c, uint32_t bar, uint32_t parity, uint32_t code) {
    if (mbar_try_wait_cluster_relaxed(bar, parity)) return true;
    return wait_mbar_cluster_slow(c, bar, parity, code);
}

// A wait on the abort path (a copy or MMA that was issued signals `bar` when
// it completes); gives up after 2 ms.
__device__ __forceinline__ void wait_mbar_drain(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity))
        if (global_timer_ns() - t0 > 2000000) return;
}

}  // namespace hk
