// bl_wait.cuh -- bounded waits of kernels whose loops run to their end whether or not a wait was given
// up (the 8-bit products, the norm's backward), and the waits for what is in flight then.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "bl_device.cuh"

namespace bl {

// As mbar_wait_bounded, but looks at the abort flag before it waits: after a wait was given up the
// ones that follow cost a poll each, not a suspension.
template <typename Limit>
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort, Limit limit_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    const unsigned long long t0 = globaltimer_ns();
    for (;;) {
        if (mbar_try_wait_sleep(bar, parity, kSuspendHintNs)) return true;
        if (*abort) return false;
        if (globaltimer_ns() - t0 > limit_ns()) {
            *abort = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort,
                                        unsigned long long limit_ns) {
    return wait_on(bar, parity, abort, [limit_ns] { return limit_ns; });
}

// Wait for what is in flight after a wait was given up: the abort flag does not end this one.
constexpr unsigned long long kDrainNs = 200000000ull;  // 0.2 s
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
    const unsigned long long t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (globaltimer_ns() - t0 > kDrainNs) return;
    }
}
// Of `issued` loads that went round `stages` stages in turn, the ones into stage s.
__device__ __forceinline__ int fills_of(int issued, int stages, int s) { return (issued - s + stages - 1) / stages; }

}  // namespace bl
