// What the steps around a projection (pq2_norm.cu, pq2_lora.cu, pq2_verify.cu)
// share beyond pq2_common.cuh.
#pragma once

#include <mutex>

#include "pq2_common.cuh"

namespace pq2 {

// Bit of the device error word (beside DEVERR_* of pq2_common.cuh): an index
// array held a value outside its range.
constexpr unsigned DEVERR_BAD_INDEX = 8u;

// mbar_wait_warp for phases that are mostly complete when asked for: all lanes
// try at once and agree by a vote, and only if that fails lane 0 polls (its
// branch and the shuffle after it take about 300 cycles in a short loop).
__device__ __forceinline__ bool mbar_ready_warp(uint64_t* bar, uint32_t parity, const DevCtl& ctl,
                                                volatile int* abort_flag = nullptr) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return mbar_wait_warp(bar, parity, ctl, abort_flag);
}

}  // namespace pq2

namespace pq2h {

// ensure_smem for kernels whose size changes from call to call, from any number
// of host threads: of two that raise one kernel's limit at once, the smaller
// could set it last, below what is noted down (later launches would then fail).
template <typename Kern>
cudaError_t raise_smem(SmemLimit& lim, Kern kern, size_t smem) {
    int dev = -1;
    if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kSmemLimitDevices &&
        lim.bytes[dev].load(std::memory_order_acquire) >= static_cast<int>(smem))
        return cudaSuccess;
    static std::mutex one_at_a_time;
    std::lock_guard<std::mutex> hold(one_at_a_time);
    return ensure_smem(lim, kern, smem);   // asks again
}

}  // namespace pq2h
