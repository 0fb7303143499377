// What the steps around a projection (pq2_norm.cu, pq2_lora.cu, pq2_verify.cu)
// share beyond pq2_common.cuh.
#pragma once

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
