// A cache of keys and values in 4 bits, in pages: its layout, and where a
// call's token rows stand in it.  See include/pq2.h for the format.
#pragma once

#include <climits>

#include "pq2_common.cuh"
#include "pq2_internal.h"
#include "pq2_step.cuh"

namespace pq2 {

constexpr int kTileTokens = 16;  // tokens of a tile

// Byte offsets within a tile of 16 tokens of one head.
__host__ __device__ constexpr int tile_bytes(int D) { return kTileTokens * (D + 8); }
__host__ __device__ constexpr int tile_codes(int D, int value) {  // value: 0 keys, 1 values
    return value * kTileTokens * D / 2;
}
__host__ __device__ constexpr int tile_pairs(int D, int value) {
    return kTileTokens * D + value * kTileTokens * 4;
}

// The sequence whose rows include `row` (all lanes of a warp ask for the same
// one): a search over row_start, 32 places at a time.  -1: none.
__device__ __forceinline__ int seq_of_row(const int32_t* start, int B, int row, int& end) {
    const int lane = threadIdx.x & 31;
    int lo = 0, size = B;
    for (;;) {
        const int step = (size + 31) >> 5;
        const int at = lane * step;
        const int v = at < size ? __ldcg(start + lo + at) : INT_MAX;
        const int n = __popc(__ballot_sync(0xffffffffu, v <= row));
        if (n == 0) return -1;
        lo += (n - 1) * step;
        size = min(step, size - (n - 1) * step);
        if (step == 1) break;
    }
    end = __ldcg(start + lo + 1);
    return row < end ? lo : -1;
}

}  // namespace pq2
