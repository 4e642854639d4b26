// kv_index.cuh -- index arithmetic of the cache operators at the ends of its
// range. Plain C++ as well, so that it is tested without a GPU.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define UZKV_INDEX __host__ __device__ __forceinline__
#else
#define UZKV_INDEX inline
#endif

namespace uzkv {

// The index `step` on from i < total, or total where that is past the end: i + step itself may not fit 32 bits.
UZKV_INDEX uint32_t next_below(uint32_t i, uint32_t step, uint32_t total) { return total - i <= step ? total : i + step; }

// x / d, by the 32-bit division where both fit.
UZKV_INDEX uint64_t divide(uint64_t x, uint64_t d) {
    return (x | d) >> 32 ? x / d : (uint64_t)((uint32_t)x / (uint32_t)d);
}

// Of `shares` equal runs of `total` positions, share c from total * c / shares (rounded down) on: the one that has
// position `at`. No share is empty: shares <= total.
UZKV_INDEX uint32_t share_of(uint64_t at, uint64_t shares, uint64_t total) {
    return (uint32_t)divide((at + 1) * shares - 1, total);
}

}  // namespace uzkv
