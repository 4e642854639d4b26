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

}  // namespace uzkv
