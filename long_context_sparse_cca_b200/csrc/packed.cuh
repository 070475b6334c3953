// Offsets of packed sequences on the device: loading them into shared
// memory with their check, and finding a row's sequence.
#pragma once

#include "common.cuh"

namespace cca {

// cu [S + 1] into scu, by the whole block; false (on every thread) unless
// 0 <= cu[0], ascending, cu[S] <= total.
__device__ __forceinline__ bool load_offsets(const int *cu, int S, int64_t total, int *scu)
{
    for (int i = threadIdx.x; i <= S; i += blockDim.x) scu[i] = cu[i];
    __syncthreads();
    bool bad = false;
    for (int i = threadIdx.x; i <= S; i += blockDim.x)
        bad |= scu[i] < 0 || scu[i] > total || (i > 0 && scu[i] < scu[i - 1]);
    return __syncthreads_or(bad) == 0;
}

// The last sequence that starts at or before row t (0 if none does).
__device__ __forceinline__ int row_sequence(const int *scu, int S, int64_t t)
{
    int lo = 0, hi = S - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (scu[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// The last sequence whose first core row cu[s] / g is at or before row c.
__device__ __forceinline__ int core_row_sequence(const int *scu, int S, int g, int c)
{
    return row_sequence(scu, S, static_cast<int64_t>(c) * g + g - 1);
}

}  // namespace cca
