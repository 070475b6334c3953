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

// The attention kernel takes (sequence, 256-row block) pairs with the most
// key tiles first, so that the last ones to finish are short.  A block's
// number within its sequence orders them (window and core rows only grow
// with it): block `blk` of sequence s comes after every block of a higher
// number and after the same block of the sequences before s.  A thread for
// each pair counts those before it; the pairs are found from the offsets
// alone, at cu[s] / 256 + s + blk (a sequence of n rows has at most
// cu[s + 1] / 256 - cu[s] / 256 + 1 blocks, so no two pairs meet; places
// that hold none are skipped).
struct PackedPair {
    int s, blk;  // blk < 0: none
};

__device__ __forceinline__ int packed_blocks(const int *scu, int s)
{
    return (scu[s + 1] - scu[s] + 255) >> 8;
}

__device__ __forceinline__ PackedPair packed_pair(const int *scu, int S, int64_t i)
{
    int lo = 0, hi = S - 1;  // the last sequence whose first place is not behind i
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((scu[mid] >> 8) + static_cast<int64_t>(mid) <= i)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int64_t blk = i - ((scu[lo] >> 8) + static_cast<int64_t>(lo));
    return {lo, blk >= 0 && blk < packed_blocks(scu, lo) ? static_cast<int>(blk) : -1};
}

__device__ __forceinline__ int packed_place(const int *scu, int S, PackedPair p)
{
    int place = 0;
    for (int s = 0; s < S; ++s) {
        const int n = packed_blocks(scu, s);
        place += max(0, n - p.blk - 1) + (s < p.s && n > p.blk ? 1 : 0);
    }
    return place;
}

}  // namespace cca
