// paging.cuh -- device helpers shared by the kernels that walk a batch of
// sequences over the paged caches.
#pragma once
#include <cstdint>

#include "common.h"

namespace dsa {

// Sequence of query token t, or -1 when t lies behind the last sequence (rows
// of a padded batch).  Sequences without new tokens are passed over: the last
// b with cu_q[b] <= t < cu_q[B] has cu_q[b + 1] > t.
__device__ __forceinline__ int query_sequence(const int32_t* cu_q, int B, int t) {
    if (t < 0 || t >= __ldg(cu_q + B)) return -1;
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(cu_q + mid) <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Cache row of position pos of sequence b through its block table, or -1 when
// the position or its page id is out of range.
__device__ __forceinline__ int64_t cache_row(const int32_t* block_table, int max_blocks, int num_blocks, int b,
                                             int64_t pos) {
    if (pos < 0 || pos / kPage >= max_blocks) return -1;
    const int blk = __ldg(block_table + (int64_t)b * max_blocks + pos / kPage);
    return blk >= 0 && blk < num_blocks ? (int64_t)blk * kPage + pos % kPage : -1;
}

}  // namespace dsa
