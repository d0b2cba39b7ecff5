// token_place.cuh -- where a token of a ragged batch lives in the cache.
#pragma once

#include <cstdint>

#include "pa_internal.h"

namespace pa {

enum class Place { kOk, kPadding, kOutOfRange };

// The sequence that holds token `tok` (the same for the whole warp) of a
// ragged batch with running offsets `cu` [batch + 1]: the last b with
// cu[b] <= tok; batch for the padding behind the last sequence, -1 before the
// first.  32 offsets are looked at per step: up to 31 sequences take one load.
__device__ __forceinline__ int warp_sequence(int tok, const int32_t* __restrict__ cu, int batch) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = batch + 1;  // candidates lo .. lo + n - 1
    while (true) {
        const int stride = (n + 31) >> 5;
        const int i = lane * stride;
        const unsigned below = __ballot_sync(0xffffffffu, i < n && __ldg(&cu[lo + i]) <= tok);
        const int count = __popc(below);  // a run from lane 0 on
        if (count == 0) return -1;        // (only in the first step)
        lo += (count - 1) * stride;
        n = min(stride, n - (count - 1) * stride);
        if (stride == 1) return lo;
    }
}

// Where token `tok` of sequence b lives: logical position
// start_pos[b] + (tok - cu[b]) is row pos % 64 of page block_table[b, pos / 64].
__device__ __forceinline__ Place token_place(int tok, int b, const int32_t* __restrict__ cu,
                                             const int32_t* __restrict__ start_pos,
                                             const int32_t* __restrict__ block_table, int batch, int max_pages,
                                             int num_pool_pages, int& page, int& row, long long& pos) {
    if (b < 0 || b >= batch) return Place::kPadding;
    pos = (long long)__ldg(&start_pos[b]) + (tok - __ldg(&cu[b]));
    if (pos < 0 || pos / kPage >= max_pages) return Place::kOutOfRange;
    page = __ldg(&block_table[(long long)b * max_pages + pos / kPage]);
    row = (int)(pos % kPage);
    return (unsigned)page < (unsigned)num_pool_pages ? Place::kOk : Place::kOutOfRange;
}

}  // namespace pa
