// token_place.cuh -- where a token of a ragged batch lives in the cache.
#pragma once

#include <cstdint>

#include "pa_internal.h"

namespace pa {

enum class Place { kOk, kPadding, kOutOfRange };

// Token `tok` of the ragged batch with running offsets `cu` [batch + 1] is
// logical position start_pos[b] + (tok - cu[b]) of its sequence b: row
// pos % 64 of page block_table[b, pos / 64].  Tokens past cu[batch] are
// padding and belong to no sequence.
__device__ __forceinline__ Place token_place(int tok, const int32_t* __restrict__ cu,
                                             const int32_t* __restrict__ start_pos,
                                             const int32_t* __restrict__ block_table, int batch, int max_pages,
                                             int num_pool_pages, int& page, int& row, long long& pos) {
    int lo = 0, hi = batch;  // last b in [0, batch] with cu[b] <= tok
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(&cu[mid]) <= tok) lo = mid;
        else hi = mid - 1;
    }
    if (lo >= batch) return Place::kPadding;
    const int into = tok - __ldg(&cu[lo]);
    if (into < 0) return Place::kPadding;  // before the first sequence
    pos = (long long)__ldg(&start_pos[lo]) + into;
    if (pos < 0 || pos / kPage >= max_pages) return Place::kOutOfRange;
    page = __ldg(&block_table[(long long)lo * max_pages + pos / kPage]);
    row = (int)(pos % kPage);
    return (unsigned)page < (unsigned)num_pool_pages ? Place::kOk : Place::kOutOfRange;
}

}  // namespace pa
