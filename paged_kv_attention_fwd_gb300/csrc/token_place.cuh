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

// A token's sequence b (batch: padding, -1: before the first), and where that
// one's tokens and positions start.
struct Sequence {
    int b, cu, start;
};

// The sequences of kTokens consecutive tokens from tok0 on, each lane asking
// for token tok0 + k; the whole warp calls it.  Up to 127 sequences the
// offsets and the start positions are fetched in one round of loads.
template <int kTokens>
__device__ __forceinline__ Sequence warp_sequences(int tok0, int k, const int32_t* __restrict__ cu,
                                                   const int32_t* __restrict__ start_pos, int batch) {
    Sequence q{-1, 0, 0};
    if (batch < 128) {
        const int lane = threadIdx.x & 31, words = (batch + 32) >> 5;
        int c[4], s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = lane + 32 * i;
            c[i] = i < words && at <= batch ? __ldg(&cu[at]) : 0x7FFFFFFF;
            s[i] = i < words && at < batch ? __ldg(&start_pos[at]) : 0;
        }
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
            int below = -1;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < words) below += __popc(__ballot_sync(0xffffffffu, c[i] <= tok0 + j));
            if (j == k) q.b = below;
        }
        const int from = max(q.b, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < words) {
                const int ci = __shfl_sync(0xffffffffu, c[i], from & 31), si = __shfl_sync(0xffffffffu, s[i], from & 31);
                if (from >> 5 == i) {
                    q.cu = ci;
                    q.start = si;
                }
            }
    } else {
        const int first = warp_sequence(tok0, cu, batch);
        int b = max(first, 0);
        if (tok0 + k >= __ldg(&cu[b])) {
            while (b < batch && __ldg(&cu[b + 1]) <= tok0 + k) ++b;
            q.b = b;
            if (b < batch) {
                q.cu = __ldg(&cu[b]);
                q.start = __ldg(&start_pos[b]);
            }
        }
    }
    return q;
}

// Where token `tok` of the sequence lives: logical position
// start + (tok - cu) is row pos % 64 of page block_table[b, pos / 64].
__device__ __forceinline__ Place token_place(int tok, const Sequence& q, const int32_t* __restrict__ block_table,
                                             int batch, int max_pages, int num_pool_pages, int& page, int& row,
                                             long long& pos) {
    if (q.b < 0 || q.b >= batch) return Place::kPadding;
    pos = (long long)q.start + (tok - q.cu);
    if (pos < 0 || pos / kPage >= max_pages) return Place::kOutOfRange;
    page = __ldg(&block_table[(long long)q.b * max_pages + pos / kPage]);
    row = (int)(pos % kPage);
    return (unsigned)page < (unsigned)num_pool_pages ? Place::kOk : Place::kOutOfRange;
}

}  // namespace pa
