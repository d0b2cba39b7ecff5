// cache4.cuh -- one 16-element block of a new row into a 4-bit page.
#pragma once

#include "fp4.cuh"
#include "pa_internal.h"

namespace pa {

// the bf16 elements of w, as floats
__device__ __forceinline__ void bf16x8_to_float(const uint4& w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint32_t absmax_bf16x8(const uint4& w) {
    return absmax_bf16x2(absmax_bf16x2(w.x, w.y), absmax_bf16x2(w.z, w.w));
}

// elements 16 piece .. 16 piece + 15 (bf16: w0, w1) of row `row` of a slab
template <int D>
__device__ __forceinline__ void fp4_store_block(uint8_t* slab, int row, int piece, const uint4& w0, const uint4& w1,
                                                float ks) {
    const uint32_t m2 = absmax_bf16x2(absmax_bf16x8(w0), absmax_bf16x8(w1));
    const uint32_t m = absmax_bf16x2(m2, m2 >> 16);
    float step;
    const uint32_t byte = fp4_block_scale(__uint_as_float(m << 16), ks, step);
    float x[8];
    uint2 codes;
    bf16x8_to_float(w0, x);
    codes.x = fp4_codes8(x, byte, step);
    bf16x8_to_float(w1, x);
    codes.y = fp4_codes8(x, byte, step);
    *reinterpret_cast<uint2*>(slab + row * (D / 2) + piece * 8) = codes;
    slab[kPage * (D / 2) + row * (D / 16) + piece] = (uint8_t)byte;
}

}  // namespace pa
