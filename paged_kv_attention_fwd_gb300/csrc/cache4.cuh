// cache4.cuh -- one 16-element block of a new row into a 4-bit page.
#pragma once

#include "fp4.cuh"
#include "pa_step.h"

namespace pa {

__device__ __forceinline__ bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

// 32 bytes of global memory: one access -- a whole sector per thread, where
// two of 16 bytes touch every sector of a warp's span twice (read-back of
// 302k rows: 238 us against 301) -- when every address is 32-byte aligned.
struct Sector {
    uint4 lo, hi;
};
__device__ __forceinline__ Sector load_sector(const void* p, bool wide) {
    Sector s;
    if (wide) {
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(s.lo.x), "=r"(s.lo.y), "=r"(s.lo.z), "=r"(s.lo.w), "=r"(s.hi.x), "=r"(s.hi.y), "=r"(s.hi.z),
                       "=r"(s.hi.w)
                     : "l"(p));
    } else {
        s.lo = __ldg(static_cast<const uint4*>(p));
        s.hi = __ldg(static_cast<const uint4*>(p) + 1);
    }
    return s;
}
__device__ __forceinline__ void store_sector(void* p, const Sector& s, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(s.lo.x), "r"(s.lo.y),
                     "r"(s.lo.z), "r"(s.lo.w), "r"(s.hi.x), "r"(s.hi.y), "r"(s.hi.z), "r"(s.hi.w)
                     : "memory");
    } else {
        static_cast<uint4*>(p)[0] = s.lo;
        static_cast<uint4*>(p)[1] = s.hi;
    }
}

// the bf16 elements of w, as floats
__device__ __forceinline__ void bf16x8_to_float(const uint4& w, F2 (&x)[4]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = f2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
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
    const uint32_t byte = fp4_block_scale(__uint_as_float((m & 0x7FFFu) << 16), ks, step);
    F2 x[4];
    uint2 codes;
    bf16x8_to_float(w0, x);
    codes.x = fp4_codes8(x, byte, step);
    bf16x8_to_float(w1, x);
    codes.y = fp4_codes8(x, byte, step);
    *reinterpret_cast<uint2*>(slab + row * (D / 2) + piece * 8) = codes;
    slab[kPage * (D / 2) + row * (D / 16) + piece] = (uint8_t)byte;
}

}  // namespace pa
