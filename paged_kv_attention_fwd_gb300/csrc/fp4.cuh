// fp4.cuh -- the 4-bit page type: e2m1 codes with one e4m3 scale per 16
// elements of a row.
//
// One (page, KV head) slab holds 64 rows of D / 2 code bytes (element 2i in
// the low nibble of byte i), then 64 rows of D / 16 scale bytes: 4.5 bits per
// element, 4608 bytes at D = 128, one contiguous copy.  An element stands for
// code * block scale * head scale.
//
// Quantising 16 elements x_i with head scale ks:
//   bs   = e4m3(max |x_i| / (6 ks)), nearest even, saturating at 448
//   S    = bs * ks                          (fp32)
//   code = e2m1(x_i / S), nearest even, saturating at 6; all codes 0 if bs = 0
// with every quotient an fp32 one (nearest even).  A NaN among the 16 makes
// the scale NaN, so the block reads back as NaN; an infinity saturates.
//
// Reading back: a code has 2 significant bits and a scale 4, so code * scale
// is exact in fp16 (at least 2^-10, at most 2688); the head scale is applied
// in fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "f32x2.cuh"

namespace pa {

constexpr int kFp4Block = 16;
__host__ __device__ constexpr int fp4_slab_bytes(int d) { return 64 * (d / 2 + d / kFp4Block); }

// e2m1 codes of 8 elements, 4 bits each, element 0 lowest
__device__ __forceinline__ uint32_t e2m1x8(const F2 (&pairs)[4]) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = split(pairs[i]);
        q[2 * i] = v.x;
        q[2 * i + 1] = v.y;
    }
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    return r;
}

// the values of byte `kByte` of w: element 2i in the low half
template <int kByte>
__device__ __forceinline__ uint32_t e2m1x2_to_half2(uint32_t w) {
    uint32_t r;
    if constexpr (kByte == 0)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (kByte == 1)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (kByte == 2)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
    else
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

// two e4m3 bytes (the low 16 bits of w) as fp16
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ float e4m3_to_float(uint32_t byte) {
    const uint32_t h2 = e4m3x2_to_half2(byte & 0xFFu);
    return __half2float(__ushort_as_half((unsigned short)(h2 & 0xFFFFu)));
}

// largest magnitude of two 16-bit lanes each, NaN if any is NaN; the signs are anything
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The scale byte of a block whose largest magnitude is `amax`, and the step
// S = scale * ks that its elements are divided by.
__device__ __forceinline__ uint32_t fp4_block_scale(float amax, float ks, float& step) {
    const uint32_t byte =
        (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(amax, __fmul_rn(ks, 6.f)), __NV_SATFINITE, __NV_E4M3);
    step = __fmul_rn(e4m3_to_float(byte), ks);
    return byte;
}

// Codes of 8 elements, 4 bits each, element 0 lowest.
//
// A division per element would cost more than the copy.  Away from the ends
// of fp32 the quotient comes from the correctly rounded reciprocal with one
// residual step (P. Markstein, IBM J. Res. Dev. 34, 1990, on division with a
// fused multiply-add), q' = q + (x - q S) r: the residual is exact, so q' is
// the fp32 quotient wherever it lies between the smallest and the largest code
// (smaller ones round to 0 either way; tested for every bf16 magnitude).  It
// is taken of -q, whose steps leave a zero of x its sign.
__device__ __forceinline__ uint32_t fp4_codes8(const F2 (&x)[4], uint32_t byte, float step) {
    F2 q[4];
    if (byte < 0x7Eu && step > 1e-30f && step < 1e30f) {
        const float r1 = __frcp_rn(step);
        const F2 minus_r = f2(-r1, -r1), s = f2(step, step);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const F2 q0 = x[i] * minus_r;
            q[i] = fma2(fma2(q0, s, x[i]), minus_r, q0);
        }
        return e2m1x8(q) ^ 0x88888888u;
    } else {
        if (byte >= 0x7Fu || !(step > 0.f)) return 0;  // a zero or NaN scale
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = split(x[i]);
            q[i] = f2(__fdiv_rn(v.x, step), __fdiv_rn(v.y, step));
        }
    }
    return e2m1x8(q);
}

}  // namespace pa
