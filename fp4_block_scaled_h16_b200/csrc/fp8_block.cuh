// fp8_block.cuh -- the codes of one E4M3 block of 128 under one FP32 scale,
// shared by the quantizer (fp8_quantize.cu) and the norms (norm_residual.cu).
//
// With m the block's largest magnitude the scale is s = RN(m / 448) (1 where that
// is below the smallest normal binary32) and the code of x is E4M3_rne(448 x / m).
// bf16 values, and products of two of them, often lie exactly in the middle of
// two codes, where a quotient that is off by one ulp takes the wrong one.  So
// 448 / m is held as an unevaluated sum of two binary32, c + d, with c a little
// below it and d >= 0 the rest (Dekker, "A floating-point technique for extending
// the available precision", 1971), within 2^-40 of it, and the quotient is
// RN(x c + RN(x d)): exact wherever binary32 holds it, and with the sign of a
// zero kept.  Two packed operations for two elements, instead of two divisions.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fp4 {

struct Fp8Block {
    float s;        // the stored scale
    float c, d;     // 448 / m
};

// RN(x / 448): a product with RN(1 / 448) corrected by its remainder (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990), where that remainder does not underflow
__device__ __forceinline__ float over_448(float x) {
    if (x < 0x1p-90f) return __fdiv_rn(x, 448.0f);
    const float q = __fmul_rn(x, 1.0f / 448.0f);
    return __fmaf_rn(__fmaf_rn(-448.0f, q, x), 1.0f / 448.0f, q);
}

// m the largest |x|, and `times` what the values still have to be multiplied by
__device__ __forceinline__ Fp8Block fp8_block(float m, float times = 1.0f) {
    Fp8Block b;
    b.s = over_448(__fmul_rn(m, times));
    if (b.s >= 1.17549435e-38f) {
        float r;                                            // 1 / m within 2^-22
        asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(m));
        b.c = __fmul_rn(448.0f * (1.0f - 0x1p-20f), r);     // below 448 / m by 2^-21 to 2^-19 of it
        b.d = __fmul_rn(__fmaf_rn(-b.c, m, 448.0f), r);
    } else {        // an all but zero block: codes of the values themselves
        b.s = 1.0f;
        b.c = times;
        b.d = 0.0f;
    }
    return b;
}

__device__ __forceinline__ float2 fp8_quotient(float2 x, const Fp8Block& b) {
    return __ffma2_rn(x, make_float2(b.c, b.c), __fmul2_rn(x, make_float2(b.d, b.d)));
}

// the codes of four elements, the first in the low byte; the conversion saturates to 448
__device__ __forceinline__ uint32_t fp8_codes4(float2 x01, float2 x23, const Fp8Block& b) {
    const float2 u = fp8_quotient(x01, b), v = fp8_quotient(x23, b);
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(u.y), "f"(u.x));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v.y), "f"(v.x));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

}  // namespace fp4
