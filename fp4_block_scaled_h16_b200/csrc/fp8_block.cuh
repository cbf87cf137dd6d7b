// fp8_block.cuh -- the codes of one E4M3 block of 128 under one FP32 scale,
// shared by the quantizer (fp8_quantize.cu) and the norms (norm_residual.cu).
//
// With m the block's largest magnitude the scale is s = RN(m / 448) (1 where that
// is below the smallest normal binary32) and the code of x is E4M3_rne(448 x / m).
// bf16 values, and products of two of them, often lie exactly in the middle of
// two codes, where a quotient that is off by one ulp takes the wrong one.  So the
// quotient is a product with the rounded 448 / m, corrected once by its remainder
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990):
//   v0 = RN(x c), c = RN(448 / m);   e = v0 (m / 512) - 7/8 x;   v = v0 - e r,
//   r = RN(512 / m)
// which is exact wherever binary32 holds the quotient and 7 x, and keeps the
// sign of a zero (e is +0 there).  Four packed operations for two elements,
// instead of two divisions.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fp4 {

struct Fp8Block {
    float s;        // the stored scale
    float c;        // 448 / m
    float m;        // m / 512
    float nr;       // -512 / m
};

// m the largest |x|, and `times` what the values still have to be multiplied by
__device__ __forceinline__ Fp8Block fp8_block(float m, float times = 1.0f) {
    Fp8Block b;
    b.s = __fdiv_rn(__fmul_rn(m, times), 448.0f);
    if (b.s >= 1.17549435e-38f) {
        b.c = __fdiv_rn(448.0f, m);
        b.m = __fmul_rn(m, 0x1p-9f);
        b.nr = -__frcp_rn(b.m);
    } else {        // an all but zero block: codes of the values themselves
        b.s = 1.0f;
        b.c = times;
        b.m = 0.0f;
        b.nr = -0.0f;
    }
    return b;
}

__device__ __forceinline__ float2 fp8_quotient(float2 x, const Fp8Block& b) {
    const float2 v = __fmul2_rn(x, make_float2(b.c, b.c));
    const float2 e = __ffma2_rn(v, make_float2(b.m, b.m), __fmul2_rn(x, make_float2(-0.875f, -0.875f)));
    return __ffma2_rn(e, make_float2(b.nr, b.nr), v);
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
