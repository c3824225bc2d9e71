// mx4.cuh -- the values of microscaled 4-bit floating point.
#pragma once

#include <stdint.h>

namespace fcm {
namespace seq {

// Two values to the nearest E2M1 codes, ties to the even code, magnitudes above 6 to 6; `lo` in the low
// four bits.
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The value of the code in the low four bits: sign, two bits of exponent, one of mantissa.  Put into a
// float's bits they stand for value * 2^-126 (the subnormal step 0.5 included).
__device__ __forceinline__ float e2m1_value(uint32_t code) {
    return __uint_as_float((code & 8u) << 28 | (code & 7u) << 22) * 0x1p126f;
}

// 2^(code - 127), NaN for 255.
__device__ __forceinline__ float power_of(unsigned code) {
    return __uint_as_float(code == 255u ? 0x7FFFFFFFu : code ? code << 23 : 0x00400000u);
}

}  // namespace seq
}  // namespace fcm
