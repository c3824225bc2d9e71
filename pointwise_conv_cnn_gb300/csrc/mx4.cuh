// mx4.cuh -- the values of microscaled 4-bit floating point.
#pragma once

#include <cuda_fp16.h>
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

// The values of the two codes in the low byte, that of the low four bits first: exact in f16.
__device__ __forceinline__ float2 e2m1_values(uint32_t codes) {
    uint32_t h;
    asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(codes));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// 2^(code - 127), NaN for 255.
__device__ __forceinline__ float power_of(unsigned code) {
    return __uint_as_float(code == 255u ? 0x7FFFFFFFu : code ? code << 23 : 0x00400000u);
}

}  // namespace seq
}  // namespace fcm
