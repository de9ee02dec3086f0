// kda_e4m3.cuh -- conversions of the 8-bit cache's numbers: 1 sign, 4 exponent and 3 mantissa
// bits, bias 7, no infinities, 0x7f the one NaN.  Every such number is an fp16 number.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kda {

constexpr float kE4m3Largest = 448.0f;

// Two numbers (the low 16 bits) as a pair of fp16, the first in the lower half.
__device__ __forceinline__ uint32_t half2_of_e4m3(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
        : "=r"(r)
        : "r"(two));
    return r;
}

// The same of the high 16 bits.
__device__ __forceinline__ uint32_t half2_of_e4m3_high(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
        : "=r"(r)
        : "r"(two));
    return r;
}

// To the nearest, ties to even, at most the largest number; the first in the low 8 bits.
__device__ __forceinline__ uint32_t e4m3_of(float first, float second) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(second), "f"(first));
    return r;
}

// The smallest power of two, 2^-60 at least, under which `largest` (finite, not negative) is
// at most 448 = 1.75 * 2^8.
__device__ __forceinline__ float e4m3_scale(float largest) {
    const uint32_t bits = __float_as_uint(largest);
    const int e = (int)(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u);   // biased by 127
    return __uint_as_float((uint32_t)(e < 67 ? 67 : e) << 23);
}

}  // namespace kda
