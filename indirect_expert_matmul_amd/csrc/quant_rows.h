// Rows to int8 codes with one float32 scale each: what the row quantizer and the int8 GEMV share.
#pragma once
#include "moe_internal.h"

namespace moe {

constexpr float kQuantMinFast = 1e-30f;   // scales whose reciprocal is a normal number

// The scale of a row whose largest magnitude has these bits (infinities and NaN sort above all numbers).
static __device__ __forceinline__ float quant_scale(uint32_t top) {
    return top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(top) / 127.0f;
}
// rint(x / d) within +-127, d > 0 and r = 1 / d. The quotient by the reciprocal is at most 3 * 2^-24 of it off, that
// is 2.3e-5: where that could move it past a half, which is one element in ten thousand, it is divided (fast false:
// always).
static __device__ __forceinline__ int quant_code(float x, float d, float r, bool fast) {
    const float t = x * r;
    float q = rintf(t);
    if (!fast || fabsf(fabsf(t - q) - 0.5f) < 1e-4f) q = rintf(x / d);
    return (int)fminf(fmaxf(q, -127.f), 127.f);
}

}  // namespace moe
