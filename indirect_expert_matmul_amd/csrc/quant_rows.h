// Rows to int8 codes with one float32 scale each: what the row quantizer and the int8 GEMV share.
#pragma once
#include <type_traits>

#include "moe_internal.h"

namespace moe {

constexpr float kQuantMinFast = 1e-30f;   // scales whose reciprocal is a normal number

// The scale of a row whose largest magnitude has these bits (infinities and NaN sort above all numbers).
static __device__ __forceinline__ float quant_scale(uint32_t top) {
    return top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(top) / 127.0f;
}
// rint(x / d) within +-127, d > 0 and r = 1 / d. The quotient by the reciprocal is at most 3 * 2^-24 of it off, that
// is 2.3e-5: where that could move it past a half, which is two elements in ten thousand, it is divided (fast false:
// always).
static __device__ __forceinline__ int quant_code(float x, float d, float r, bool fast) {
    const float t = x * r;
    float q = rintf(t);
    if (!fast || fabsf(fabsf(t - q) - 0.5f) < 1e-4f) q = rintf(x / d);
    return (int)fminf(fmaxf(q, -127.f), 127.f);
}

// Rows of a source type, read 16 bytes at a time from anywhere.
template <int SRC>
struct QuantSrc {
    using Elem = std::conditional_t<SRC == kElemF32, float, std::conditional_t<SRC == kElemBf16, __bf16, _Float16>>;
    static constexpr int EC = 16 / (int)sizeof(Elem);   // elements of a load
    typedef Elem Vec __attribute__((ext_vector_type(EC)));
    static __device__ __forceinline__ Vec load(const Elem* p) {
        Vec v;
        __builtin_memcpy(&v, p, 16);
        return v;
    }
};

static __device__ __forceinline__ uint32_t quant_wave_max(uint32_t v) {
    for (int m = 32; m; m >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, m));
    return v;
}
// Codes of one load.
template <int SRC>
__device__ __forceinline__ void quant_store(int8_t* o, const typename QuantSrc<SRC>::Vec& v, float d, float r, bool fast, bool some) {
    constexpr int EC = QuantSrc<SRC>::EC;
    uint32_t w[EC / 4];
#pragma unroll
    for (int i = 0; i < EC / 4; i++) {
        w[i] = 0;
#pragma unroll
        for (int u = 0; u < 4; u++) w[i] |= ((uint32_t)quant_code((float)v[4 * i + u], d, r, fast) & 255u) << (8 * u);
        if (!some) w[i] = 0;
    }
    __builtin_memcpy(o, w, EC);
}

// A wave quantizes a row of at least one load, reading it twice.
template <int SRC>
__device__ __forceinline__ void quant_row_twice(const QuantRowsArgs& a, int64_t row, int lane) {
    using S = QuantSrc<SRC>;
    constexpr int EC = S::EC;
    const typename S::Elem* x = (const typename S::Elem*)a.src + row * a.K;
    int8_t* q = a.q + row * a.K;
    const int64_t last = a.K - EC;
    uint32_t top = 0;
    for (int64_t at = lane * EC; at < a.K; at += 64 * EC) {
        const typename S::Vec v = S::load(x + (at < last ? at : last));
#pragma unroll
        for (int u = 0; u < EC; u++) top = max(top, __float_as_uint((float)v[u]) & 0x7fffffffu);
    }
    top = quant_wave_max(top);
    const float d = quant_scale(top), r = 1.0f / d;
    const bool some = d > 0.f, fast = d > kQuantMinFast;
    for (int64_t at = lane * EC; at < a.K; at += 64 * EC) {
        const int64_t p = at < last ? at : last;
        quant_store<SRC>(q + p, S::load(x + p), d, r, fast, some);
    }
    if (lane == 0) a.d[row] = d;
}

}  // namespace moe
