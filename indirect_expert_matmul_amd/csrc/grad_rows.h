// The rows of d_dst as the gradients' products of mul_mat_id read them: device code of thread blocks
// beside the row ids. A pass of memory (16384 slots of 2880 bf16 from 4096 rows, with their factors, two terms: 41 us, three 58;
// from float32 rows 40, and 16384 float32 rows rounded 42).
#pragma once
#include <type_traits>

#include "moe_internal.h"

namespace moe {

// The elements that a float32 number is the sum of: each takes the leading bits of what is left (8 of bf16, 11 of f16), the
// last one is rounded. Two are off by at most 2^-15 (bf16) or 2^-21 (f16) of the number, three hold it; f16 adds up to its
// smallest number, 2^-24. An infinity or a NaN is all of them. All have the number's sign and none is zero, so that an
// infinity of the other operand meets neither a zero nor both signs: a bf16 term of zero is 2^-133 instead; that is too
// little to count, which 2^-24 is not beside small numbers, so f16's leading bits are those of the next number towards
// zero and leave something (but for numbers of one or two times 2^-24).
template <class Elem>
__device__ __forceinline__ Elem cut_off(float v) {
    if constexpr (std::is_same<Elem, __bf16>::value) {
        return __builtin_bit_cast(__bf16, (uint16_t)(__float_as_uint(v) >> 16));
    } else {
        const float less = v == 0.f ? v : __uint_as_float(__float_as_uint(v) - 1u);
        return __builtin_bit_cast(_Float16, (uint16_t)__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(less, 0.f)));
    }
}
template <class Elem>
__device__ __forceinline__ Elem next_term(float v, float& rest, bool last) {   // selects: a branch an element costs more
    Elem t = last ? (Elem)rest : cut_off<Elem>(rest);
    rest -= (float)t;
    const uint32_t bits = __float_as_uint(v), small = v != 0.f ? bits >> 31 << 15 | 1u : 0u;
    const bool none = (float)t == 0.f && (std::is_same<Elem, __bf16>::value || last);
    const uint32_t some = none ? small : __builtin_bit_cast(uint16_t, t);
    return __builtin_bit_cast(Elem, (uint16_t)((bits & 0x7f800000u) == 0x7f800000u ? __builtin_bit_cast(uint16_t, (Elem)v) : some));
}

// Block `block` of `blocks`: eight columns a thread, in the element type, and with the slots' factors.
template <class Elem, int THREADS>
__device__ __forceinline__ void prepare_rows(const GradInArgs& a, int64_t block, int64_t blocks) {
    typedef Elem Vec __attribute__((ext_vector_type(8)));
    const uint32_t chunks = (uint32_t)(a.ld / 8);
    const int64_t all = a.rows * chunks;
    const bool whole = !a.f32 && a.N % 8 == 0 && ((uintptr_t)a.src & 15) == 0;
    float scale = 1.f;
    if (a.tops) {   // every wave joins the parts by itself
        float top = 0.f;
        for (int i = threadIdx.x & 63; i < a.n_tops; i += 64) top = fmaxf(top, a.tops[i]);
#pragma unroll
        for (int m = 32; m; m >>= 1) top = fmaxf(top, __shfl_xor(top, m));
        // exponents below -112 would take the factor past float32
        const int e = top > 0.f ? max((int)(__float_as_uint(top) >> 23) - 127, -112) - 14 : 0;
        scale = __uint_as_float((uint32_t)(127 - e) << 23);
        if (block == 0 && threadIdx.x == 0) *a.unscale = __uint_as_float((uint32_t)(127 + e) << 23);
    }
    for (int64_t i = block * THREADS + threadIdx.x; i < all; i += blocks * THREADS) {
        const int64_t row = i >> 32 ? i / chunks : (int64_t)((uint32_t)i / chunks), c = (i - row * chunks) * 8;
        float v[8];
        if (whole) {
            const Vec in = *(const Vec*)((const Elem*)a.src + row * a.N + c);
#pragma unroll
            for (int u = 0; u < 8; u++) v[u] = (float)in[u];
        } else if (a.f32) {
            typedef float f32x4 __attribute__((ext_vector_type(4), aligned(4)));   // rows start anywhere
            const float* in = (const float*)a.src + row * a.N + c;
            if (c + 8 <= a.N) {
                const f32x4 lo = *(const f32x4*)in, hi = *(const f32x4*)(in + 4);
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    v[u] = lo[u];
                    v[4 + u] = hi[u];
                }
            } else {
#pragma unroll
                for (int u = 0; u < 8; u++) v[u] = c + u < a.N ? in[u] : 0.f;
            }
        } else {
            const Elem* in = (const Elem*)a.src + row * a.N + c;
#pragma unroll
            for (int u = 0; u < 8; u++) v[u] = c + u < a.N ? (float)in[u] : 0.f;
        }
        Vec o;
        if (a.dst) {
#pragma unroll
            for (int u = 0; u < 8; u++) o[u] = (Elem)v[u];
            *(Vec*)((Elem*)a.dst + row * a.ld + c) = o;
        }
        if (a.scaled) {
            for (int s = 0; s < a.k; s++) {
                const float w = a.route_w[row * a.k + s];
                float p[8], rest[8];
#pragma unroll
                for (int u = 0; u < 8; u++) rest[u] = p[u] = c + u < a.N ? w * v[u] * scale : 0.f;
                Elem* to = (Elem*)a.scaled + (row * a.k + s) * a.ld + c;
                for (int t = 0; t < a.terms; t++, to += a.rows * a.k * a.ld) {
#pragma unroll
                    for (int u = 0; u < 8; u++) o[u] = next_term<Elem>(p[u], rest[u], t + 1 == a.terms);
                    *(Vec*)to = o;
                }
            }
        }
    }
}

}  // namespace moe
