// The rows of d_dst as the gradients' products of mul_mat_id read them: device code of thread blocks
// beside the row ids. A pass of memory (16384 slots of 2880 bf16 from 4096 rows, with their factors: 24 us).
#pragma once
#include "moe_internal.h"

namespace moe {

// Block `block` of `blocks`: eight columns a thread, in the element type, and with the slots' factors.
template <class Elem, int THREADS>
__device__ __forceinline__ void prepare_rows(const GradInArgs& a, int64_t block, int64_t blocks) {
    typedef Elem Vec __attribute__((ext_vector_type(8)));
    const uint32_t chunks = (uint32_t)(a.ld / 8);
    const int64_t all = a.rows * chunks;
    const bool whole = !a.f32 && a.N % 8 == 0 && ((uintptr_t)a.src & 15) == 0;
    for (int64_t i = block * THREADS + threadIdx.x; i < all; i += blocks * THREADS) {
        const int64_t row = i >> 32 ? i / chunks : (int64_t)((uint32_t)i / chunks), c = (i - row * chunks) * 8;
        float v[8];
        if (whole) {
            const Vec in = *(const Vec*)((const Elem*)a.src + row * a.N + c);
#pragma unroll
            for (int u = 0; u < 8; u++) v[u] = (float)in[u];
        } else {
#pragma unroll
            for (int u = 0; u < 8; u++) {
                const int64_t at = row * a.N + c + u;
                v[u] = c + u >= a.N ? 0.f : a.f32 ? ((const float*)a.src)[at] : (float)((const Elem*)a.src)[at];
            }
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
#pragma unroll
                for (int u = 0; u < 8; u++) o[u] = c + u < a.N ? (Elem)(w * v[u]) : (Elem)0.f;
                *(Vec*)((Elem*)a.scaled + (row * a.k + s) * a.ld + c) = o;
            }
        }
    }
}

}  // namespace moe
