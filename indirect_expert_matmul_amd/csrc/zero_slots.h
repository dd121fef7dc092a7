// Per-slot output: rows of slots whose id is out of range are zero. One wave looks at kZeroSlots
// slots, a lane each, and writes its piece of kZeroCols columns of the rows that need it, 16 bytes
// a lane. (One thread per output element spent 75 us on 32768 x 2048 just reading ids: 6 us now. One
// wave for whole rows took 27 us for 8 slots of 7168 columns and 109 for 8 of 32768; pieces take 6.2 and 7.4,
// most of it the launch.)
#pragma once
#include "moe_internal.h"

namespace moe {

constexpr int kZeroSlots = 8, kZeroCols = 2048;
// Thread blocks along the slots at most, which take several groups of slots then: with up to 2^31 slots
// one group each would be more work-items than a dispatch holds.
constexpr int64_t kZeroGrid = 1 << 16;

inline __host__ __device__ int zero_pieces(const ZeroSlots& a) { return (a.N - 1) / kZeroCols + 1; }
inline int64_t zero_slots_grid(const ZeroSlots& a, int threads) {
    const int64_t per = threads / 64 * kZeroSlots, groups = (a.n + per - 1) / per, most = kZeroGrid / zero_pieces(a);
    return (groups < most ? groups : most > 1 ? most : groups > 0) * zero_pieces(a);
}

// Thread block `block` of the `grid` blocks of THREADS threads.
template <int THREADS>
__device__ __forceinline__ void zero_invalid_slots(const ZeroSlots& a, uint32_t block, uint32_t grid) {
    typedef float f32x4 __attribute__((ext_vector_type(4), aligned(4)));   // rows start anywhere
    const uint32_t lane = threadIdx.x & 63, pieces = zero_pieces(a);
    const int c0 = (int)(block % pieces) * kZeroCols, cols = min(kZeroCols, a.N - c0);
    constexpr int kWaves = THREADS / 64;
    int64_t s0 = ((int64_t)(block / pieces) * kWaves + (threadIdx.x >> 6)) * kZeroSlots;
    for (; s0 < a.n; s0 += (int64_t)(grid / pieces) * kWaves * kZeroSlots) {
        const int32_t e = lane < kZeroSlots && s0 + lane < a.n ? a.ids[s0 + lane] : 0;
        uint64_t bad = __ballot(e < 0 || e >= a.E);
        for (; bad; bad &= bad - 1) {
            float* o = a.out + (s0 + __builtin_ctzll(bad)) * a.N + c0;
            for (int c = 4 * (int)lane; c + 4 <= cols; c += 256) *(f32x4*)(o + c) = f32x4{0.f, 0.f, 0.f, 0.f};
            if ((int)lane < (cols & 3)) o[(cols & ~3) + lane] = 0.f;
        }
    }
}

}  // namespace moe
