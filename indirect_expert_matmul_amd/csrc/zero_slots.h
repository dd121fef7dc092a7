// Per-slot output: rows of slots whose id is out of range are zero. One wave looks at kZeroSlots
// slots, a lane each, and writes the rows that need it (one thread per output element
// spent 75 us on 32768 x 2048 just reading ids: 6 us now).
#pragma once
#include "moe_internal.h"

namespace moe {

constexpr int kZeroSlots = 8;

inline int64_t zero_slots_grid(int64_t n, int threads) {
    const int64_t per = threads / 64 * kZeroSlots;
    return (n + per - 1) / per;
}

// Thread block `block` of THREADS threads.
template <int THREADS>
__device__ __forceinline__ void zero_invalid_slots(const ZeroSlots& a, int64_t block) {
    const int lane = threadIdx.x & 63;
    const int64_t s0 = (block * (THREADS / 64) + (threadIdx.x >> 6)) * kZeroSlots;
    if (s0 >= a.n) return;
    const int32_t e = lane < kZeroSlots && s0 + lane < a.n ? a.ids[s0 + lane] : 0;
    uint64_t bad = __ballot(e < 0 || e >= a.E);
    for (; bad; bad &= bad - 1) {
        float* o = a.out + (s0 + __builtin_ctzll(bad)) * a.N;
        for (int c = lane; c < a.N; c += 64) o[c] = 0.f;
    }
}

}  // namespace moe
