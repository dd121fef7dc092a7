// Rows to int8 with one float32 scale a row: d = max|x| / 127 and q = rint(x / d), both in
// float32 (IEEE division, ties to even); a row of zeros has d = 0 and q = 0, a row with an
// infinity or a NaN d = NaN and q = 0.
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256, kRows = kThreads / 64;
constexpr int64_t kMaxGrid = 1 << 22;   // blocks take several rows past it

template <int SRC>
__device__ __forceinline__ float load(const void* p, int64_t i) {
    if constexpr (SRC == kElemF32) return ((const float*)p)[i];
    else if constexpr (SRC == kElemBf16) return (float)((const __bf16*)p)[i];
    else return (float)((const _Float16*)p)[i];
}

// One wave a row.
template <int SRC>
__global__ __launch_bounds__(kThreads) void k_quant_rows(QuantRowsArgs a) {
    const int lane = threadIdx.x & 63;
    for (int64_t row = (int64_t)blockIdx.x * kRows + (threadIdx.x >> 6); row < a.rows; row += (int64_t)gridDim.x * kRows) {
        const int64_t base = row * a.K;
        uint32_t top = 0;   // largest magnitude as bits: infinities and NaN sort above all numbers
        for (int64_t c = lane; c < a.K; c += 64) top = max(top, __float_as_uint(load<SRC>(a.src, base + c)) & 0x7fffffffu);
        for (int m = 32; m; m >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
        const float d = top >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float(top) / 127.0f;
        const bool some = d > 0.f;
        for (int64_t c = lane; c < a.K; c += 64) {
            const float v = some ? fminf(fmaxf(rintf(load<SRC>(a.src, base + c) / d), -127.f), 127.f) : 0.f;
            a.q[base + c] = (int8_t)(int)v;
        }
        if (lane == 0) a.d[row] = d;
    }
}

}  // namespace

hipError_t launch_quant_rows(const QuantRowsArgs& a, hipStream_t st) {
    if (a.rows <= 0) return hipSuccess;
    const int64_t blocks = (a.rows + kRows - 1) / kRows;
    const unsigned grid = (unsigned)(blocks < kMaxGrid ? blocks : kMaxGrid);
    if (a.src_type == kElemF32) k_quant_rows<kElemF32><<<grid, kThreads, 0, st>>>(a);
    else if (a.src_type == kElemBf16) k_quant_rows<kElemBf16><<<grid, kThreads, 0, st>>>(a);
    else k_quant_rows<kElemF16><<<grid, kThreads, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace moe
