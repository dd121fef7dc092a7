// Rows to int8 with one float32 scale a row: d = max|x| / 127 and q = rint(x / d), both in
// float32 (IEEE division, ties to even); a row of zeros has d = 0 and q = 0, a row with an
// infinity or a NaN d = NaN and q = 0.
//
// A pass of memory: one wave a row, 16 bytes a lane and load, the row held in registers between
// its maximum and its codes (up to 16 loads; longer rows are read again, from the caches). Rows may
// start anywhere and have any length: the loads need no alignment, and the last of a row ends with
// it, so that some elements are done twice, with the same result.
// Measured (one MI355X): TODO
#include "quant_rows.h"

namespace moe {
namespace {

constexpr int kThreads = 256, kRows = kThreads / 64;
constexpr int64_t kMaxGrid = 1 << 22;   // blocks take several rows past it

// CH: loads a lane holds; 0: the row is read twice.
template <int SRC, int CH>
__global__ __launch_bounds__(kThreads) void k_quant_rows(QuantRowsArgs a) {
    using S = QuantSrc<SRC>;
    constexpr int EC = S::EC;
    const int lane = threadIdx.x & 63;
    for (int64_t row = (int64_t)blockIdx.x * kRows + (threadIdx.x >> 6); row < a.rows; row += (int64_t)gridDim.x * kRows) {
        const typename S::Elem* x = (const typename S::Elem*)a.src + row * a.K;
        int8_t* q = a.q + row * a.K;
        const int64_t last = a.K - EC;
        uint32_t top = 0;   // largest magnitude as bits: infinities and NaN sort above all numbers
        auto grow = [&](const typename S::Vec& v) {
#pragma unroll
            for (int u = 0; u < EC; u++) top = max(top, __float_as_uint((float)v[u]) & 0x7fffffffu);
        };
        if constexpr (CH > 0) {
            typename S::Vec v[CH];
#pragma unroll
            for (int c = 0; c < CH; c++) {
                const int at = (c * 64 + lane) * EC;
                v[c] = S::load(x + (at < last ? at : last));
            }
#pragma unroll
            for (int c = 0; c < CH; c++) grow(v[c]);
            top = quant_wave_max(top);
            const float d = quant_scale(top), r = 1.0f / d;
            const bool some = d > 0.f, fast = d > kQuantMinFast;
#pragma unroll
            for (int c = 0; c < CH; c++) {
                const int at = (c * 64 + lane) * EC;
                if (at < a.K) quant_store<SRC>(q + (at < last ? at : last), v[c], d, r, fast, some);
            }
            if (lane == 0) a.d[row] = d;
        } else {
            quant_row_twice<SRC>(a, row, lane);
        }
    }
}

// Rows shorter than a load.
template <int SRC>
__global__ __launch_bounds__(kThreads) void k_quant_short(QuantRowsArgs a) {
    using Elem = typename QuantSrc<SRC>::Elem;
    for (int64_t row = (int64_t)blockIdx.x * kThreads + threadIdx.x; row < a.rows; row += (int64_t)gridDim.x * kThreads) {
        const Elem* x = (const Elem*)a.src + row * a.K;
        uint32_t top = 0;
        for (int c = 0; c < a.K; c++) top = max(top, __float_as_uint((float)x[c]) & 0x7fffffffu);
        const float d = quant_scale(top);
        for (int c = 0; c < a.K; c++) a.q[row * a.K + c] = d > 0.f ? (int8_t)quant_code((float)x[c], d, 0.f, false) : 0;
        a.d[row] = d;
    }
}

template <int SRC>
void launch(const QuantRowsArgs& a, hipStream_t st) {
    const auto grid = [](int64_t blocks) { return (unsigned)(blocks < kMaxGrid ? blocks : kMaxGrid); };
    const unsigned g = grid((a.rows + kRows - 1) / kRows);
    const int64_t ch = (a.K + 64 * QuantSrc<SRC>::EC - 1) / (64 * QuantSrc<SRC>::EC);
    if (a.K < QuantSrc<SRC>::EC) k_quant_short<SRC><<<grid((a.rows + kThreads - 1) / kThreads), kThreads, 0, st>>>(a);
    else if (ch <= 1) k_quant_rows<SRC, 1><<<g, kThreads, 0, st>>>(a);
    else if (ch <= 2) k_quant_rows<SRC, 2><<<g, kThreads, 0, st>>>(a);
    else if (ch <= 4) k_quant_rows<SRC, 4><<<g, kThreads, 0, st>>>(a);
    else if (ch <= 8) k_quant_rows<SRC, 8><<<g, kThreads, 0, st>>>(a);
    else if (ch <= 12) k_quant_rows<SRC, 12><<<g, kThreads, 0, st>>>(a);
    else if (ch <= 16) k_quant_rows<SRC, 16><<<g, kThreads, 0, st>>>(a);
    else k_quant_rows<SRC, 0><<<g, kThreads, 0, st>>>(a);
}

}  // namespace

hipError_t launch_quant_rows(const QuantRowsArgs& a, hipStream_t st) {
    if (a.rows <= 0) return hipSuccess;
    if (a.src_type == kElemF32) launch<kElemF32>(a, st);
    else if (a.src_type == kElemBf16) launch<kElemBf16>(a, st);
    else launch<kElemF16>(a, st);
    return hipGetLastError();
}

}  // namespace moe
