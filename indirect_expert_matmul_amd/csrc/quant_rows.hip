// Rows to int8 with one float32 scale a row: d = max|x| / 127 and q = rint(x / d), both in
// float32 (IEEE division, ties to even); a row of zeros has d = 0 and q = 0, a row with an
// infinity or a NaN d = NaN and q = 0.
//
// A pass of memory: the lanes of a row load 16 bytes each and hold them in registers between the
// row's maximum and its codes (rows past 64 loads a lane of a wave are read again, from the caches).
// A row has the lanes that it needs: 4 to 32 up to 32 loads, a wave up to 256, then a block. Rows may
// start anywhere and have any length: the loads need no alignment, and the last of a row ends with
// it, so that some elements are done twice, with the same result.
// Measured (one MI355X, per call): 92160 x 2880 float32 237 us, 5.6 TB/s; 30000 x 2048 bf16 31, 5.9 TB/s; 8192 x 16384
// bf16 84, 4.8 TB/s; 4096 x 7168 bf16 19, 4.6 TB/s; 4096 x 2880 bf16 11 to 13, of which an empty call is 10.
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

// Rows of more than 256 loads: the block's four waves share one, so that a lane holds few loads and many waves run
// (one wave a row: 4096 x 7168 bf16 29 us instead of 19, 8192 x 16384 197 instead of 84, 92160 x 2880 float32 231 instead
// of 237. Below, a wave is better: 200000 x 2048 bf16 248 us, 406 by blocks).
template <int SRC, int CH>
__global__ __launch_bounds__(kThreads) void k_quant_block(QuantRowsArgs a) {
    using S = QuantSrc<SRC>;
    constexpr int EC = S::EC;
    __shared__ uint32_t tops[2][kRows];   // of this row and of the one before
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const typename S::Elem* x = (const typename S::Elem*)a.src + row * a.K;
        int8_t* q = a.q + row * a.K;
        const int last = (int)a.K - EC;
        uint32_t top = 0;
        typename S::Vec v[CH];
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int at = (c * kThreads + (int)threadIdx.x) * EC;
            v[c] = S::load(x + (at < last ? at : last));
        }
#pragma unroll
        for (int c = 0; c < CH; c++)
#pragma unroll
            for (int u = 0; u < EC; u++) top = max(top, __float_as_uint((float)v[c][u]) & 0x7fffffffu);
        top = quant_wave_max(top);
        if ((threadIdx.x & 63) == 0) tops[turn][threadIdx.x >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kRows; w++) top = max(top, tops[turn][w]);
        const float d = quant_scale(top), r = 1.0f / d;
        const bool some = d > 0.f, fast = d > kQuantMinFast;
#pragma unroll
        for (int c = 0; c < CH; c++) {
            const int at = (c * kThreads + (int)threadIdx.x) * EC;
            if (at < a.K) quant_store<SRC>(q + (at < last ? at : last), v[c], d, r, fast, some);
        }
        if (threadIdx.x == 0) a.d[row] = d;
    }
}

// Rows of up to L loads, L lanes each (one wave a row left most lanes idle: 606776 rows of 120 bf16 236 us, now 49).
template <int SRC, int L>
__global__ __launch_bounds__(kThreads) void k_quant_narrow(QuantRowsArgs a) {
    using S = QuantSrc<SRC>;
    constexpr int EC = S::EC, kPer = kThreads / L;
    const int l = threadIdx.x % L;
    for (int64_t row = (int64_t)blockIdx.x * kPer + threadIdx.x / L; row < a.rows; row += (int64_t)gridDim.x * kPer) {
        const int last = (int)a.K - EC, at = l * EC < last ? l * EC : last;
        const typename S::Vec v = S::load((const typename S::Elem*)a.src + row * a.K + at);
        uint32_t top = 0;
#pragma unroll
        for (int u = 0; u < EC; u++) top = max(top, __float_as_uint((float)v[u]) & 0x7fffffffu);
#pragma unroll
        for (int m = L / 2; m; m >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
        const float d = quant_scale(top), r = 1.0f / d;
        if (l * EC < a.K) quant_store<SRC>(a.q + row * a.K + at, v, d, r, d > kQuantMinFast, d > 0.f);
        if (l == 0) a.d[row] = d;
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
    constexpr int EC = QuantSrc<SRC>::EC;
    const auto grid = [&](int64_t rows) {   // blocks of so many rows
        const int64_t blocks = (a.rows + rows - 1) / rows;
        return (unsigned)(blocks < kMaxGrid ? blocks : kMaxGrid);
    };
    const int64_t loads = (a.K + EC - 1) / EC, ch = (loads + 63) / 64;
    if (a.K < EC) k_quant_short<SRC><<<grid(kThreads), kThreads, 0, st>>>(a);
    else if (loads <= 4) k_quant_narrow<SRC, 4><<<grid(kThreads / 4), kThreads, 0, st>>>(a);
    else if (loads <= 8) k_quant_narrow<SRC, 8><<<grid(kThreads / 8), kThreads, 0, st>>>(a);
    else if (loads <= 16) k_quant_narrow<SRC, 16><<<grid(kThreads / 16), kThreads, 0, st>>>(a);
    else if (loads <= 32) k_quant_narrow<SRC, 32><<<grid(kThreads / 32), kThreads, 0, st>>>(a);
    else if (ch <= 1) k_quant_rows<SRC, 1><<<grid(kRows), kThreads, 0, st>>>(a);
    else if (ch <= 2) k_quant_rows<SRC, 2><<<grid(kRows), kThreads, 0, st>>>(a);
    else if (ch <= 4) k_quant_rows<SRC, 4><<<grid(kRows), kThreads, 0, st>>>(a);
    else if (ch <= 8) k_quant_block<SRC, 2><<<grid(1), kThreads, 0, st>>>(a);
    else if (ch <= 12) k_quant_block<SRC, 3><<<grid(1), kThreads, 0, st>>>(a);
    else if (ch <= 16) k_quant_block<SRC, 4><<<grid(1), kThreads, 0, st>>>(a);
    else if (ch <= 24) k_quant_block<SRC, 6><<<grid(1), kThreads, 0, st>>>(a);
    else if (ch <= 32) k_quant_block<SRC, 8><<<grid(1), kThreads, 0, st>>>(a);
    else if (ch <= 64) k_quant_block<SRC, 16><<<grid(1), kThreads, 0, st>>>(a);
    else k_quant_rows<SRC, 0><<<grid(kRows), kThreads, 0, st>>>(a);
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
