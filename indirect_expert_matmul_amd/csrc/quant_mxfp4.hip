// The launch of moe_quantize_mxfp4.
#include "quant_mxfp4.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <bool BF16>
__global__ __launch_bounds__(kThreads) void k_quant_mxfp4(QuantFp4Args a) {
    quantize_mxfp4_blocks<BF16, kThreads>(a, blockIdx.x);
}

}  // namespace

hipError_t launch_quant_mxfp4(const QuantFp4Args& a, hipStream_t st) {
    const int64_t grid = quant_fp4_grid(a, kThreads);
    if (grid <= 0) return hipSuccess;
    if (a.src_bf16) k_quant_mxfp4<true><<<(unsigned)grid, kThreads, 0, st>>>(a);
    else k_quant_mxfp4<false><<<(unsigned)grid, kThreads, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace moe
