// Quantization to MXFP4: blocks of 32 columns -> 32 E2M1 codes and one E8M0 scale byte.
//
//     byte = max(expfield(max|x|) - 2, 0)        (expfield: the float32 exponent field)
//     code = nearest E2M1 to x * 2^(127 - byte), ties to the even code, saturated at 6
//
// expfield - 127 = floor(log2 m) for normal m, and E2M1's largest exponent is 2, so the
// largest magnitude of a block lands in [4, 8). Subnormal maxima have field 0 and take
// byte 0 (2^-127), as do all blocks with fields 0 to 2. v_cvt_scalef32_pk_fp4_* divides
// by the scale and rounds as the code line says, for every finite input and scale
// (checked value by value against the comparison form over all exponents, ties and
// subnormals). A field of 255 (infinity or NaN) makes the whole block NaN.
//
// First form: one thread per block.
#include "moe_internal.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

// Value of E2M1 code c (0..15) in units of the scale.
__device__ __forceinline__ float e2m1(int c) {
    const int m = c & 7;
    const float v = m < 4 ? 0.5f * m : (m < 6 ? (float)(m - 2) : (float)(2 * m - 8));
    return (c & 8) ? -v : v;
}

template <bool BF16>
__global__ __launch_bounds__(kThreads) void k_quant_mxfp4(QuantFp4Args args) {
    const bool second = (int64_t)blockIdx.x >= args.blocks0;
    const QuantFp4Part& a = args.part[second ? 1 : 0];
    const int64_t blk = ((int64_t)blockIdx.x - (second ? args.blocks0 : 0)) * kThreads + threadIdx.x;
    const int64_t KB = a.K >> 5;
    if (blk >= a.rows * KB) return;
    float v[32];
    if constexpr (BF16) {
        const i32x4* src = (const i32x4*)((const uint16_t*)a.src + blk * 32);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const i32x4 w = src[i];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                v[8 * i + 2 * j] = __builtin_bit_cast(float, (uint32_t)w[j] << 16);
                v[8 * i + 2 * j + 1] = __builtin_bit_cast(float, (uint32_t)w[j] & 0xffff0000u);
            }
        }
    } else {
        const f32x4* src = (const f32x4*)((const float*)a.src + blk * 32);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const f32x4 w = src[i];
#pragma unroll
            for (int j = 0; j < 4; j++) v[4 * i + j] = w[j];
        }
    }
    uint32_t top = 0;   // largest magnitude as bits: NaN and infinity sort above all numbers
#pragma unroll
    for (int i = 0; i < 32; i++) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    const int field = (int)(top >> 23);
    const bool bad = field == 255;
    const int byte = bad ? 255 : max(field - 2, 0);
    // the scale as a float32: subnormal 2^-127 for byte 0
    const float scale = __uint_as_float(byte ? (uint32_t)byte << 23 : 0x00400000u);
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        uint32_t p = 0;
        p = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(p, v[8 * i], v[8 * i + 1], scale, 0);
        p = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(p, v[8 * i + 2], v[8 * i + 3], scale, 1);
        p = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(p, v[8 * i + 4], v[8 * i + 5], scale, 2);
        p = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(p, v[8 * i + 6], v[8 * i + 7], scale, 3);
        q[i] = bad ? 0u : p;
    }
    *(i32x4*)(a.q + blk * 16) = i32x4{(int)q[0], (int)q[1], (int)q[2], (int)q[3]};
    a.s[blk] = (uint8_t)byte;
    if (a.values) {
#pragma unroll
        for (int i = 0; i < 32; i++) {
            const float y = bad ? __uint_as_float(0x7fc00000u) : e2m1((q[i >> 3] >> (4 * (i & 7))) & 15) * scale;
            if constexpr (BF16) ((uint16_t*)a.values)[blk * 32 + i] = (uint16_t)(__float_as_uint(y) >> 16);
            else ((float*)a.values)[blk * 32 + i] = y;
        }
    }
}

}  // namespace

hipError_t launch_quant_mxfp4(const QuantFp4Args& a0, hipStream_t st) {
    QuantFp4Args a = a0;
    int64_t grid[2] = {0, 0};
    for (int i = 0; i < a.n_part; i++) grid[i] = (a.part[i].rows * (a.part[i].K >> 5) + kThreads - 1) / kThreads;
    a.blocks0 = grid[0];
    const int64_t total = grid[0] + grid[1];
    if (total <= 0) return hipSuccess;
    if (a.src_bf16) k_quant_mxfp4<true><<<(unsigned)total, kThreads, 0, st>>>(a);
    else k_quant_mxfp4<false><<<(unsigned)total, kThreads, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace moe
