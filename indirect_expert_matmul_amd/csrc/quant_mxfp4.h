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
// Memory bound: a wave reads 1 KB at a time, each lane 16 bytes, so a block's maximum is a
// few lane shuffles (4 lanes of bf16, 8 of float32) and every access of the wave, the
// codes' 2 or 4 bytes a lane included, is one contiguous run. Each thread has kU such
// pieces in flight. With values, read and written: 92160 x 2880 float32 372 us, 6.1 TB/s;
// 4096 x 2880 bf16 10.2 us, 5.2 TB/s.
// Used by a launch of its own (moe_quantize_mxfp4) and by the row-id pass's first launch, whose
// further thread blocks quantize a call's activations.
#pragma once
#include "moe_internal.h"

namespace moe {

constexpr int kQuantFp4Pieces = 4;   // 16-byte pieces per thread
// Blocks of 32 columns that one thread block takes.
inline constexpr int quant_fp4_per(bool bf16, int threads) { return threads / (bf16 ? 4 : 8) * kQuantFp4Pieces; }
inline int64_t quant_fp4_grid(const QuantFp4Args& a, int threads) {
    const int per = quant_fp4_per(a.src_bf16, threads);
    return (a.rows * (a.K >> 5) + per - 1) / per;
}

// Thread block `block` of THREADS threads: its quant_fp4_per(BF16, THREADS) blocks of 32.
template <bool BF16, int THREADS>
__device__ __forceinline__ void quantize_mxfp4_blocks(const QuantFp4Args& a, int64_t block) {
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    constexpr int kU = kQuantFp4Pieces;
    constexpr int LANES = BF16 ? 4 : 8;                        // lanes per block of 32
    constexpr int PER = THREADS / LANES;                      // blocks per piece row
    const int64_t base = block * (PER * kU) + threadIdx.x / LANES;
    const uint32_t KB = (uint32_t)(a.K >> 5);
    const int64_t total = a.rows * KB;                         // < 2^31
    const int sub = threadIdx.x % LANES;
    i32x4 x[kU];
#pragma unroll
    for (int u = 0; u < kU; u++) {
        const int64_t blk = min(base + u * PER, total - 1);    // spare lanes repeat the last block
        x[u] = __builtin_nontemporal_load((const i32x4*)a.src + blk * LANES + sub);
    }
#pragma unroll
    for (int u = 0; u < kU; u++) {
        const int64_t blk = base + u * PER;
        uint32_t top = 0;   // largest magnitude as bits: NaN and infinity sort above all numbers
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t w = (uint32_t)x[u][i];
            if constexpr (BF16) top = max(top, max((w << 16) & 0x7fffffffu, w & 0x7fff0000u));
            else top = max(top, w & 0x7fffffffu);
        }
#pragma unroll
        for (int m = 1; m < LANES; m <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
        const int field = (int)(top >> 23);
        const bool bad = field == 255;
        const uint32_t byte = bad ? 255u : (uint32_t)max(field - 2, 0);
        // the scale as a float32: subnormal 2^-127 for byte 0
        const float scale = __uint_as_float(byte ? byte << 23 : 0x00400000u);
        uint32_t q = 0;
        if constexpr (BF16) {
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, (uint32_t)x[u][0]), scale, 0);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, (uint32_t)x[u][1]), scale, 1);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, (uint32_t)x[u][2]), scale, 2);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, (uint32_t)x[u][3]), scale, 3);
        } else {
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __int_as_float(x[u][0]), __int_as_float(x[u][1]), scale, 0);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __int_as_float(x[u][2]), __int_as_float(x[u][3]), scale, 1);
        }
        if (bad) q = 0;
        if (blk >= total) continue;
        int64_t cb = blk;        // where the block's codes and scale byte go, in blocks
        int64_t sb = blk;
        if (a.padded) {
            const uint32_t r = (uint32_t)blk / KB, b = (uint32_t)blk - r * KB;
            const uint32_t KBc = (KB + 3) & ~3u;   // blocks in whole stages
            cb = r * (fp4_code_row(a.K) / 16) + b;
            sb = r * fp4_scale_row(a.K) + b;
            if (b == KB - 1)
                for (uint32_t p = 1; p < KBc - b; p++) {
                    if constexpr (BF16) ((uint32_t*)a.q)[(cb + p) * LANES + sub] = 0;
                    else ((uint16_t*)a.q)[(cb + p) * LANES + sub] = 0;
                    if (sub == 0) a.s[sb + p] = 127;
                }
        }
        if constexpr (BF16) ((uint32_t*)a.q)[cb * LANES + sub] = q;
        else ((uint16_t*)a.q)[cb * LANES + sub] = (uint16_t)q;
        if (sub == 0) a.s[sb] = (uint8_t)byte;
        if (a.values) {
            i32x4 y;
            const uint32_t nan = BF16 ? 0x7fc07fc0u : 0x7fc00000u;
            if constexpr (BF16) {
                y[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0));
                y[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1));
                y[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2));
                y[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3));
            } else {
                const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 0);
                const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, scale, 1);
                y = i32x4{__float_as_int(lo[0]), __float_as_int(lo[1]), __float_as_int(hi[0]), __float_as_int(hi[1])};
            }
            if (bad) y = i32x4{(int)nan, (int)nan, (int)nan, (int)nan};
            __builtin_nontemporal_store(y, (i32x4*)a.values + blk * LANES + sub);
        }
    }
}

}  // namespace moe
