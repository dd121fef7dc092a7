// GEMV (decode) path of MXFP4 activations and MXFP4 experts (act_quant = 2) for small
// batches: gate/up with silu(gate) * up, down and mul_mat_id, over the selected experts
// only, the shared experts in the same launch.
//
// Decode is a weight stream: the selected experts' codes are read once. The block scaled
// MFMA makes the arithmetic free: v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 weight rows with
// the activations of up to 16 slots of their expert, so a wave that reads 1 KB of codes
// issues one instruction for it whatever the number of slots.
//   * A unit is one distinct expert (found from ids by wave ballots, no row-id launch) and
//     16 rg of its rows; its columns are split over kp waves, whose partial sums meet in LDS
//     and are added in a fixed order.
//   * Codes go straight into the MFMA's registers, 16 bytes a lane: a load covers 64
//     contiguous bytes of 16 rows. A superstep is 512 columns, four MFMAs, whose scale bytes
//     of a row are one 16-byte load; step j of lane group g takes byte g of word j.
//   * Activations are quantized where they are used (a separate pass over x would cost a
//     launch): the wave reads a slot's 512 columns with one load per lane, finds each block's
//     maximum over 4 lanes, and puts the codes and scale bytes into LDS, from where they come
//     back in the MFMA's layout. (Each lane reading its own blocks took 16 loads a superstep,
//     four of them one after the other.)
//   * A block that does not sum keeps the partial sums of one pass (up to 16 slots of its expert)
//     in LDS, so that two to four blocks share a CU (room for every slot of the call left one: 64
//     slots of 2048 x 7168 took 130 us, then 106; 64 of 4096 x 4096, 8 experts, 32, then 23).
//   * A wave holds one group's codes and no next ones: other waves cover the loads. (Loading a
//     group ahead took 141 and 221 registers instead of 109 and 156: gate/up of one token, 2880 x
//     2880, 4 experts, 21 us instead of 15; 64 slots of 2048 x 7168 106 instead of 92.)
//   * The weighted sum over a token's slots is fused where one block can take all the experts
//     of its 16 rows in a few rounds of its waves (one token 2880 x 2880, 4 experts: 11.8 us, against
//     9.1 and 4 for the sum's launch); else the per-slot rows go through the workspace to the
//     reduce kernel.
// Measured: 4 experts of 2880 x 2880 9.3 us (17.6 MB: the launch and two memory
// round trips, the ids and then codes and activations), 8
// tokens x 4 of 32 28 us (3.3 TB/s, one round of blocks), 64 slots of 128 experts of 2048 x 7168
// 92 us (4.4 TB/s).
#include <algorithm>

#include "moe_internal.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 8;        // waves of a block at most
constexpr int kFuseItems = 16;   // work items of a block that sums the slots at most
constexpr int kXRow = 256 + 16;  // a slot's superstep in LDS: codes, scale bytes
// Waves that fill the chip (8 a CU): units of more rows once there are so many (with 4096 for it,
// 64 slots of 4096 x 4096, 8 experts, took 28 us instead of 23.7; with 1024 one token 10.1 for 9.1).
constexpr int kManyWaves = 2048;

__device__ __forceinline__ i32x8 operand(i32x4 v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

template <class V>
__device__ __forceinline__ V load_unaligned(const uint8_t* p) {
    V v;
    __builtin_memcpy(&v, p, sizeof(V));
    return v;
}

// This lane's 8 columns of a superstep; the block of 32 is lanes 4 i .. 4 i + 3.
template <bool F32>
struct Cols {
    i32x4 v[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ uint32_t quantize(const Cols<F32>& x, uint32_t& byte) {
    uint32_t top = 0;   // largest magnitude as bits: NaN and infinity sort above all numbers
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); i++) {
        const uint32_t w = (uint32_t)x.v[i / 4][i % 4];
        if constexpr (F32) top = max(top, w & 0x7fffffffu);
        else top = max(top, max((w << 16) & 0x7fffffffu, w & 0x7fff0000u));
    }
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2));
    const int field = (int)(top >> 23);
    byte = field == 255 ? 255u : (uint32_t)max(field - 2, 0);
    const float scale = __uint_as_float(byte ? byte << 23 : 0x00400000u);   // 2^-127 for byte 0
    uint32_t c = 0;
    if constexpr (F32) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __int_as_float(x.v[0][0]), __int_as_float(x.v[0][1]), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __int_as_float(x.v[0][2]), __int_as_float(x.v[0][3]), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __int_as_float(x.v[1][0]), __int_as_float(x.v[1][1]), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __int_as_float(x.v[1][2]), __int_as_float(x.v[1][3]), scale, 3);
    } else {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)x.v[0][0]), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)x.v[0][1]), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)x.v[0][2]), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, (uint32_t)x.v[0][3]), scale, 3);
    }
    return byte == 255u ? 0u : c;
}

// A lane's part of a superstep of one weight row: blocks 4 j + g of its 16, and the row's 16
// scale bytes.
struct Piece {
    i32x4 q[4], s;
};
// q, s: the row (at least 4 blocks); b: the superstep's first block. Blocks past the row's end read block 0 (the
// activation codes there are 0), words past it its last 4 bytes.
__device__ __forceinline__ Piece load_piece(const uint8_t* q, const uint8_t* s, int b, int g, int KB) {
    Piece p;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const int at = b + 4 * j + g;
        p.q[j] = __builtin_nontemporal_load((const i32x4*)(q + (at < KB ? at : 0) * 16));
    }
    if (b + 16 <= KB) {
        p.s = load_unaligned<i32x4>(s + b);
    } else {
#pragma unroll
        for (int j = 0; j < 4; j++) p.s[j] = load_unaligned<int>(s + min(b + 4 * j, KB - 4));
    }
    return p;
}
// Scale byte of step j, in byte 0 (past the row's end: 0, a finite scale).
__device__ __forceinline__ int piece_scale(const Piece& p, int j, int b, int g, int KB) {
    uint32_t w = (uint32_t)p.s[j];
    const int past = b + 4 * j - (KB - 4);
    if (past > 0) w = past < 4 ? w >> (8 * past) : 0u;
    return (int)(w >> (8 * g));
}

template <int MODE, bool F32, bool FUSE>
__global__ __launch_bounds__(64 * kWaves) void k_decode_fp4(DecFp4Args a) {
    // partial sums [slots][kp][rg][16 rows] (gate/up: twice), then each wave's quantized activations;
    // slots: all of them in a block that sums, else those of one pass
    extern __shared__ __attribute__((aligned(16))) float s_part[];
    __shared__ int s_list[kWaves][kDecFp4Slots];                 // per wave: the unit's slots
    __shared__ uint8_t s_mine[FUSE ? kDecFp4Slots : 1];              // routed slots with an expert
    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, g4 = lane >> 4;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6), waves = (int)blockDim.x >> 6;
    const int n = a.T * a.k, n_all = n + a.sw.n_mat * a.T;
    const int row_first = (int)blockIdx.x * 16 * a.rg;
    const int y = (int)blockIdx.y;
    constexpr int kRows = MODE == 1 ? 32 : 16;
    uint8_t* s_x = (uint8_t*)(s_part + (FUSE ? n_all : a.xs) * a.kp * a.rg * kRows) +
                   wv * 2 * a.xs * kXRow;   // [2 supersteps][xs slots]
    // row r (of the block's 16 rg) of a slot's product
    auto total = [&](int at, int r, int m) -> float {
        float v = 0.f;
        for (int p = 0; p < a.kp; p++)
            v += s_part[(((int64_t)at * a.kp + p) * a.rg + (r >> 4)) * kRows + 16 * m + (r & 15)];
        return v;
    };
    const int rows = 16 * a.rg, shift = a.rg == 1 ? 4 : a.rg == 2 ? 5 : 6;   // rg: 1, 2 or 4

    // each lane its slot's expert; lanes with the same one; the first lane of each distinct expert
    int my_e = lane < n ? a.ids[lane] : -1;
    if (my_e >= a.E) my_e = -1;
    const uint64_t valid = __ballot(my_e >= 0);
    uint64_t same = valid;
    for (int v = a.E - 1, bit = 0; v >> bit; bit++) {   // by the bits of the ids
        const uint64_t set = __ballot((my_e >> bit) & 1);
        same &= (my_e >> bit) & 1 ? set : ~set;
    }
    const uint64_t firsts = __ballot(my_e >= 0 && (same & ((1ull << lane) - 1)) == 0);
    const int nd = __popcll(firsts);
    // Work items of a wave: (unit, part p of its columns). A block that does not sum has one unit,
    // expert number y of the distinct ones or shared expert y - d_max, and a wave for each part.
    if (!FUSE && y < a.d_max && y >= nd && y > 0) return;
    if (FUSE) {
        for (int i = tid; i < n; i += (int)blockDim.x) s_mine[i] = (valid >> i) & 1;
    }
    const int units = FUSE ? nd + a.sw.n_mat : (y < a.d_max ? (y < nd) : 1);
    for (int it = wv; it < units * a.kp; it += waves) {
        const int u = FUSE ? it / a.kp : y, p = FUSE ? it - u * a.kp : it;
        const bool sh = FUSE ? u >= nd : y >= a.d_max;
        const int sj = u - (FUSE ? nd : a.d_max);   // shared expert
        const DecFp4Weights& W = sh ? a.sw : a.rw;
        int e;
        uint64_t mask;   // the unit's slots (shared: tokens)
        if (sh) {
            e = sj;
            mask = a.T >= 64 ? ~0ull : (1ull << a.T) - 1;
        } else {
            uint64_t m = firsts;
            for (int d = u; d > 0; d--) m &= m - 1;
            e = __builtin_amdgcn_readlane(my_e, __builtin_ctzll(m));
            mask = __ballot(my_e == e);
        }
        const int cnt = __popcll(mask);
        if ((mask >> lane) & 1) s_list[wv][__popcll(mask & ((1ull << lane) - 1))] = lane;
        __builtin_amdgcn_wave_barrier();
        const int N = W.N, KB = W.K >> 5;
        if (row_first >= N) continue;
        const int groups = min(a.rg, (N - row_first + 15) >> 4);
        const int nss = (KB + 15) >> 4, per = (nss + a.kp - 1) / a.kp;
        const int ss0 = p * per, ss1 = min(ss0 + per, nss);
        struct Weights {
            Piece a[2], b[2];   // two supersteps; b: the up rows
        };
        auto load = [&](Weights& w, int rg, int ss) __attribute__((always_inline)) {
            const int64_t row = (int64_t)e * N + min(row_first + 16 * rg + r16, N - 1);
#pragma unroll
            for (int z = 0; z < 2; z++) {
                const int b = 16 * min(ss + z, ss1 - 1);
                w.a[z] = load_piece(W.q1 + row * (KB * 16), W.s1 + row * KB, b, g4, KB);
                if (MODE == 1) w.b[z] = load_piece(W.q2 + row * (KB * 16), W.s2 + row * KB, b, g4, KB);
            }
        };
        // xs slots at a time (more of one expert read its rows again)
        uint64_t left = mask;
        for (int sg = 0; sg < cnt; sg += a.xs) {
            const int some = min(cnt - sg, a.xs);
            const bool on = r16 < some;
            const int slot = on ? s_list[wv][sg + r16] : 0;
            const int at = !FUSE ? r16 : sh ? n + sj * a.T + slot : slot;
            float* part = s_part + ((int64_t)at * a.kp + p) * a.rg * kRows + 4 * g4;
            uint64_t here = left;
            // two supersteps at a time: all of the wave's up to K = 8192
            for (int ss = ss0; ss < ss1 || ss == ss0; ss += 2) {
                Weights w;
                if (ss0 < ss1) load(w, 0, ss);
                here = left;
                for (int i = 0; i < some; i += 2) {   // two slots' activations at a time
                    Cols<F32> x[2][2];
#pragma unroll
                    for (int d = 0; d < 2; d++) {
                        const int s = here ? __builtin_ctzll(here) : 0;   // wave-uniform
                        if (i + d < some) here &= here - 1;
                        const int64_t xr = sh ? (int64_t)sj * a.sact_jstride + s : a.act_B == 1 ? s / a.k : s;
                        const char* xp = (const char*)(sh ? a.sact : a.act) + xr * W.K * (F32 ? 4 : 2);
#pragma unroll
                        for (int z = 0; z < 2; z++) {
                            const int c0 = 512 * (ss + z) + 8 * lane;
                            const i32x4* src = (const i32x4*)(xp + (int64_t)(c0 < W.K ? c0 : 0) * (F32 ? 4 : 2));
#pragma unroll
                            for (int r = 0; r < (F32 ? 2 : 1); r++) x[d][z].v[r] = src[r];
                        }
                    }
#pragma unroll
                    for (int d = 0; d < 2; d++)
#pragma unroll
                        for (int z = 0; z < 2; z++) {
                            uint32_t byte;
                            uint32_t q = quantize(x[d][z], byte);
                            if (512 * (ss + z) + 8 * lane >= W.K) {   // past the row's end: 0 under scale 1
                                q = 0;
                                byte = 127;
                            }
                            if (i + d < some) {
                                uint8_t* o = s_x + (z * a.xs + i + d) * kXRow;
                                ((uint32_t*)o)[lane] = q;
                                if ((lane & 3) == 0) o[256 + (lane >> 2)] = (uint8_t)byte;
                            }
                        }
                }
                __builtin_amdgcn_wave_barrier();
                for (int rg = 0; rg < groups; rg++) {
                    if (rg > 0 && ss0 < ss1) load(w, rg, ss);
                    f32x4 acc[MODE + 1];
#pragma unroll
                    for (int m = 0; m <= MODE; m++) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int z = 0; z < 2; z++) {
                        if (ss + z >= ss1) break;
                        const int b = 16 * (ss + z);
                        // lanes without a slot take the last one's: their results go nowhere
                        const uint8_t* o = s_x + (z * a.xs + min(r16, some - 1)) * kXRow;
                        const i32x4 xs = *(const i32x4*)(o + 256);
#define STEP(j)                                                                                            \
    {                                                                                                      \
        const i32x8 xq = operand(*(const i32x4*)(o + (4 * j + g4) * 16));                                  \
        const int sx = (int)((uint32_t)xs[j] >> (8 * g4));                                                 \
        acc[0] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w.a[z].q[j]), xq, acc[0], 4, 4, \
                                                                  0, piece_scale(w.a[z], j, b, g4, KB), 0, sx); \
        if (MODE == 1)                                                                                     \
            acc[MODE] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(                                  \
                operand(w.b[z].q[j]), xq, acc[MODE], 4, 4, 0, piece_scale(w.b[z], j, b, g4, KB), 0, sx);   \
    }
                        STEP(0)
                        STEP(1)
                        STEP(2)
                        STEP(3)
#undef STEP
                    }
                    // element u of lane l: weight row 4 (l / 16) + u, slot l % 16
                    if (on) {
                        float* d = part + rg * kRows;
#pragma unroll
                        for (int m = 0; m <= MODE; m++) {
                            if (ss > ss0) acc[m] += *(const f32x4*)(d + 16 * m);
                            *(f32x4*)(d + 16 * m) = acc[m];
                        }
                    }
                }
                __builtin_amdgcn_wave_barrier();
            }
            left = here;
            if (!FUSE) {   // all the block's waves are at this pass of the one unit
                __syncthreads();
                for (int i = tid; i < some * rows; i += (int)blockDim.x) {
                    const int z = i >> shift, r = i & (rows - 1), s = s_list[wv][sg + z];
                    if (row_first + r >= N) continue;
                    float v = total(z, r, 0);
                    if (MODE == 1) v = v / (1.0f + expf(-v)) * total(z, r, MODE);
                    ((sh ? a.sout + ((int64_t)sj * a.T + s) * N : a.out + (int64_t)s * N) + row_first)[r] = v;
                }
                __syncthreads();
            }
        }
    }
    if (FUSE) {   // out_tok[t] = sum over s ascending of route_w * row, then the shared experts
        __syncthreads();
        for (int i = tid; i < a.T * rows; i += (int)blockDim.x) {
            const int t = i >> shift, r = i & (rows - 1);
            if (row_first + r >= a.rw.N) continue;
            float v = 0.f;
            for (int s = 0; s < a.k; s++)
                if (s_mine[t * a.k + s]) v = fmaf(a.route_w[t * a.k + s], total(t * a.k + s, r, 0), v);
            for (int j = 0; j < a.sw.n_mat; j++) v += total(n + j * a.T + t, r, 0);
            a.out_tok[(int64_t)t * a.rw.N + row_first + r] = v;
        }
        return;
    }
    if (MODE == 0 && y == 0) {   // rows of slots whose id is out of range are zero
        uint64_t bad = ~valid & (n >= 64 ? ~0ull : (1ull << n) - 1);
        for (; bad; bad &= bad - 1)
            if (tid < rows && row_first + tid < a.rw.N) a.out[(int64_t)__builtin_ctzll(bad) * a.rw.N + row_first + tid] = 0.f;
    }
}

template <int MODE, bool F32, bool FUSE = false>
hipError_t launch(const DecFp4Args& a, dim3 grid, int waves, size_t lds, hipStream_t st) {
    static PerDeviceOnce cap;
    if (const hipError_t e = set_lds_cap(cap, (const void*)k_decode_fp4<MODE, F32, FUSE>, kDecFp4Lds)) return e;
    k_decode_fp4<MODE, F32, FUSE><<<grid, 64 * waves, lds, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_decode_fp4(const DecFp4Args& a0, hipStream_t st) {
    DecFp4Args a = a0;
    const int n = a.T * a.k, n_all = n + a.sw.n_mat * a.T;
    const int n_rows = a.sw.n_mat && a.sw.N > a.rw.N ? a.sw.N : a.rw.N;
    const int K = a.sw.n_mat && a.sw.K > a.rw.K ? a.sw.K : a.rw.K;
    const int nss = (K + 511) / 512;   // supersteps
    const int d_max = n < a.E ? n : a.E;
    // slots of one expert at a time: those of distinct ids (others take another round)
    a.xs = a.T < kDecFp4Pass ? a.T : kDecFp4Pass;
    const size_t per_wave = (size_t)2 * a.xs * kXRow;
    const int units = d_max + a.sw.n_mat;
    // two supersteps a wave; rows per unit: up to four groups of 16 while that leaves enough waves
    int kp = (nss + 1) / 2;
    if (kp > kWaves) kp = kWaves;
    a.rg = 1;
    while (!a.fuse && a.rg < 4 && (int64_t)units * kp * ((n_rows + 32 * a.rg - 1) / (32 * a.rg)) >= kManyWaves) a.rg *= 2;
    int waves = kp;
    a.d_max = d_max;
    if (a.fuse) {   // all experts of 16 rows in one block
        waves = units * kp < kWaves ? units * kp : kWaves;
    }
    auto lds_of = [&]() {
        return (size_t)(a.fuse ? n_all : a.xs) * a.rg * 16 * 4 * (a.mode == 1 ? 2 : 1) * kp + per_wave * waves;
    };
    while (lds_of() > (size_t)kDecFp4Lds) {
        if (a.fuse && waves > 4) waves--;
        else if (kp > 1) kp--;
        else return hipErrorInvalidConfiguration;
        if (!a.fuse) waves = kp;
    }
    a.kp = kp;
    const dim3 grid((unsigned)((n_rows + 16 * a.rg - 1) / (16 * a.rg)), (unsigned)(a.fuse ? 1 : units));
    const size_t lds = lds_of();
    if (a.mode == 1) return launch<1, false>(a, grid, waves, lds, st);   // x is bf16
    if (a.fuse) return a.f32 ? launch<0, true, true>(a, grid, waves, lds, st) : launch<0, false, true>(a, grid, waves, lds, st);
    return a.f32 ? launch<0, true>(a, grid, waves, lds, st) : launch<0, false>(a, grid, waves, lds, st);
}

bool decode_fp4_fuses(int64_t n, int64_t E, int64_t S, int64_t K) {
    const int64_t kp = std::min<int64_t>(((K + 511) / 512 + 1) / 2, kWaves);
    return (std::min(n, E) + S) * kp <= kFuseItems;
}

}  // namespace moe
