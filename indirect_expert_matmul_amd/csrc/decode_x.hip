// GEMV (decode) path of mul_mat_id with bf16, f16 and int8 experts, for small batches: the
// selected experts' rows are read once, straight from ids (no row-id launch), and multiplied with
// the activations of their slots.
//
//   * A wave takes kR rows of one distinct expert (found from ids by wave ballots), 16 bytes a lane
//     and load: 1 KB in a row for each of kR rows, the next one asked for when one has been used. That
//     keeps few registers, and so many waves, busy: two loads of a row under way took 160 registers instead
//     of 130 (8 tokens, 6 of 64 experts of 2048 x 1408, weighted 46 us instead of 36), three 200. Its lanes'
//     sums meet in a tree of fixed order.
//   * Up to kP of the expert's slots are done at a time; more read the rows again, from the caches.
//   * 16-bit elements are widened and summed by float32 FMAs (the instructions for pairs of them
//     need not keep subnormals). int8: v_dot4_i32_i8 on the codes. A single token's are made by every
//     block, in LDS, while its first weights are on their way; more tokens' by a launch of their own.
//   * The weighted sum over a token's slots (FUSE) is taken in the same launch: a block has kR
//     rows of every selected expert, its waves an expert each in turn, and the slots' values in LDS.
// Bound by memory: the selected experts' rows, once. Measured (one MI355X, per call): one token with 4 experts of 2880 x
// 2880 bf16 12.3 us (5.4 TB/s; of int8 10.2, an empty call's time); 8 tokens with 6 of 64 experts of 2048 x 1408 bf16,
// weighted, 36 to 37 us (5.5 TB/s); 8 tokens with 8 of 128 experts of 2048 x 7168 bf16 213 us (7.0 TB/s), int8 125.
#include <type_traits>

#include "quant_rows.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kR = 4;         // rows of a wave
constexpr int kP = 4;         // slots of a pass at most
constexpr int kRowWaves = 4;  // waves of a block that does not sum
constexpr int kSumWaves = 8;  // of one that does, at most

// One 16-byte piece as float32 numbers.
template <int TYPE>
__device__ __forceinline__ void widen(const i32x4& v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t w = (uint32_t)v[i];
        if constexpr (TYPE == kElemBf16) {
            f[2 * i] = __uint_as_float(w << 16);
            f[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
        } else {
            f[2 * i] = (float)__builtin_bit_cast(_Float16, (uint16_t)w);
            f[2 * i + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16));
        }
    }
}

// Sums of four values over the wave: lane l gets that of value (l / 32) + 2 (l / 16 % 2).
template <class V>
__device__ __forceinline__ V sum4(V r0, V r1, V r2, V r3, int lane) {
    const bool hi = lane & 32, mid = lane & 16;
    V a = (hi ? r1 : r0) + __shfl_xor(hi ? r0 : r1, 32);
    const V b = (hi ? r3 : r2) + __shfl_xor(hi ? r2 : r3, 32);
    a = (mid ? b : a) + __shfl_xor(mid ? a : b, 16);
#pragma unroll
    for (int m = 8; m; m >>= 1) a += __shfl_xor(a, m);
    return a;
}

// Eight neighbours of a row of activations (16-byte aligned).
__device__ __forceinline__ void src8(const void* p, int32_t type, int64_t i, float (&f)[8]) {
    if (type == kElemF32) {
        const f32x4 a = *(const f32x4*)((const float*)p + i), b = *(const f32x4*)((const float*)p + i + 4);
#pragma unroll
        for (int u = 0; u < 4; u++) {
            f[u] = a[u];
            f[4 + u] = b[u];
        }
    } else {
        const i32x4 v = *(const i32x4*)((const uint16_t*)p + i);
        if (type == kElemBf16) widen<kElemBf16>(v, f);
        else widen<kElemF16>(v, f);
    }
}
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// TYPE: of the experts (and, 16-bit, of the activations). MAKE: int8 codes are made here, else they are given.
template <int TYPE, bool FUSE, bool MAKE>
__global__ __launch_bounds__(64 * kSumWaves) void k_decode_x(DecXArgs a) {
    constexpr bool I8 = TYPE == kElemI8;
    constexpr int EC = I8 ? 16 : 8, STEP = 64 * EC;   // columns of a lane's load, of a wave's
    using Acc = std::conditional_t<I8, int, float>;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    // MAKE: codes of xs rows, their scales, the waves' maxima; FUSE: kR values of every slot
    int8_t* s_q = (int8_t*)smem;
    float* s_d = (float*)(smem + (MAKE ? (size_t)a.xs * a.K : 0));
    uint32_t* s_top = (uint32_t*)s_d + (MAKE ? kDecXSlots : 0);
    float* s_y = (float*)s_top + (MAKE ? kDecXSlots * kSumWaves : 0);
    const int tid = threadIdx.x, lane = tid & 63, waves = (int)blockDim.x >> 6;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = a.T * a.k, K = a.K, N = a.N;
    const int unit = (int)blockIdx.y;
    const int row0 = (int)blockIdx.x * kR * (FUSE ? 1 : kRowWaves) + (FUSE ? 0 : kR * wv);

    // each lane its slot's expert; the first lane of each distinct one
    int my_e = lane < n ? a.ids[lane] : -1;
    if (my_e < 0 || my_e >= a.E) my_e = -1;
    const uint64_t valid = __ballot(my_e >= 0);
    uint64_t same = valid;
    for (int v = a.E - 1, bit = 0; v >> bit; bit++) {   // by the bits of the ids
        const uint64_t set = __ballot((my_e >> bit) & 1);
        same &= (my_e >> bit) & 1 ? set : ~set;
    }
    const uint64_t firsts = __ballot(my_e >= 0 && (same & ((1ull << lane) - 1)) == 0);
    const int nd = __popcll(firsts);
    if (!FUSE && unit >= nd && unit > 0) return;

    auto src_row = [&](int slot) -> int64_t { return a.act_B == 1 ? slot / a.k : slot; };
    // Codes of cnt rows of activations, row_of(i) each, by all waves of the block.
    auto make = [&](int cnt, auto row_of) {
        for (int i = 0; i < cnt; i++) {
            const int64_t first = row_of(i) * K;
            uint32_t top = 0;
            for (int c = 8 * tid; c < K; c += 8 * (int)blockDim.x) {
                float f[8];
                src8(a.src, a.src_type, first + c, f);
#pragma unroll
                for (int u = 0; u < 8; u++) top = max(top, __float_as_uint(f[u]) & 0x7fffffffu);
            }
#pragma unroll
            for (int m = 32; m; m >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
            if (lane == 0) s_top[i * waves + wv] = top;
        }
        lds_barrier();
        for (int i = 0; i < cnt; i++) {
            const int64_t first = row_of(i) * K;
            uint32_t top = 0;
            for (int v = 0; v < waves; v++) top = max(top, s_top[i * waves + v]);
            const float d = quant_scale(top), r = 1.0f / d;
            const bool some = d > 0.f, fast = d > kQuantMinFast;
            for (int c = 8 * tid; c < K; c += 8 * (int)blockDim.x) {
                float f[8];
                src8(a.src, a.src_type, first + c, f);
                uint32_t w[2] = {0, 0};
#pragma unroll
                for (int u = 0; u < 8; u++) w[u >> 2] |= ((uint32_t)quant_code(f[u], d, r, fast) & 255u) << (8 * (u & 3));
                *(uint2*)(s_q + (size_t)i * K + c) = some ? make_uint2(w[0], w[1]) : make_uint2(0, 0);
            }
            if (tid == 0) s_d[i] = d;
        }
        lds_barrier();
    };

    const uint8_t* w[kR];
    i32x4 wq[kR];
    // what a lane would read past the row's end is a piece of its beginning, and counts as zero
    auto load = [&](int r, int c0) __attribute__((always_inline)) -> i32x4 {
        const int64_t at = c0 + lane * EC < K ? (int64_t)c0 * (I8 ? 1 : 2) : -(int64_t)lane * 16;
        return __builtin_nontemporal_load((const i32x4*)(w[r] + at));
    };
    auto loads = [&](int c0) __attribute__((always_inline)) {
#pragma unroll
        for (int r = 0; r < kR; r++) wq[r] = load(r, c0);
    };
    auto expert_of = [&](int u) -> int {
        uint64_t m = firsts;
        for (int d = u; d > 0; d--) m &= m - 1;
        return __builtin_amdgcn_readlane(my_e, __builtin_ctzll(m));
    };
    auto rows_of = [&](int e) __attribute__((always_inline)) {
#pragma unroll
        for (int r = 0; r < kR; r++)
            w[r] = (const uint8_t*)a.W + ((int64_t)e * N + min(row0 + r, N - 1)) * K * (I8 ? 1 : 2) + lane * 16;
    };
    const int u0 = FUSE ? wv : unit;
    if (u0 < nd) {   // the first weights, before anything that takes time
        rows_of(expert_of(u0));
        loads(0);
    }
    if (FUSE && MAKE) make(a.xs, [](int i) { return (int64_t)i; });   // all rows of activations

    for (int u = u0; u < nd; u += FUSE ? waves : nd) {
        const int e = expert_of(u);
        uint64_t left = __ballot(my_e == e);   // the expert's slots
        const int64_t w0 = (int64_t)e * N;
        if (u != u0) {
            rows_of(e);
            loads(0);
        }
        for (bool again = false; left; again = true) {
            if (again) loads(0);
            int cnt = min(__popcll(left), kP);
            if (MAKE && !FUSE) cnt = min(cnt, a.xs);
            int slot[kP];
#pragma unroll
            for (int p = 0; p < kP; p++) {
                slot[p] = left ? __builtin_ctzll(left) : slot[p > 0 ? p - 1 : 0];
                if (p < cnt) left &= left - 1;
            }
            if (MAKE && !FUSE) {   // every wave of the block has the same slots
                if (again) lds_barrier();
                make(cnt, [&](int i) {
                    int s = slot[0];
#pragma unroll
                    for (int z = 1; z < kP; z++) s = i == z ? slot[z] : s;
                    return src_row(s);
                });
            }
            Acc acc[kP][kR];
#pragma unroll
            for (int p = 0; p < kP; p++)
#pragma unroll
                for (int r = 0; r < kR; r++) acc[p][r] = 0;
            auto run = [&](auto p_c) __attribute__((always_inline)) {
                constexpr int P = decltype(p_c)::value;
                const uint8_t* x[P];
#pragma unroll
                for (int p = 0; p < P; p++)
                    x[p] = MAKE ? (const uint8_t*)s_q + (size_t)(FUSE ? src_row(slot[p]) : min(p, cnt - 1)) * K
                                : (const uint8_t*)a.src + src_row(slot[p]) * K * (I8 ? 1 : 2);
                for (int c = 0; c < K; c += STEP) {
                    const bool in = c + lane * EC < K;
                    i32x4 xv[P];
#pragma unroll
                    for (int p = 0; p < P; p++) xv[p] = *(const i32x4*)(x[p] + (int64_t)(in ? c + lane * EC : 0) * (I8 ? 1 : 2));
                    if (c + STEP > K) {   // the row's end
#pragma unroll
                        for (int r = 0; r < kR; r++)
                            if (!in) wq[r] = i32x4{0, 0, 0, 0};
#pragma unroll
                        for (int p = 0; p < P; p++)
                            if (!in) xv[p] = i32x4{0, 0, 0, 0};
                    }
                    if constexpr (I8) {
#pragma unroll
                        for (int p = 0; p < P; p++)
#pragma unroll
                            for (int r = 0; r < kR; r++)
#pragma unroll
                                for (int i = 0; i < 4; i++) acc[p][r] = __builtin_amdgcn_sdot4(wq[r][i], xv[p][i], acc[p][r], false);
                    } else {
                        float wf[kR][8];
#pragma unroll
                        for (int r = 0; r < kR; r++) widen<TYPE>(wq[r], wf[r]);
#pragma unroll
                        for (int p = 0; p < P; p++) {
                            float xf[8];
                            widen<TYPE>(xv[p], xf);
#pragma unroll
                            for (int r = 0; r < kR; r++)
#pragma unroll
                                for (int i = 0; i < 8; i++) acc[p][r] = fmaf(wf[r][i], xf[i], acc[p][r]);
                        }
                    }
                    if (c + STEP < K) loads(c + STEP);
                }
            };
            if (cnt > 2) run(std::integral_constant<int, kP>{});
            else if (cnt == 2) run(std::integral_constant<int, 2>{});
            else run(std::integral_constant<int, 1>{});
            const int r = (lane >> 5) + 2 * ((lane >> 4) & 1);   // the row whose sum this lane gets
            const bool writer = (lane & 15) == 0 && row0 + r < N;
#pragma unroll
            for (int p = 0; p < kP; p++) {
                if (p >= cnt) break;
                const Acc s = sum4(acc[p][0], acc[p][1], acc[p][2], acc[p][3], lane);
                if (!writer) continue;
                float y;
                if constexpr (I8) {
                    const float d = !MAKE ? a.src_scale[src_row(slot[p])] : s_d[FUSE ? src_row(slot[p]) : p];
                    y = (float)s * (d * a.w_scale[w0 + row0 + r]);
                }
                else y = s;
                if (FUSE) s_y[slot[p] * kR + r] = y;
                else a.out[(int64_t)slot[p] * N + row0 + r] = y;
            }
        }
    }
    if (FUSE) {   // out_tok[t] = sum over s ascending of route_w * row
        lds_barrier();
        for (int i = tid; i < a.T * kR; i += (int)blockDim.x) {
            const int t = i / kR, r = i % kR;
            if (row0 + r >= N) continue;
            float v = 0.f;
            for (int s = t * a.k; s < (t + 1) * a.k; s++)
                if ((valid >> s) & 1) v = fmaf(a.route_w[s], s_y[s * kR + r], v);
            a.out_tok[(int64_t)t * N + row0 + r] = v;
        }
    } else if (unit == 0) {   // rows of slots whose id is out of range are zero
        uint64_t bad = ~valid & (n >= 64 ? ~0ull : (1ull << n) - 1);
        for (; bad; bad &= bad - 1)
            if (lane < kR && row0 + lane < N) a.out[(int64_t)__builtin_ctzll(bad) * N + row0 + lane] = 0.f;
    }
}

template <int TYPE, bool FUSE, bool MAKE>
hipError_t launch(const DecXArgs& a, dim3 grid, int waves, size_t lds, hipStream_t st) {
    static PerDeviceOnce cap;
    if (const hipError_t e = set_lds_cap(cap, (const void*)k_decode_x<TYPE, FUSE, MAKE>, kDecXLds)) return e;
    k_decode_x<TYPE, FUSE, MAKE><<<grid, 64 * waves, lds, st>>>(a);
    return hipGetLastError();
}
// Waves of a block, and blocks along the rows.
struct Shape {
    int waves;
    int64_t blocks;
    int64_t work_items() const { return 64 * waves * blocks; }
};
Shape shape(int64_t N, int d_max, bool fuse) {
    Shape s{fuse ? 1 : kRowWaves, 0};
    const int rows = kR * (fuse ? 1 : kRowWaves);
    s.blocks = (N + rows - 1) / rows;
    if (fuse)   // a wave an expert, as far as a dispatch of so many rows holds them
        while (s.waves < d_max && s.waves < kSumWaves && 2 * s.work_items() < 1ll << 32) s.waves *= 2;
    return s;
}
int distinct_max(const DecXArgs& a) { return a.T * a.k < a.E ? a.T * a.k : a.E; }

template <int TYPE, bool MAKE>
hipError_t launch(DecXArgs a, hipStream_t st) {
    const int n = a.T * a.k, d_max = distinct_max(a);
    const bool fuse = a.out_tok != nullptr;
    const Shape g = shape(a.N, d_max, fuse);
    const int waves = g.waves;
    a.xs = a.T * a.act_B;
    if (!fuse && a.xs > kP) a.xs = kP;
    const size_t lds = (MAKE ? (size_t)a.xs * a.K + kDecXSlots * 4 * (1 + kSumWaves) : 0) + (fuse ? (size_t)n * kR * 4 : 0);
    const dim3 grid((unsigned)g.blocks, (unsigned)(fuse ? 1 : d_max));
    return fuse ? launch<TYPE, true, MAKE>(a, grid, waves, lds, st) : launch<TYPE, false, MAKE>(a, grid, waves, lds, st);
}

}  // namespace

bool decode_x_makes(int64_t T) { return T == 1; }
bool decode_x_fuses(ElemType type, int64_t T, int64_t B, int64_t K) {
    return type != kElemI8 || !decode_x_makes(T) || T * B * K <= 64 * 1024;
}

int64_t decode_x_work_items(const DecXArgs& a) { return shape(a.N, distinct_max(a), a.out_tok != nullptr).work_items(); }

hipError_t launch_decode_x(const DecXArgs& a, hipStream_t st) {
    if (a.type == kElemBf16) return launch<kElemBf16, false>(a, st);
    if (a.type == kElemF16) return launch<kElemF16, false>(a, st);
    return a.src_scale ? launch<kElemI8, false>(a, st) : launch<kElemI8, true>(a, st);
}

}  // namespace moe
