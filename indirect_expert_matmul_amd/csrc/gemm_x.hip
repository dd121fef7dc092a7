// Grouped products over expert segments of 16-bit experts (bf16, f16) and their gradients, and of
// int8 experts with a scale per output row, on gfx950.
//
//   product       out[i][n] = sum_k A[r][k] W_e[n][k]            (int8: times the scales of row r and of n)
//   row gradient  out[i][k] = sum_n dY[r][n] W_e[n][k]
//   expert grad.  dW_e[n][k] = sum over e's positions j of dY[r_j][n] X[r'_j][k]
//
// i a slot of expert e and r its activation row (section 1.2 of "CUDA: better MoE implementation"
// has the product; the gradients follow from it). Positions j, their rows and the M tiles come from
// the row-id pass.
#include <type_traits>

#include "lds_dma.h"
#include "moe_internal.h"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// An element type: its 32x32 MFMA takes 16 bytes a lane of each operand, lane half h the bytes
// 16 h .. +15 of a 32-byte step of the row.
struct Bf16 {
    using Elem = __bf16;
    using Acc = f32x16;
    static __device__ __forceinline__ Acc mfma(i32x4 a, i32x4 b, Acc c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
};
struct F16 {
    using Elem = _Float16;
    using Acc = f32x16;
    static __device__ __forceinline__ Acc mfma(i32x4 a, i32x4 b, Acc c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
};
struct I8 {
    using Elem = int8_t;
    using Acc = i32x16;
    static __device__ __forceinline__ Acc mfma(i32x4 a, i32x4 b, Acc c) {
        return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
    }
};

__device__ __attribute__((aligned(16))) const uint32_t g_zero[4] = {0, 0, 0, 0};   // what lies past an end

constexpr int kMChunk = 4;   // M tiles sharing each weight slab in turn

// 16-byte chunk c of row r sits at c ^ swz(r): the rows of a phase of ds_read_b128 cover the banks once.
template <int RB>
__device__ __forceinline__ int swz(int r) { return RB == 64 ? (r >> 2) & 3 : (r & 7) ^ ((r >> 3) & 1); }
// Rows that are read transposed (four rows, 32 or 64 bytes of each, at a time): the four rows'
// chunks are apart in both 128 and 256 bytes.
__device__ __forceinline__ int swz_t(int r) { return ((r & 3) << 2) | (r & 2); }

// Eight elements down a column of an LDS tile (rows r .. r + 7 of it) for each of 32 columns and
// the next eight rows for the upper lane half: two transposing reads of four rows, 16 lanes a
// 4 x 16 block. p: this lane's address of the first (row l16 / 4 of the block, 8-byte piece l16 % 4).
template <int ROW>
__device__ __forceinline__ i32x4 read_t(const uint8_t* p) {
    typedef __attribute__((address_space(3))) i16x4* Lds;
    const i32x2 lo = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)p));
    const i32x2 hi = __builtin_bit_cast(i32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p + 4 * ROW)));
    return i32x4{lo[0], lo[1], hi[0], hi[1]};
}

// Geometry: WM x WN waves, each SM x SN tiles of 32 x 32 at most; a ring of NS slots, RB bytes of every row in
// each; OCC waves a SIMD.
template <int WM_, int WN_, int SM_, int SN_, int RB_, int NS_, int OCC_>
struct Tile {
    static constexpr int WM = WM_, WN = WN_, SM = SM_, SN = SN_, RB = RB_, NS = NS_, OCC = OCC_;
    static constexpr int waves = WM * WN, threads = 64 * waves;
    static constexpr int BM = 32 * WM * SM, BN = 32 * WN * SN;
    static constexpr int stage = (BM + BN) * RB;
    static constexpr int lds = NS * stage;
};
template <int N>
using Int = std::integral_constant<int, N>;

// M tile and column tile of this block: tiles ordered by expert, chunk of M tiles, column tile,
// an eighth of them to each XCD. False: none.
struct Where {
    int e, m0, m_len, nt;
};
template <int BM>
__device__ __forceinline__ bool find_tile(const ExpertGemm& P, int n_nt, Where& w) {
    const int b = (int)blockIdx.x;
    const int total = P.tile_off[P.E] * n_nt;
    const int part = (total + 7) >> 3, q = b >> 3, t = (b & 7) * part + q;
    if (q >= part || t >= total) return false;
    const int4 ti = *(const int4*)(P.tile_tab + 4 * (int64_t)(t / n_nt));
    w.e = __builtin_amdgcn_readfirstlane(ti.x);
    const int first = __builtin_amdgcn_readfirstlane(ti.y);
    const int row0 = __builtin_amdgcn_readfirstlane(ti.z);
    const int rows = __builtin_amdgcn_readfirstlane(ti.w);
    const int tiles = (rows + BM - 1) / BM;
    const int r = t - n_nt * first;
    const int c = r / (kMChunk * n_nt);
    const int g = min(kMChunk, tiles - c * kMChunk);
    const int rr = r - c * kMChunk * n_nt;
    w.nt = rr / g;
    const int j = c * kMChunk + (rr - w.nt * g);
    const int height = ((rows + tiles - 1) / tiles + 31) & ~31;   // equal tiles rather than full ones and a rest
    w.m0 = row0 + j * height;
    w.m_len = min(height, rows - j * height);
    return w.m_len > 0;
}

// TR 0: the product (reduction along W's columns); 1: the row gradient (along its rows).
// OUT16: rows of the element type, else float32.
template <class T, int TR, bool OUT16, class G>
__global__ __launch_bounds__(G::threads, G::OCC) void k_gemm_x(ExpertGemm P) {
    using Elem = typename T::Elem;
    constexpr int RB = G::RB, W = G::waves;
    constexpr int KS = RB / (int)sizeof(Elem);    // reduction elements per stage
    constexpr int EC = 16 / (int)sizeof(Elem);    // elements of a chunk
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int cols = TR ? P.K : P.N, depth = TR ? P.N : P.K;
    Where at;
    if (!find_tile<G::BM>(P, (cols + G::BN - 1) / G::BN, at)) return;
    const int e = at.e, m0 = at.m0, m_len = at.m_len, col0 = at.nt * G::BN;

    const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wv % G::WM, wn = wv / G::WM;
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
    const int nst = (depth + KS - 1) / KS;
    const void* zero = g_zero;

    // ---- copies of a stage, 1 KB each: activation rows, 1024 / RB a copy and dealt out to the waves in turn (so
    // that a shorter tile's rows are the first copies of all of them), then weights
    constexpr int CR = 1024 / RB, CL = RB / 16;   // rows of a copy, lanes of a row
    constexpr int CA = (G::BM / CR + W - 1) / W, CB = G::BN / CR / W;
    static_assert(CB * CR * W == G::BN, "whole copies per wave");
    const uint8_t* ap[CA];
    const int a_k = ((lane % CL) ^ swz<RB>(lane / CL + (CR == 8 ? 8 * (wv & 1) : 0))) * EC;   // of this lane's chunk
    static_assert(CR == 16 || W % 2 == 0, "a wave's copies differ in multiples of 16 rows");
#pragma unroll
    for (int i = 0; i < CA; i++) {
        const int R = (i * W + wv) * CR + lane / CL;
        const int j = m0 + min(R, m_len - 1);
        const int64_t row = P.a_rows ? P.a_rows[j] : j;
        ap[i] = (const uint8_t*)P.A + (row * P.lda + a_k) * (int64_t)sizeof(Elem);
    }
    constexpr int BROW = TR ? G::BN * 2 : RB;        // bytes of a row of the weight tile in LDS
    constexpr int BLR = BROW / 16;                   // lanes of a row
    const uint8_t* bp[CB];
    int b_k[CB];   // reduction element of this lane's chunk
    const int64_t bstep = TR ? (int64_t)KS * P.K * (int)sizeof(Elem) : RB;
#pragma unroll
    for (int i = 0; i < CB; i++) {
        const int R = (wv * CB + i) * (64 / BLR) + lane / BLR;
        if (TR) {
            const int c = min(col0 + (((lane % BLR) ^ swz_t(R)) * EC), cols - EC);
            b_k[i] = R;
            bp[i] = (const uint8_t*)P.W + (((int64_t)e * P.N + R) * P.K + c) * (int64_t)sizeof(Elem);
        } else {
            b_k[i] = ((lane % CL) ^ swz<RB>(R)) * EC;
            bp[i] = (const uint8_t*)P.W + (((int64_t)e * P.N + min(col0 + R, cols - 1)) * P.K + b_k[i]) * (int64_t)sizeof(Elem);
        }
    }
    // copies of stage s; TA: the tile's activation copies
    auto issue = [&](int s, int slot, auto ta_c) __attribute__((always_inline)) {
        constexpr int TA = decltype(ta_c)::value;
        const uint32_t st = lds0 + (uint32_t)(slot * G::stage);
        const int k0 = s * KS;
        const bool full = k0 + KS <= depth;   // what passes the end is zero on both sides
        const bool a_in = full || k0 + a_k < depth;
#pragma unroll
        for (int i = 0; i < (TA + W - 1) / W; i++) {
            if (i * W + W <= TA || i * W + wv < TA) {
                dma16v(a_in ? (const void*)ap[i] : zero, st + (i * W + wv) * 1024);
                ap[i] += RB;
            }
        }
#pragma unroll
        for (int i = 0; i < CB; i++) {
            dma16v(full || k0 + b_k[i] < depth ? (const void*)bp[i] : zero, st + G::BM * RB + (wv * CB + i) * 1024);
            bp[i] += bstep;
        }
    };

    typename T::Acc acc[G::SM][G::SN];
    const int l16 = lane & 15;
    const uint32_t a_lane = (wm * 32 + l32) * RB;
    uint32_t b_lane[G::SN];
#pragma unroll
    for (int c = 0; c < G::SN; c++)
        b_lane[c] = TR ? (8 * h + (l16 >> 2)) * BROW + (l16 & 1) * 8 +
                             ((((wn * G::SN + c) * 4 + ((lane >> 4) & 1) * 2 + ((l16 >> 1) & 1)) ^ swz_t(l16 >> 2)) << 4)
                       : ((wn * G::SN + c) * 32 + l32) * RB;
    struct Frag {
        i32x4 a[G::SM], b[G::SN];
    };
    // operands of 32-byte step q of the stage in a slot
    auto read = [&](Frag& f, int slot, int q, auto n_c) __attribute__((always_inline)) {
        const uint8_t* st = smem + slot * G::stage;
        const uint32_t ch = (uint32_t)((2 * q + h) ^ swz<RB>(l32)) << 4;
#pragma unroll
        for (int c = 0; c < G::SN; c++) {
            if (TR) f.b[c] = read_t<BROW>(st + G::BM * RB + b_lane[c] + q * 16 * BROW);
            else f.b[c] = *(const i32x4*)(st + G::BM * RB + b_lane[c] + ch);
        }
#pragma unroll
        for (int i = 0; i < decltype(n_c)::value; i++) f.a[i] = *(const i32x4*)(st + a_lane + i * G::WM * 32 * RB + ch);
    };
    auto multiply = [&](const Frag& f, auto n_c) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < decltype(n_c)::value; i++)
#pragma unroll
            for (int c = 0; c < G::SN; c++) acc[i][c] = T::mfma(f.a[i], f.b[c], acc[i][c]);
    };
    auto k_loop = [&](auto n_c) __attribute__((always_inline)) {
        constexpr int MACT = decltype(n_c)::value, TA = MACT * 32 * G::WM / CR, Q = RB / 32;
        constexpr int few = (TA / W + CB) * (G::NS - 2), more = ((TA + W - 1) / W + CB) * (G::NS - 2);
        using NA = Int<TA>;
        static_assert(MACT * 32 * G::WM % CR == 0, "a sub-tile's copies are whole");
#pragma unroll
        for (int i = 0; i < MACT; i++)
#pragma unroll
            for (int c = 0; c < G::SN; c++) acc[i][c] = typename T::Acc{};
        // stage s landed; of the copies only those of the NS - 2 stages after it may be in flight
        auto landed = [&](int s) __attribute__((always_inline)) {
            if (s + G::NS - 2 >= nst) wait_vm<0>();
            else if (few == more || wv < TA % W) wait_vm<more>();
            else wait_vm<few>();
            wait_stage_and_barrier<63>();
        };
        for (int s = 0; s < G::NS - 1 && s < nst; s++) issue(s, s, NA{});
        landed(0);
        if (G::NS - 1 < nst) issue(G::NS - 1, G::NS - 1, NA{});
        Frag f0, f1;
        read(f0, 0, 0, n_c);
        int slot = 0;
        // at the loop's head: step 0 of stage s in f0, stage s + NS - 1 on its way
        for (int s = 0; s < nst; s++) {
#pragma unroll
            for (int q = 0; q + 1 < Q; q++) {
                read(q & 1 ? f0 : f1, slot, q + 1, n_c);
                multiply(q & 1 ? f1 : f0, n_c);
                __builtin_amdgcn_sched_barrier(0);
            }
            // this wave's reads of stage s are done, the other waves' too after the barrier
            const int next = slot == G::NS - 1 ? 0 : slot + 1;
            if (s + 1 < nst) {
                landed(s + 1);
                if (s + G::NS < nst) issue(s + G::NS, slot, NA{});
                read(f0, next, 0, n_c);
            }
            slot = next;
            multiply(f1, n_c);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    const int mact = (m_len + 32 * G::WM - 1) / (32 * G::WM);   // occupied sub-tiles (block-uniform)
    if (G::SM >= 4 && mact >= 4) k_loop(Int<(G::SM >= 4 ? 4 : 1)>{});
    else if (G::SM >= 3 && mact == 3) k_loop(Int<(G::SM >= 3 ? 3 : 1)>{});
    else if (G::SM >= 2 && mact == 2) k_loop(Int<(G::SM >= 2 ? 2 : 1)>{});
    else k_loop(Int<1>{});

    // ---- output rows (and what scales them) into the now idle ring
    int32_t* s_row = (int32_t*)smem;
    float* s_scale = (float*)(smem + G::BM * 4);
    __syncthreads();
    for (int r = tid; r < G::BM; r += G::threads) {
        const int j = m0 + min(r, m_len - 1);
        const int o = P.out_rows ? P.out_rows[j] : j;
        s_row[r] = o;
        if constexpr (std::is_same<T, I8>::value) s_scale[r] = P.a_scale[P.a_rows ? P.a_rows[j] : j];
        else if (OUT16) s_scale[r] = P.row_w ? P.row_w[o] : 1.f;
    }
    __syncthreads();

    // ---- element 4 g + u of lane l: row 8 g + 4 (l / 32) + u of the sub-tile, column l % 32
#pragma unroll
    for (int c = 0; c < G::SN; c++) {
        const int col = col0 + (wn * G::SN + c) * 32 + l32;
        if (col >= cols) continue;
        float ws = 1.f;
        if constexpr (std::is_same<T, I8>::value) ws = P.w_scale[(int64_t)e * P.N + col];
#pragma unroll
        for (int i = 0; i < G::SM; i++) {
            const int base = (i * G::WM + wm) * 32 + 4 * h;
            if (base >= m_len) continue;
#pragma unroll
            for (int v = 0; v < 16; v++) {
                const int m = base + 8 * (v >> 2) + (v & 3);
                if (m >= m_len) continue;
                const int64_t o = (int64_t)s_row[m] * cols + col;
                if constexpr (std::is_same<T, I8>::value) ((float*)P.out)[o] = (float)acc[i][c][v] * (s_scale[m] * ws);
                else if (OUT16) ((Elem*)P.out)[o] = (Elem)(acc[i][c][v] * s_scale[m]);
                else ((float*)P.out)[o] = acc[i][c][v];
            }
        }
    }
}

// ---------------------------------------------------------------- expert gradient
// dW_e tile of BM rows (n) x BN columns (k); the reduction runs along e's positions, KS a stage, both operands
// read transposed. WEIGHTED: dY row j times route_w of its slot, rounded to the element type.
constexpr int kMapRows = 512;   // ring of positions whose rows are in LDS, refilled by halves

template <class T, bool WEIGHTED, class G>
__global__ __launch_bounds__(G::threads, G::OCC) void k_grad_w(ExpertGradW P) {
    using Elem = typename T::Elem;
    constexpr int W = G::waves, NS = G::NS;
    constexpr int KS = G::RB / 2, Q = KS / 16, kHalf = kMapRows / 2 / KS;   // positions and MFMA steps of a stage; stages of half a map
    static_assert(NS < kHalf && kMapRows % (2 * KS) == 0, "the map covers the stages in flight");
    constexpr int AROW = G::BM * 2, BROW = G::BN * 2, ALR = AROW / 16, BLR = BROW / 16;
    constexpr int stage = KS * (AROW + BROW);
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    int32_t* s_dy = (int32_t*)(smem + NS * stage);   // rows of dY and X of the positions
    int32_t* s_x = s_dy + kMapRows;
    float* s_w = (float*)(s_x + kMapRows);           // WEIGHTED: their routing weights

    const int n_nt = (P.N + G::BM - 1) / G::BM, n_kt = (P.K + G::BN - 1) / G::BN;
    const int64_t total = (int64_t)P.E * n_nt * n_kt, part = (total + 7) >> 3;
    const int64_t t = (int64_t)(blockIdx.x & 7) * part + (blockIdx.x >> 3);
    if ((int64_t)(blockIdx.x >> 3) >= part || t >= total) return;
    const int e = (int)(t / (n_nt * n_kt)), tt = (int)(t - (int64_t)e * n_nt * n_kt);
    const int row0 = tt / n_kt * G::BM, col0 = tt % n_kt * G::BN;
    const int j0 = P.bounds[e], len = P.bounds[e + 1] - j0;

    const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, l16 = lane & 15, h = lane >> 5;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wv % G::WM, wn = wv / G::WM;
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
    const int nst = (len + KS - 1) / KS;
    const void* zero = g_zero;

    // rows of half a map from position `from` of the segment on: 64 a copy
    auto map = [&](int from) __attribute__((always_inline)) {
        const uint32_t at = lds0 + NS * stage + (from & (kMapRows - 1)) * 4;
        for (int i = wv; i < kMapRows / 128; i += W) {
            const int p = from + 64 * i + lane;
            const bool in = p < len;
            dma4v(in ? (const void*)(P.dy_rows + j0 + p) : zero, at + 256 * i);
            dma4v(in ? (const void*)(P.x_rows + j0 + p) : zero, at + kMapRows * 4 + 256 * i);
            if (WEIGHTED) dma4v(in ? (const void*)(P.pos_w + j0 + p) : zero, at + kMapRows * 8 + 256 * i);
        }
    };
    constexpr int CA = KS * ALR / 64 / W, CB = KS * BLR / 64 / W;
    static_assert(CA * 64 * W == KS * ALR && CB * 64 * W == KS * BLR, "whole copies per wave");
    auto issue = [&](int s, int slot) __attribute__((always_inline)) {
        const uint32_t st = lds0 + (uint32_t)(slot * stage);
#pragma unroll
        for (int i = 0; i < CA; i++) {
            const int R = (wv * CA + i) * (64 / ALR) + lane / ALR, j = s * KS + R;
            const int c = min(row0 + ((lane % ALR) ^ swz_t(R)) * 8, P.ldy - 8);
            const uint8_t* p = (const uint8_t*)P.dY + ((int64_t)s_dy[j & (kMapRows - 1)] * P.ldy + c) * 2;
            dma16v(j < len ? (const void*)p : zero, st + (wv * CA + i) * 1024);
        }
#pragma unroll
        for (int i = 0; i < CB; i++) {
            const int R = (wv * CB + i) * (64 / BLR) + lane / BLR, j = s * KS + R;
            const int c = min(col0 + ((lane % BLR) ^ swz_t(R)) * 8, P.K - 8);
            const uint8_t* p = (const uint8_t*)P.X + ((int64_t)s_x[j & (kMapRows - 1)] * P.K + c) * 2;
            dma16v(j < len ? (const void*)p : zero, st + KS * AROW + (wv * CB + i) * 1024);
        }
    };

    f32x16 acc[G::SM][G::SN];
#pragma unroll
    for (int i = 0; i < G::SM; i++)
#pragma unroll
        for (int c = 0; c < G::SN; c++) acc[i][c] = f32x16{};
    uint32_t a_lane[G::SM], b_lane[G::SN];
    const int r4 = 8 * h + (l16 >> 2), piece = ((lane >> 4) & 1) * 2 + ((l16 >> 1) & 1);
#pragma unroll
    for (int i = 0; i < G::SM; i++)
        a_lane[i] = r4 * AROW + (l16 & 1) * 8 + ((((wm * G::SM + i) * 4 + piece) ^ swz_t(l16 >> 2)) << 4);
#pragma unroll
    for (int c = 0; c < G::SN; c++)
        b_lane[c] = r4 * BROW + (l16 & 1) * 8 + ((((wn * G::SN + c) * 4 + piece) ^ swz_t(l16 >> 2)) << 4);
    struct Frag {
        i32x4 a[G::SM], b[G::SN];
    };
    auto read = [&](Frag& f, int s, int slot, int q) __attribute__((always_inline)) {
        const uint8_t* st = smem + slot * stage;
#pragma unroll
        for (int c = 0; c < G::SN; c++) f.b[c] = read_t<BROW>(st + KS * AROW + b_lane[c] + q * 16 * BROW);
#pragma unroll
        for (int i = 0; i < G::SM; i++) f.a[i] = read_t<AROW>(st + a_lane[i] + q * 16 * AROW);
        if (WEIGHTED) {
            typedef Elem Vec __attribute__((ext_vector_type(8)));
            const float* w = s_w + ((s * KS) & (kMapRows - 1)) + q * 16 + 8 * h;
#pragma unroll
            for (int i = 0; i < G::SM; i++) {
                Vec v = __builtin_bit_cast(Vec, f.a[i]);
#pragma unroll
                for (int u = 0; u < 8; u++) v[u] = (Elem)((float)v[u] * w[u]);
                f.a[i] = __builtin_bit_cast(i32x4, v);
            }
        }
    };
    auto multiply = [&](const Frag& f) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < G::SM; i++)
#pragma unroll
            for (int c = 0; c < G::SN; c++) acc[i][c] = T::mfma(f.a[i], f.b[c], acc[i][c]);
    };
    if (nst > 0) {
        // stage s landed; of the copies only those of the NS - 2 stages after it may be in flight (a map's copies
        // among them make it wait for more)
        auto landed = [&](int s) __attribute__((always_inline)) {
            if (s + NS - 2 >= nst) wait_stage_and_barrier<0>();
            else wait_stage_and_barrier<(CA + CB) * (NS - 2)>();
        };
        map(0);
        if (len > kMapRows / 2) map(kMapRows / 2);
        wait_stage_and_barrier<0>();
        for (int s = 0; s < NS - 1 && s < nst; s++) issue(s, s);
        landed(0);
        if (NS - 1 < nst) issue(NS - 1, NS - 1);
        Frag f0, f1;
        read(f0, 0, 0, 0);
        int slot = 0;
        for (int s = 0; s < nst; s++) {
#pragma unroll
            for (int q = 0; q + 1 < Q; q++) {
                read(q & 1 ? f0 : f1, s, slot, q + 1);
                multiply(q & 1 ? f1 : f0);
                __builtin_amdgcn_sched_barrier(0);
            }
            const int next = slot == NS - 1 ? 0 : slot + 1;
            if (s + 1 < nst) {
                landed(s + 1);
                if (s + NS < nst) {
                    issue(s + NS, slot);
                    // The half of the map that holds stage s and the kHalf - 1 before it has served, once s is its
                    // last stage: the rows two halves on take its place, needed kHalf - NS + 1 stages from now.
                    if ((s + 1) % kHalf == 0 && (s + 1 + kHalf) * KS < len) map((s + 1 + kHalf) * KS);
                }
                read(f0, s + 1, next, 0);
            }
            slot = next;
            multiply(f1);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // ---- element 4 g + u of lane l: row 8 g + 4 (l / 32) + u of the tile, column l % 32
#pragma unroll
    for (int c = 0; c < G::SN; c++) {
        const int col = col0 + (wn * G::SN + c) * 32 + l32;
        const bool in = col < P.K;
#pragma unroll
        for (int i = 0; i < G::SM; i++) {
            const int row = row0 + (wm * G::SM + i) * 32 + 4 * h;
#pragma unroll
            for (int v = 0; v < 16; v += 2) {
                const int r = row + 8 * (v >> 2) + (v & 3);
                const int64_t o = ((int64_t)e * P.N + r) * P.K + col;
                if (P.f32) {
                    if (in && r < P.N) ((float*)P.dW)[o] = acc[i][c][v];
                    if (in && r + 1 < P.N) ((float*)P.dW)[o + P.K] = acc[i][c][v + 1];
                } else {
                    // two columns a store: even lanes take row r of both, odd lanes row r + 1
                    const bool odd = lane & 1;
                    const float give = odd ? acc[i][c][v] : acc[i][c][v + 1];
                    const float got = __shfl_xor(give, 1);
                    typedef Elem Pair __attribute__((ext_vector_type(2)));
                    const Pair pair = {(Elem)(odd ? got : acc[i][c][v]), (Elem)(odd ? acc[i][c][v + 1] : got)};
                    if (in && r + odd < P.N) *(Pair*)((Elem*)P.dW + o + (odd ? P.K - 1 : 0)) = pair;
                }
            }
        }
    }
}

using Wide = Tile<2, 4, 4, 2, 64, 5, 2>;      // 256 x 256, one block a CU
using Narrow = Tile<1, 4, 2, 1, 128, 3, 2>;   // 64 x 128, two blocks a CU
using GradW = Tile<1, 4, 4, 2, 64, 3, 2>;     // 128 x 256, two blocks a CU

template <class T, int TR, bool OUT16, class G>
hipError_t launch(const ExpertGemm& a, hipStream_t st) {
    const int64_t grid = expert_gemm_grid(a, TR ? 1 : 0);
    if (grid <= 0) return hipSuccess;
    static PerDeviceOnce cap;
    if (const hipError_t e = set_lds_cap(cap, (const void*)k_gemm_x<T, TR, OUT16, G>, G::lds)) return e;
    k_gemm_x<T, TR, OUT16, G><<<(unsigned)grid, G::threads, G::lds, st>>>(a);
    return hipGetLastError();
}
template <class T, int TR, bool OUT16>
hipError_t launch_tile(const ExpertGemm& a, hipStream_t st) {
    return a.tile_m == Wide::BM ? launch<T, TR, OUT16, Wide>(a, st) : launch<T, TR, OUT16, Narrow>(a, st);
}

template <class T, bool WEIGHTED>
hipError_t launch_w(const ExpertGradW& a, hipStream_t st) {
    using G = GradW;
    constexpr int lds = G::lds + kMapRows * (WEIGHTED ? 12 : 8);
    static PerDeviceOnce cap;
    if (const hipError_t e = set_lds_cap(cap, (const void*)k_grad_w<T, WEIGHTED, G>, lds)) return e;
    k_grad_w<T, WEIGHTED, G><<<(unsigned)expert_grad_w_grid(a), G::threads, lds, st>>>(a);
    return hipGetLastError();
}

}  // namespace

int expert_gemm_tile_m(double avg_rows) { return avg_rows > 64 ? Wide::BM : Narrow::BM; }

int64_t expert_gemm_grid(const ExpertGemm& a, int grad) {
    const int64_t cols = grad ? a.K : a.N, bn = a.tile_m == Wide::BM ? Wide::BN : Narrow::BN;
    return ((int64_t)a.m_tiles_max * ((cols + bn - 1) / bn) + 7) / 8 * 8;
}

int64_t expert_grad_w_grid(const ExpertGradW& a) {
    const int64_t n = (a.N + GradW::BM - 1) / GradW::BM, k = (a.K + GradW::BN - 1) / GradW::BN;
    return (a.E * n * k + 7) / 8 * 8;
}

hipError_t launch_expert_gemm(const ExpertGemm& a, hipStream_t st) {
    switch (a.type) {
        case kElemBf16: return launch_tile<Bf16, 0, false>(a, st);
        case kElemF16: return launch_tile<F16, 0, false>(a, st);
        default: return launch_tile<I8, 0, false>(a, st);
    }
}

hipError_t launch_expert_grad_x(const ExpertGemm& a, hipStream_t st) {
    if (a.type == kElemBf16) return a.out16 ? launch_tile<Bf16, 1, true>(a, st) : launch_tile<Bf16, 1, false>(a, st);
    return a.out16 ? launch_tile<F16, 1, true>(a, st) : launch_tile<F16, 1, false>(a, st);
}

hipError_t launch_expert_grad_w(const ExpertGradW& a, hipStream_t st) {
    if (a.type == kElemBf16) return a.pos_w ? launch_w<Bf16, true>(a, st) : launch_w<Bf16, false>(a, st);
    return a.pos_w ? launch_w<F16, true>(a, st) : launch_w<F16, false>(a, st);
}

}  // namespace moe
