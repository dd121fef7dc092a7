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

// 16-byte chunk c of row r sits at c ^ swz(r). Rows of 128 bytes: 16 rows reading the same chunk
// cover all 64 banks.
__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }
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

// Geometry: WM x WN waves, each SM x SN tiles of 32 x 32 at most; NS ring slots.
template <int WM_, int WN_, int SM_, int SN_, int NS_, int OCC_>
struct Tile {
    static constexpr int WM = WM_, WN = WN_, SM = SM_, SN = SN_, NS = NS_, OCC = OCC_;
    static constexpr int waves = WM * WN, threads = 64 * waves;
    static constexpr int BM = 32 * WM * SM, BN = 32 * WN * SN;
    static constexpr int stage = (BM + BN) * 128;   // a stage is 128 bytes of every row
    static constexpr int lds = NS * stage;
};

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
    constexpr int KS = 128 / (int)sizeof(Elem);   // reduction elements per stage
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

    // ---- copies of a stage, 1 KB each: activation rows (8 a copy), weights
    constexpr int CA = G::BM / 8 / G::waves, CB = G::BN / 8 / G::waves;
    static_assert(CA * 8 * G::waves == G::BM && CB * 8 * G::waves == G::BN, "whole copies per wave");
    const uint8_t* ap[CA];
    int a_k[CA];   // first reduction element of this lane's chunk
#pragma unroll
    for (int i = 0; i < CA; i++) {
        // copies i of all the waves together are rows 8 waves i .. +8 waves - 1: the first MACT of them hold the
        // rows of the first MACT sub-tiles
        const int R = (i * G::waves + wv) * 8 + (lane >> 3), lc = (lane & 7) ^ swz(R);
        const int j = m0 + min(R, m_len - 1);
        const int64_t row = P.a_rows ? P.a_rows[j] : j;
        a_k[i] = lc * EC;
        ap[i] = (const uint8_t*)P.A + (row * P.lda + lc * EC) * (int64_t)sizeof(Elem);
    }
    constexpr int BROW = TR ? G::BN * 2 : 128;        // bytes of a row of the weight tile in LDS
    constexpr int BLR = BROW / 16;                    // lanes of a row
    const uint8_t* bp[CB];
    int b_k[CB];
    const int64_t bstep = TR ? (int64_t)KS * P.K * (int)sizeof(Elem) : 128;
#pragma unroll
    for (int i = 0; i < CB; i++) {
        const int R = (wv * CB + i) * (64 / BLR) + lane / BLR;
        if (TR) {
            const int c = min(col0 + (((lane % BLR) ^ swz_t(R)) * EC), cols - EC);
            b_k[i] = R;
            bp[i] = (const uint8_t*)P.W + (((int64_t)e * P.N + R) * P.K + c) * (int64_t)sizeof(Elem);
        } else {
            const int lc = (lane & 7) ^ swz(R);
            b_k[i] = lc * EC;
            bp[i] = (const uint8_t*)P.W + (((int64_t)e * P.N + min(col0 + R, cols - 1)) * P.K + lc * EC) * (int64_t)sizeof(Elem);
        }
    }
    auto issue = [&](int s, int slot, auto n_c) __attribute__((always_inline)) {
        const uint32_t st = lds0 + (uint32_t)(slot * G::stage);
        const int k0 = s * KS;
        const bool full = k0 + KS <= depth;   // what passes the end is zero on both sides
#pragma unroll
        for (int i = 0; i < decltype(n_c)::value; i++) {
            dma16v(full || k0 + a_k[i] < depth ? (const void*)ap[i] : zero, st + (i * G::waves + wv) * 1024);
            ap[i] += 128;
        }
#pragma unroll
        for (int i = 0; i < CB; i++) {
            dma16v(full || k0 + b_k[i] < depth ? (const void*)bp[i] : zero, st + G::BM * 128 + (wv * CB + i) * 1024);
            bp[i] += bstep;
        }
    };

    typename T::Acc acc[G::SM][G::SN];
    auto k_loop = [&](auto n_c) __attribute__((always_inline)) {
        constexpr int MACT = decltype(n_c)::value;
        constexpr int copies = MACT * CA / G::SM + CB;
        using NA = std::integral_constant<int, MACT * CA / G::SM>;
        static_assert(CA % G::SM == 0, "a sub-tile's copies are whole");
#pragma unroll
        for (int i = 0; i < MACT; i++)
#pragma unroll
            for (int c = 0; c < G::SN; c++) acc[i][c] = typename T::Acc{};
        const int l16 = lane & 15;
        const uint32_t a_lane = l32 * 128 + wm * 4096;
        uint32_t b_lane[G::SN];
#pragma unroll
        for (int c = 0; c < G::SN; c++)
            b_lane[c] = TR ? (8 * h + (l16 >> 2)) * BROW + (l16 & 1) * 8 +
                                 ((((wn * G::SN + c) * 4 + ((lane >> 4) & 1) * 2 + ((l16 >> 1) & 1)) ^ swz_t(l16 >> 2)) << 4)
                           : ((wn * G::SN + c) * 32 + l32) * 128;
        for (int s = 0; s < G::NS - 1 && s < nst; s++) issue(s, s, NA{});
        int slot = 0;
        for (int s = 0; s < nst; s++) {
            // stage s landed (the copies of NS - 2 later stages may be in flight), and every wave is past stage s - 1
            if (s + G::NS - 2 < nst) wait_stage_and_barrier<(G::NS - 2) * copies>();
            else wait_stage_and_barrier<0>();
            if (s + G::NS - 1 < nst) issue(s + G::NS - 1, slot == 0 ? G::NS - 1 : slot - 1, NA{});
            const uint8_t* st = smem + slot * G::stage;
            slot = slot == G::NS - 1 ? 0 : slot + 1;
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const uint32_t ch = (uint32_t)((2 * q + h) ^ swz(l32)) << 4;
                i32x4 a[MACT], b[G::SN];
#pragma unroll
                for (int c = 0; c < G::SN; c++) {
                    if (TR) b[c] = read_t<BROW>(st + G::BM * 128 + b_lane[c] + q * 16 * BROW);
                    else b[c] = *(const i32x4*)(st + G::BM * 128 + b_lane[c] + ch);
                }
#pragma unroll
                for (int i = 0; i < MACT; i++) a[i] = *(const i32x4*)(st + a_lane + i * G::WM * 4096 + ch);
#pragma unroll
                for (int i = 0; i < MACT; i++)
#pragma unroll
                    for (int c = 0; c < G::SN; c++) acc[i][c] = T::mfma(a[i], b[c], acc[i][c]);
            }
        }
    };
    const int mact = (m_len + 32 * G::WM - 1) / (32 * G::WM);   // occupied sub-tiles (block-uniform)
    if (G::SM >= 4 && mact >= 4) k_loop(std::integral_constant<int, G::SM >= 4 ? 4 : 1>{});
    else if (G::SM >= 3 && mact == 3) k_loop(std::integral_constant<int, G::SM >= 3 ? 3 : 1>{});
    else if (G::SM >= 2 && mact == 2) k_loop(std::integral_constant<int, G::SM >= 2 ? 2 : 1>{});
    else k_loop(std::integral_constant<int, 1>{});

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
// dW_e tile of BM rows (n) x BN columns (k); the reduction runs along e's positions, 64 a stage, both operands
// read transposed. WEIGHTED: dY row j times route_w of its slot, rounded to the element type.
constexpr int kMapRows = 1024;   // positions whose rows are in LDS at a time

template <class T, bool WEIGHTED, class G>
__global__ __launch_bounds__(G::threads, G::OCC) void k_grad_w(ExpertGradW P) {
    using Elem = typename T::Elem;
    constexpr int KS = 64;
    constexpr int AROW = G::BM * 2, BROW = G::BN * 2, ALR = AROW / 16, BLR = BROW / 16;
    constexpr int stage = KS * (AROW + BROW);
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    int32_t* s_dy = (int32_t*)(smem + G::NS * stage);   // rows of dY and X of positions j0 ..
    int32_t* s_x = s_dy + kMapRows;
    float* s_w = (float*)(s_x + kMapRows);              // WEIGHTED: their routing weights

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

    constexpr int CA = KS * ALR / 64 / G::waves, CB = KS * BLR / 64 / G::waves;
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
    // rows of positions jb .. of the segment (jb a multiple of kMapRows), row 0 past its end
    auto map = [&](int jb) {
        for (int i = tid; i < kMapRows; i += G::threads) {
            const int j = j0 + jb + i;
            const bool in = jb + i < len;
            s_dy[i] = in ? P.dy_rows[j] : 0;
            s_x[i] = in ? P.x_rows[j] : 0;
            if (WEIGHTED) s_w[i] = in ? P.route_w[P.slots[j]] : 0.f;
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

    for (int s = 0; s < nst; s++) {
        if ((s & (kMapRows / KS - 1)) == 0) {   // a ring of two slots: the copies of a stage ahead end at the map's end
            __syncthreads();
            map(s * KS);
            __syncthreads();
            issue(s, s & 1);
        }
        wait_stage_and_barrier<0>();
        if (s + 1 < nst && ((s + 1) & (kMapRows / KS - 1))) issue(s + 1, (s + 1) & 1);
        const uint8_t* st = smem + (s & 1) * stage;
#pragma unroll
        for (int q = 0; q < KS / 16; q++) {
            i32x4 a[G::SM], b[G::SN];
#pragma unroll
            for (int c = 0; c < G::SN; c++) b[c] = read_t<BROW>(st + KS * AROW + b_lane[c] + q * 16 * BROW);
#pragma unroll
            for (int i = 0; i < G::SM; i++) a[i] = read_t<AROW>(st + a_lane[i] + q * 16 * AROW);
            if (WEIGHTED) {
                typedef Elem Vec __attribute__((ext_vector_type(8)));
                const float* w = s_w + ((s * KS) & (kMapRows - 1)) + q * 16 + 8 * h;
#pragma unroll
                for (int i = 0; i < G::SM; i++) {
                    Vec v = __builtin_bit_cast(Vec, a[i]);
#pragma unroll
                    for (int u = 0; u < 8; u++) v[u] = (Elem)((float)v[u] * w[u]);
                    a[i] = __builtin_bit_cast(i32x4, v);
                }
            }
#pragma unroll
            for (int i = 0; i < G::SM; i++)
#pragma unroll
                for (int c = 0; c < G::SN; c++) acc[i][c] = T::mfma(a[i], b[c], acc[i][c]);
        }
    }
#pragma unroll
    for (int c = 0; c < G::SN; c++) {
        const int col = col0 + (wn * G::SN + c) * 32 + l32;
        if (col >= P.K) continue;
#pragma unroll
        for (int i = 0; i < G::SM; i++) {
#pragma unroll
            for (int v = 0; v < 16; v++) {
                const int row = row0 + (wm * G::SM + i) * 32 + 8 * (v >> 2) + 4 * h + (v & 3);
                if (row >= P.N) continue;
                const int64_t o = ((int64_t)e * P.N + row) * P.K + col;
                if (P.f32) ((float*)P.dW)[o] = acc[i][c][v];
                else ((Elem*)P.dW)[o] = (Elem)acc[i][c][v];
            }
        }
    }
}

using Wide = Tile<2, 4, 4, 2, 2, 2>;     // 256 x 256, one block a CU
using Narrow = Tile<1, 4, 2, 1, 3, 2>;   // 64 x 128, two blocks a CU
using GradW = Tile<2, 4, 4, 2, 2, 2>;

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
    constexpr int lds = G::NS * 64 * 2 * (G::BM + G::BN) + kMapRows * 12;
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
    if (a.type == kElemBf16) return a.route_w ? launch_w<Bf16, true>(a, st) : launch_w<Bf16, false>(a, st);
    return a.route_w ? launch_w<F16, true>(a, st) : launch_w<F16, false>(a, st);
}

}  // namespace moe
