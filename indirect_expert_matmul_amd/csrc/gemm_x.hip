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
//
// Product and row gradient, k_gemm_x: a block has up to 320 rows of a segment and 256 columns (8 waves,
// one block a CU; 64 x 128 and two blocks where the segments are short; 64 x 32, four waves that take parts of the depth in
// turn, where that makes few blocks). Both operands come to LDS by direct copies,
// 128 bytes of a row a stage (64 bytes a row reach half the rate), the rows of activations through the row map. Weights
// have a ring of three stages, activations of two: two stages of weights, which come from HBM, are under
// way while one is multiplied. Chunks of 16 bytes are swizzled so that the reads of LDS have no
// bank conflicts; the row gradient reads its weights, whose reduction axis is the slow one, by transposing reads. The
// operands of the next step are read before the products of this one, and the copies are issued
// between products: a wave issues in order. A segment's tiles are of equal height, in steps of 32 rows: 2 rows of
// waves take them in turn, and those of a SIMD share the columns, so that an odd step costs half.
// Measured (one MI355X): 32768 slots, 128 experts of 2048 x 7168: bf16 1120 to 1160 us, 830 to 860 TFLOP/s, with 4.5 GB of
// memory traffic (4.1 at least); the products alone took 660, the copies alone 850, so that a part of them does not
// overlap; the clock is down to 1.5 to 1.9 GHz and the matrix units are busy half of its cycles. int8 615 us, 1560 TOP/s. One expert of 8192 x 8192 with 4096 slots: row gradient 1054 TFLOP/s. 3054
// slots, 64 experts of 1408 x 2048 (the narrow tile): 80 to 90 us for 388 MB, 4.6 TB/s.
// Tried without gain: deeper rings of 64-byte stages, 256 x 128 tiles, wave priorities, three narrow blocks a CU, the row
// gradient's 16-bit rows through LDS, streaming stores of the rows.
//
// Experts' gradient, k_grad_w: 128 x 256 tiles, two blocks a CU, so that one multiplies while the other
// starts or stores; both operands are read transposed, through a map of the positions' rows in LDS.
// Measured: 32 experts of 2880 x 2880, 16384 slots to bf16 375 us, 725 TFLOP/s (256 x 256 tiles of one block a CU were no
// faster; the stores alone take 104, all but the stores 319); 64 experts of 1408 x 2048, 24576
// slots to float32 228 us, of which writing 738 MB alone takes 132. Weighted, with rows of two terms: the former 604 us,
// matrix units busy half of the cycles (reading X's operand once for both terms made no difference).
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
typedef float f32x4 __attribute__((ext_vector_type(4)));
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

// Geometry: WM x WN waves, each SM x SN tiles of 32 x 32; RB bytes of every row a stage, rings of NSA slots for the
// first operand (activations) and NSB >= NSA for the second (weights); OCC waves a SIMD. TX: rows that a segment's
// tiles may have beyond BM (the last ring slot of the weights makes room for them). KW: groups of those waves that
// take RB bytes of the rows in turn, each with rings of its own, and add up their sums at the end.
template <int WM_, int WN_, int SM_, int SN_, int RB_, int NSA_, int NSB_, int OCC_, int TX_ = 0, int KW_ = 1>
struct Tile {
    static constexpr int WM = WM_, WN = WN_, SM = SM_, SN = SN_, RB = RB_, NSA = NSA_, NSB = NSB_, OCC = OCC_, TX = TX_, KW = KW_;
    static constexpr int waves = WM * WN, threads = 64 * waves * KW;
    static constexpr int BM = 32 * WM * SM, BN = 32 * WN * SN, MX = SM + TX / (32 * WM);
    static constexpr int a_slot = BM * RB, b_slot = BN * RB;
    static constexpr int rings = NSA * a_slot + NSB * b_slot, lds = KW * rings;
    static_assert(NSA * TX * RB <= (NSB - NSA) * b_slot, "room for the taller tiles");
};
template <int N>
using Int = std::integral_constant<int, N>;

// The neighbour's value (lane ^ 1).
__device__ __forceinline__ float swap1(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0xb1, 0xf, 0xf, true));
}
// Two columns a store: of the values of rows r and r + 1 in columns c (even lanes) and c + 1 (odd lanes), even lanes
// get row r of both columns, odd lanes row r + 1.
struct Pair {
    float lo, hi;
};
__device__ __forceinline__ Pair pair_up(float a, float b, bool odd) {
    const float got = swap1(odd ? a : b);
    return Pair{odd ? got : a, odd ? b : got};
}
template <class Elem>
__device__ __forceinline__ uint32_t packed(Pair p) {
    typedef Elem Two __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, Two{(Elem)p.lo, (Elem)p.hi});
}

// M tile and column tile of this block: tiles ordered by expert, chunk of M tiles, column tile,
// an eighth of them to each XCD. False: none.
struct Where {
    int e, m0, m_len, nt;
};
template <int BM, int TX>
__device__ __forceinline__ bool find_tile(const ExpertGemm& P, int b, int n_nt, Where& w) {
    const int total = P.tile_off[P.E] * n_nt;
    const int part = (total + 7) >> 3, q = b >> 3, t = (b & 7) * part + q;
    if (q >= part || t >= total) return false;
    const int4 ti = *(const int4*)(P.tile_tab + 4 * (int64_t)(t / n_nt));
    w.e = __builtin_amdgcn_readfirstlane(ti.x);
    const int first = __builtin_amdgcn_readfirstlane(ti.y);
    const int row0 = __builtin_amdgcn_readfirstlane(ti.z);
    const int rows = __builtin_amdgcn_readfirstlane(ti.w);
    const int tiles = tiles_of(rows, BM, TX);
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
__device__ __forceinline__ void gemm_x(const ExpertGemm& P, int block) {
    using Elem = typename T::Elem;
    constexpr int RB = G::RB, W = G::waves;
    constexpr int KS = RB / (int)sizeof(Elem), KA = KS * G::KW;   // reduction elements of a group of waves and of all, per stage
    constexpr int EC = 16 / (int)sizeof(Elem);    // elements of a chunk
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int cols = TR ? P.K : P.N, depth = TR ? P.N : P.K;
    Where at;
    if (!find_tile<G::BM, G::TX>(P, block, (cols + G::BN - 1) / G::BN, at)) return;
    const int e = at.e, m0 = at.m0, m_len = at.m_len, col0 = at.nt * G::BN;

    const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wv = wave % W, wk = wave / W;
    const int wm = wv / G::WN, wn = wv % G::WN;   // waves of a SIMD (wv, wv + 4) share the columns: uneven rows meet there
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
    const int nst = (depth + KA - 1) / KA;
    const int subs = (m_len + 31) >> 5;           // 32-row sub-tiles: of wave row wm, wm, wm + WM, ...
    const void* zero = g_zero;

    // ---- copies of a stage, 1 KB each: activation rows, 1024 / RB a copy and dealt out to the waves in turn (so
    // that a shorter tile's rows are the first copies of all of them), then weights
    constexpr int CR = 1024 / RB, CL = RB / 16;   // rows of a copy, lanes of a row
    constexpr int CA = ((G::BM + G::TX) / CR + W - 1) / W, CB = G::BN / CR / W;
    const int n_copies = subs * (32 / CR);
    static_assert(CB * CR * W == G::BN, "whole copies per wave");
    const uint8_t* ap[CA];
    // of this lane's chunk, of copies i with i % 2 = 0 and 1: the swizzle goes by the row mod 16
    const auto chunk_k = [&](int i) { return wk * KS + ((lane % CL) ^ swz<RB>(lane / CL + (CR == 8 ? 8 * ((i * W + wv) & 1) : 0))) * EC; };
    const int a_k[2] = {chunk_k(0), chunk_k(1)};
    auto find_rows = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < CA; i++) {
            const int R = (i * W + wv) * CR + lane / CL;
            const int j = m0 + min(R, m_len - 1);
            const int64_t row = P.a_rows ? P.a_rows[j] : j;
            ap[i] = (const uint8_t*)P.A + (row * P.lda + a_k[i & 1]) * (int64_t)sizeof(Elem);
        }
    };
    constexpr int BROW = TR ? G::BN * 2 : RB;        // bytes of a row of the weight tile in LDS
    constexpr int BLR = BROW / 16;                   // lanes of a row
    const uint8_t* bp[CB];
    int b_k[CB];   // reduction element of this lane's chunk
    static_assert(!TR || G::KW == 1, "the groups' parts are of the rows' bytes");
    const int64_t bstep = TR ? (int64_t)KS * P.K * (int)sizeof(Elem) : RB * G::KW;
#pragma unroll
    for (int i = 0; i < CB; i++) {
        const int R = (wv * CB + i) * (64 / BLR) + lane / BLR;
        if (TR) {
            const int c = min(col0 + (((lane % BLR) ^ swz_t(R)) * EC), cols - EC);
            b_k[i] = R;
            bp[i] = (const uint8_t*)P.W + (((int64_t)e * P.N + R) * P.K + c) * (int64_t)sizeof(Elem);
        } else {
            b_k[i] = wk * KS + ((lane % CL) ^ swz<RB>(R)) * EC;
            bp[i] = (const uint8_t*)P.W + (((int64_t)e * P.N + min(col0 + R, cols - 1)) * P.K + b_k[i]) * (int64_t)sizeof(Elem);
        }
    }
    // copy i of a wave's: of a stage's activations, of its weights; to: the ring slot
    auto copy_a = [&](int i, int s, uint32_t to) __attribute__((always_inline)) {
        if (i * W + wv < n_copies) {
            const bool in = s * KA + a_k[i & 1] < depth;   // what passes the end is zero on both sides
            dma16v(in ? (const void*)ap[i] : zero, lds0 + to + (i * W + wv) * 1024);
            ap[i] += RB * G::KW;
        }
    };
    auto copy_b = [&](int i, int s, uint32_t to) __attribute__((always_inline)) {
        const bool in = s * KA + b_k[i] < depth;
        dma16v(in ? (const void*)bp[i] : zero, lds0 + to + (wv * CB + i) * 1024);
        bp[i] += bstep;
    };

    typename T::Acc acc[G::MX][G::SN];
    const int l16 = lane & 15;
    const uint32_t a_lane = (wm * 32 + l32) * RB;
    uint32_t b_lane[G::SN];
#pragma unroll
    for (int c = 0; c < G::SN; c++)
        b_lane[c] = TR ? (8 * h + (l16 >> 2)) * BROW + (l16 & 1) * 8 +
                             ((((wn * G::SN + c) * 4 + ((lane >> 4) & 1) * 2 + ((l16 >> 1) & 1)) ^ swz_t(l16 >> 2)) << 4)
                       : ((wn * G::SN + c) * 32 + l32) * RB;
    struct Frag {
        i32x4 a[G::MX], b[G::SN];
    };
    // operands of 32-byte step q of the stage in these slots
    auto read = [&](Frag& f, uint32_t sa, uint32_t sb, int q, auto n_c) __attribute__((always_inline)) {
        const uint8_t *pa = smem + sa + a_lane, *pb = smem + sb;
        const uint32_t ch = (uint32_t)((2 * q + h) ^ swz<RB>(l32)) << 4;
#pragma unroll
        for (int c = 0; c < G::SN; c++) {
            if (TR) f.b[c] = read_t<BROW>(pb + b_lane[c] + q * 16 * BROW);
            else f.b[c] = *(const i32x4*)(pb + b_lane[c] + ch);
        }
#pragma unroll
        for (int i = 0; i < decltype(n_c)::value; i++) f.a[i] = *(const i32x4*)(pa + i * G::WM * 32 * RB + ch);
    };
    auto multiply = [&](const Frag& f, int from, int to) __attribute__((always_inline)) {
#pragma unroll
        for (int i = from; i < to; i++)
#pragma unroll
            for (int c = 0; c < G::SN; c++) acc[i][c] = T::mfma(f.a[i], f.b[c], acc[i][c]);
    };
    // n_c: sub-tiles of this wave; tall_c: of a tile of more than BM rows
    auto k_loop = [&](auto n_c, auto tall_c) __attribute__((always_inline)) {
        constexpr int MACT = decltype(n_c)::value, Q = RB / 32, NSA = G::NSA;
        constexpr bool tall = decltype(tall_c)::value;
        constexpr int NSB = tall ? NSA : G::NSB, a_slot = tall ? (G::BM + G::TX) * RB : G::a_slot;
        constexpr int NCA = tall ? CA : (G::BM / CR + W - 1) / W;   // activation copies of a wave at most
        static_assert(NSA == 2 && NSA * a_slot + NSB * G::b_slot <= G::rings, "");
        auto slot_a = [&](int i) { return (uint32_t)(wk * G::rings + i * a_slot); };
        auto slot_b = [&](int i) { return (uint32_t)(wk * G::rings + NSA * a_slot + i * G::b_slot); };
#pragma unroll
        for (int i = 0; i < MACT; i++)
#pragma unroll
            for (int c = 0; c < G::SN; c++) acc[i][c] = typename T::Acc{};
        // stage s landed; the weights of NSB - 2 stages after it may be in flight (its activations are the newest
        // but for those)
        auto landed = [&](int s) __attribute__((always_inline)) {
            if (NSB == 2 || s + NSB - 2 >= nst) wait_stage_and_barrier<0>();
            else wait_stage_and_barrier<(NSB - 2) * CB>();
        };
        // copies into the slots of stage s: stage s + NSA's activations, then stage s + NSB's weights
        auto copies = [&](int s, int sa, int sb) __attribute__((always_inline)) {
            if (s + NSA < nst) {
#pragma unroll
                for (int i = 0; i < NCA; i++) copy_a(i, s + NSA, slot_a(sa));
            }
            if (s + NSB < nst) {
#pragma unroll
                for (int i = 0; i < CB; i++) copy_b(i, s + NSB, slot_b(sb));
            }
        };
#pragma unroll
        for (int s = 0; s < NSB - 1; s++) {   // weights before the row map has arrived
#pragma unroll
            for (int i = 0; i < CB; i++)
                if (s < nst) copy_b(i, s, slot_b(s));
        }
        find_rows();
#pragma unroll
        for (int i = 0; i < NCA; i++) copy_a(i, 0, slot_a(0));
        wait_stage_and_barrier<0>();
        Frag f0, f1;
        read(f0, slot_a(0), slot_b(0), 0, n_c);
        copies(-1, NSA - 1, NSB - 1);
        int sa = 0, sb = 0;
        auto step = [&](auto q_c, Frag& now, Frag& next) __attribute__((always_inline)) {
            read(next, slot_a(sa), slot_b(sb), decltype(q_c)::value + 1, n_c);
            __builtin_amdgcn_sched_barrier(0);   // or they sink behind the products and are waited for at once
            multiply(now, 0, MACT);
            __builtin_amdgcn_sched_barrier(0);
        };
        // at the loop's head: step 0 of stage s in f0, the copies into the slots of stage s - 1 on their way
        for (int s = 0; s < nst; s++) {
            static_assert(Q == 4, "");
            step(Int<0>{}, f0, f1);
            step(Int<1>{}, f1, f0);
            step(Int<2>{}, f0, f1);
            const int pa = sa, pb = sb;
            sa ^= 1;
            sb = sb == NSB - 1 ? 0 : sb + 1;
            if (s + 1 < nst) {
                landed(s + 1);   // and every wave's reads of stage s are done
                read(f0, slot_a(sa), slot_b(sb), 0, n_c);
                __builtin_amdgcn_sched_barrier(0);
            }
            // products before the copies: a wave issues in order, and the copies take a while
            multiply(f1, 0, (MACT + 1) / 2);
            __builtin_amdgcn_sched_barrier(0);
            copies(s, pa, pb);
            multiply(f1, (MACT + 1) / 2, MACT);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    const int mine = (subs + G::WM - 1 - wm) / G::WM;   // this wave's
    using No = std::false_type;
    if (G::TX && m_len > G::BM) {
        if (mine > G::SM) k_loop(Int<G::MX>{}, std::integral_constant<bool, (G::TX > 0)>{});
        else k_loop(Int<G::SM>{}, std::integral_constant<bool, (G::TX > 0)>{});
    } else if (G::SM >= 4 && mine >= 4) k_loop(Int<(G::SM >= 4 ? 4 : 1)>{}, No{});
    else if (G::SM >= 3 && mine == 3) k_loop(Int<(G::SM >= 3 ? 3 : 1)>{}, No{});
    else if (G::SM >= 2 && mine == 2) k_loop(Int<(G::SM >= 2 ? 2 : 1)>{}, No{});
    else if (G::WM == 1 || mine == 1) k_loop(Int<1>{}, No{});
    else k_loop(Int<0>{}, No{});

    // ---- output rows (and what scales them) into the now idle ring
    int32_t* s_row = (int32_t*)smem;
    float* s_scale = (float*)(smem + (G::BM + G::TX) * 4);
    __syncthreads();
    for (int r = tid; r < G::BM + G::TX; r += G::threads) {
        const int j = m0 + min(r, m_len - 1);
        const int o = P.out_rows ? P.out_rows[j] : j;
        s_row[r] = o;
        if constexpr (std::is_same<T, I8>::value) s_scale[r] = P.a_scale[P.a_rows ? P.a_rows[j] : j];
        else if (OUT16) s_scale[r] = P.row_w ? P.row_w[o] : 1.f;
    }
    __syncthreads();

    if constexpr (G::KW > 1) {   // the groups' sums, added in order by the waves for a part of the rows each
        static_assert(G::KW == 4 && W == 1 && G::SN == 1 && !OUT16, "a wave a group, eight rows of a sub-tile a wave");
        typedef std::conditional_t<std::is_same<T, I8>::value, int32_t, float> Sum;
        Sum* part = (Sum*)(smem + (G::BM + G::TX) * 8);
        static_assert((G::BM + G::TX) * 8 + G::KW * G::SM * 4096 <= G::lds, "the ring has room");
#pragma unroll
        for (int i = 0; i < G::SM; i++)
            if (32 * i < m_len) {
#pragma unroll
                for (int v = 0; v < 16; v++) part[((wk * G::SM + i) * 16 + v) * 64 + lane] = acc[i][0][v];
            }
        __syncthreads();
        const int col = col0 + l32;
        float scale = 1.f;
        if constexpr (std::is_same<T, I8>::value) scale = P.w_scale[(int64_t)e * P.N + min(col, cols - 1)];
#pragma unroll
        for (int i = 0; i < G::SM; i++) {
            if (32 * i >= m_len) break;
            const int base = 32 * i + 8 * wk + 4 * h;
#pragma unroll
            for (int u = 0; u < 4; u++) {
                Sum sum = part[(i * 16 + 4 * wk + u) * 64 + lane];
#pragma unroll
                for (int w = 1; w < G::KW; w++) sum += part[((w * G::SM + i) * 16 + 4 * wk + u) * 64 + lane];
                float v = (float)sum;
                if constexpr (std::is_same<T, I8>::value) v *= s_scale[base + u] * scale;
                if (base + u < m_len && col < cols) ((float*)P.out)[(uint64_t)(uint32_t)s_row[base + u] * (uint32_t)cols + col] = v;
            }
        }
        return;
    }

    // ---- element 4 g + u of lane l: row 8 g + 4 (l / 32) + u of the sub-tile, column l % 32. A tile's edges are told
    // apart once: 128 stores a lane with their own conditions took as long as the products of 20 stages.
    const int col = col0 + wn * G::SN * 32 + l32, col_left = cols - col;
    const bool odd = lane & 1;
    float ws[G::SN];
    if constexpr (std::is_same<T, I8>::value) {
#pragma unroll
        for (int c = 0; c < G::SN; c++) ws[c] = P.w_scale[(int64_t)e * P.N + min(col + 32 * c, cols - 1)];
    }
    auto put = [&](int i, auto rows_c, auto cols_c) __attribute__((always_inline)) {
        constexpr bool all_rows = decltype(rows_c)::value, all_cols = decltype(cols_c)::value;
        const int base = (i * G::WM + wm) * 32 + 4 * h;
        float dot[8];   // OUT16: of this lane's 8 rows with those of x, over its columns
        uint32_t x[8][G::SN];
        if (OUT16 && P.dots) {   // all loads before the first use
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const int m = base + 4 * j - 2 * (j & 1) + odd;   // 8 (j / 2) + 2 (j % 2)
                const Elem* from = (const Elem*)P.x + (uint64_t)(uint32_t)s_row[min(m, m_len - 1)] * (uint32_t)cols + (col - odd);
#pragma unroll
                for (int c = 0; c < G::SN; c++) x[j][c] = all_cols || 32 * c < col_left ? *(const uint32_t*)(from + 32 * c) : 0u;
            }
        }
#pragma unroll
        for (int g = 0; g < 4; g++) {
            const i32x4 row = *(const i32x4*)(s_row + base + 8 * g);
            f32x4 sc;
            if (std::is_same<T, I8>::value || OUT16) sc = *(const f32x4*)(s_scale + base + 8 * g);
            if constexpr (OUT16) {
#pragma unroll
                for (int u = 0; u < 4; u += 2) {
                    const bool in = all_rows || base + 8 * g + u + odd < m_len;
                    const uint64_t from = (uint64_t)(uint32_t)(odd ? row[u + 1] : row[u]) * (uint32_t)cols + (col - odd);
                    const float scale = odd ? sc[u + 1] : sc[u];
                    float d = 0.f;
#pragma unroll
                    for (int c = 0; c < G::SN; c++) {
                        const Pair v = pair_up(acc[i][c][4 * g + u], acc[i][c][4 * g + u + 1], odd);
                        if (!(in && (all_cols || 32 * c < col_left))) continue;   // columns are even
                        if (P.dots) {
                            typedef Elem Two __attribute__((ext_vector_type(2)));
                            const Two w = __builtin_bit_cast(Two, x[2 * g + u / 2][c]);
                            d = fmaf(v.lo, (float)w[0], fmaf(v.hi, (float)w[1], d));
                        }
                        if (P.out) *(uint32_t*)((Elem*)P.out + from + 32 * c) = packed<Elem>(Pair{v.lo * scale, v.hi * scale});
                    }
                    dot[2 * g + u / 2] = d;
                }
            } else {
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    if (!all_rows && base + 8 * g + u >= m_len) continue;
                    float* o = (float*)P.out + (uint64_t)(uint32_t)row[u] * (uint32_t)cols + col;
#pragma unroll
                    for (int c = 0; c < G::SN; c++) {
                        float v;
                        if constexpr (std::is_same<T, I8>::value) v = (float)acc[i][c][4 * g + u] * (sc[u] * ws[c]);
                        else v = acc[i][c][4 * g + u];
                        if (all_cols || 32 * c < col_left) o[32 * c] = v;
                    }
                }
            }
        }
        if (OUT16 && P.dots) {   // the 16 lanes of one parity: halve the rows a lane holds, then add the last two lanes
            const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
#pragma unroll
            for (int j = 0; j < 4; j++) dot[j] = (b4 ? dot[j + 4] : dot[j]) + __shfl_xor(b4 ? dot[j] : dot[j + 4], 16);
#pragma unroll
            for (int j = 0; j < 2; j++) dot[j] = (b3 ? dot[j + 2] : dot[j]) + __shfl_xor(b3 ? dot[j] : dot[j + 2], 8);
            dot[0] = (b2 ? dot[1] : dot[0]) + __shfl_xor(b2 ? dot[0] : dot[1], 4);
            dot[0] += __shfl_xor(dot[0], 2);
            const int m = base + 8 * (2 * b4 + b3) + 2 * b2 + odd;
            if (!(lane & 2) && m < m_len) P.dots[(int64_t)s_row[m] * P.dot_parts + at.nt * G::WN + wn] = dot[0];
        }
    };
    const bool wide = col0 + G::BN <= cols;
#pragma unroll
    for (int i = 0; i < G::MX; i++) {
        const int left = m_len - (i * G::WM + wm) * 32;
        if (left <= 0) break;
        if (left >= 32 && wide) put(i, std::true_type{}, std::true_type{});
        else put(i, std::false_type{}, std::false_type{});
    }
}

template <class T, int TR, bool OUT16, class G>
__global__ __launch_bounds__(G::threads, G::OCC) void k_gemm_x(ExpertGemm P) {
    gemm_x<T, TR, OUT16, G>(P, (int)blockIdx.x);
}

// ---------------------------------------------------------------- expert gradient
// dW_e tile of BM rows (n) x BN columns (k); the reduction runs along e's positions, KS a stage, both operands
// read transposed. Weighted calls bring rows of dY times their factors (scaling them here, between
// the LDS and the products, took 575 us for 32 experts of 2880 x 2880 and 16384 slots, against 437 without it) as
// TERMS rows of the type each, whose sum they are: rounded to one 16-bit row, they would leave d_w with half again
// the error of its own rounding, or of 16 bits where it is float32. A stage has the terms of its positions behind one another
// and their rows of X once.
constexpr int kMapRows = 512;   // ring of positions whose rows are in LDS, refilled by halves

template <class G, int TERMS>
struct GradWGeometry {
    static constexpr int KS = TERMS == 1 ? G::RB / 2 : 16;   // positions of a stage
    static constexpr int stage = KS * (TERMS * G::BM + G::BN) * 2;
    static constexpr int NS = TERMS == 2 ? G::NSA + 1 : G::NSA;
    static constexpr int lds = NS * stage + kMapRows * 8;
};

template <class T, class G, int TERMS>
__device__ __forceinline__ void grad_w(const ExpertGradW& P, int block, int part) {
    using Elem = typename T::Elem;
    using Geo = GradWGeometry<G, TERMS>;
    constexpr int W = G::waves, NS = Geo::NS, KS = Geo::KS, stage = Geo::stage;
    static_assert(G::NSA == G::NSB, "one ring");
    constexpr int KA = TERMS * KS, Q = KA / 16, kHalf = kMapRows / 2 / KS;   // rows of dY and MFMA steps of a stage; stages of half a map
    static_assert(NS + 2 <= kHalf && kMapRows % (2 * KS) == 0, "the map covers the stages in flight");
    constexpr int AROW = G::BM * 2, BROW = G::BN * 2, ALR = AROW / 16, BLR = BROW / 16;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    int32_t* s_dy = (int32_t*)(smem + NS * stage);   // rows of dY and X of the positions
    int32_t* s_x = s_dy + kMapRows;

    // every expert's tiles in eight parts, one to each XCD and another for the next expert: experts are of very
    // different lengths (an eighth of all tiles each left the XCDs with the long ones working when the others were
    // done: 64 experts of 1408 x 2048 with Zipf(1.1) ids 337 us against 303). A part is a rectangle, which reads fewer
    // rows than a strip (24576 slots to float32, 64 experts of 1408 x 2048: 241 us by strips, now 228)
    const int n_nt = (P.N + G::BM - 1) / G::BM, n_kt = (P.K + G::BN - 1) / G::BN, pn = 8 / P.pk;
    const int per_k = (n_kt + P.pk - 1) / P.pk, per = (n_nt + pn - 1) / pn * per_k;
    const int q = block >> 3, e = q / per, xcd = (block + e) & 7, xn = xcd / P.pk, xk = xcd % P.pk;
    const int tn = xn * n_nt / pn + (q - e * per) / per_k, tk = xk * n_kt / P.pk + (q - e * per) % per_k;
    if (e >= P.E || tn >= (xn + 1) * n_nt / pn || tk >= (xk + 1) * n_kt / P.pk) return;
    const int row0 = tn * G::BM, col0 = tk * G::BN;
    int j0 = P.bounds[e], len = P.bounds[e + 1] - j0;
    if (P.splits > 1) {   // a part of the segment's stages, summed up by the pass that joins the parts
        const int per = expert_split_len(len, P.splits), from = part * per;
        if (from >= len) return;
        j0 += from;
        len = min(len - from, per);
    }

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
        }
    };
    constexpr int CA = KA * ALR / 64 / W, CB = KS * BLR / 64 / W;
    static_assert(CA * 64 * W == KA * ALR && CB * 64 * W == KS * BLR, "whole copies per wave");
    // Where a stage's copies read: the rows come from the map in LDS two stages ahead of the copies and become
    // addresses a stage ahead, between the products (a copy that waits for its address keeps the products waiting).
    int row_a[CA], row_b[CB];
    const uint8_t *from_a[CA], *from_b[CB];
    const uint8_t *base_a[CA], *base_b[CB];
    const uint32_t step_a = (uint32_t)P.ldy * 2, step_b = (uint32_t)P.K * 2;
#pragma unroll
    for (int i = 0; i < CA; i++) {
        const int R = (wv * CA + i) * (64 / ALR) + lane / ALR;
        base_a[i] = (const uint8_t*)P.dY + (R / KS * P.term_stride + min(row0 + ((lane % ALR) ^ swz_t(R)) * 8, P.ldy - 8)) * 2ll;
    }
#pragma unroll
    for (int i = 0; i < CB; i++) {
        const int R = (wv * CB + i) * (64 / BLR) + lane / BLR;
        base_b[i] = (const uint8_t*)P.X + min(col0 + ((lane % BLR) ^ swz_t(R)) * 8, P.K - 8) * 2ll;
    }
    auto rows = [&](int s) __attribute__((always_inline)) {
        const int at = (s * KS) & (kMapRows - 1);
#pragma unroll
        for (int i = 0; i < CA; i++) {
            const int R = (wv * CA + i) * (64 / ALR) + lane / ALR;
            row_a[i] = s_dy[at + R % KS];
        }
#pragma unroll
        for (int i = 0; i < CB; i++) row_b[i] = s_x[at + (wv * CB + i) * (64 / BLR) + lane / BLR];
    };
    auto locate = [&](int s) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < CA; i++) from_a[i] = base_a[i] + (uint64_t)(uint32_t)row_a[i] * step_a;
#pragma unroll
        for (int i = 0; i < CB; i++) from_b[i] = base_b[i] + (uint64_t)(uint32_t)row_b[i] * step_b;
        if ((s + 1) * KS > len) {   // the segment's end: zeros past it
#pragma unroll
            for (int i = 0; i < CA; i++)
                if (s * KS + ((wv * CA + i) * (64 / ALR) + lane / ALR) % KS >= len) from_a[i] = (const uint8_t*)zero;
#pragma unroll
            for (int i = 0; i < CB; i++)
                if (s * KS + (wv * CB + i) * (64 / BLR) + lane / BLR >= len) from_b[i] = (const uint8_t*)zero;
        }
    };
    auto issue = [&](int slot) __attribute__((always_inline)) {
        const uint32_t st = lds0 + (uint32_t)(slot * stage);
#pragma unroll
        for (int i = 0; i < CA; i++) dma16v(from_a[i], st + (wv * CA + i) * 1024);
#pragma unroll
        for (int i = 0; i < CB; i++) dma16v(from_b[i], st + KA * AROW + (wv * CB + i) * 1024);
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
    auto read = [&](Frag& f, int slot, int q) __attribute__((always_inline)) {
        const uint8_t* st = smem + slot * stage;
#pragma unroll
        for (int c = 0; c < G::SN; c++) f.b[c] = read_t<BROW>(st + KA * AROW + b_lane[c] + (TERMS == 1 ? q : 0) * 16 * BROW);
#pragma unroll
        for (int i = 0; i < G::SM; i++) f.a[i] = read_t<AROW>(st + a_lane[i] + q * 16 * AROW);
    };
    auto multiply = [&](const Frag& f, int from = 0, int to = G::SM) __attribute__((always_inline)) {
#pragma unroll
        for (int i = from; i < to; i++)
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
        for (int s = 0; s < NS - 1 && s < nst; s++) {
            rows(s);
            locate(s);
            issue(s);
        }
        rows(NS - 1);
        locate(NS - 1);
        landed(0);
        if (NS - 1 < nst) issue(NS - 1);
        rows(NS);   // past the end: rows that are not copied
        locate(NS);
        Frag f0, f1;
        read(f0, 0, 0);
        int slot = 0;
        // stage s, its first step's operands in f; the next stage's go to f where it has an even number of steps, else to g
        auto one = [&](int s, Frag& f, Frag& g) __attribute__((always_inline)) {
            auto step = [&](auto q_c, Frag& now, Frag& next) __attribute__((always_inline)) {
                constexpr int q = decltype(q_c)::value;
                read(next, slot, q + 1);
                if (q == 0) rows(s + NS + 1);
                __builtin_amdgcn_sched_barrier(0);
                multiply(now);
                __builtin_amdgcn_sched_barrier(0);
            };
            static_assert(Q == 2 || Q == 3, "");
            step(Int<0>{}, f, g);
            if constexpr (Q == 3) step(Int<1>{}, g, f);
            Frag &last = Q == 3 ? f : g, &first = Q == 3 ? g : f;
            const int was = slot;
            slot = slot == NS - 1 ? 0 : slot + 1;
            if (s + 1 < nst) {
                landed(s + 1);
                read(first, slot, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
            multiply(last, 0, G::SM / 2);
            __builtin_amdgcn_sched_barrier(0);
            if (s + NS < nst) {
                issue(was);
                // The half of the map that holds stage s and the kHalf - 1 before it has served, once s is its
                // last stage: the rows two halves on take its place, needed kHalf - NS stages from now.
                if ((s + 1) % kHalf == 0 && (s + 1 + kHalf) * KS < len) map((s + 1 + kHalf) * KS);
            }
            multiply(last, G::SM / 2, G::SM);
            locate(s + NS + 1);
            __builtin_amdgcn_sched_barrier(0);
        };
        for (int s = 0; s < nst; s++) {
            one(s, f0, f1);
            if constexpr (Q == 3)
                if (++s < nst) one(s, f1, f0);
        }
    }
    if (TERMS > 1 && P.unscale) {
        const float u = *P.unscale;
#pragma unroll
        for (int i = 0; i < G::SM; i++)
#pragma unroll
            for (int c = 0; c < G::SN; c++) acc[i][c] *= u;
    }

    // ---- element 4 g + u of lane l: row 8 g + 4 (l / 32) + u of the tile, column l % 32
    const int row = row0 + wm * G::SM * 32 + 4 * h, col = col0 + wn * G::SN * 32 + l32;
    const bool odd = lane & 1;
    auto put = [&](auto all_c) __attribute__((always_inline)) {
        constexpr bool all = decltype(all_c)::value;
        const int row_left = P.N - row, col_left = P.K - col;
        float* o = (P.splits > 1 ? P.parts + (int64_t)part * P.E * P.N * P.K : (float*)P.dW) + ((int64_t)e * P.N + row) * P.K + col;
#pragma unroll
        for (int i = 0; i < G::SM; i++)
#pragma unroll
            for (int v = 0; v < 16; v++) {
                const int r = i * 32 + 8 * (v >> 2) + (v & 3);
                if (all || r < row_left) {
#pragma unroll
                    for (int c = 0; c < G::SN; c++)
                        if (all || 32 * c < col_left) __builtin_nontemporal_store(acc[i][c][v], o + (int64_t)r * P.K + 32 * c);
                }
            }
    };
    if (P.f32 || P.splits > 1) {
        if (row0 + G::BM <= P.N && col0 + G::BN <= P.K) put(std::true_type{});
        else put(std::false_type{});
        return;
    }
    // 16-bit rows go through the ring's LDS, to be stored as whole lines
    if constexpr (TERMS < 3) {   // three terms: of a float32 d_w alone
        static_assert(G::BM * BROW <= NS * stage, "the tile's rows");
        uint8_t* tile = smem;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < G::SM; i++)
#pragma unroll
            for (int v = 0; v < 16; v += 2) {
                const int r = wm * G::SM * 32 + 4 * h + i * 32 + 8 * (v >> 2) + (v & 3) + odd;
#pragma unroll
                for (int c = 0; c < G::SN; c++) {
                    const int piece = ((wn * G::SN + c) ^ (r & 7)) * 64;   // of 64 bytes, apart in neighbouring rows
                    *(uint32_t*)(tile + r * BROW + piece + (l32 >> 1) * 4) = packed<Elem>(pair_up(acc[i][c][v], acc[i][c][v + 1], odd));
                }
            }
        __syncthreads();
        constexpr int RL = BROW / 16;   // lanes of a row
        const int col_out = col0 + tid % RL * 8;
        Elem* o = (Elem*)P.dW + ((int64_t)e * P.N + row0) * P.K + col_out;
#pragma unroll 4
        for (int r = tid / RL; r < G::BM; r += G::threads / RL) {
            const int at = ((tid % RL * 16) ^ ((r & 7) * 64));
            const i32x4 v = *(const i32x4*)(tile + r * BROW + at);
            if (row0 + r < P.N && col_out < P.K) __builtin_nontemporal_store(v, (i32x4*)(o + (int64_t)r * P.K));
        }
    }
}

template <class T, class G, int TERMS>
__global__ __launch_bounds__(G::threads, G::OCC) void k_grad_w(ExpertGradW P) {
    grad_w<T, G, TERMS>(P, (int)blockIdx.x, (int)blockIdx.y);
}

using Wide = Tile<2, 4, 4, 2, 128, 2, 3, 2, 64>;   // up to 320 x 256, one block a CU
using Narrow = Tile<1, 4, 2, 1, 128, 2, 3, 2>;    // 64 x 128, two blocks a CU
using Deep = Tile<1, 1, 2, 1, 128, 2, 3, 1, 0, 4>;   // 64 x 32, four waves along the rows, one block a CU
using GradW = Tile<1, 4, 4, 2, 64, 3, 3, 2>;      // 128 x 256, two blocks a CU

// Both gradients in one launch, blocks of the experts' first: neither fills the chip when they are small (both gradients,
// us per call in one launch against two: E8 k2 300 x 200, 30 tokens 20.0 / 22.8; E8 k2 512 x 512, 2000 tokens 29.0 / 36.6;
// E32 k4 2880 x 2880, 100 tokens 226 / 238; E64 k6 1408 x 2048, 500 tokens 189 / 189).
template <class T, bool OUT16, int TERMS>
__global__ __launch_bounds__(GradW::threads, GradW::OCC) void k_grads(ExpertGradW w, ExpertGemm g, int w_grid) {
    static_assert(GradW::threads == Narrow::threads && GradW::OCC == Narrow::OCC, "one launch");
    const int block = (int)blockIdx.x, w_blocks = w_grid * w.splits;
    if (block < w_blocks) grad_w<T, GradW, TERMS>(w, block % w_grid, block / w_grid);
    else gemm_x<T, 1, OUT16, Narrow>(g, block - w_blocks);
}

// Few blocks of the narrow tile: four times as many, whose waves share the depth (mul_mat_id by the grouped path, narrow /
// deep in us on one MI355X, by narrow blocks: 32, E8 k2 512 x 512, 20 tokens 10.1 / 8.3; 70, E4 k1 256 x 7168, 2000 tokens
// 57.6 / 48.5; 72, E5 k2 943 x 4192, 141 tokens 43.3 / 22.4; 80, E72 k8 74 x 2608, 68 tokens 23.7 / 14.8; 152, E16 k2 1024 x
// 1024, 100 tokens 15.0 / 16.6; 184, E8 k2 1024 x 4096, 500 tokens 41.2 / 48.6; 320, E8 k2 4096 x 4096, 64 tokens 68 / 69; int8
// 72 34.9 / 24.7, 80 22.4 / 17.5, 184 34.9 / 42.3).
bool deep_tile(const ExpertGemm& a) {
    return (int64_t)a.m_tiles_max * ((a.N + Narrow::BN - 1) / Narrow::BN) <= 96;
}

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
    if (a.tile_m == Wide::BM) return launch<T, TR, OUT16, Wide>(a, st);
    if constexpr (!TR)
        if (deep_tile(a)) return launch<T, TR, OUT16, Deep>(a, st);
    return launch<T, TR, OUT16, Narrow>(a, st);
}

// Parts of an expert's columns, of eight parts of its tiles, that read the fewest rows of dY and X.
int grad_w_pk(int64_t N, int64_t K) {
    const int64_t n = (N + GradW::BM - 1) / GradW::BM, k = (K + GradW::BN - 1) / GradW::BN;
    int best = 1;
    int64_t least = INT64_MAX;
    for (int pk = 1; pk <= 8; pk *= 2) {
        const int64_t pn = 8 / pk, read = (n + pn - 1) / pn * GradW::BM + (k + pk - 1) / pk * GradW::BN;
        if (read < least) least = read, best = pk;
    }
    return best;
}

template <class T, bool OUT16, int TERMS>
hipError_t launch_both(const ExpertGemm& a, ExpertGradW w, hipStream_t st) {
    w.pk = grad_w_pk(w.N, w.K);
    constexpr int w_lds = GradWGeometry<GradW, TERMS>::lds, lds = w_lds > Narrow::lds ? w_lds : Narrow::lds;
    static PerDeviceOnce cap;
    if (const hipError_t e = set_lds_cap(cap, (const void*)k_grads<T, OUT16, TERMS>, lds)) return e;
    const int64_t w_grid = expert_grad_w_grid(w), grid = w_grid * w.splits + expert_gemm_grid(a, 1);
    k_grads<T, OUT16, TERMS><<<(unsigned)grid, GradW::threads, lds, st>>>(w, a, (int)w_grid);
    return hipGetLastError();
}
template <class T, bool OUT16>
hipError_t launch_both(const ExpertGemm& a, const ExpertGradW& w, hipStream_t st) {
    return w.terms == 1 ? launch_both<T, OUT16, 1>(a, w, st) : w.terms == 2 ? launch_both<T, OUT16, 2>(a, w, st) : launch_both<T, OUT16, 3>(a, w, st);
}

template <class T, int TERMS>
hipError_t launch_w(ExpertGradW a, hipStream_t st) {
    using G = GradW;
    constexpr int lds = GradWGeometry<G, TERMS>::lds;
    a.pk = grad_w_pk(a.N, a.K);
    static PerDeviceOnce cap;
    if (const hipError_t e = set_lds_cap(cap, (const void*)k_grad_w<T, G, TERMS>, lds)) return e;
    const dim3 grid((unsigned)expert_grad_w_grid(a), (unsigned)a.splits);
    k_grad_w<T, G, TERMS><<<grid, G::threads, lds, st>>>(a);
    return hipGetLastError();
}
template <class T>
hipError_t launch_w(const ExpertGradW& a, hipStream_t st) {
    return a.terms == 1 ? launch_w<T, 1>(a, st) : a.terms == 2 ? launch_w<T, 2>(a, st) : launch_w<T, 3>(a, st);
}

}  // namespace

int expert_gemm_tile_x(int tile_m) { return tile_m == Wide::BM ? Wide::TX : Narrow::TX; }

// The wide tile from 48 rows an expert on, where there are blocks enough for it (mul_mat_id, wide against narrow in us
// per call on one MI355X: E128 k8 2048 x 7168 T = 384 645 / 647, T = 768 665 / 724, T = 1536 713 / 914; E64 k4
// 1408 x 2048 T = 512 98 / 100, T = 2048 117 / 135; E16 k4 2880 x 2880 T = 256, 192 blocks, 53 / 81; E8 k2 4096 x 4096
// T = 512, 128 blocks, 78 / 73; E8 k2 1024 x 4096 T = 2048, 64 blocks, 110 / 59; E1 4096 x 4096 T = 256, 16, 105 / 41).
int expert_gemm_tile_m(int64_t slots, int64_t E, int64_t cols) {
    const int64_t rows = slots / E, blocks = E * ((rows + Wide::BM - 1) / Wide::BM) * ((cols + Wide::BN - 1) / Wide::BN);
    return rows >= 48 && blocks >= 160 ? Wide::BM : Narrow::BM;
}

int64_t expert_gemm_grid(const ExpertGemm& a, int grad) {
    const int64_t cols = grad ? a.K : a.N;
    const int64_t bn = a.tile_m == Wide::BM ? Wide::BN : !grad && deep_tile(a) ? Deep::BN : Narrow::BN;
    return ((int64_t)a.m_tiles_max * ((cols + bn - 1) / bn) + 7) / 8 * 8;
}

int expert_dot_parts(const ExpertGemm& a) {
    const int bn = a.tile_m == Wide::BM ? Wide::BN : Narrow::BN, wn = a.tile_m == Wide::BM ? Wide::WN : Narrow::WN;
    return (a.K + bn - 1) / bn * wn;
}

// Two blocks a CU, where that takes 32 stages of an expert's 32 positions or more off its longest row of products: the
// parts and their join cost some 15 us (us per call, in parts against whole: E1 1024 x 1024, 32768 slots 135 / 586;
// E8 278 x 128, 14905 slots with Zipf(1.1) ids 61 / 82; in two parts E8 1024 x 1024, 8192 slots 57 / 41, which is left
// whole).
int expert_grad_w_splits(int64_t slots, int64_t E, int64_t N, int64_t K) {
    const int64_t blocks = E * ((N + GradW::BM - 1) / GradW::BM) * ((K + GradW::BN - 1) / GradW::BN);
    const int64_t stages = slots / E / 32;
    int64_t s = 512 / blocks;
    s = s > 16 ? 16 : s;
    return s > 1 && stages - stages / s >= 32 ? (int)s : 1;
}

int64_t expert_grad_w_grid(const ExpertGradW& a) {
    const int64_t n = (a.N + GradW::BM - 1) / GradW::BM, k = (a.K + GradW::BN - 1) / GradW::BN;
    const int pk = grad_w_pk(a.N, a.K), pn = 8 / pk;
    return 8ll * a.E * ((n + pn - 1) / pn) * ((k + pk - 1) / pk);
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

hipError_t launch_expert_grads(const ExpertGemm& a, const ExpertGradW& w, hipStream_t st) {
    if (a.type == kElemBf16) return a.out16 ? launch_both<Bf16, true>(a, w, st) : launch_both<Bf16, false>(a, w, st);
    return a.out16 ? launch_both<F16, true>(a, w, st) : launch_both<F16, false>(a, w, st);
}
bool expert_grads_share(const ExpertGemm& a) { return a.tile_m == Narrow::BM; }

hipError_t launch_expert_grad_w(const ExpertGradW& a, hipStream_t st) {
    return a.type == kElemBf16 ? launch_w<Bf16>(a, st) : launch_w<F16>(a, st);
}

}  // namespace moe
