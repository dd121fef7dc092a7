// Grouped GEMM of MXFP4 experts with MXFP4 activations on gfx950 (act_quant = 2).
//
//     out[m][n] = sum over blocks b of 2^(xa[m][b] + xw[n][b] - 254) * sum_{32} a * w
//
// over expert segments, a and w the E2M1 values of activation row m and weight row n. The
// block scaled MFMA v_mfma_scale_f32_32x32x64_f8f6f4 takes both rows' codes and scale
// bytes as they are stored: lane l holds row l % 32 and columns 32 (l / 32) .. +31 of
// each operand, 16 bytes of codes and one scale byte, and sums in float32. (The
// 16x16x128 form runs at half its rate: 4.8 against 9.5 PFLOP/s from registers.)
//
// Block tile: up to 128 activation rows x 256 weight rows, 4 waves; wave w owns 64 weight
// rows (gate/up mode: 32 gate rows and the 32 up rows of the same outputs) and all
// activation rows. A stage is 128 columns, 64 bytes of codes a row.
//   * Codes go global -> LDS by direct copies into a ring of three slots, two stages
//     ahead; the gather through the row map is the copies' addresses. Loading the weights
//     straight into MFMA registers would save LDS traffic, but neighbouring lanes then
//     hold neighbouring rows, and such loads run at 16 bytes a clock and CU against 57
//     for rows of 64 bytes.
//   * LDS rows are 64 bytes; 16-byte chunk c of row r sits at c ^ ((r >> 2) & 3), so the
//     8 lanes of a ds_read_b128 phase hit different banks.
//   * Scale bytes come 16 a row (four stages) into registers, one row a thread, and go to
//     LDS as one word per row and stage; the MFMA step j of lane half h takes byte
//     2 j + h of its row's word.
//   * Activation rows are padded to whole stages (codes 0), so the row ends need no care
//     beyond addresses that stay inside the weight rows.
//   * Gate/up mode quantizes h in its epilogue, from the float32 accumulators.
//   * An expert's rows are split into equal tiles (of whole 32-row MFMA columns) rather
//     than full ones and a rest: a block's time goes with its rows.
//   * Output rows that no further kernel of the call reads are stored past the caches
//     (32768 rows x 2048: 482 -> 474 us); before a weighted sum the plain stores are better,
//     which leave part of the rows in the caches (sum: 40 us against 43).
//
// Measured (this kernel alone): 4096 tokens x 8 slots, 128 experts of 2048 x 7168, 474 us, 2030
// TFLOP/s; 4096 x 4, 32 experts of 2880 x 2880, 189 us, 1440 TFLOP/s. No pipe is full in the first: MFMA
// pipes busy 23 % of the cycles, LDS 12 %, L2 to LDS 15 bytes a clock and CU of the 57 that such rows
// reach (3.5 GB in requests of 64 bytes, 1.4 GB from HBM). It takes 297 us without the copies and 450 with
// them and one MFMA in eight: what bounds it is waiting for them, once per 128 columns, with 512 cycles
// of MFMA per wave between two waits. Segments of a few rows over a multiple of 128 take one more tile, with
// all of its weight copies (uniform ids: 320 tiles for 256, 146 for 128). Tried and slower at these two
// sizes: 128 x 128 tiles 507 and 196;
// weights from global memory straight into MFMA registers 604 and 210; 256 x 256 tiles with
// 8 waves 497 and 183; persistent blocks 506 and 185.
#include <type_traits>

#include "lds_dma.h"
#include "moe_internal.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kBM = kFp4TileM;   // activation rows per block tile
constexpr int kW = 4;            // waves, along the weight rows
constexpr int kThreads = 64 * kW;
constexpr int kKS = 128;         // columns per stage
constexpr int kRow = kKS / 2;    // code bytes of a row per stage
constexpr int kNS = 3;           // ring slots
constexpr int kSS = 4;           // stages whose scale bytes are in LDS
constexpr int kNT = 2;           // 32-row MFMA tiles of weight rows per wave
constexpr int kBN = 32 * kNT * kW;       // weight rows per block tile
constexpr int kRows = kBM + kBN;         // rows of a ring slot: activations, weights
constexpr int kStage = kRows * kRow;     // bytes of a ring slot
constexpr int kLds = kNS * kStage + kSS * kRows * 4;
constexpr int kMChunk = 8;       // M tiles sharing each weight slab in turn (4: 195 against 186 us)

__device__ __forceinline__ i32x8 operand(i32x4 v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }
__device__ __forceinline__ int swz(int r) { return (r >> 2) & 3; }

template <class V>
__device__ __forceinline__ V load_unaligned(const uint8_t* p) {
    V v;
    __builtin_memcpy(&v, p, sizeof(V));
    return v;
}
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

constexpr int out_cols(int mode) { return mode == 1 ? kBN / 2 : kBN; }

template <int MODE>
__global__ __launch_bounds__(kThreads, 2) void k_gemm_fp4(GemmArgs args) {
    constexpr int NTW = out_cols(MODE);
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    uint32_t* s_scale = (uint32_t*)(smem + kNS * kStage);       // [kSS][kRows]

    // ---- tile of this block (the XCD-aware order of the bf16 grouped GEMM)
    int b = (int)blockIdx.x, pi = 0;
    {
        const GemmProblem& P0 = args.p[0];
        const int reg0 = ((P0.m_tiles_max * ((P0.N + NTW - 1) / NTW) + 7) >> 3) * 8;
        if (b >= reg0) {
            pi = 1;
            b -= reg0;
        }
    }
    const GemmProblem& P = args.p[pi];
    const int N = P.N, KB = P.K >> 5;
    const int n_nt = (N + NTW - 1) / NTW;
    int e, m0, m_len, nt;
    {
        const int m_tiles = P.bounds ? P.tile_off[P.n_seg] : P.n_seg * ((P.seg_len + kBM - 1) / kBM);
        const int total = m_tiles * n_nt;
        const int part = (total + 7) >> 3;
        const int q = b >> 3;
        const int t = (b & 7) * part + q;
        if (q >= part || t >= total) return;
        int first, tiles, row0, rows;
        if (P.bounds) {
            const int4 ti = *(const int4*)(P.tile_tab + 4 * (int64_t)(t / n_nt));
            e = __builtin_amdgcn_readfirstlane(ti.x);
            first = __builtin_amdgcn_readfirstlane(ti.y);
            row0 = __builtin_amdgcn_readfirstlane(ti.z);
            rows = __builtin_amdgcn_readfirstlane(ti.w);
            tiles = (rows + kBM - 1) / kBM;
        } else {
            tiles = (P.seg_len + kBM - 1) / kBM;
            e = t / (n_nt * tiles);
            first = e * tiles;
            row0 = e * P.seg_len;
            rows = P.seg_len;
        }
        const int r = t - n_nt * first;
        const int c = r / (kMChunk * n_nt);
        const int g = min(kMChunk, tiles - c * kMChunk);
        const int rr = r - c * kMChunk * n_nt;
        nt = rr / g;
        const int j = c * kMChunk + (rr - nt * g);
        const int height = ((rows + tiles - 1) / tiles + 31) & ~31;
        m0 = row0 + j * height;
        m_len = min(height, rows - j * height);
        if (m_len <= 0) return;   // the last tiles of a long segment may be empty
    }
    const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
    const int nst = (P.K + kKS - 1) / kKS;

    // Row of the weight tensor of block-local weight row R (gate/up mode: each wave's 32 gate
    // rows, then the 32 up rows of the same outputs).
    auto is_up = [&](int R) -> bool { return MODE == 1 && (R & 32); };
    auto wrow = [&](int R) -> int {
        return min(MODE == 1 ? nt * NTW + (R >> 6) * 32 + (R & 31) : nt * NTW + R, N - 1);
    };
    // Activation row of tile row R, relative to act_row0 (rows that are not gathered are counted
    // from the tile's first).
    const int64_t act_row0 = P.a_rows ? 0 : (P.a_row_mod ? m0 % P.a_row_mod : m0);
    auto act_row = [&](int R) -> uint32_t {
        const int j = min(R, m_len - 1);
        return P.a_rows ? (uint32_t)P.a_rows[m0 + j] : (uint32_t)j;
    };
    // ---- copies: copy i of wave w covers rows 16 (w * n + i) .. +15, 4 lanes a row
    constexpr int CA = kBM / 16 / kW, CW = kBN / 16 / kW;   // per wave and stage
    constexpr int kCopies = CA + CW;
    const uint32_t KH = (uint32_t)KB * 16, KHp = (uint32_t)fp4_code_row(P.K);
    const int64_t w0 = (int64_t)e * N + wrow(0);
    const uint8_t* aq = (const uint8_t*)uniform_ptr(P.Aq + act_row0 * KHp);
    const uint8_t* q1 = (const uint8_t*)uniform_ptr(P.qs1 + w0 * KH);
    const uint8_t* q2 = MODE == 1 ? (const uint8_t*)uniform_ptr(P.qs2 + w0 * KH) : q1;
    uint32_t a_off[CA], w_off[CW];
#pragma unroll
    for (int i = 0; i < CA; i++) {
        const int R = (wv * CA + i) * 16 + (lane >> 2);
        a_off[i] = act_row(R) * KHp + (((lane & 3) ^ swz(R)) << 4);
    }
#pragma unroll
    for (int i = 0; i < CW; i++) {
        const int R = (wv * CW + i) * 16 + (lane >> 2);
        w_off[i] = (uint32_t)(wrow(R) - wrow(0)) * KH + (((lane & 3) ^ swz(R)) << 4);
    }
    auto issue = [&](int s, int slot) __attribute__((always_inline)) {
        const uint32_t st = lds0 + (uint32_t)(slot * kStage);
#pragma unroll
        for (int i = 0; i < CA; i++) dma16(aq + s * kRow, a_off[i], st + (wv * CA + i) * 1024);
#pragma unroll
        for (int i = 0; i < CW; i++) {
            // a chunk past the row's end re-reads the stage's first one (the activation codes there are 0)
            const int lc = (lane & 3) ^ swz((wv * CW + i) * 16 + (lane >> 2));
            const uint32_t adj = 4 * s + lc >= KB ? (uint32_t)(lc << 4) : 0u;
            dma16((is_up((wv * CW + i) * 16) ? q2 : q1) + s * kRow, w_off[i] - adj,
                  st + kBM * kRow + (wv * CW + i) * 1024);
        }
    };
    // ---- scale bytes of kSS stages: weight row tid (the first kBN threads) and activation row tid
    const bool has_w = tid < kBN, has_a = tid < kBM;
    const uint8_t* sw = (const uint8_t*)(is_up(tid & (kBN - 1)) ? P.d2 : P.d1) +
                        ((int64_t)e * N + wrow(tid & (kBN - 1))) * KB;
    const uint8_t* sa = P.As + (act_row0 + act_row(tid & (kBM - 1))) * fp4_scale_row(P.K);
    i32x4 rw, ra;
    // Raw loads only: what depends on the row's end is done when the words are stored. Weight words
    // that would pass the row's end are read from its last 4 bytes; activation rows are padded.
    auto load_scales = [&](int S) __attribute__((always_inline)) {
        const int o = 16 * S;
        ra = *(const i32x4*)(sa + o);
        if (o + 16 <= KB) {
            rw = load_unaligned<i32x4>(sw + o);
        } else if (KB >= 4) {
#pragma unroll
            for (int d = 0; d < 4; d++) rw[d] = load_unaligned<int>(sw + min(o + 4 * d, KB - 4));
        } else {
            rw = i32x4{0, 0, 0, 0};
            for (int i = 0; i < KB; i++) rw[0] |= (int)sw[i] << (8 * i);
        }
    };
    // Bytes past the row's end: 0, a finite scale (the codes of the activations there are 0).
    auto store_scales = [&](int S) __attribute__((always_inline)) {
        const int o = 16 * S;
        if (o + 16 > KB && KB >= 4) {
#pragma unroll
            for (int d = 0; d < 4; d++) {
                const int past = o + 4 * d - (KB - 4);
                if (past > 0) rw[d] = past < 4 ? (int)((uint32_t)rw[d] >> (8 * past)) : 0;
            }
        }
        if (has_a) {
#pragma unroll
            for (int d = 0; d < 4; d++) s_scale[d * kRows + tid] = (uint32_t)ra[d];
        }
        if (has_w) {
#pragma unroll
            for (int d = 0; d < 4; d++) s_scale[d * kRows + kBM + tid] = (uint32_t)rw[d];
        }
    };

    // ---- a wave's operands: MFMA step j of a stage, and the stage's scale words
    struct Frag {
        i32x4 a[4], w[kNT];
    };
    struct Scale {
        int a[4], w[kNT];
    };
    f32x16 acc[4][kNT];
    auto read = [&](Frag& f, int slot, int j, auto n_c) __attribute__((always_inline)) {
        const uint8_t* st = smem + slot * kStage + (((2 * j + h) ^ swz(l32)) << 4) + l32 * kRow;
#pragma unroll
        for (int c = 0; c < kNT; c++) f.w[c] = *(const i32x4*)(st + (kBM + wv * 32 * kNT + c * 32) * kRow);
#pragma unroll
        for (int i = 0; i < decltype(n_c)::value; i++) f.a[i] = *(const i32x4*)(st + i * 32 * kRow);
    };
    auto read_scale = [&](Scale& v, int s, auto n_c) __attribute__((always_inline)) {
        const uint32_t* sc = s_scale + (s & (kSS - 1)) * kRows + l32;
#pragma unroll
        for (int c = 0; c < kNT; c++) v.w[c] = (int)(sc[kBM + wv * 32 * kNT + c * 32] >> (8 * h));
#pragma unroll
        for (int i = 0; i < decltype(n_c)::value; i++) v.a[i] = (int)(sc[i * 32] >> (8 * h));
    };
    auto multiply = [&](const Frag& f, const Scale& v, auto j_c, auto n_c) __attribute__((always_inline)) {
        constexpr int SEL = decltype(j_c)::value * 2;
#pragma unroll
        for (int i = 0; i < decltype(n_c)::value; i++)
#pragma unroll
            for (int c = 0; c < kNT; c++) {
                // gate/up: weights as the row operand, so that a lane holds one activation row's columns
                if (MODE == 1)
                    acc[i][c] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        operand(f.w[c]), operand(f.a[i]), acc[i][c], 4, 4, SEL, v.w[c], SEL, v.a[i]);
                else
                    acc[i][c] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                        operand(f.a[i]), operand(f.w[c]), acc[i][c], 4, 4, SEL, v.a[i], SEL, v.w[c]);
            }
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    auto k_loop = [&](auto n_c) __attribute__((always_inline)) {
        constexpr int MACT = decltype(n_c)::value;
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int c = 0; c < kNT; c++) acc[i][c] = f32x16{};
        load_scales(0);
        issue(0, 0);
        if (nst > 1) issue(1, 1);
        if (nst > 2) issue(2, 2);
        store_scales(0);
        if (nst > kSS) load_scales(1);
        wait_stage_and_barrier<0>();
        Frag f0, f1;
        Scale v0, v1;
        read_scale(v0, 0, n_c);
        read(f0, 0, 0, n_c);
        int slot = 0;
        // at the loop's head: step 0 of stage s in f0, its scales in v0; copies up to stage s + 2 issued
        for (int s = 0; s < nst; s++) {
            read(f1, slot, 1, n_c);
            multiply(f0, v0, I0{}, n_c);
            v1 = v0;
            __builtin_amdgcn_sched_barrier(0);
            // stage s + 1 landed (of the copies, only those of s + 2 may be in flight), this wave's
            // reads of stage s are done, and so are the other waves' after the barrier
            if (s + 2 < nst) wait_stage_and_barrier<kCopies>();
            else wait_stage_and_barrier<0>();
            if (s + 3 < nst) issue(s + 3, slot);
            slot = slot == 2 ? 0 : slot + 1;
            if (s + 1 < nst) {
                if (((s + 1) & (kSS - 1)) == 0) {
                    store_scales((s + 1) / kSS);
                    lds_barrier();
                    if (s + 1 + kSS < nst) load_scales((s + 1) / kSS + 1);
                }
                read_scale(v0, s + 1, n_c);
                read(f0, slot, 0, n_c);
            }
            multiply(f1, v1, I1{}, n_c);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    const int mact = (m_len + 31) >> 5;   // occupied 32-row sub-tiles (block-uniform)
    if (mact >= 4) k_loop(std::integral_constant<int, 4>{});
    else if (mact == 3) k_loop(std::integral_constant<int, 3>{});
    else if (mact == 2) k_loop(std::integral_constant<int, 2>{});
    else k_loop(std::integral_constant<int, 1>{});

    // ---- output rows into the (now idle) ring
    int32_t* s_orow = (int32_t*)smem;
    if (MODE == 0) {
        __syncthreads();
        if (tid < kBM) {
            const int j = m0 + min(tid, m_len - 1);
            s_orow[tid] = P.out_rows ? P.out_rows[j] : j;
        }
        __syncthreads();
    }

    // ---- epilogue: element 4 g + u of lane l is row 8 g + 4 (l / 32) + u of the row operand's
    // 32 and column l % 32
    if (MODE == 1) {
        // h = silu(gate) * up, quantized where it is: the wave's 32 outputs of a row are one
        // block, 16 of them in this lane and 16 in lane l ^ 32. Blocks past N are the padding
        // of the rows the down product reads.
        const int blk = nt * (NTW / 32) + wv;
        const bool pad = blk * 32 >= N;
        const int64_t cr = fp4_code_row(N), sr = fp4_scale_row(N);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (i * 32 >= m_len) continue;
            const int m = i * 32 + l32;
            float hv[16];
            uint32_t top = 0;
#pragma unroll
            for (int v = 0; v < 16; v++) {
                const float gv = acc[i][0][v];
                hv[v] = pad ? 0.f : gv / (1.0f + expf(-gv)) * acc[i][kNT - 1][v];
                top = max(top, __float_as_uint(hv[v]) & 0x7fffffffu);
            }
            top = max(top, (uint32_t)__shfl_xor((int)top, 32));
            const int field = (int)(top >> 23);
            const bool bad = field == 255;
            const uint32_t byte = bad ? 255u : (uint32_t)max(field - 2, 0);
            const float scale = __uint_as_float(byte ? byte << 23 : 0x00400000u);
            uint32_t q[4];   // codes of columns 8 g + 4 h .. +3
#pragma unroll
            for (int g = 0; g < 4; g++) {
                uint32_t c = 0;
                c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, hv[4 * g], hv[4 * g + 1], scale, 0);
                c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, hv[4 * g + 2], hv[4 * g + 3], scale, 1);
                q[g] = bad ? 0u : c & 0xffffu;
            }
            // lane half h keeps columns 16 h .. +15: it gets the partner's part of them for its own of the others
            const uint32_t give = h ? q[0] | q[1] << 16 : q[2] | q[3] << 16;
            const uint32_t got = (uint32_t)__shfl_xor((int)give, 32);
            uint2 d;
            d.x = h ? (got & 0xffffu) | q[2] << 16 : q[0] | got << 16;
            d.y = h ? got >> 16 | q[3] << 16 : q[1] | (got & 0xffff0000u);
            if (m < m_len) {
                const int64_t row = m0 + m;
                *(uint2*)((uint8_t*)P.out + row * cr + blk * 16 + 8 * h) = d;
                if (h == 0) P.out_s[row * sr + blk] = pad ? 127 : (uint8_t)byte;
            }
        }
    } else {
        // this lane's rows are 4 h + constants: one base and one limit for all of them
        const int left = m_len - 4 * h;
        const int32_t* orow_h = s_orow + 4 * h;
        float* o = (float*)P.out + nt * NTW + wv * 32 * kNT + l32;
        const int n_left = N - (nt * NTW + wv * 32 * kNT + l32);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (i * 32 >= m_len) continue;
#pragma unroll
            for (int v = 0; v < 16; v++) {
                const int m = i * 32 + 8 * (v >> 2) + (v & 3);
                if (m >= left) continue;
                float* r = o + orow_h[m] * P.ldo;
#pragma unroll
                for (int c = 0; c < kNT; c++)
                    if (32 * c < n_left) {
                        if (args.stream_out) __builtin_nontemporal_store(acc[i][c][v], r + 32 * c);
                        else r[32 * c] = acc[i][c][v];
                    }
            }
        }
    }
}

template <int MODE>
hipError_t launch(const GemmArgs& a, int64_t total, hipStream_t st) {
    static PerDeviceOnce lds_cap;
    if (const hipError_t e = set_lds_cap(lds_cap, (const void*)k_gemm_fp4<MODE>, kLds)) return e;
    k_gemm_fp4<MODE><<<(unsigned)total, kThreads, kLds, st>>>(a);
    return hipGetLastError();
}

int64_t grid_of(const GemmArgs& a) {
    const int ntw = out_cols(a.mode);
    int64_t total = 0;
    for (int i = 0; i < a.n_prob; i++) {
        const GemmProblem& p = a.p[i];
        total += ((int64_t)p.m_tiles_max * ((p.N + ntw - 1) / ntw) + 7) / 8 * 8;
    }
    return total;
}

}  // namespace

hipError_t launch_gemm_fp4(const GemmArgs& a0, hipStream_t st) {
    GemmArgs a = a0;
    if (a.n_prob < 2) a.p[1] = GemmProblem{};
    const int64_t total = grid_of(a);
    if (total <= 0) return hipSuccess;
    a.grid_real = (int32_t)total;
    return a.mode == 1 ? launch<1>(a, total, st) : launch<0>(a, total, st);
}

int64_t gemm_fp4_max_threads(const GemmArgs& a) { return grid_of(a) * kThreads; }

}  // namespace moe
