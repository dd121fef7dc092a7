// Grouped GEMM of MXFP4 experts with MXFP4 activations on gfx950 (act_quant = 2).
//
//     out[m][n] = sum over blocks b of 2^(xa[m][b] + xw[n][b] - 254) * sum_{32} a * w
//
// over expert segments, a and w the E2M1 values of activation row m and weight row n. The
// block scaled MFMA v_mfma_scale_f32_16x16x128_f8f6f4 takes both rows' codes and scale
// bytes as they are stored: lane l holds row l % 16 and columns 32 (l / 16) .. +31 of
// each operand, 16 bytes of codes and one scale byte, and sums in float32.
//
// First form: operands straight from global memory into the MFMA layout. Block tile 64
// activation rows x 128 weight rows, 4 waves, each 32 weight rows (gate/up mode: 16 gate
// rows and the 16 up rows of the same outputs) and all 64 activation rows.
#include "moe_internal.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kBM = kFp4TileM;   // activation rows per block tile
constexpr int kW = 4;            // waves
constexpr int kBN = 32 * kW;     // weight rows per block tile
constexpr int kMChunk = 4;       // M tiles sharing each weight slab in turn

template <int MODE>
constexpr int out_cols() { return MODE == 1 ? kBN / 2 : kBN; }

__device__ __forceinline__ i32x8 operand(i32x4 v) { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

template <int MODE>
__global__ __launch_bounds__(64 * kW) void k_gemm_fp4(GemmArgs args) {
    constexpr int NTW = out_cols<MODE>();
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
    const int N = P.N, K = P.K;
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
            const int mt = t / n_nt;
            const int4 ti = *(const int4*)(P.tile_tab + 4 * (int64_t)mt);
            e = ti.x;
            first = ti.y;
            row0 = ti.z;
            rows = ti.w;
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
        m0 = row0 + j * kBM;
        m_len = min(kBM, rows - j * kBM);
    }
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, r16 = lane & 15, g4 = lane >> 4;
    const int KB = K >> 5, KH = K >> 1;
    // weight rows of this lane: MFMA tile i of the wave
    const uint8_t *wq[2], *ws[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int n = min(MODE == 1 ? nt * NTW + wv * 16 + r16 : nt * NTW + wv * 32 + i * 16 + r16, N - 1);
        const int64_t row = (int64_t)e * N + n;
        wq[i] = (const uint8_t*)(MODE == 1 && i ? P.qs2 : P.qs1) + row * KH;
        ws[i] = (const uint8_t*)(MODE == 1 && i ? P.d2 : P.d1) + row * KB;
    }
    const uint8_t *aq[4], *as[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int j = m0 + min(i * 16 + r16, m_len - 1);
        const int64_t row = P.a_rows ? (int64_t)P.a_rows[j] : (P.a_row_mod ? j % P.a_row_mod : j);
        aq[i] = (const uint8_t*)P.Aq + row * KH;
        as[i] = P.As + row * KB;
    }
    f32x4 acc[2][4];
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int b0 = 0; b0 < KB; b0 += 4) {
        // block b0 + l / 16; past the row's end: codes 0 and scale 1
        const bool in = b0 + g4 < KB;
        const int bb = in ? b0 + g4 : 0;
        i32x4 vw[2], va[4];
        int sw[2], sa[4];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            vw[i] = *(const i32x4*)(wq[i] + bb * 16);
            sw[i] = ws[i][bb];
            if (!in) {
                vw[i] = i32x4{0, 0, 0, 0};
                sw[i] = 127;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            va[i] = *(const i32x4*)(aq[i] + bb * 16);
            sa[i] = as[i][bb];
            if (!in) {
                va[i] = i32x4{0, 0, 0, 0};
                sa[i] = 127;
            }
        }
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int j = 0; j < 4; j++)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(vw[i]), operand(va[j]), acc[i][j],
                                                                             4, 4, 0, sw[i], 0, sa[j]);
    }
    // ---- epilogue: element u of lane l is weight row 4 (l / 16) + u, activation row l % 16
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const int m = j * 16 + r16;
        if (m >= m_len) continue;
        const int64_t row = P.out_rows ? P.out_rows[m0 + m] : m0 + m;
        float* o = (float*)P.out + row * P.ldo;
        if (MODE == 1) {
#pragma unroll
            for (int u = 0; u < 4; u++) {
                const int n = nt * NTW + wv * 16 + 4 * g4 + u;
                const float gv = acc[0][j][u];
                if (n < N) o[n] = gv / (1.0f + expf(-gv)) * acc[1][j][u];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    const int n = nt * NTW + wv * 32 + i * 16 + 4 * g4 + u;
                    if (n < N) o[n] = acc[i][j][u];
                }
        }
    }
}

int64_t grid_of(const GemmArgs& a) {
    const int ntw = a.mode == 1 ? kBN / 2 : kBN;
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
    if (a.mode == 1) k_gemm_fp4<1><<<(unsigned)total, 64 * kW, 0, st>>>(a);
    else k_gemm_fp4<0><<<(unsigned)total, 64 * kW, 0, st>>>(a);
    return hipGetLastError();
}

int64_t gemm_fp4_max_threads(const GemmArgs& a) { return grid_of(a) * 64 * kW; }

}  // namespace moe
