// What the gradients of mul_mat_id do after the grouped products, joining the slots' gradient rows g:
//   d_src1[r] = sum over r's slots, ascending, of route_w * g   (float32, rounded once)
//   d_route_w[i] = sum over the columns of g[i] * src1[r]
#include "quant_rows.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int64_t kMaxGrid = 1 << 22;   // blocks take several rows past it

// One block a row of d_src1 and its k slots; the dot products' parts of a wave are in LDS.
template <class Elem>
__global__ __launch_bounds__(kThreads) void k_grad_rows(GradRowsArgs a) {
    extern __shared__ float s_dot[];   // [kWaves][k]
    typedef Elem Vec __attribute__((ext_vector_type(4)));
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        if (a.d_route_w) {
            for (int i = tid; i < kWaves * a.k; i += kThreads) s_dot[i] = 0.f;
            __syncthreads();
        }
        for (int c0 = 0; c0 < a.K; c0 += 4 * kThreads) {
            const int c = c0 + 4 * tid;
            const bool in = c < a.K;
            f32x4 acc = {0.f, 0.f, 0.f, 0.f}, x = acc;
            if (in && a.d_route_w) {
                const Vec v = *(const Vec*)((const Elem*)a.x + r * a.K + c);
#pragma unroll
                for (int u = 0; u < 4; u++) x[u] = (float)v[u];
            }
            for (int s = 0; s < a.k; s++) {
                const int64_t i = r * a.k + s;
                const int32_t e = a.ids[i];
                if (e < 0 || e >= a.E) continue;
                const f32x4 g = in ? *(const f32x4*)(a.g + i * a.K + c) : f32x4{0.f, 0.f, 0.f, 0.f};
                const float w = a.route_w ? a.route_w[i] : 1.f;
#pragma unroll
                for (int u = 0; u < 4; u++) acc[u] = fmaf(w, g[u], acc[u]);
                if (a.d_route_w) {
                    float d = in ? g[0] * x[0] + g[1] * x[1] + g[2] * x[2] + g[3] * x[3] : 0.f;
                    for (int m = 32; m; m >>= 1) d += __shfl_xor(d, m);
                    if (lane == 0) s_dot[wv * a.k + s] += d;
                }
            }
            if (in && a.d_x) {
                Vec v;
#pragma unroll
                for (int u = 0; u < 4; u++) v[u] = (Elem)acc[u];
                *(Vec*)((Elem*)a.d_x + r * a.K + c) = v;
            }
        }
        if (a.d_route_w) {
            __syncthreads();
            for (int s = tid; s < a.k; s += kThreads) {
                float d = 0.f;
                for (int w = 0; w < kWaves; w++) d += s_dot[w * a.k + s];
                a.d_route_w[r * a.k + s] = d;
            }
        }
        __syncthreads();
    }
}

// 16 lanes a slot.
__global__ __launch_bounds__(kThreads) void k_join_dots(JoinDotsArgs a) {
    constexpr int kLanes = 16;
    const int l = threadIdx.x % kLanes;
    for (int64_t i = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes; i < a.n;
         i += (int64_t)gridDim.x * (kThreads / kLanes)) {
        const int32_t e = a.ids[i];
        float d = 0.f;
        if (e >= 0 && e < a.E)
            for (int p = l; p < a.parts; p += kLanes) d += a.dots[i * a.parts + p];
#pragma unroll
        for (int m = kLanes / 2; m; m >>= 1) d += __shfl_xor(d, m);
        if (l == 0) a.out[i] = d;
    }
}

// dW from the parts of its sums, ascending; eight neighbours a thread (an expert's elements are a multiple of 8).
template <class Elem>
__global__ __launch_bounds__(kThreads) void k_join_w(ExpertGradW a) {
    const int64_t per = (int64_t)a.N * a.K, all = per * a.E;
    for (int64_t i = 8 * ((int64_t)blockIdx.x * kThreads + threadIdx.x); i < all; i += 8 * (int64_t)gridDim.x * kThreads) {
        const int e = (int)(i / per);
        const int len = a.bounds[e + 1] - a.bounds[e];
        f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
        if (len > 0) {
            const int parts = (len - 1) / expert_split_len(len, a.splits) + 1;
            for (int p = 0; p < parts; p++) {
                const f32x4* v = (const f32x4*)(a.parts + p * all + i);
                lo += v[0];
                hi += v[1];
            }
        }
        if (a.f32) {
            f32x4* o = (f32x4*)((float*)a.dW + i);
            o[0] = lo;
            o[1] = hi;
        } else {
            typedef Elem Vec __attribute__((ext_vector_type(8)));
            Vec v;
#pragma unroll
            for (int u = 0; u < 4; u++) {
                v[u] = (Elem)lo[u];
                v[4 + u] = (Elem)hi[u];
            }
            *(Vec*)((Elem*)a.dW + i) = v;
        }
    }
}

// A wave takes the largest finite magnitude of a row of d_dst, then of its products with the row's factors.
template <int SRC>
__global__ __launch_bounds__(kThreads) void k_grad_top(GradTopArgs a) {
    using S = QuantSrc<SRC>;
    constexpr int EC = S::EC;
    __shared__ float tops[kWaves];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    float top = 0.f;
    for (int64_t r = (int64_t)blockIdx.x * kWaves + wv; r < a.rows; r += (int64_t)gridDim.x * kWaves) {
        const typename S::Elem* row = (const typename S::Elem*)a.src + r * a.N;
        float most = 0.f;
        const auto grow = [&](float v) {
            const float m = fabsf(v);
            if (m < __builtin_inff()) most = fmaxf(most, m);
        };
        for (int64_t c = lane * EC; c < a.N; c += 64 * EC) {
            if (c + EC <= a.N) {
                const typename S::Vec v = S::load(row + c);
#pragma unroll
                for (int u = 0; u < EC; u++) grow((float)v[u]);
            } else {
                for (int64_t u = c; u < a.N; u++) grow((float)row[u]);
            }
        }
#pragma unroll
        for (int m = 32; m; m >>= 1) most = fmaxf(most, __shfl_xor(most, m));
        for (int s = lane; s < a.k; s += 64) {
            const int32_t e = a.ids[r * a.k + s];
            const float w = fabsf(a.route_w[r * a.k + s]);
            if (e >= 0 && e < a.E && w < __builtin_inff()) top = fmaxf(top, fminf(w * most, 3.402823466e38f));
        }
    }
#pragma unroll
    for (int m = 32; m; m >>= 1) top = fmaxf(top, __shfl_xor(top, m));
    if (lane == 0) tops[wv] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kWaves; w++) top = fmaxf(top, tops[w]);
        a.tops[blockIdx.x] = top;
    }
}

}  // namespace

int grad_tops(int64_t rows) {
    const int64_t blocks = (rows + kWaves - 1) / kWaves;
    return (int)(blocks < kGradTops ? blocks : kGradTops);
}
hipError_t launch_grad_top(const GradTopArgs& a, hipStream_t st) {
    if (a.rows <= 0) return hipSuccess;
    if (a.f32) k_grad_top<kElemF32><<<(unsigned)grad_tops(a.rows), kThreads, 0, st>>>(a);
    else k_grad_top<kElemF16><<<(unsigned)grad_tops(a.rows), kThreads, 0, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_join_w(const ExpertGradW& a, hipStream_t st) {
    const int64_t blocks = ((int64_t)a.E * a.N * a.K / 8 + kThreads - 1) / kThreads;
    const unsigned grid = (unsigned)(blocks < kMaxGrid ? blocks : kMaxGrid);
    if (a.type == kElemBf16) k_join_w<__bf16><<<grid, kThreads, 0, st>>>(a);
    else k_join_w<_Float16><<<grid, kThreads, 0, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_join_dots(const JoinDotsArgs& a, hipStream_t st) {
    if (a.n <= 0) return hipSuccess;
    const int64_t blocks = (a.n + kThreads / 16 - 1) / (kThreads / 16);
    k_join_dots<<<(unsigned)(blocks < kMaxGrid ? blocks : kMaxGrid), kThreads, 0, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_grad_rows(const GradRowsArgs& a, hipStream_t st) {
    if (a.rows <= 0) return hipSuccess;
    const unsigned grid = (unsigned)(a.rows < kMaxGrid ? a.rows : kMaxGrid);
    const size_t lds = a.d_route_w ? (size_t)kWaves * a.k * 4 : 0;
    if (a.type == kElemBf16) k_grad_rows<__bf16><<<grid, kThreads, lds, st>>>(a);
    else k_grad_rows<_Float16><<<grid, kThreads, lds, st>>>(a);
    return hipGetLastError();
}

}  // namespace moe
