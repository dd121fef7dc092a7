// Scored routing and its gradient (moe_router_scored, moe_router_scored_backward).
//
// Forward, first form: one wavefront per token, lane l holds experts l, l + 64, ...
// Choices are float64 numbers turned into 64-bit keys that order as they do (0: never
// picked), so a pick does not depend on how a float32 exp rounds.
#include <type_traits>

#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kWaves = 4;  // tokens per block

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v = fmaxf(v, __shfl_xor(v, m));
    return v;
}
// Largest key of the wave and the lowest index that holds it.
__device__ __forceinline__ void wave_best(uint64_t& key, int& idx) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) {
        const uint64_t k2 = __shfl_xor((unsigned long long)key, m);
        const int i2 = __shfl_xor(idx, m);
        if (k2 > key || (k2 == key && i2 < idx)) {
            key = k2;
            idx = i2;
        }
    }
}
// Order key of a choice: larger numbers give larger keys, -0 counts as +0; NaN and -inf
// give 0 (never picked).
__device__ __forceinline__ uint64_t order_key(double c) {
    if (!(c > -INFINITY)) return 0;
    const uint64_t u = c == 0.0 ? 0ull : __builtin_bit_cast(uint64_t, c);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_value(uint64_t k) {
    return __builtin_bit_cast(double, (k >> 63) ? k & 0x7fffffffffffffffull : ~k);
}

__device__ __forceinline__ float load_logit(const void* p, bool bf16, int64_t i) {
    return bf16 ? __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i];
}

// Ratio of the sigmoids of l and of lmax >= l, without overflow or 0 / 0.
__device__ __forceinline__ float sigmoid_ratio(float l, float lmax) {
    if (lmax > 0.f) return (1.f + expf(-lmax)) / (1.f + expf(-l));
    return expf(l - lmax) * ((1.f + expf(lmax)) / (1.f + expf(l)));
}

template <int NC>
__global__ __launch_bounds__(64 * kWaves) void k_router_scored(RouterScoredArgs a) {
    __shared__ uint64_t s_key[kWaves][64 * NC];
    __shared__ uint64_t s_grp[kWaves][64 * NC];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int64_t t0 = (int64_t)blockIdx.x * kWaves + wv;
    const bool live_t = t0 < a.T;
    const int64_t t = live_t ? t0 : a.T - 1;    // spare waves repeat the last token and write nothing
    const int E = a.E, k = a.k, per = E / a.n_group;
    float l[NC];   // NaN taken as -inf
    float top = -INFINITY;
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int e = lane + 64 * c;
        const float x = e < E ? load_logit(a.logits, a.bf16, t * E + e) : -INFINITY;
        l[c] = x != x ? -INFINITY : x;
        top = fmaxf(top, l[c]);
    }
    top = wave_max(top);
    const bool none = top == -INFINITY, inf = top == INFINITY;
    // scores: softmax as exp(l - top) / den; infinite logits share the sum
    double den = 0;
    double s[NC];
#pragma unroll
    for (int c = 0; c < NC; c++) {
        if (a.sigmoid) s[c] = 1.0 / (1.0 + exp(-(double)l[c]));
        else s[c] = none ? 0.0 : inf ? (l[c] == INFINITY ? 1.0 : 0.0) : exp((double)l[c] - (double)top);
        den += s[c];
    }
    if (!a.sigmoid) {
        den = wave_sum(den);
#pragma unroll
        for (int c = 0; c < NC; c++) s[c] = none ? 0.0 : s[c] / den;
    }
    if (a.scores && live_t) {
#pragma unroll
        for (int c = 0; c < NC; c++) {
            const int e = lane + 64 * c;
            if (e < E) a.scores[t * E + e] = (float)s[c];
        }
    }
    uint64_t key[NC];
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int e = lane + 64 * c;
        key[c] = 0;
        if (e < E && l[c] > -INFINITY) key[c] = order_key(a.bias ? s[c] + (double)a.bias[e] : (double)l[c]);
    }
    if (a.topk_group < a.n_group) {
#pragma unroll
        for (int c = 0; c < NC; c++)
            if (lane + 64 * c < E) s_key[wv][lane + 64 * c] = key[c];
        if (a.group_top == 2 && !a.bias) {   // sums are of scores, not of logits
            __syncthreads();
#pragma unroll
            for (int c = 0; c < NC; c++)
                if (lane + 64 * c < E) s_key[wv][lane + 64 * c] = key[c] ? order_key(s[c]) : 0;
        }
        __syncthreads();
        for (int g = lane; g < a.n_group; g += 64) {
            uint64_t b1 = 0, b2 = 0;
            for (int i = 0; i < per; i++) {
                const uint64_t x = s_key[wv][g * per + i];
                if (x > b1) {
                    b2 = b1;
                    b1 = x;
                } else if (x > b2) {
                    b2 = x;
                }
            }
            uint64_t v = b1;
            if (a.group_top == 2 && b2) v = order_key(key_value(b1) + key_value(b2));
            s_grp[wv][g] = v;
        }
        __syncthreads();
        // keep the best groups: a kept group's key becomes all ones, which no key is
        for (int r = 0; r < a.topk_group; r++) {
            uint64_t bk = 0;
            int bi = 0x7fffffff;
            for (int g = lane; g < a.n_group; g += 64) {
                const uint64_t v = s_grp[wv][g];
                if (v != ~0ull && v > bk) {
                    bk = v;
                    bi = g;
                }
            }
            wave_best(bk, bi);
            if (bk && lane == (bi & 63)) s_grp[wv][bi] = ~0ull;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < NC; c++) {
            const int e = lane + 64 * c;
            if (e < E && s_grp[wv][e / per] != ~0ull) key[c] = 0;
        }
    }
    // picks: round r's logit and score are parked in lane r % 64 of slot r / 64
    float pl[NC];
    float ps[NC];
#pragma unroll
    for (int c = 0; c < NC; c++) {
        pl[c] = -INFINITY;
        ps[c] = 0.f;
    }
    for (int r = 0; r < k; r++) {
        uint64_t bk = 0;
        int bi = 0x7fffffff;
        float bl = -INFINITY, bs = 0.f;
#pragma unroll
        for (int c = 0; c < NC; c++)
            if (key[c] > bk) {
                bk = key[c];
                bi = lane + 64 * c;
                bl = l[c];
                bs = (float)s[c];
            }
        wave_best(bk, bi);
        const int own = bi & 63;
        const float vl = __shfl(bl, own), vs = __shfl(bs, own);
        if (bk) {
#pragma unroll
            for (int c = 0; c < NC; c++)
                if (bi == lane + 64 * c) key[c] = 0;
        }
        if (lane == 0 && live_t) a.ids[t * k + r] = bk ? bi : -1;
#pragma unroll
        for (int c = 0; c < NC; c++)
            if (bk && lane + 64 * c == r) {
                pl[c] = vl;
                ps[c] = vs;
            }
    }
    if (a.renorm) {
        float m = -INFINITY;
#pragma unroll
        for (int c = 0; c < NC; c++) m = fmaxf(m, pl[c]);
        m = wave_max(m);
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < NC; c++) {
            if (!(pl[c] > -INFINITY)) ps[c] = 0.f;
            else if (m == INFINITY && !a.sigmoid) ps[c] = pl[c] == m ? 1.f : 0.f;
            else ps[c] = a.sigmoid ? sigmoid_ratio(pl[c], m) : expf(pl[c] - m);
            sum += ps[c];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int c = 0; c < NC; c++) ps[c] = sum > 0.f ? ps[c] / sum : 0.f;
    }
#pragma unroll
    for (int c = 0; c < NC; c++)
        if (lane + 64 * c < k && live_t) a.w[t * k + lane + 64 * c] = a.scale * ps[c];
}

// Gradient, first form: one wavefront per token. With w'_j the weight of pick j without
// the scale (s_j / sum of the picks' s with renorm, else s_j) and g_j its gradient,
//     q_e = s_e dS_e + sum over picks j of e:  scale * w'_j * (g_j - sum_m w'_m g_m)  (renorm)
//                                              scale * w'_j * g_j                     (else)
// which is s_e * dL/ds_e, and
//     softmax: dl_e = q_e - s_e * sum_f q_f        sigmoid: dl_e = q_e * (1 - s_e).
// With renorm the picks' part of sum_f q_f is zero, so only dS enters it.
template <int NC>
__global__ __launch_bounds__(64 * kWaves) void k_router_grad(RouterGradArgs a) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kWaves + wv;
    if (t >= a.T) return;
    const int E = a.E, k = a.k;
    float l[NC];
    float top = -INFINITY;
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int e = lane + 64 * c;
        const float x = e < E ? load_logit(a.logits, a.bf16, t * E + e) : -INFINITY;
        l[c] = x != x ? -INFINITY : x;
        top = fmaxf(top, l[c]);
    }
    top = wave_max(top);
    const bool none = top == -INFINITY, inf = top == INFINITY;
    float s[NC], rest[NC];   // rest: 1 - s of a sigmoid, without its cancellation
    float den = 0.f;
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const float z = expf(-fabsf(l[c])), r = 1.f / (1.f + z);
        rest[c] = l[c] > 0.f ? z * r : r;
        if (a.sigmoid) s[c] = l[c] > 0.f ? r : z * r;
        else s[c] = none ? 0.f : inf ? (l[c] == INFINITY ? 1.f : 0.f) : expf(l[c] - top);
        den += s[c];
    }
    if (!a.sigmoid) {
        den = wave_sum(den);
#pragma unroll
        for (int c = 0; c < NC; c++) s[c] = none ? 0.f : s[c] / den;
    }
    float q[NC], sum_q = 0.f;
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int e = lane + 64 * c;
        q[c] = a.ds && e < E && l[c] > -INFINITY ? s[c] * a.ds[t * a.ds_stride + e] : 0.f;
        sum_q += q[c];
    }
    // picks in chunks of 64: lane j of a chunk holds pick j
    auto logit_of = [&](int e) -> float {
        const bool ok = e >= 0 && e < E;
        const float x = ok ? load_logit(a.logits, a.bf16, t * E + e) : -INFINITY;
        return x != x ? -INFINITY : x;
    };
    float pmax = -INFINITY, psum = 0.f, dot = 0.f;
    auto weight = [&](float x) -> float {   // of a pick with logit x, up to the renorm sum
        if (!(x > -INFINITY)) return 0.f;
        if (a.renorm) {
            if (a.sigmoid) return sigmoid_ratio(x, pmax);
            return pmax == INFINITY ? (x == pmax ? 1.f : 0.f) : expf(x - pmax);
        }
        if (a.sigmoid) return 1.f / (1.f + expf(-x));
        return inf ? (x == INFINITY ? 1.f : 0.f) / den : expf(x - top) / den;
    };
    if (a.renorm) {
        for (int j = lane; j < k; j += 64) pmax = fmaxf(pmax, logit_of(a.ids[t * k + j]));
        pmax = wave_max(pmax);
        for (int j = lane; j < k; j += 64) {
            const float w = weight(logit_of(a.ids[t * k + j]));
            psum += w;
            if (w > 0.f) dot += w * a.dw[t * k + j];
        }
        psum = wave_sum(psum);
        dot = wave_sum(dot);
        dot = psum > 0.f ? dot / psum : 0.f;
    }
    for (int j0 = 0; j0 < k; j0 += 64) {
        const int j = j0 + lane;
        int e = j < k ? a.ids[t * k + j] : -1;
        float w = j < k ? weight(logit_of(e)) : 0.f;
        if (!(w > 0.f)) e = -1;
        float v = 0.f;
        if (e >= 0 && e < E) {
            if (a.renorm) v = a.scale * (w / psum) * (a.dw[t * k + j] - dot);
            else v = a.scale * w * a.dw[t * k + j];
        }
        if (!a.renorm) sum_q += v;
        const int n = min(64, k - j0);
        for (int i = 0; i < n; i++) {
            const int ei = __builtin_amdgcn_readlane(e, i);
            const float vi = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), i));
#pragma unroll
            for (int c = 0; c < NC; c++)
                if (ei == lane + 64 * c) q[c] += vi;
        }
    }
    if (!a.sigmoid) sum_q = wave_sum(sum_q);
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int e = lane + 64 * c;
        if (e >= E) continue;
        const float d = !(l[c] > -INFINITY) ? 0.f : a.sigmoid ? q[c] * rest[c] : q[c] - s[c] * sum_q;
        if (a.bf16) ((__bf16*)a.dl)[t * E + e] = (__bf16)d;
        else ((float*)a.dl)[t * E + e] = d;
    }
}

template <class A, class F>
hipError_t by_width(const A& a, F&& f) {
    const int nc = (a.E + 63) / 64;
    const unsigned grid = (unsigned)((a.T + kWaves - 1) / kWaves);
    if (nc <= 1) f(std::integral_constant<int, 1>{}, grid);
    else if (nc <= 2) f(std::integral_constant<int, 2>{}, grid);
    else if (nc <= 4) f(std::integral_constant<int, 4>{}, grid);
    else if (nc <= 8) f(std::integral_constant<int, 8>{}, grid);
    else f(std::integral_constant<int, 16>{}, grid);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_router_scored(const RouterScoredArgs& a, hipStream_t st) {
    if (a.T <= 0) return hipSuccess;
    return by_width(a, [&](auto nc, unsigned grid) {
        k_router_scored<decltype(nc)::value><<<grid, 64 * kWaves, 0, st>>>(a);
    });
}

hipError_t launch_router_grad(const RouterGradArgs& a, hipStream_t st) {
    if (a.T <= 0) return hipSuccess;
    return by_width(a, [&](auto nc, unsigned grid) {
        k_router_grad<decltype(nc)::value><<<grid, 64 * kWaves, 0, st>>>(a);
    });
}

}  // namespace moe
