// Scored routing and its gradient (moe_router_scored, moe_router_scored_backward).
//
// Choices are compared as float64 numbers, so a pick does not depend on how a float32
// exponential rounds. Two kernels:
//   * k_route_rows (up to 512 experts, 15 picks, 16 groups; every usual router): 16 lanes a
//     token, four tokens a wave, so that every reduction is four row rotations and no LDS
//     crossbar. Choices are float32 first: each is at most kErr from the exact one, so
//     picks and groups whose neighbours in the order are further apart than twice that are
//     the exact ones. The rest are routed again in float64 by the whole wave: about one token
//     in a thousand of random float32 logits; with a bias also every token whose last pick ties
//     with the first expert left, or whose last group does, exactly (65536 x 256 bf16 with a
//     bias of zeros 67 us against 42 with a random one, 8 groups 98 against 65; all logits
//     equal 186 and 273).
//       - a lane holds chunks of four experts (chunk lane + 16 q), loaded 16 bytes at a time;
//       - a choice and its expert become one float64 integer, key * 1024 + 1023 - e, whose
//         order is that of the choices, lower expert first: one v_max_f64 compares both;
//       - a lane sorts its own with a merge-exchange network, and each round takes the
//         largest head of the 16 lanes and shifts that lane's list;
//       - group scores: choices through LDS, one lane a group; groups are ranked by
//         comparing with the 15 rotations;
//       - without a bias the order is that of the logits, which is exact as it stands, and
//         renormalised weights need the picks' exponentials only.
//   * k_router_scored (all other sizes, and the function the first one falls back on): one
//     wave a token, lane l takes experts l, l + 64, ..., float64 throughout, the choices'
//     64-bit keys in LDS, k rounds of a wave maximum.
#include <type_traits>

#include "moe_internal.h"

namespace moe {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;  // waves per block
// Twice how far a float32 choice may be from the exact one (k_route_rows). Sigmoid: z = exp(-|l|) is
// off by |l| 2^-23 + 2^-22 relative, which moves the score by s (1 - s) of that, and the quotient
// rounds three times: under 2^-21 in all. Softmax, in units of 2^-23 relative: exp(x), x = l - top, off
// by 1.13 |x| + 1 (the difference, the product with log2(e) and that constant, 2^x); the sum by the mean
// of that over the scores, where the mean of |x| is under 3.9 for 512 experts, so 5.4, and by half a unit
// for each of 35 additions (31 of a lane's 32 experts, 4 across the lanes), 17.5; reciprocal and product
// 1; the score's own s (1.13 |x| + 1) at most 1.1. In all 25, or 2^-18.3, of which twice is 0.78 of
// kErrSoftmax. Adding the bias rounds once more, relative to the sum.
constexpr float kErrSigmoid = 0x1p-20f, kErrSoftmax = 0x1p-17f, kErrSum = 0x1p-22f;

template <int N>
__device__ __forceinline__ int row_ror(int v) {   // lane i of a row of 16 gets lane i - N's
    return __builtin_amdgcn_mov_dpp(v, 0x120 + N, 0xf, 0xf, true);
}
template <int N>
__device__ __forceinline__ float row_ror(float v) { return __int_as_float(row_ror<N>(__float_as_int(v))); }
template <int N>
__device__ __forceinline__ double row_ror(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)row_ror<N>((int)(uint32_t)u), hi = (uint32_t)row_ror<N>((int)(uint32_t)(u >> 32));
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// The lanes' values exchanged across the rows of 16: one result has those of the even rows (half
// 0) in both rows of a pair (both halves of the wave), the other those of the odd ones (half 1).
struct Pair {
    uint32_t x, y;
};
template <int ROWS>
__device__ __forceinline__ Pair across(uint32_t v) {
    if constexpr (ROWS == 1) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return {r[0], r[1]};
    } else {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return {r[0], r[1]};
    }
}
template <int ROWS, class F>
__device__ __forceinline__ float across(float v, F f) {
    const Pair p = across<ROWS>(__float_as_uint(v));
    return f(__uint_as_float(p.x), __uint_as_float(p.y));
}
template <int ROWS, class F>
__device__ __forceinline__ double across(double v, F f) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const Pair lo = across<ROWS>((uint32_t)u), hi = across<ROWS>((uint32_t)(u >> 32));
    return f(__builtin_bit_cast(double, ((uint64_t)hi.x << 32) | lo.x), __builtin_bit_cast(double, ((uint64_t)hi.y << 32) | lo.y));
}
// Reductions over the wave, the same bits in every lane; no LDS.
template <class V, class F>
__device__ __forceinline__ V wave_reduce(V v, F f) {
    v = f(v, row_ror<8>(v));
    v = f(v, row_ror<4>(v));
    v = f(v, row_ror<2>(v));
    v = f(v, row_ror<1>(v));
    v = across<1>(v, f);
    return across<2>(v, f);
}
template <class V>
__device__ __forceinline__ V wave_sum(V v) {
    return wave_reduce(v, [](V a, V b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float v) {
    return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}
// Largest key of the wave and the lowest index that holds it.
__device__ __forceinline__ void wave_best(uint64_t& key, int& idx) {
    auto better = [](uint64_t k1, int i1, uint64_t k2, int i2) { return k2 > k1 || (k2 == k1 && i2 < i1); };
    auto rotated = [&](auto n) {
        constexpr int N = decltype(n)::value;
        const uint32_t lo = (uint32_t)row_ror<N>((int)(uint32_t)key), hi = (uint32_t)row_ror<N>((int)(uint32_t)(key >> 32));
        const uint64_t k2 = ((uint64_t)hi << 32) | lo;
        const int i2 = row_ror<N>(idx);
        const bool t = better(key, idx, k2, i2);
        key = t ? k2 : key;
        idx = t ? i2 : idx;
    };
    auto crossed = [&](auto n) {
        constexpr int N = decltype(n)::value;
        const Pair lo = across<N>((uint32_t)key), hi = across<N>((uint32_t)(key >> 32)), i = across<N>((uint32_t)idx);
        const uint64_t k1 = ((uint64_t)hi.x << 32) | lo.x, k2 = ((uint64_t)hi.y << 32) | lo.y;
        const bool t = better(k1, (int)i.x, k2, (int)i.y);
        key = t ? k2 : k1;
        idx = t ? (int)i.y : (int)i.x;
    };
    rotated(std::integral_constant<int, 8>{});
    rotated(std::integral_constant<int, 4>{});
    rotated(std::integral_constant<int, 2>{});
    rotated(std::integral_constant<int, 1>{});
    crossed(std::integral_constant<int, 1>{});
    crossed(std::integral_constant<int, 2>{});
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

// LDS words of route_wave beside the keys: groups, then picks.
__host__ __device__ __forceinline__ int route_extra(const RouterScoredArgs& a) {
    const int p = (a.k + 1) / 2;
    return a.n_group > p ? a.n_group : p;
}

// Ratio of the sigmoids of l and of lmax >= l, without overflow or 0 / 0.
__device__ __forceinline__ float sigmoid_ratio(float l, float lmax) {
    if (lmax > 0.f) return (1.f + expf(-lmax)) / (1.f + expf(-l));
    return expf(l - lmax) * ((1.f + expf(lmax)) / (1.f + expf(l)));
}

// Routes token t with one wave, in float64; writes its scores if asked to. s_key: E words of LDS of
// this wave's own, s_grp: max(n_group, (k + 1) / 2) more. Loops over a lane's experts stay loops: as the fallback of
// k_route_rows this runs rarely and from a cold instruction cache: a launch that needs it for any
// token ends 11 us later (65536 x 256: 67 against 56 us), so its loops are kept small.
__device__ __forceinline__ void route_wave(const RouterScoredArgs& a, int64_t t, bool scores, uint64_t* s_key,
                                           uint64_t* s_grp) {
    const int lane = threadIdx.x & 63;
    const int E = a.E, k = a.k, per = E / a.n_group;
    auto logit = [&](int e) -> float {   // NaN taken as -inf
        const float x = load_logit(a.logits, a.bf16, t * E + e);
        return x != x ? -INFINITY : x;
    };
    float top = -INFINITY;
#pragma unroll 4
    for (int e = lane; e < E; e += 64) {   // the logits wait in the keys' places
        const float l = logit(e);
        s_key[e] = __float_as_uint(l);
        top = fmaxf(top, l);
    }
    top = wave_max(top);
    const bool none = top == -INFINITY, inf = top == INFINITY;
    // softmax as exp(l - top) / den; infinite logits share the sum
    double den = 1.0;
    auto score = [&](float l) -> double {
        if (a.sigmoid) return 1.0 / (1.0 + exp(-(double)l));
        return (none ? 0.0 : inf ? (l == INFINITY ? 1.0 : 0.0) : exp((double)l - (double)top)) / den;
    };
    if (!a.sigmoid && !none) {
        double sum = 0.0;
#pragma unroll 1
        for (int e = lane; e < E; e += 64) sum += score(__uint_as_float((uint32_t)s_key[e]));
        den = wave_sum(sum);
    }
    const bool grouped = a.topk_group < a.n_group;
    // sums of scores rank the groups, while the experts' order without a bias is that of the logits
    const bool two_orders = grouped && a.group_top == 2 && !a.bias;
#pragma unroll 1
    for (int e = lane; e < E; e += 64) {
        const float l = __uint_as_float((uint32_t)s_key[e]);
        const double s = a.bias || two_orders || scores ? score(l) : 0.0;
        if (scores) a.scores[t * E + e] = (float)s;
        s_key[e] = !(l > -INFINITY) ? 0 : order_key(a.bias ? s + (double)a.bias[e] : two_orders ? s : (double)l);
    }
    __builtin_amdgcn_wave_barrier();
    if (grouped) {
        for (int g = lane; g < a.n_group; g += 64) {
            uint64_t b1 = 0, b2 = 0;
#pragma unroll 4
            for (int i = 0; i < per; i++) {
                const uint64_t x = s_key[g * per + i];
                const bool first = x > b1;
                b2 = first ? b1 : x > b2 ? x : b2;
                b1 = first ? x : b1;
            }
            uint64_t v = b1;
            if (a.group_top == 2 && b2) v = order_key(key_value(b1) + key_value(b2));
            s_grp[g] = v;
        }
        __builtin_amdgcn_wave_barrier();
        // keep the best groups: a kept group's key becomes all ones, which no key is
#pragma unroll 1
        for (int r = 0; r < a.topk_group; r++) {
            uint64_t bk = 0;
            int bi = 0x7fffffff;
            for (int g = lane; g < a.n_group; g += 64) {
                const uint64_t v = s_grp[g];
                if (v != ~0ull && v > bk) {
                    bk = v;
                    bi = g;
                }
            }
            wave_best(bk, bi);
            if (bk && lane == (bi & 63)) s_grp[bi] = ~0ull;
            __builtin_amdgcn_wave_barrier();
        }
#pragma unroll 1
        for (int e = lane; e < E; e += 64) {
            if (s_grp[e / per] != ~0ull) {
                s_key[e] = 0;
            } else if (two_orders) {
                const float l = logit(e);
                s_key[e] = l > -INFINITY ? order_key((double)l) : 0;
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
    int* s_pick = (int*)s_grp;
#pragma unroll 1
    for (int r = 0; r < k; r++) {
        uint64_t bk = 0;
        int bi = 0x7fffffff;
#pragma unroll 4
        for (int e = lane; e < E; e += 64) {
            const uint64_t v = s_key[e];
            bi = v > bk ? e : bi;
            bk = v > bk ? v : bk;
        }
        wave_best(bk, bi);
        if (bk && lane == (bi & 63)) s_key[bi] = 0;
        if (lane == 0) {
            s_pick[r] = bk ? bi : -1;
            a.ids[t * k + r] = bk ? bi : -1;
        }
        __builtin_amdgcn_wave_barrier();
    }
    // weights: renormalised ones from the logits, without 0 / 0
    float m = -INFINITY, sum = 0.f;
    auto weight = [&](int j) -> float {
        const int e = s_pick[j];
        if (e < 0) return 0.f;
        const float l = logit(e);
        if (!a.renorm) return (float)score(l);
        if (m == INFINITY && !a.sigmoid) return l == m ? 1.f : 0.f;
        return a.sigmoid ? sigmoid_ratio(l, m) : expf(l - m);
    };
    if (a.renorm) {
#pragma unroll 1
        for (int j = lane; j < k; j += 64) m = fmaxf(m, s_pick[j] < 0 ? -INFINITY : logit(s_pick[j]));
        m = wave_max(m);
#pragma unroll 1
        for (int j = lane; j < k; j += 64) sum += weight(j);
        sum = wave_sum(sum);
    }
#pragma unroll 1
    for (int j = lane; j < k; j += 64) {
        const float w = weight(j);
        a.w[t * k + j] = a.scale * (!a.renorm ? w : sum > 0.f ? w / sum : 0.f);
    }
}

__global__ __launch_bounds__(64 * kWaves) void k_router_scored(RouterScoredArgs a) {
    extern __shared__ uint64_t s_dyn[];
    const int wv = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kWaves + wv;
    uint64_t* mine = s_dyn + wv * (a.E + route_extra(a));
    if (t < a.T) route_wave(a, t, a.scores != nullptr, mine, mine + a.E);
}

// ---------------------------------------------------------------- 16 lanes a token
constexpr int kRowExperts = 512, kRowPicks = 15, kRowGroups = 16;
static_assert(kRowExperts <= 512, "kErrSoftmax counts the additions and the mean for 512 experts");

// No NaN comes here, so the instructions need no quieting of their inputs before them.
__device__ __forceinline__ double bigger(double a, double b) {
    double d;
    asm("v_max_f64 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
    return d;
}
__device__ __forceinline__ double smaller(double a, double b) {
    double d;
    asm("v_min_f64 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
    return d;
}
__device__ __forceinline__ float bigger(float a, float b) { return fmaxf(a, b); }
template <class V>
__device__ __forceinline__ V row_max(V v) {
    v = bigger(v, row_ror<8>(v));
    v = bigger(v, row_ror<4>(v));
    v = bigger(v, row_ror<2>(v));
    return bigger(v, row_ror<1>(v));
}
__device__ __forceinline__ float row_sum(float v) {   // the same bits in every lane
    v += row_ror<8>(v);
    v += row_ror<4>(v);
    v += row_ror<2>(v);
    return v + row_ror<1>(v);
}
// exp of x <= 0 to an ulp, subnormal results included: x log2(e) = n + t with n whole and |t| <= 1/2,
// then 2^t and n into the exponent. 8 instructions (expf: 13, for the range that does not come here;
// 65536 x 256 sigmoid gradients 45 us with this, 47 with expf); __expf rounds x log2(e), which is off by
// |x| 2^-24 relative.
__device__ __forceinline__ float exp_neg(float x) {
    x = fmaxf(x, -110.f);   // 0 from here on
    const float n = __builtin_rintf(x * 0x1.715476p+0f);
    const float t = fmaf(x, 0x1.4ae0cp-26f, fmaf(x, 0x1.715476p+0f, -n));   // log2(e) in two parts
    return ldexpf(__builtin_amdgcn_exp2f(t), (int)n);
}
// 1 / d of d in [1, 2]: v_rcp (an ulp) and a Newton step, which leaves the rounding of the last fma. (A
// quotient takes 10 instructions, for operands that do not come here: 65536 x 256 sigmoid gradients 45.3
// us, with this 43.6.)
__device__ __forceinline__ float recip_1_2(float d) {
    const float f = __builtin_amdgcn_rcpf(d);
    return fmaf(f, fmaf(-d, f, 1.f), f);
}
// Order key of a float32 choice as above; float of a key.
__device__ __forceinline__ uint32_t order_key(float c) {
    const uint32_t u = c == 0.f ? 0u : __float_as_uint(c);
    return !(c > -INFINITY) ? 0u : (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_float(uint32_t k) { return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k); }

// Descending, by Batcher's merge exchange.
template <int C>
__device__ __forceinline__ void sort_desc(double (&v)[C]) {
#pragma unroll
    for (int p = 1; p < C; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < C; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; i++)
                    if (i + j + k < C && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const double x = v[i + j], y = v[i + j + k];
                        v[i + j] = bigger(x, y);
                        v[i + j + k] = smaller(x, y);
                    }
}

// C: experts of a lane (a multiple of 4); KL: picks a call may take.
template <int C, int KL>
__global__ __launch_bounds__(64 * kWaves) void k_route_rows(RouterScoredArgs a) {
    constexpr int Q = C / 4;
    constexpr int LIST = C < KL + 1 ? C : KL + 1;
    // choices of the wave's tokens (float32, four rows of 16 C + 4), or the fallback's keys and groups
    // (at most 16 C + 16 words: kRowGroups)
    static_assert(16 * C + kRowGroups <= 2 * (16 * C + 4), "room for the fallback");
    __shared__ uint64_t s_mem[kWaves][2 * (16 * C + 4)];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, r = lane & 15, row = lane >> 4;
    const int64_t t0 = ((int64_t)blockIdx.x * kWaves + wv) * 4;
    if (t0 >= a.T) return;
    const int64_t t = t0 + row;
    const bool live = t < a.T;               // spare rows repeat the last token and write nothing
    const int64_t tt = live ? t : a.T - 1;
    const int E = a.E, k = a.k;
    const bool grouped = a.topk_group < a.n_group;
    const bool approx = a.bias != nullptr;   // choices are float32 sums, not exact
    const bool sums = grouped && a.group_top == 2;
    // scores of all experts are needed; otherwise the logits alone decide
    const bool all_scores = a.scores || approx || sums || (!a.renorm && !a.sigmoid);

    float l[C];   // NaN as -inf; -inf past E
#pragma unroll
    for (int q = 0; q < Q; q++) {
        const int e = 4 * (r + 16 * q);
        if ((E & 3) == 0) {
            const int64_t at = tt * E + (e < E ? e : 0);
            if (a.bf16) {
                const uint2 v = *(const uint2*)((const uint16_t*)a.logits + at);
                l[4 * q] = __uint_as_float(v.x << 16);
                l[4 * q + 1] = __uint_as_float(v.x & 0xffff0000u);
                l[4 * q + 2] = __uint_as_float(v.y << 16);
                l[4 * q + 3] = __uint_as_float(v.y & 0xffff0000u);
            } else {
                const float4 v = *(const float4*)((const float*)a.logits + at);
                l[4 * q] = v.x;
                l[4 * q + 1] = v.y;
                l[4 * q + 2] = v.z;
                l[4 * q + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) l[4 * q + i] = load_logit(a.logits, a.bf16, tt * E + min(e + i, E - 1));
        }
    }
    float top = -INFINITY;
#pragma unroll
    for (int c = 0; c < C; c++) {
        const int e = 4 * (r + 16 * (c / 4)) + c % 4;
        if (e >= E || l[c] != l[c]) l[c] = -INFINITY;
        top = fmaxf(top, l[c]);
    }
    top = row_max(top);
    const bool limit = top == INFINITY;      // limits are left to the exact form
    bool doubt = limit;
    const float base = top > -INFINITY ? top : 0.f;
    float den = 0.f;
    float v[C];                              // scores, then choices
    if (all_scores) {
        // scores that leave the kernel, and a sum that weights are divided by, with full exponentials;
        // choices alone with the short ones (z = exp(-|l|) off by |l| 2^-23), which their bound covers
        const bool full = a.scores || (!a.renorm && !a.sigmoid);
        if (a.sigmoid && full) {
#pragma unroll
            for (int c = 0; c < C; c++) {
                const float z = exp_neg(-fabsf(l[c]));
                v[c] = (l[c] > 0.f ? 1.f : z) / (1.f + z);
            }
        } else if (a.sigmoid) {
#pragma unroll
            for (int c = 0; c < C; c++) {
                const float z = __expf(-fabsf(l[c])), f = __builtin_amdgcn_rcpf(1.f + z);
                v[c] = l[c] > 0.f ? f : z * f;
            }
        } else {
#pragma unroll
            for (int c = 0; c < C; c++) v[c] = l[c] - base;
            if (full) {
#pragma unroll
                for (int c = 0; c < C; c++) den += v[c] = exp_neg(v[c]);
            } else {
#pragma unroll
                for (int c = 0; c < C; c++) den += v[c] = __expf(v[c]);
            }
        }
        if (!a.sigmoid) {
            den = row_sum(den);
            const float f = den > 0.f ? 1.f / den : 0.f;
#pragma unroll
            for (int c = 0; c < C; c++) v[c] *= f;
        }
        if (a.scores && live && !limit) {
#pragma unroll
            for (int q = 0; q < Q; q++) {
                const int e = 4 * (r + 16 * q);
                float* o = a.scores + t * E + e;
                if ((E & 3) == 0 && ((uintptr_t)a.scores & 15) == 0) {
                    if (e < E) *(float4*)o = float4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
                } else {
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        if (e + i < E) o[i] = v[4 * q + i];
                }
            }
        }
    }
    // choices of masked experts: -inf
    if (approx) {
        const bool vec = (E & 3) == 0 && ((uintptr_t)a.bias & 15) == 0;
#pragma unroll
        for (int q = 0; q < Q; q++) {
            const int e = 4 * (r + 16 * q);
            float b[4];
            if (vec) {
                const float4 x = *(const float4*)(a.bias + (e < E ? e : 0));
                b[0] = x.x;
                b[1] = x.y;
                b[2] = x.z;
                b[3] = x.w;
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++) b[i] = a.bias[min(e + i, E - 1)];
            }
#pragma unroll
            for (int i = 0; i < 4; i++)
                v[4 * q + i] = l[4 * q + i] > -INFINITY && b[i] > -INFINITY ? v[4 * q + i] + b[i] : -INFINITY;
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; c++)
            if (!sums || !(l[c] > -INFINITY)) v[c] = l[c];
    }
    uint32_t kept = 0xffffffffu;             // groups of this row's token that stay
    const int per = E / a.n_group;
    if (grouped) {
        float* s = (float*)s_mem[wv] + row * (16 * C + 4);
#pragma unroll
        for (int q = 0; q < Q; q++)
            *(float4*)(s + 4 * (r + 16 * q)) = float4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
        __builtin_amdgcn_wave_barrier();
        float b1 = -INFINITY, b2 = -INFINITY;
        if (r < a.n_group) {
            int i = (r + 4 * row) % per;     // each lane from another place: fewer bank conflicts
            auto see = [&](float x) {
                b2 = __builtin_amdgcn_fmed3f(b1, b2, x);   // the middle one: b2 <= b1
                b1 = fmaxf(b1, x);
            };
            int n = 0;
            for (; n + 4 <= per; n += 4) {   // four reads in flight
                float x[4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    x[j] = s[r * per + i];
                    i = i + 1 == per ? 0 : i + 1;
                }
#pragma unroll
                for (int j = 0; j < 4; j++) see(x[j]);
            }
            for (; n < per; n++) {
                see(s[r * per + i]);
                i = i + 1 == per ? 0 : i + 1;
            }
        }
        const float g = sums && b2 > -INFINITY ? b1 + b2 : b1;   // lanes past n_group: -inf, last in rank
        int rank = 0;
        auto against = [&](float x, int n) {  // lane r - n (mod 16) has x
            const int other = (r - n) & 15;
            rank += x > g || (x == g && other < r);
        };
        against(row_ror<1>(g), 1);
        against(row_ror<2>(g), 2);
        against(row_ror<3>(g), 3);
        against(row_ror<4>(g), 4);
        against(row_ror<5>(g), 5);
        against(row_ror<6>(g), 6);
        against(row_ror<7>(g), 7);
        against(row_ror<8>(g), 8);
        against(row_ror<9>(g), 9);
        against(row_ror<10>(g), 10);
        against(row_ror<11>(g), 11);
        against(row_ror<12>(g), 12);
        against(row_ror<13>(g), 13);
        against(row_ror<14>(g), 14);
        against(row_ror<15>(g), 15);
        const bool keep = rank < a.topk_group && r < a.n_group;
        kept = (uint32_t)(__ballot(keep) >> (16 * row)) & 0xffffu;
        if (approx || sums) {                // the last one kept and the first one left too near to tell
            const float in = -row_max(keep ? -g : -INFINITY), out = row_max(!keep && r < a.n_group ? g : -INFINITY);
            // both choices were rounded, and a sum can be far smaller than they are
            const float size = (b1 > -INFINITY ? fabsf(b1) : 0.f) + (sums && b2 > -INFINITY ? fabsf(b2) : 0.f);
            const float err = (a.sigmoid ? kErrSigmoid : kErrSoftmax) * 2.f + kErrSum * row_max(size);
            if (out > -INFINITY && !(in - out > err)) doubt = true;
            // a sum past float32's range: no order against the others, and none against an empty group
            if (sums && b2 > -INFINITY && !(fabsf(g) < INFINITY)) doubt = true;
        }
    }
    // one number per expert: its choice's key and itself, in the order of picking
    double list[C];
#pragma unroll
    for (int c = 0; c < C; c++) {
        const int e = 4 * (r + 16 * (c / 4)) + c % 4;
        uint32_t key = order_key(approx ? v[c] : l[c]);
        if (grouped && !((kept >> ((e / per) & 31)) & 1)) key = 0;   // past E: key is 0 as it is
        list[c] = key ? (double)key * 1024.0 + (double)(1023 - e) : 0.0;
    }
    sort_desc(list);
    // round n's pick is parked in lane n; one round more than picks, for the distance to the next
    int pe = -1;
    float pc = -INFINITY;
    for (int n = 0; n <= k; n++) {
        const double m = row_max(list[0]);
        const bool mine = list[0] == m;
#pragma unroll
        for (int i = 0; i + 1 < LIST; i++) {
            double next = list[i + 1];
            asm("" : "+v"(next));   // a value, not an element: the select must not become an index
            list[i] = mine ? next : list[i];
        }
        list[LIST - 1] = mine && LIST == C ? 0.0 : list[LIST - 1];
        if (r == n && m > 0.0) {
            const uint32_t key = (uint32_t)(m * (1.0 / 1024.0));
            pe = 1023 - (int)(m - (double)key * 1024.0);
            pc = key_float(key);
        }
    }
    const float pl0 = pe >= 0 ? load_logit(a.logits, a.bf16, tt * E + pe) : -INFINITY;
    if (approx) {
        // neighbours in the order too near to tell, unless logit and bias are the same: then the tie
        // is exact (but a third one may be near the last pick and the first one left)
        const float pb = pe >= 0 ? a.bias[pe] : 0.f;
        const float nc = row_ror<15>(pc), nl = row_ror<15>(pl0), nb = row_ror<15>(pb);   // of lane r + 1
        const float err = (a.sigmoid ? kErrSigmoid : kErrSoftmax) + kErrSum * fabsf(pc);
        if (r < k && nc > -INFINITY && !(pc - nc > err) && !(nl == pl0 && nb == pb && r + 1 < k)) doubt = true;
    }
    // weights of the picks (lanes r < k)
    const bool pick = r < k && pe >= 0;
    const float pl = pick ? pl0 : -INFINITY;
    float w;
    if (a.renorm) {
        const float m = row_max(pl);
        w = !pick ? 0.f : a.sigmoid ? sigmoid_ratio(pl, m) : expf(pl - m);
        const float sum = row_sum(w);
        w = sum > 0.f ? w / sum : 0.f;
    } else if (a.sigmoid) {
        w = pick ? 1.f / (1.f + expf(-pl)) : 0.f;
    } else {
        w = pick ? expf(pl - base) / den : 0.f;
    }
    // the exact form for tokens in doubt, one after the other: their picks, and scores only where they
    // are a limit, so that no score depends on the bias and nothing is written twice
    uint64_t again = __ballot(doubt && live);
    const uint64_t limits = a.scores ? __ballot(limit) : 0;
    if (live && r < k && ((again >> (16 * row)) & 0xffff) == 0) {
        a.ids[t * k + r] = pick ? pe : -1;
        a.w[t * k + r] = a.scale * w;
    }
    while (again) {
        const int which = __builtin_ctzll(again) >> 4;
        again &= ~(0xffffull << (16 * which));
        __builtin_amdgcn_wave_barrier();
        route_wave(a, t0 + which, (limits >> (16 * which)) & 1, s_mem[wv], s_mem[wv] + E);
    }
}

// ---------------------------------------------------------------- gradient
// With w'_j the weight of pick j without
// the scale (s_j / sum of the picks' s with renorm, else s_j) and g_j its gradient,
//     q_e = s_e dS_e + sum over picks j of e:  scale * w'_j * (g_j - sum_m w'_m g_m)  (renorm)
//                                              scale * w'_j * g_j                     (else)
// which is s_e * dL/ds_e, and
//     softmax: dl_e = q_e - s_e * sum_f q_f        sigmoid: dl_e = q_e * (1 - s_e).
// With renorm the picks' part of sum_f q_f is zero, so only dS enters it.
// k_grad_rows (the sizes of k_route_rows): 16 lanes a token, chunks of four experts a lane. Lane
// j has pick j; picks of one expert are added up by the first of them (in a fixed order) and
// each pick's value goes to its expert through a row of LDS. Without dS only the picks of a
// sigmoid or of renormalised weights have a gradient, so the logits' rows are not read.
// Bound by memory: 65536 x 256 float32 with a full dS move 206 MB in 44 us, 4.7 TB/s (one wave
// a token with the experts strided over its lanes took 88).
// k_router_grad (other sizes): one wave a token.
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

// The gradient of 16 lanes a token; C experts a lane.
template <int C>
__global__ __launch_bounds__(64 * kWaves) void k_grad_rows(RouterGradArgs a) {
    constexpr int Q = C / 4;
    __shared__ float s_mem[kWaves][4][16 * C];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, r = lane & 15, row = lane >> 4;
    const int64_t t0 = ((int64_t)blockIdx.x * kWaves + wv) * 4;
    if (t0 >= a.T) return;
    const int64_t t = t0 + row;
    const bool live = t < a.T;               // spare rows repeat the last token and write nothing
    const int64_t tt = live ? t : a.T - 1;
    const int E = a.E, k = a.k;
    const bool vec = (E & 3) == 0 && ((uintptr_t)a.dl & (a.bf16 ? 7 : 15)) == 0;
    // every expert has a gradient
    const bool dense = a.ds || (!a.sigmoid && !a.renorm);

    // the pick of this lane
    int e = r < k ? a.ids[tt * k + r] : -1;
    float g = r < k ? a.dw[tt * k + r] : 0.f;
    if (e >= E) e = -1;
    float pl = e >= 0 ? load_logit(a.logits, a.bf16, tt * E + e) : -INFINITY;
    if (!(pl > -INFINITY)) e = -1;

    float l[C], d[C];   // logits (NaN as -inf, -inf past E), dS
    float top = -INFINITY;
    if (dense) {
#pragma unroll
        for (int q = 0; q < Q; q++) {
            const int e0 = 4 * (r + 16 * q);
            if ((E & 3) == 0) {
                const int64_t at = tt * E + (e0 < E ? e0 : 0);
                if (a.bf16) {
                    const uint2 v = *(const uint2*)((const uint16_t*)a.logits + at);
                    l[4 * q] = __uint_as_float(v.x << 16);
                    l[4 * q + 1] = __uint_as_float(v.x & 0xffff0000u);
                    l[4 * q + 2] = __uint_as_float(v.y << 16);
                    l[4 * q + 3] = __uint_as_float(v.y & 0xffff0000u);
                } else {
                    const float4 v = *(const float4*)((const float*)a.logits + at);
                    l[4 * q] = v.x;
                    l[4 * q + 1] = v.y;
                    l[4 * q + 2] = v.z;
                    l[4 * q + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++) l[4 * q + i] = load_logit(a.logits, a.bf16, tt * E + min(e0 + i, E - 1));
            }
        }
        if (a.ds) {
            const bool dvec = (((uintptr_t)a.ds & 15) | (E & 3) | (a.ds_stride & 3)) == 0;
            const float* ds = a.ds + tt * a.ds_stride;
#pragma unroll
            for (int q = 0; q < Q; q++) {
                const int e0 = 4 * (r + 16 * q);
                if (dvec) {
                    const f32x4 v = __builtin_nontemporal_load((const f32x4*)(ds + (e0 < E ? e0 : 0)));
#pragma unroll
                    for (int i = 0; i < 4; i++) d[4 * q + i] = v[i];
                } else {
#pragma unroll
                    for (int i = 0; i < 4; i++) d[4 * q + i] = ds[min(e0 + i, E - 1)];
                }
            }
        }
#pragma unroll
        for (int c = 0; c < C; c++) {
            if (4 * (r + 16 * (c / 4)) + c % 4 >= E || l[c] != l[c]) l[c] = -INFINITY;
            if (!a.ds) d[c] = 0.f;
            top = fmaxf(top, l[c]);
        }
        top = row_max(top);
    }
    // scores and 1 - s (without its cancellation); softmax of infinite logits shares the sum
    const bool inf = top == INFINITY;
    const float base = top > -INFINITY ? top : 0.f;
    float den = 0.f;
    float s[C], rest[C];
    if (dense) {
#pragma unroll
        for (int c = 0; c < C; c++) {
            if (a.sigmoid) {
                const float z = exp_neg(-fabsf(l[c])), f = recip_1_2(1.f + z);
                s[c] = l[c] > 0.f ? f : z * f;
                rest[c] = l[c] > 0.f ? z * f : f;
            } else {
                s[c] = inf ? (l[c] == INFINITY ? 1.f : 0.f) : exp_neg(l[c] - base);
                den += s[c];
            }
        }
        if (!a.sigmoid) {
            den = row_sum(den);
            const float f = den > 0.f ? 1.f / den : 0.f;
#pragma unroll
            for (int c = 0; c < C; c++) s[c] *= f;
        }
    }
    // this pick's part of q
    float v = 0.f;
    if (a.renorm) {
        const float m = row_max(e >= 0 ? pl : -INFINITY);
        float w = e < 0 ? 0.f : a.sigmoid ? sigmoid_ratio(pl, m) : m == INFINITY ? (pl == m ? 1.f : 0.f) : expf(pl - m);
        const float sum = row_sum(w);
        w = sum > 0.f ? w / sum : 0.f;
        const float dot = row_sum(w > 0.f ? w * g : 0.f);
        v = w > 0.f ? a.scale * w * (g - dot) : 0.f;
    } else if (e >= 0) {
        const float w = a.sigmoid ? 1.f / (1.f + expf(-pl)) : inf ? (pl == INFINITY ? 1.f : 0.f) / den : expf(pl - base) / den;
        v = w > 0.f ? a.scale * w * g : 0.f;
    }
    float sum_q = a.sigmoid || a.renorm ? 0.f : v;
    if (a.sigmoid) {   // straight to the logit's gradient: times 1 - s
        const float z = expf(-fabsf(pl));
        v *= pl > 0.f ? z / (1.f + z) : 1.f / (1.f + z);
        if (e < 0) v = 0.f;
    }
    // picks of one expert: the first lane adds the others' values, which then have no expert
    {
        float add = 0.f;
        bool later = false;
        auto from = [&](int oe, float ov, int n) {   // of lane r - n (mod 16)
            const int o = (r - n) & 15;
            if (oe == e && e >= 0) {
                if (o < r) later = true;
                else add += ov;
            }
        };
        from(row_ror<15>(e), row_ror<15>(v), 15);
        from(row_ror<14>(e), row_ror<14>(v), 14);
        from(row_ror<13>(e), row_ror<13>(v), 13);
        from(row_ror<12>(e), row_ror<12>(v), 12);
        from(row_ror<11>(e), row_ror<11>(v), 11);
        from(row_ror<10>(e), row_ror<10>(v), 10);
        from(row_ror<9>(e), row_ror<9>(v), 9);
        from(row_ror<8>(e), row_ror<8>(v), 8);
        from(row_ror<7>(e), row_ror<7>(v), 7);
        from(row_ror<6>(e), row_ror<6>(v), 6);
        from(row_ror<5>(e), row_ror<5>(v), 5);
        from(row_ror<4>(e), row_ror<4>(v), 4);
        from(row_ror<3>(e), row_ror<3>(v), 3);
        from(row_ror<2>(e), row_ror<2>(v), 2);
        from(row_ror<1>(e), row_ror<1>(v), 1);
        v += add;
        if (later) e = -1;
    }
    float* m = s_mem[wv][row];
#pragma unroll
    for (int q = 0; q < Q; q++) *(float4*)(m + 4 * (r + 16 * q)) = float4{0.f, 0.f, 0.f, 0.f};
    __builtin_amdgcn_wave_barrier();
    if (e >= 0) m[e] = v;
    __builtin_amdgcn_wave_barrier();
    float o[C];
#pragma unroll
    for (int q = 0; q < Q; q++) {
        const float4 x = *(const float4*)(m + 4 * (r + 16 * q));
        o[4 * q] = x.x;
        o[4 * q + 1] = x.y;
        o[4 * q + 2] = x.z;
        o[4 * q + 3] = x.w;
    }
    if (dense) {
        if (!a.sigmoid) {
            float aux = 0.f;
#pragma unroll
            for (int c = 0; c < C; c++) {
                const float x = l[c] > -INFINITY ? s[c] * d[c] : 0.f;
                aux += x;
                o[c] += x;
            }
            sum_q = row_sum(sum_q + aux);
#pragma unroll
            for (int c = 0; c < C; c++) o[c] = l[c] > -INFINITY ? o[c] - s[c] * sum_q : 0.f;
        } else {
#pragma unroll
            for (int c = 0; c < C; c++) o[c] = l[c] > -INFINITY ? o[c] + s[c] * d[c] * rest[c] : 0.f;
        }
    }
    if (!live) return;
#pragma unroll
    for (int q = 0; q < Q; q++) {
        const int e0 = 4 * (r + 16 * q);
        if (a.bf16) {
            __bf16* p = (__bf16*)a.dl + t * E + e0;
            const __bf16 x[4] = {(__bf16)o[4 * q], (__bf16)o[4 * q + 1], (__bf16)o[4 * q + 2], (__bf16)o[4 * q + 3]};
            if (vec) {
                if (e0 < E) *(uint2*)p = __builtin_bit_cast(uint2, x);
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++)
                    if (e0 + i < E) p[i] = x[i];
            }
        } else {
            float* p = (float*)a.dl + t * E + e0;
            if (vec) {
                if (e0 < E)
                    __builtin_nontemporal_store(f32x4{o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]}, (f32x4*)p);
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++)
                    if (e0 + i < E) p[i] = o[4 * q + i];
            }
        }
    }
}

template <int C>
hipError_t launch_grad_rows(const RouterGradArgs& a, hipStream_t st) {
    k_grad_rows<C><<<(unsigned)((a.T + 4 * kWaves - 1) / (4 * kWaves)), 64 * kWaves, 0, st>>>(a);
    return hipGetLastError();
}

template <int C>
hipError_t launch_rows(const RouterScoredArgs& a, hipStream_t st) {
    const unsigned grid = (unsigned)((a.T + 4 * kWaves - 1) / (4 * kWaves));
    if (a.k <= 8) k_route_rows<C, 8><<<grid, 64 * kWaves, 0, st>>>(a);
    else k_route_rows<C, kRowPicks><<<grid, 64 * kWaves, 0, st>>>(a);
    return hipGetLastError();
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
    // vector loads of four logits need their alignment
    const bool aligned = (a.E & 3) != 0 || ((uintptr_t)a.logits & (a.bf16 ? 7 : 15)) == 0;
    if (aligned && a.E <= kRowExperts && a.k <= kRowPicks && (a.n_group <= kRowGroups || a.topk_group == a.n_group)) {
        if (a.E <= 64) return launch_rows<4>(a, st);
        if (a.E <= 128) return launch_rows<8>(a, st);
        if (a.E <= 256) return launch_rows<16>(a, st);
        return launch_rows<32>(a, st);
    }
    const size_t lds = (size_t)kWaves * (a.E + route_extra(a)) * 8;   // 64 KB at most
    k_router_scored<<<(unsigned)((a.T + kWaves - 1) / kWaves), 64 * kWaves, lds, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_router_grad(const RouterGradArgs& a, hipStream_t st) {
    if (a.T <= 0) return hipSuccess;
    const bool aligned = (a.E & 3) != 0 || ((uintptr_t)a.logits & (a.bf16 ? 7 : 15)) == 0;
    if (aligned && a.E <= kRowExperts && a.k <= 16) {
        if (a.E <= 64) return launch_grad_rows<4>(a, st);
        if (a.E <= 128) return launch_grad_rows<8>(a, st);
        if (a.E <= 256) return launch_grad_rows<16>(a, st);
        return launch_grad_rows<32>(a, st);
    }
    return by_width(a, [&](auto nc, unsigned grid) {
        k_router_grad<decltype(nc)::value><<<grid, 64 * kWaves, 0, st>>>(a);
    });
}

}  // namespace moe
