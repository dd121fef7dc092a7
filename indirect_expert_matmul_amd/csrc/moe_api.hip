// libmoe C ABI: argument validation, limits, workspace carving, path selection and
// the launch sequence of each entry point (declared and documented in moe.h).
//
// Host-side rules taken from the pages' account of the CUDA implementation
// ("CUDA: better MoE implementation"):
//   * the three row maps are built on the device, so no host buffer has to outlive
//     an asynchronous copy (section 5 discusses exactly that hazard with host-side
//     mapping buffers) -- this file never copies host data to the device and never
//     synchronises;
//   * the grouped (GEMM) path serves batches whose token count is large relative to
//     the expert count, the mat-vec path the small ones (section 2.1's threshold
//     test, read here as n_tokens >= tau * n_experts);
//   * the packing limits n_tokens < 2^22 and n_used < 2^10 (section 2.1).
#include <cstdarg>
#include <cstdio>
#include <string>

#include "moe.h"
#include "moe_internal.h"

using namespace moe;

namespace {

thread_local std::string g_err;
thread_local int32_t g_stages = 0;   // kernels timed by the last call

moe_status fail(moe_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_err = buf;
    return s;
}

struct Carve {
    char* base;
    size_t off = 0;
    explicit Carve(void* b) : base((char*)b) {}
    void* take(size_t bytes) {
        off = (off + kAlign - 1) / kAlign * kAlign;
        void* p = base ? base + off : nullptr;
        off += bytes;
        return p;
    }
};

struct Timer {
    void* const* ev;
    int n;
    int stage = 0;
    hipStream_t st;
    Timer(const moe_options* o, hipStream_t s)
        : ev(o ? o->timing_events : nullptr), n(o ? o->n_timing_events : 0), st(s) {}
    void begin() {
        if (ev && 2 * stage + 1 < n) (void)hipEventRecord((hipEvent_t)ev[2 * stage], st);
    }
    void end() {
        if (ev && 2 * stage + 1 < n) (void)hipEventRecord((hipEvent_t)ev[2 * stage + 1], st);
        stage++;
    }
};

moe_status hip_check(hipError_t e, const char* what) {
    if (e != hipSuccess) return fail(MOE_EHIP, "%s: %s", what, hipGetErrorString(e));
    return MOE_OK;
}

moe_status check_tokens(int64_t T, int32_t k) {
    if (T < 0) return fail(MOE_EINVAL, "n_tokens must be >= 0 (got %lld)", (long long)T);
    if (k <= 0) return fail(MOE_EINVAL, "n_used must be > 0 (got %d)", k);
    if (T >= (1LL << 22)) return fail(MOE_ELIMIT, "n_tokens must be < 2^22 (got %lld)", (long long)T);
    if (k >= (1 << 10)) return fail(MOE_ELIMIT, "n_used must be < 2^10 (got %d)", k);
    if (T * (int64_t)k >= (1LL << 31))
        return fail(MOE_ELIMIT, "n_tokens * n_used must be < 2^31");
    return MOE_OK;
}

moe_status check_experts(int64_t E) {
    if (E <= 0) return fail(MOE_EINVAL, "n_experts must be > 0 (got %lld)", (long long)E);
    if (E > kMaxExperts) return fail(MOE_ELIMIT, "n_experts must be <= %d (got %lld)", kMaxExperts, (long long)E);
    return MOE_OK;
}

// Experts of the 16-bit and int8 products.
bool is_elem(moe_dtype t) { return t == MOE_BF16 || t == MOE_F16 || t == MOE_I8; }
ElemType elem_of(moe_dtype t) {
    return t == MOE_BF16 ? kElemBf16 : t == MOE_F16 ? kElemF16 : t == MOE_I8 ? kElemI8 : kElemF32;
}
const char* type_name(moe_dtype t) {
    return t == MOE_BF16 ? "BF16" : t == MOE_F16 ? "F16" : t == MOE_I8 ? "I8" : t == MOE_F32 ? "F32" : "another type";
}
constexpr int64_t kElemMaxSize = 1 << 30;   // rows, cols: tile ends stay in int32
constexpr int64_t kI8MaxCols = 131072;      // 128 * 127 * cols < 2^31
moe_status check_aligned(const void* p, const char* name) {
    if ((uintptr_t)p % 16) return fail(MOE_EINVAL, "%s must be 16-byte aligned", name);
    return MOE_OK;
}
// Device memory of a call; nullptr or no bytes: none.
struct Span {
    const void* p;
    int64_t bytes;
};
bool overlap(const Span& a, const Span& b) {
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return a.p && b.p && a.bytes > 0 && b.bytes > 0 && (x < y ? y - x < (uint64_t)a.bytes : x - y < (uint64_t)b.bytes);
}
moe_status check_elem_weights(const moe_weights* w, const char* name) {
    moe_status s;
    const int64_t unit = w->type == MOE_I8 ? 16 : 8;
    if (w->type == MOE_I8 && !w->scales) return fail(MOE_EINVAL, "%s: I8 scales are NULL", name);
    if (w->cols % unit)
        return fail(MOE_ELIMIT, "%s: %s needs cols %% %lld == 0 (got %lld)", name, type_name(w->type),
                    (long long)unit, (long long)w->cols);
    if (w->rows >= kElemMaxSize || w->cols >= kElemMaxSize)
        return fail(MOE_ELIMIT, "%s: rows and cols must be < 2^30", name);
    if (w->type == MOE_I8 && w->cols > kI8MaxCols)
        return fail(MOE_ELIMIT, "%s: I8 needs cols <= %lld (got %lld)", name, (long long)kI8MaxCols, (long long)w->cols);
    if ((s = check_aligned(w->data, name))) return s;
    if (w->type == MOE_I8 && (uintptr_t)w->scales % 4) return fail(MOE_EINVAL, "%s: I8 scales must be 4-byte aligned", name);
    return MOE_OK;
}

moe_status check_weights(const moe_weights* w, const char* name, bool allow_f32) {
    if (!w) return fail(MOE_EINVAL, "%s: weights struct is NULL", name);
    if (!w->data) return fail(MOE_EINVAL, "%s: data is NULL", name);
    if (w->n_mat <= 0 || w->rows <= 0 || w->cols <= 0)
        return fail(MOE_EINVAL, "%s: sizes must be > 0", name);
    if (w->rows > INT32_MAX || w->cols > INT32_MAX)
        return fail(MOE_ELIMIT, "%s: rows and cols must fit in int32", name);
    if (w->type == MOE_Q8_0 || w->type == MOE_MXFP4 || w->type == MOE_IQ4_NL || w->type == MOE_IQ4_XS) {
        const char* fmt = w->type == MOE_Q8_0 ? "Q8_0"
                          : w->type == MOE_MXFP4 ? "MXFP4" : w->type == MOE_IQ4_NL ? "IQ4_NL" : "IQ4_XS";
        const int64_t unit = w->type == MOE_IQ4_XS ? 256 : 32;   // columns per scale unit
        if (!w->scales) return fail(MOE_EINVAL, "%s: %s scales are NULL", name, fmt);
        if (w->cols % unit)
            return fail(MOE_ELIMIT, "%s: %s needs cols %% %lld == 0 (got %lld)", name, fmt, (long long)unit,
                        (long long)w->cols);
        if (w->type == MOE_IQ4_XS && ((uintptr_t)w->scales & 7))
            return fail(MOE_EINVAL, "%s: IQ4_XS super-block records must be 8-byte aligned", name);
    } else if (w->type == MOE_F32) {
        if (!allow_f32) return fail(MOE_EINVAL, "%s: float32 weights are not supported here", name);
    } else if (allow_f32 && is_elem(w->type)) {
        return check_elem_weights(w, name);
    } else {
        return fail(MOE_EINVAL, "%s: unsupported weight type %d", name, (int)w->type);
    }
    return MOE_OK;
}

// Weight format code of the kernels: 0 Q8_0, 1 MXFP4, 2 IQ4_NL, 3 IQ4_XS.
int32_t kernel_fmt(moe_dtype t) {
    return t == MOE_MXFP4 ? 1 : t == MOE_IQ4_NL ? 2 : t == MOE_IQ4_XS ? 3 : 0;
}

float tau_of(const moe_options* o) { return (o && o->tau > 0.f) ? o->tau : 1.0f; }

// 1 = GEMM, 2 = GEMV, or a negative status.
int select_path(int64_t T, int32_t k, int32_t E, int64_t act_width, const moe_options* o) {
    const int32_t force = o ? o->path : 0;
    const bool dec_ok = T * (int64_t)k <= kDecMaxSlots && act_width <= kDecMaxWidth;
    if (force == 1) return 1;
    if (force == 2) {
        if (!dec_ok)
            return fail(MOE_EINVAL, "GEMV path needs n_tokens*n_used <= %d and activation width <= %lld",
                        kDecMaxSlots, (long long)kDecMaxWidth);
        return 2;
    }
    if (force != 0) return fail(MOE_EINVAL, "options.path must be 0, 1 or 2 (got %d)", force);
    // Automatic choice: the GEMV's wave-level kernels up to kDecAutoSlots slots, its block
    // kernel (wider rows, more slots) for a single token only. Past those the block kernel
    // streams an expert's rows once per slot and the grouped GEMM wins (measured on one
    // MI355X, Q8_0, GEMV against GEMM per layer call: V3-shaped T = 2 155 / 156 us, T = 16
    // 2,868 / 941 us; Lite-shaped T = 10 126 / 106 us, T = 42 1,249 / 149 us; GPT-OSS-shaped
    // T = 16 235 / 225 us; T = 8 127 / 153 us).
    const bool wave_ok = T * (int64_t)k <= kDecAutoSlots && act_width <= 4096;
    return ((double)T < (double)tau_of(o) * (double)E && dec_ok && (wave_ok || T == 1)) ? 2 : 1;
}

// 4-bit experts (MXFP4, IQ4_NL, IQ4_XS): the GEMV path only through its wave-level kernels
// (n_tokens * n_used <= 64 and every activation width <= 4096); otherwise the grouped GEMM.
// Automatically up to auto_slots slots: MXFP4 32 (GPT-OSS-shaped, GEMV against GEMM per layer
// call on one MI355X: 16 slots 79 / 91 us, 32 slots 119 / 112, 48 slots 165 / 141, 64 slots
// 200 / 162), the IQ formats 64 (IQ4_XS E128 k8 at 64 slots 70 / 77 us; IQ4_NL
// GPT-OSS-shaped at 48 and 64 slots 189 / 189 and 227 / 219, Lite-shaped at 48 84 / 93).
int select_path_fmt(int64_t T, int32_t k, int32_t E, int64_t act_width, bool fp4, const moe_options* o,
                    int auto_slots = 64) {
    if (!fp4) return select_path(T, k, E, act_width, o);
    const int32_t force = o ? o->path : 0;
    const bool dec_ok = T * (int64_t)k <= 64 && act_width <= 4096;
    if (force == 1) return 1;
    if (force == 2) {
        if (!dec_ok)
            return fail(MOE_EINVAL, "GEMV path with 4-bit (MXFP4, IQ4_NL, IQ4_XS) experts needs n_tokens*n_used <= 64 "
                        "and widths <= 4096");
        return 2;
    }
    if (force != 0) return fail(MOE_EINVAL, "options.path must be 0, 1 or 2 (got %d)", force);
    return ((double)T < (double)tau_of(o) * (double)E && dec_ok && T * (int64_t)k <= auto_slots) ? 2 : 1;
}

// With options.act_quant = 1: 3 (the quantized-activation grouped GEMM, Q8_0 experts
// only, whatever the batch size), with 2 (MXFP4 experts only): 4 (the MXFP4-activation
// grouped GEMM) or 5 (its GEMV), else the choice above; or a negative status. S: shared
// experts; min_width: the narrowest activation row.
// With MXFP4 activations the GEMV is taken wherever it can run, up to 16 slots an expert on
// average, which is one of its passes (mul_mat_id, GEMV against GEMM in us per call on one MI355X, weight
// copies in turn: E32 k4 2880 x 2880 T = 1 10.9 / 21.7, T = 16 42.8 / 51.0; E64 k6 1408 x 2048 T = 10
// 18.1 / 24.7; E128 k8 2048 x 7168 T = 1 20.2 / 47.4, T = 8 98 / 104; E8 k2 4096 x 4096 T = 32
// 23.2 / 32.3; 16 slots an expert, E4 k1 2880 x 2880 T = 64, 23.7 / 30.6; 32 of them, E2 k2 1024 x 1024
// T = 32, 20.9 / 14.4).
int select_path_aq(int64_t T, int32_t k, int32_t E, int64_t act_width, int32_t wtype,
                   const moe_options* o, int64_t S, int64_t min_width) {
    const int32_t aq = o ? o->act_quant : 0;
    if (aq < 0 || aq > 2) return fail(MOE_EINVAL, "options.act_quant must be 0, 1 or 2 (got %d)", aq);
    if (aq == 2) {
        if (wtype != MOE_MXFP4) return fail(MOE_EINVAL, "MXFP4 activations (act_quant = 2) need MXFP4 experts");
        const bool dec_ok = T * (int64_t)k <= kDecFp4Slots && S * T <= kDecFp4Slots && min_width >= 128;
        if (o->path == 1) return 4;
        if (o->path == 2) {
            if (!dec_ok)
                return fail(MOE_EINVAL, "GEMV path with MXFP4 activations needs n_tokens*n_used and "
                            "n_tokens*shared experts <= %d and widths >= 128", kDecFp4Slots);
            return 5;
        }
        if (o->path != 0) return fail(MOE_EINVAL, "options.path must be 0, 1 or 2 (got %d)", o->path);
        return dec_ok && T * (int64_t)k <= kDecFp4Pass * (int64_t)E ? 5 : 4;
    }
    if (!aq)
        return select_path_fmt(T, k, E, act_width,
                               wtype == MOE_MXFP4 || wtype == MOE_IQ4_NL || wtype == MOE_IQ4_XS, o,
                               wtype == MOE_MXFP4 ? 32 : 64);
    if (wtype != MOE_Q8_0) return fail(MOE_EINVAL, "quantized activations (act_quant = 1) need Q8_0 experts");
    if (o->path != 0 && o->path != 1)
        return fail(MOE_EINVAL, "quantized activations run on the grouped GEMM only: options.path must "
                    "be 0 or 1 (got %d)", o->path);
    return 3;
}

int64_t m_tiles_bound(int64_t n, int64_t E, int bm) { return n / bm + (n < E ? n : E); }

// ---------------------------------------------------------------- workspace plans
struct RowIdsPlan {
    int32_t *ids_src1, *ids_dst, *bounds, *tile_a, *tile_tab;
    void* scratch;   // multi-block scratch of the row-id pass (row_ids_scratch_bytes)
    int32_t tile_cap;
};
// tile_m > 0: also room for the GEMM's M-tile prefix and per-tile table (tiles of
// tile_m rows)
RowIdsPlan carve_row_ids(Carve& c, int64_t n, int32_t E, bool maps, int tile_m) {
    RowIdsPlan p{};
    const bool tiles = tile_m > 0;
    if (maps) {
        p.ids_src1 = (int32_t*)c.take(sizeof(int32_t) * n);
        p.ids_dst = (int32_t*)c.take(sizeof(int32_t) * n);
        p.bounds = (int32_t*)c.take(sizeof(int32_t) * (E + 1));
    }
    if (tiles) {
        p.tile_a = (int32_t*)c.take(sizeof(int32_t) * (E + 1));
        p.tile_cap = (int32_t)m_tiles_bound(n, E, tile_m);
        p.tile_tab = (int32_t*)c.take(sizeof(int32_t) * 4 * (size_t)p.tile_cap);
    }
    const size_t sb = row_ids_scratch_bytes(n, E);
    if (sb) p.scratch = c.take(sb);
    return p;
}

struct FfnDims {
    int64_t T;
    int32_t k, E, n_embd, n_ff, S, n_ff_sh;
    int32_t fmt;   // kernel weight format: 0 Q8_0, 1 MXFP4, 2 IQ4_NL, 3 IQ4_XS
};

struct FfnPlan {
    int path;
    int msub;
    RowIdsPlan r;
    void *h, *hsh, *y, *ysh;
    // quantized-activation path: codes and block scales of x, h and the shared h
    int8_t *xq, *hq, *hshq;
    float *xd, *hd, *hshd;
    uint8_t *xs, *hs, *hshs;   // MXFP4 activations: E8M0 scale bytes (codes in xq, hq, hshq)
    bool fuse;                 // path 5: the down GEMV writes out itself
};

FfnPlan carve_ffn(Carve& c, const FfnDims& d, int path) {
    FfnPlan p{};
    p.path = path;
    const int64_t n = d.T * d.k;
    if (path == 3) {
        p.r = carve_row_ids(c, n, d.E, true, kQ8aTileM);
        p.xq = (int8_t*)c.take((size_t)d.T * d.n_embd);
        p.xd = (float*)c.take((size_t)d.T * (d.n_embd / 32) * 4);
        p.h = c.take((size_t)n * d.n_ff * 2);
        p.hsh = c.take((size_t)d.S * d.T * d.n_ff_sh * 2);
        p.hq = (int8_t*)c.take((size_t)n * d.n_ff);
        p.hd = (float*)c.take((size_t)n * (d.n_ff / 32) * 4);
        p.hshq = (int8_t*)c.take((size_t)d.S * d.T * d.n_ff_sh);
        p.hshd = (float*)c.take((size_t)d.S * d.T * (d.n_ff_sh / 32) * 4);
    } else if (path == 4) {
        p.r = carve_row_ids(c, n, d.E, true, kFp4TileM);
        p.xq = (int8_t*)c.take((size_t)d.T * fp4_code_row(d.n_embd));
        p.xs = (uint8_t*)c.take((size_t)d.T * fp4_scale_row(d.n_embd));
        p.hq = (int8_t*)c.take((size_t)n * fp4_code_row(d.n_ff));
        p.hs = (uint8_t*)c.take((size_t)n * fp4_scale_row(d.n_ff));
        p.hshq = (int8_t*)c.take((size_t)d.S * d.T * fp4_code_row(d.n_ff_sh));
        p.hshs = (uint8_t*)c.take((size_t)d.S * d.T * fp4_scale_row(d.n_ff_sh));
    } else if (path == 5) {   // h in float32; a small batch's down sums the slots itself
        p.h = c.take((size_t)n * d.n_ff * 4);
        p.hsh = c.take((size_t)d.S * d.T * d.n_ff_sh * 4);
        p.fuse = decode_fp4_fuses(n, d.E, d.S, d.n_ff > d.n_ff_sh ? d.n_ff : d.n_ff_sh);
        if (p.fuse) return p;
    } else if (path == 1) {
        p.msub = gemm_pick_msub((double)n / d.E);
        p.r = carve_row_ids(c, n, d.E, true, gemm_tile_m(p.msub));
        p.h = c.take((size_t)n * d.n_ff * 2);
        p.hsh = c.take((size_t)d.S * d.T * d.n_ff_sh * 2);
    } else {
        p.h = c.take((size_t)n * d.n_ff * 4);
        p.hsh = c.take((size_t)d.S * d.T * d.n_ff_sh * 4);
    }
    p.y = c.take((size_t)n * d.n_embd * 4);
    p.ysh = c.take((size_t)d.S * d.T * d.n_embd * 4);
    return p;
}

struct MmidPlan {
    int path;
    int msub;
    RowIdsPlan r;
    void* y;
    int8_t* aq;   // quantized-activation path: src1 codes [T*B][K] and block scales
    float* ad;
    uint8_t* as;  // MXFP4 activations: E8M0 scale bytes (codes [T*B][K/2] in aq)
    bool fuse;    // path 5: the GEMV writes the weighted sum itself
};

MmidPlan carve_mmid(Carve& c, int64_t T, int32_t k, int32_t E, int64_t N, bool weighted, bool q8, int path,
                    int32_t B = 1, int64_t K = 0) {
    MmidPlan p{};
    p.path = path;
    const int64_t n = T * k;
    if (path == 3) {
        p.r = carve_row_ids(c, n, E, true, kQ8aTileM);
        p.aq = (int8_t*)c.take((size_t)(T * B) * K);
        p.ad = (float*)c.take((size_t)(T * B) * (K / 32) * 4);
    } else if (path == 4) {
        p.r = carve_row_ids(c, n, E, true, kFp4TileM);
        p.aq = (int8_t*)c.take((size_t)(T * B) * fp4_code_row(K));
        p.as = (uint8_t*)c.take((size_t)(T * B) * fp4_scale_row(K));
    } else if (path == 5) {
        p.fuse = weighted && decode_fp4_fuses(n, E, 0, K);
        if (p.fuse) return p;
    } else if (!q8 || path == 1) {
        p.msub = gemm_pick_msub((double)n / E);
        p.r = carve_row_ids(c, n, E, true, q8 ? gemm_tile_m(p.msub) : 0);
    }
    if (weighted) p.y = c.take((size_t)n * N * 4);
    return p;
}

moe_status validate_ffn(const moe_weights* gate, const moe_weights* up, const moe_weights* down,
                        const moe_weights* sg, const moe_weights* su, const moe_weights* sd,
                        moe_dtype x_type, int64_t T, int32_t k, FfnDims* d) {
    moe_status s;
    if ((s = check_tokens(T, k))) return s;
    if ((s = check_weights(gate, "gate", false))) return s;
    if ((s = check_weights(up, "up", false))) return s;
    if ((s = check_weights(down, "down", false))) return s;
    if ((s = check_experts(gate->n_mat))) return s;
    if (x_type != MOE_BF16) return fail(MOE_EINVAL, "x must be BF16 (Q8_0 experts run bf16 activations)");
    if (up->type != gate->type || down->type != gate->type)
        return fail(MOE_EINVAL, "gate, up and down must have the same weight type");
    if (up->n_mat != gate->n_mat || down->n_mat != gate->n_mat || up->rows != gate->rows ||
        up->cols != gate->cols || down->rows != gate->cols || down->cols != gate->rows)
        return fail(MOE_EINVAL, "gate/up must be [E][n_ff][n_embd] and down [E][n_embd][n_ff]");
    d->T = T;
    d->k = k;
    d->E = (int32_t)gate->n_mat;
    d->n_ff = (int32_t)gate->rows;
    d->n_embd = (int32_t)gate->cols;
    d->fmt = kernel_fmt(gate->type);
    const bool any_sh = (sg && sg->n_mat) || (su && su->n_mat) || (sd && sd->n_mat);
    d->S = 0;
    d->n_ff_sh = 0;
    if (any_sh) {
        if (!sg || !su || !sd || !sg->n_mat || !su->n_mat || !sd->n_mat)
            return fail(MOE_EINVAL, "shared experts: give all of sh_gate, sh_up and sh_down, or none");
        if ((s = check_weights(sg, "sh_gate", false))) return s;
        if ((s = check_weights(su, "sh_up", false))) return s;
        if ((s = check_weights(sd, "sh_down", false))) return s;
        if (sg->type != gate->type || su->type != gate->type || sd->type != gate->type)
            return fail(MOE_EINVAL, "shared experts must have the routed experts' weight type");
        if (su->n_mat != sg->n_mat || sd->n_mat != sg->n_mat || su->rows != sg->rows ||
            su->cols != sg->cols || sg->cols != gate->cols || sd->rows != gate->cols ||
            sd->cols != sg->rows)
            return fail(MOE_EINVAL, "shared gate/up must be [S][n_ff_sh][n_embd], shared down [S][n_embd][n_ff_sh]");
        if (sg->n_mat > 64) return fail(MOE_ELIMIT, "at most 64 shared experts");
        d->S = (int32_t)sg->n_mat;
        d->n_ff_sh = (int32_t)sg->rows;
    }
    return MOE_OK;
}

int64_t ffn_min_width(const FfnDims& d) {
    int64_t w = d.n_embd < d.n_ff ? d.n_embd : d.n_ff;
    return d.S && d.n_ff_sh < w ? d.n_ff_sh : w;
}

int64_t ffn_act_width(const FfnDims& d) {
    int64_t w = d.n_embd > d.n_ff ? d.n_embd : d.n_ff;
    return w > d.n_ff_sh ? w : d.n_ff_sh;
}

moe_status validate_mmid(const moe_weights* w, moe_dtype st, int32_t B, int64_t T, int32_t k) {
    moe_status s;
    if ((s = check_tokens(T, k))) return s;
    if ((s = check_weights(w, "w", true))) return s;
    if ((s = check_experts(w->n_mat))) return s;
    if (B != 1 && B != k) return fail(MOE_EINVAL, "src1_rows_per_token must be 1 or n_used (got %d)", B);
    if (w->type == MOE_Q8_0 && st != MOE_BF16) return fail(MOE_EINVAL, "Q8_0 weights need BF16 src1");
    if (w->type == MOE_MXFP4 && st != MOE_BF16) return fail(MOE_EINVAL, "MXFP4 weights need BF16 src1");
    if (w->type == MOE_IQ4_NL && st != MOE_BF16) return fail(MOE_EINVAL, "IQ4_NL weights need BF16 src1");
    if (w->type == MOE_IQ4_XS && st != MOE_BF16) return fail(MOE_EINVAL, "IQ4_XS weights need BF16 src1");
    if (w->type == MOE_F32 && st != MOE_F32) return fail(MOE_EINVAL, "F32 weights need F32 src1");
    if ((w->type == MOE_BF16 || w->type == MOE_F16) && st != w->type)
        return fail(MOE_EINVAL, "%s weights need %s src1", type_name(w->type), type_name(w->type));
    if (w->type == MOE_I8 && st != MOE_BF16 && st != MOE_F16 && st != MOE_F32)
        return fail(MOE_EINVAL, "I8 weights need BF16, F16 or F32 src1");
    return MOE_OK;
}

RowIdsArgs row_ids_args(const int32_t* ids, int64_t n, int32_t k, int32_t E, int32_t B,
                        const RowIdsPlan& p) {
    RowIdsArgs a{};
    a.ids = ids;
    a.n = n;
    a.k = k;
    a.E = E;
    a.B = B;
    a.ids_src1 = p.ids_src1;
    a.ids_dst = p.ids_dst;
    a.bounds = p.bounds;
    if (p.scratch) row_ids_carve_scratch(a, p.scratch);
    return a;
}

constexpr int64_t k4GiB = 1LL << 32;

// Launch limits of the grouped GEMM path, checked before anything is enqueued:
// activation rows gathered through the row map are addressed by 32-bit byte offsets
// from the tensor's start, and one dispatch holds fewer than 2^32 work-items.
moe_status check_gemm_limits(const GemmArgs& g, int msub, int64_t gathered_rows, int64_t lda,
                             const char* what) {
    if (gathered_rows * lda * 2 > k4GiB - 256)
        return fail(MOE_ELIMIT, "%s: the gathered bf16 activation tensor must be under 4 GiB "
                    "(%lld rows x %lld columns)", what, (long long)gathered_rows, (long long)lda);
    if (gemm_q8_max_threads(g, msub) >= k4GiB)
        return fail(MOE_ELIMIT, "%s: the grouped GEMM grid exceeds 2^32 work-items", what);
    return MOE_OK;
}

moe_status check_q8a_limits(const GemmArgs& g, int64_t gathered_rows, int64_t K, const char* what) {
    if (gathered_rows * K > k4GiB - 256)
        return fail(MOE_ELIMIT, "%s: the gathered int8 activation tensor must be under 4 GiB "
                    "(%lld rows x %lld columns)", what, (long long)gathered_rows, (long long)K);
    if (gemm_q8a_max_threads(g) >= k4GiB)
        return fail(MOE_ELIMIT, "%s: the grouped GEMM grid exceeds 2^32 work-items", what);
    return MOE_OK;
}

// One activation quantization part: rows x K of bf16 -> codes and block scales.
QuantPart qpart(const void* src, int64_t rows, int64_t K, int8_t* q, float* d) {
    QuantPart p{};
    p.src = src;
    p.rows = rows;
    p.K = K;
    p.q = q;
    p.d = d;
    return p;
}

// ---------------------------------------------------------------- MXFP4 activations
constexpr int64_t kFp4MaxBlocks = 1LL << 31;   // 32-column blocks one quantization takes

// Quantization of a call's bf16 activations into rows as the grouped GEMM reads them.
QuantFp4Args fp4_act(const void* src, int64_t rows, int64_t K, int8_t* q, uint8_t* s) {
    QuantFp4Args p{};
    p.src_bf16 = 1;
    p.src = src;
    p.rows = rows;
    p.K = K;
    p.q = (uint8_t*)q;
    p.s = s;
    p.padded = 1;
    return p;
}

// One side of an MXFP4-activation GEMM launch: the routed experts' segments ...
GemmProblem fp4_routed(const moe_weights* w1, const moe_weights* w2, const RowIdsPlan& r, int64_t n,
                       const int8_t* aq, const uint8_t* as, void* out) {
    GemmProblem p{};
    p.qs1 = (const int8_t*)w1->data;
    p.d1 = (const uint16_t*)w1->scales;
    if (w2) {
        p.qs2 = (const int8_t*)w2->data;
        p.d2 = (const uint16_t*)w2->scales;
    }
    p.N = (int32_t)w1->rows;
    p.K = (int32_t)w1->cols;
    p.bounds = r.bounds;
    p.tile_off = r.tile_a;
    p.tile_tab = r.tile_tab;
    p.n_seg = (int32_t)w1->n_mat;
    p.m_tiles_max = (int32_t)m_tiles_bound(n, w1->n_mat, kFp4TileM);
    p.Aq = aq;
    p.As = as;
    p.out = out;
    p.ldo = w1->rows;
    return p;
}
// ... and the shared experts', each over all T tokens.
GemmProblem fp4_shared(const moe_weights* w1, const moe_weights* w2, int64_t T, const int8_t* aq,
                       const uint8_t* as, void* out) {
    GemmProblem p = fp4_routed(w1, w2, RowIdsPlan{}, 0, aq, as, out);
    p.seg_len = (int32_t)T;
    p.m_tiles_max = (int32_t)(w1->n_mat * ((T + kFp4TileM - 1) / kFp4TileM));
    return p;
}

moe_status check_fp4_act(const void* x, const char* name) {
    if ((uintptr_t)x % 16) return fail(MOE_EINVAL, "MXFP4 activations: %s must be 16-byte aligned", name);
    return MOE_OK;
}
moe_status check_fp4_weights(const moe_weights* w, const char* name) {
    if (!w || !w->n_mat) return MOE_OK;
    if ((uintptr_t)w->data % 16)
        return fail(MOE_EINVAL, "MXFP4 activations: the codes of %s must be 16-byte aligned", name);
    if (w->cols >= (1 << 24) || w->rows > INT32_MAX - 512)   // row numbers of the last tile stay in int32
        return fail(MOE_ELIMIT, "MXFP4 activations: %s must have cols < 2^24 and rows < 2^31 - 512 (got %lld, %lld)",
                    name, (long long)w->cols, (long long)w->rows);
    return MOE_OK;
}
// gathered_rows: rows of the activation tensor that is addressed through the row map.
moe_status check_fp4_limits(const GemmArgs& g, int64_t act_blocks, int64_t gathered_rows, const char* what) {
    if (gathered_rows * fp4_code_row(g.p[0].K) > k4GiB - 256)
        return fail(MOE_ELIMIT, "%s: the gathered MXFP4 activation codes must be under 4 GiB", what);
    if (act_blocks >= kFp4MaxBlocks)
        return fail(MOE_ELIMIT, "%s: too many activation blocks (rows * K / 32 must be under 2^31)", what);
    if (gemm_fp4_max_threads(g) >= k4GiB)
        return fail(MOE_ELIMIT, "%s: the grouped GEMM grid exceeds 2^32 work-items", what);
    return MOE_OK;
}
void fp4_tiles(RowIdsArgs& ra, const RowIdsPlan& r) {
    ra.tile_off[0] = r.tile_a;
    ra.tile_m[0] = kFp4TileM;
    ra.tile_tab[0] = r.tile_tab;
    ra.tile_cap[0] = r.tile_cap;
}

// The fused FFN up to the per-slot rows (p.y, p.ysh): row ids, x -> codes, gate/up (whose
// epilogue quantizes the float32 h), down.
moe_status ffn_fp4(const FfnDims& d, const FfnPlan& p, const moe_weights* gate, const moe_weights* up,
                   const moe_weights* down, const moe_weights* sg, const moe_weights* su,
                   const moe_weights* sd, const void* x, const int32_t* ids, Timer& tm, hipStream_t st) {
    moe_status s;
    const int64_t n = d.T * d.k;
    const bool shared = d.S > 0;
    if ((s = check_fp4_act(x, "x")) || (s = check_fp4_weights(gate, "gate")) ||
        (s = check_fp4_weights(up, "up")) || (s = check_fp4_weights(down, "down")))
        return s;
    if (shared && ((s = check_fp4_weights(sg, "sh_gate")) || (s = check_fp4_weights(su, "sh_up")) ||
                   (s = check_fp4_weights(sd, "sh_down"))))
        return s;
    RowIdsArgs ra = row_ids_args(ids, n, d.k, d.E, 1, p.r);
    fp4_tiles(ra, p.r);
    BesideRowIds beside{};
    beside.quant = fp4_act(x, d.T, d.n_embd, p.xq, p.xs);
    GemmArgs g{}, g2{};
    g.mode = 1;
    g.n_prob = g2.n_prob = shared ? 2 : 1;
    g.p[0] = fp4_routed(gate, up, p.r, n, p.xq, p.xs, p.hq);
    g.p[0].out_s = p.hs;
    g.p[0].a_rows = p.r.ids_src1;
    g2.p[0] = fp4_routed(down, nullptr, p.r, n, p.hq, p.hs, p.y);
    g2.p[0].out_rows = p.r.ids_dst;
    if (shared) {
        g.p[1] = fp4_shared(sg, su, d.T, p.xq, p.xs, p.hshq);
        g.p[1].out_s = p.hshs;
        g.p[1].a_row_mod = (int32_t)d.T;
        g2.p[1] = fp4_shared(sd, nullptr, d.T, p.hshq, p.hshs, p.ysh);
    }
    if ((s = check_fp4_limits(g, d.T * (d.n_embd / 32), d.T, "gate/up"))) return s;
    if ((s = check_fp4_limits(g2, n * (d.n_ff / 32) + (int64_t)d.S * d.T * (d.n_ff_sh / 32), 0, "down"))) return s;
    tm.begin();
    if ((s = hip_check(launch_row_ids(ra, st, nullptr, &beside), "row ids, quantize x"))) return s;
    tm.end();
    tm.begin();
    if ((s = hip_check(launch_gemm_fp4(g, st), "gate/up grouped GEMM (MXFP4)"))) return s;
    tm.end();
    tm.begin();
    if ((s = hip_check(launch_gemm_fp4(g2, st), "down grouped GEMM (MXFP4)"))) return s;
    tm.end();
    return MOE_OK;
}

// moe_mul_mat_id up to the per-slot rows: row ids, src1 -> codes, grouped GEMM.
moe_status mmid_fp4(const MmidPlan& p, const moe_weights* w, const void* src1, int32_t B,
                    const int32_t* ids, int64_t T, int32_t k, float* slot_out, bool weighted, Timer& tm,
                    hipStream_t st) {
    moe_status s;
    const int64_t n = T * k;
    if ((s = check_fp4_act(src1, "src1")) || (s = check_fp4_weights(w, "w"))) return s;
    RowIdsArgs ra = row_ids_args(ids, n, k, (int32_t)w->n_mat, B, p.r);
    fp4_tiles(ra, p.r);
    BesideRowIds beside{};
    beside.quant = fp4_act(src1, T * B, w->cols, p.aq, p.as);
    if (!weighted) beside.zero = ZeroSlots{ids, slot_out, n, (int32_t)w->n_mat, (int32_t)w->rows};
    GemmArgs g{};
    g.n_prob = 1;
    g.stream_out = !weighted;
    g.p[0] = fp4_routed(w, nullptr, p.r, n, p.aq, p.as, slot_out);
    g.p[0].a_rows = p.r.ids_src1;
    g.p[0].out_rows = p.r.ids_dst;
    if ((s = check_fp4_limits(g, T * B * (w->cols / 32), T * B, "mul_mat_id"))) return s;
    tm.begin();
    if ((s = hip_check(launch_row_ids(ra, st, nullptr, &beside), "row ids, quantize src1"))) return s;
    tm.end();
    tm.begin();
    if ((s = hip_check(launch_gemm_fp4(g, st), "grouped GEMM (MXFP4)"))) return s;
    tm.end();
    return MOE_OK;
}

DecFp4Weights fp4_dec_weights(const moe_weights* w1, const moe_weights* w2) {
    DecFp4Weights d{};
    if (!w1 || !w1->n_mat) return d;
    d.q1 = (const uint8_t*)w1->data;
    d.s1 = (const uint8_t*)w1->scales;
    if (w2) {
        d.q2 = (const uint8_t*)w2->data;
        d.s2 = (const uint8_t*)w2->scales;
    }
    d.n_mat = (int32_t)w1->n_mat;
    d.N = (int32_t)w1->rows;
    d.K = (int32_t)w1->cols;
    return d;
}

// The fused FFN by GEMV: gate/up (float32 h), then down (p.fuse: with the sum over the slots).
moe_status ffn_dec_fp4(const FfnDims& d, const FfnPlan& p, const moe_weights* gate, const moe_weights* up,
                       const moe_weights* down, const moe_weights* sg, const moe_weights* su,
                       const moe_weights* sd, const void* x, const int32_t* ids, const float* route_w,
                       float* out, Timer& tm, hipStream_t st) {
    moe_status s;
    const bool shared = d.S > 0;
    if ((s = check_fp4_act(x, "x")) || (s = check_fp4_weights(gate, "gate")) ||
        (s = check_fp4_weights(up, "up")) || (s = check_fp4_weights(down, "down")))
        return s;
    if (shared && ((s = check_fp4_weights(sg, "sh_gate")) || (s = check_fp4_weights(su, "sh_up")) ||
                   (s = check_fp4_weights(sd, "sh_down"))))
        return s;
    DecFp4Args a{};
    a.ids = ids;
    a.T = (int32_t)d.T;
    a.k = d.k;
    a.E = d.E;
    DecFp4Args b = a;
    a.rw = fp4_dec_weights(gate, up);
    if (shared) a.sw = fp4_dec_weights(sg, su);
    a.act = a.sact = x;
    a.act_B = 1;
    a.mode = 1;
    a.out = (float*)p.h;
    a.sout = (float*)p.hsh;
    b.rw = fp4_dec_weights(down, nullptr);
    if (shared) b.sw = fp4_dec_weights(sd, nullptr);
    b.act = p.h;
    b.sact = p.hsh;
    b.f32 = 1;
    b.act_B = d.k;
    b.sact_jstride = d.T;
    b.fuse = p.fuse;
    b.route_w = route_w;
    b.out_tok = out;
    b.out = (float*)p.y;
    b.sout = (float*)p.ysh;
    tm.begin();
    if ((s = hip_check(launch_decode_fp4(a, st), "gate/up GEMV (MXFP4)"))) return s;
    tm.end();
    tm.begin();
    if ((s = hip_check(launch_decode_fp4(b, st), "down GEMV (MXFP4)"))) return s;
    tm.end();
    return MOE_OK;
}

// moe_mul_mat_id by GEMV: per-slot rows to slot_out, or (p.fuse) the weighted sum to dst.
moe_status mmid_dec_fp4(const MmidPlan& p, const moe_weights* w, const void* src1, int32_t B,
                        const int32_t* ids, int64_t T, int32_t k, const float* route_w, float* slot_out,
                        float* dst, Timer& tm, hipStream_t st) {
    moe_status s;
    if ((s = check_fp4_act(src1, "src1")) || (s = check_fp4_weights(w, "w"))) return s;
    DecFp4Args a{};
    a.ids = ids;
    a.T = (int32_t)T;
    a.k = k;
    a.E = (int32_t)w->n_mat;
    a.rw = fp4_dec_weights(w, nullptr);
    a.act = src1;
    a.act_B = B;
    a.out = slot_out;
    a.fuse = p.fuse;
    a.route_w = route_w;
    a.out_tok = dst;
    tm.begin();
    if ((s = hip_check(launch_decode_fp4(a, st), "GEMV (MXFP4)"))) return s;
    tm.end();
    return MOE_OK;
}

// ---------------------------------------------------------------- 16-bit and int8 experts
// Options of their calls: act_quant 0, a path the call has.
moe_status check_elem_options(const moe_options* o, int max_path, const char* what) {
    if (o && o->act_quant)
        return fail(MOE_EINVAL, "%s with BF16, F16 or I8 experts: options.act_quant must be 0 (got %d)", what, o->act_quant);
    if (o && (o->path < 0 || o->path > max_path))
        return fail(MOE_EINVAL, "%s with BF16, F16 or I8 experts: options.path must be 0 to %d (got %d)", what, max_path,
                    o->path);
    return MOE_OK;
}

// 1 grouped GEMM, 2 GEMV, or a negative status.
int elem_path(int64_t T, int32_t k, int32_t E, int64_t K, moe_dtype type, const moe_options* o) {
    const moe_status s = check_elem_options(o, 2, "mul_mat_id");
    if (s) return s;
    const bool dec_ok = T * (int64_t)k <= kDecXSlots && (type != MOE_I8 || K <= kDecXMaxK);
    const int32_t force = o ? o->path : 0;
    if (force == 1) return 1;
    if (force == 2) {
        if (!dec_ok)
            return fail(MOE_EINVAL, "GEMV path with BF16, F16 or I8 experts needs n_tokens*n_used <= %d, and I8 cols <= %d",
                        kDecXSlots, kDecXMaxK);
        return 2;
    }
    // The GEMV up to four slots an expert on average, which is one of its passes, and always for a dozen slots
    // (mul_mat_id, GEMV against GEMM in us per call on one MI355X, weight copies in turn, bf16: E32 k4 2880 x 2880
    // T = 1 12.2 / 26.5, T = 16 82 / 104; E128 k8 2048 x 7168 T = 8 213 / 257; four slots an expert, E16 k1 2048 x 2048
    // T = 64, 37.5 / 38.1, int8 27.3 / 25.6; eight, E8 k8 2880 x 2880 T = 8, 51.6 / 34.5; E1 4096 x 4096 T = 12
    // 30.7 / 37.9, T = 16 39.9 / 38.1)
    return dec_ok && (T * (int64_t)k <= 4 * (int64_t)E || T * (int64_t)k <= 12) ? 2 : 1;
}

struct ElemPlan {
    bool fuse;    // the GEMV writes the weighted sum itself
    RowIdsPlan r;
    int tile_m;
    int8_t* q;    // I8: src1 codes and row scales
    float* d;
    float* y;     // weighted: per-slot rows
};
ElemPlan carve_elem(Carve& c, const moe_weights* w, int64_t T, int32_t k, int32_t B, bool weighted, int path) {
    ElemPlan p{};
    const int64_t n = T * k;
    if (path == 2) {
        p.fuse = weighted && decode_x_fuses(elem_of(w->type), T, B, w->cols);
        if (w->type == MOE_I8 && !decode_x_makes(T)) {
            p.q = (int8_t*)c.take((size_t)(T * B) * w->cols);
            p.d = (float*)c.take((size_t)(T * B) * 4);
        }
        if (weighted && !p.fuse) p.y = (float*)c.take((size_t)n * w->rows * 4);
        return p;
    }
    p.tile_m = expert_gemm_tile_m(n, w->n_mat, w->rows);
    p.r = carve_row_ids(c, n, (int32_t)w->n_mat, true, p.tile_m);
    if (w->type == MOE_I8) {
        p.q = (int8_t*)c.take((size_t)(T * B) * w->cols);
        p.d = (float*)c.take((size_t)(T * B) * 4);
    }
    if (weighted) p.y = (float*)c.take((size_t)n * w->rows * 4);
    return p;
}
ExpertGemm elem_gemm(const moe_weights* w, const RowIdsPlan& r, int tile_m, int64_t n) {
    ExpertGemm g{};
    g.type = elem_of(w->type);
    g.W = w->data;
    g.w_scale = w->type == MOE_I8 ? (const float*)w->scales : nullptr;
    g.N = (int32_t)w->rows;
    g.K = (int32_t)w->cols;
    g.E = (int32_t)w->n_mat;
    g.tile_off = r.tile_a;
    g.tile_tab = r.tile_tab;
    g.tile_m = tile_m;
    g.m_tiles_max = (int32_t)m_tiles_bound(n, w->n_mat, tile_m);
    return g;
}
void elem_tiles(RowIdsArgs& ra, const RowIdsPlan& r, int tile_m) {
    ra.tile_off[0] = r.tile_a;
    ra.tile_m[0] = tile_m;
    ra.tile_x[0] = expert_gemm_tile_x(tile_m);
    ra.tile_tab[0] = r.tile_tab;
    ra.tile_cap[0] = r.tile_cap;
}
moe_status check_grid(int64_t blocks, const char* what) {
    if (blocks * 512 >= k4GiB) return fail(MOE_ELIMIT, "%s: the grid exceeds 2^32 work-items", what);
    return MOE_OK;
}

// Activations (elements) that are quantized beside the row ids, where they save a launch (4.3 M: 8.1 us instead of 6.6
// and 6.5); more go through the quantizer's own kernel, which reads them once (7.3 M: no difference).
constexpr int64_t kRowsBesideMax = 6 << 20;

// moe_mul_mat_id up to the per-slot rows (slot_out; weighted: those of invalid slots are not written).
moe_status mmid_elem(const ElemPlan& p, const moe_weights* w, const void* src1, moe_dtype src1_type, int32_t B,
                     const int32_t* ids, int64_t T, int32_t k, float* slot_out, bool weighted, Timer& tm, hipStream_t st) {
    moe_status s;
    const int64_t n = T * k;
    RowIdsArgs ra = row_ids_args(ids, n, k, (int32_t)w->n_mat, B, p.r);
    elem_tiles(ra, p.r, p.tile_m);
    ExpertGemm g = elem_gemm(w, p.r, p.tile_m, n);
    g.A = w->type == MOE_I8 ? (const void*)p.q : src1;
    g.lda = w->cols;
    g.a_scale = p.d;
    g.a_rows = p.r.ids_src1;
    g.out = slot_out;
    g.out_rows = p.r.ids_dst;
    if ((s = check_grid(expert_gemm_grid(g, 0), "mul_mat_id"))) return s;
    const QuantRowsArgs q{src1, elem_of(src1_type), T * B, w->cols, p.q, p.d};
    const bool apart = w->type == MOE_I8 && T * B * w->cols > kRowsBesideMax;
    BesideRowIds beside{};
    if (w->type == MOE_I8 && !apart) beside.rows = q;
    if (!weighted) beside.zero = ZeroSlots{ids, slot_out, n, (int32_t)w->n_mat, (int32_t)w->rows};
    tm.begin();
    if ((s = hip_check(launch_row_ids(ra, st, nullptr, &beside), "row ids"))) return s;
    tm.end();
    if (apart) {
        tm.begin();
        if ((s = hip_check(launch_quant_rows(q, st), "quantize src1"))) return s;
        tm.end();
    }
    tm.begin();
    if ((s = hip_check(launch_expert_gemm(g, st), "grouped GEMM"))) return s;
    tm.end();
    return MOE_OK;
}

moe_status mul_mat_id_elem(const moe_weights* w, const void* src1, moe_dtype src1_type, int32_t B, const int32_t* ids,
                           int64_t T, int32_t k, const float* route_w, float* dst, const moe_options* opt, void* ws,
                           size_t ws_bytes, hipStream_t st) {
    moe_status s;
    const int path = elem_path(T, k, (int32_t)w->n_mat, w->cols, w->type, opt);
    if (path < 0) return (moe_status)path;
    const bool weighted = route_w != nullptr;
    if ((s = check_aligned(src1, "src1"))) return s;
    if (weighted && (s = check_grid((w->rows + 1023) / 1024 * T, "the weighted sum"))) return s;
    Carve sz(nullptr);
    carve_elem(sz, w, T, k, B, weighted, path);
    if (sz.off > ws_bytes || (sz.off && !ws)) return fail(MOE_EWORKSPACE, "workspace needs %zu bytes", sz.off);
    if ((s = check_aligned(ws, "the workspace"))) return s;
    Carve c(ws);
    const ElemPlan p = carve_elem(c, w, T, k, B, weighted, path);
    Timer tm(opt, st);
    float* slot_out = weighted ? p.y : dst;
    if (path == 2) {
        DecXArgs a{};
        a.type = elem_of(w->type);
        a.W = w->data;
        a.w_scale = (const float*)w->scales;
        a.N = (int32_t)w->rows;
        a.K = (int32_t)w->cols;
        a.E = (int32_t)w->n_mat;
        a.T = (int32_t)T;
        a.k = k;
        a.act_B = B;
        a.ids = ids;
        a.src = p.q ? (const void*)p.q : src1;
        a.src_type = elem_of(src1_type);
        a.src_scale = p.d;
        a.out = slot_out;
        a.route_w = route_w;
        a.out_tok = p.fuse ? dst : nullptr;
        if (decode_x_work_items(a) >= k4GiB) return fail(MOE_ELIMIT, "mul_mat_id: the GEMV's grid exceeds 2^32 work-items");
        if (p.q) {
            const QuantRowsArgs q{src1, elem_of(src1_type), T * B, w->cols, p.q, p.d};
            tm.begin();
            if ((s = hip_check(launch_quant_rows(q, st), "quantize src1"))) return s;
            tm.end();
        }
        tm.begin();
        if ((s = hip_check(launch_decode_x(a, st), "GEMV"))) return s;
        tm.end();
        if (p.fuse || !weighted) {   // written in full, rows of invalid slots too
            g_stages = tm.stage;
            return MOE_OK;
        }
    } else {
        if ((s = mmid_elem(p, w, src1, src1_type, B, ids, T, k, slot_out, weighted, tm, st))) return s;
        if (!weighted) {
            g_stages = tm.stage;
            return MOE_OK;
        }
    }
    ReduceArgs rd{};
    rd.ids = ids;
    rd.route_w = route_w;
    rd.T = (int32_t)T;
    rd.k = k;
    rd.E = (int32_t)w->n_mat;
    rd.N = (int32_t)w->rows;
    rd.y = slot_out;
    rd.out = dst;
    tm.begin();
    if ((s = hip_check(launch_reduce(rd, st), "reduce"))) return s;
    tm.end();
    g_stages = tm.stage;
    return MOE_OK;
}

enum Want { kWantX = 1, kWantW = 2, kWantR = 4 };
struct GradPlan {
    RowIdsPlan r;
    int tile_m;
    bool direct;    // the row gradients go to d_src1 as they are
    int64_t ld;     // row length of dY
    void* dy;       // d_dst in the experts' type, rows of ld (nullptr: d_dst itself)
    float* g;       // per-slot rows of g (not direct)
    float* dots;    // direct: parts of d_route_w
    int dot_parts;
    int terms;      // of which rows route_w * dY are the sums
    void* scaled;   // weighted d_w: those rows by slot, [terms][n][ld]
    float* tops;    // float16: parts of their largest, then their scale's inverse
    int splits;     // of the positions of each expert, for d_w
    float* parts;
};
// dy_as_is: d_dst can be read in place (its type, and rows of whole 16-byte chunks at aligned addresses). w_f32: d_w is
// float32, for which the scaled rows keep all bits (three terms); two hold more than twice the bits of a 16-bit d_w.
GradPlan carve_grad(Carve& c, const moe_weights* w, int64_t T, int32_t k, int32_t B, bool weighted, int want,
                    bool dy_as_is, bool w_f32) {
    GradPlan p{};
    const int64_t n = T * k;
    p.tile_m = expert_gemm_tile_m(n, w->n_mat, w->cols);
    p.direct = B == k;   // a slot a row of d_src1
    p.r = carve_row_ids(c, n, (int32_t)w->n_mat, true, p.tile_m);
    p.ld = (w->rows + 7) / 8 * 8;
    if (!dy_as_is && (!weighted || (want & (kWantX | kWantR)))) p.dy = c.take((size_t)(weighted ? T : n) * p.ld * 2);
    p.terms = !weighted ? 1 : w_f32 ? 3 : 2;
    if (weighted && (want & kWantW)) {
        p.scaled = c.take((size_t)n * p.ld * 2 * p.terms);
        if (w->type == MOE_F16) p.tops = (float*)c.take((kGradTops + 1) * 4);
    }
    p.splits = want & kWantW ? expert_grad_w_splits(n, w->n_mat, w->rows, w->cols) : 1;
    if (p.splits > 1) p.parts = (float*)c.take((size_t)p.splits * w->n_mat * w->rows * w->cols * 4);
    if ((want & (kWantX | kWantR)) && !p.direct) p.g = (float*)c.take((size_t)n * w->cols * 4);
    if ((want & kWantR) && p.direct) {
        p.dot_parts = expert_dot_parts(elem_gemm(w, p.r, p.tile_m, n));
        p.dots = (float*)c.take((size_t)n * p.dot_parts * 4);
    }
    return p;
}
moe_status validate_grad(const moe_weights* w, moe_dtype src1_type, moe_dtype d_dst_type, int32_t B, int64_t T,
                         int32_t k, bool weighted, int want, const moe_options* opt) {
    moe_status s;
    if ((s = check_tokens(T, k))) return s;
    if ((s = check_weights(w, "w", true))) return s;
    if (w->type != MOE_BF16 && w->type != MOE_F16)
        return fail(MOE_EINVAL, "gradients of mul_mat_id need BF16 or F16 experts");
    if ((s = check_experts(w->n_mat))) return s;
    if (B != 1 && B != k) return fail(MOE_EINVAL, "src1_rows_per_token must be 1 or n_used (got %d)", B);
    if (src1_type != w->type) return fail(MOE_EINVAL, "src1 must be of the experts' type (%s)", type_name(w->type));
    if (d_dst_type != w->type && d_dst_type != MOE_F32)
        return fail(MOE_EINVAL, "d_dst must be of the experts' type (%s) or F32", type_name(w->type));
    if (!want || (want & ~7)) return fail(MOE_EINVAL, "at least one of d_src1, d_w and d_route_w is needed");
    if ((want & kWantR) && !weighted) return fail(MOE_EINVAL, "d_route_w needs route_w");
    return check_elem_options(opt, 1, "gradients of mul_mat_id");
}

moe_status check_router(const moe_router_config* c, int64_t T, int32_t E, int32_t k, bool choose) {
    moe_status s;
    if ((s = check_tokens(T, k))) return s;
    if ((s = check_experts(E))) return s;
    if (!c) return fail(MOE_EINVAL, "router config is NULL");
    if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID)
        return fail(MOE_EINVAL, "router config: score must be 0 (softmax) or 1 (sigmoid) (got %d)", c->score);
    if (c->renorm != 0 && c->renorm != 1)
        return fail(MOE_EINVAL, "router config: renorm must be 0 or 1 (got %d)", c->renorm);
    if (!(c->scale - c->scale == 0.f)) return fail(MOE_EINVAL, "router config: scale must be finite");
    if (!choose) return MOE_OK;
    if (c->n_group < 1 || E % c->n_group)
        return fail(MOE_EINVAL, "router config: n_group (%d) must divide n_experts (%d)", c->n_group, E);
    if (c->topk_group < 1 || c->topk_group > c->n_group)
        return fail(MOE_EINVAL, "router config: topk_group must be 1 to n_group (got %d)", c->topk_group);
    if (c->group_top != 1 && c->group_top != 2)
        return fail(MOE_EINVAL, "router config: group_top must be 1 or 2 (got %d)", c->group_top);
    if ((int64_t)k * c->n_group > (int64_t)c->topk_group * E)
        return fail(MOE_EINVAL, "n_used (%d) exceeds the experts of %d kept groups", k, c->topk_group);
    return MOE_OK;
}

}  // namespace

void moe::set_last_error(const char* msg) { g_err = msg; }

extern "C" {

const char* moe_status_string(moe_status s) {
    switch (s) {
        case MOE_OK: return "MOE_OK";
        case MOE_EINVAL: return "MOE_EINVAL: invalid argument";
        case MOE_ELIMIT: return "MOE_ELIMIT: size limit exceeded";
        case MOE_EWORKSPACE: return "MOE_EWORKSPACE: workspace too small";
        case MOE_EHIP: return "MOE_EHIP: HIP launch failed";
    }
    return "unknown moe_status";
}

const char* moe_last_error(void) { return g_err.c_str(); }
int32_t moe_last_stage_count(void) { return g_stages; }

int32_t moe_select_path(int64_t n_tokens, int32_t n_used, int32_t n_experts, int64_t act_width,
                        const moe_options* opt) {
    moe_status s;
    if ((s = check_tokens(n_tokens, n_used))) return s;
    if ((s = check_experts(n_experts))) return s;
    if (act_width <= 0) return fail(MOE_EINVAL, "act_width must be > 0");
    return select_path(n_tokens, n_used, n_experts, act_width, opt);
}

int32_t moe_select_path_typed(int64_t n_tokens, int32_t n_used, int32_t n_experts, int64_t act_width,
                              moe_dtype weight_type, const moe_options* opt) {
    moe_status s;
    if ((s = check_tokens(n_tokens, n_used))) return s;
    if ((s = check_experts(n_experts))) return s;
    if (act_width <= 0) return fail(MOE_EINVAL, "act_width must be > 0");
    if (is_elem(weight_type)) return elem_path(n_tokens, n_used, n_experts, act_width, weight_type, opt);
    if (weight_type != MOE_Q8_0 && weight_type != MOE_MXFP4 && weight_type != MOE_IQ4_NL &&
        weight_type != MOE_IQ4_XS)
        return fail(MOE_EINVAL, "weight_type must be Q8_0, MXFP4, IQ4_NL, IQ4_XS, BF16, F16 or I8 (got %d)", (int)weight_type);
    return select_path_aq(n_tokens, n_used, n_experts, act_width, weight_type, opt, 0, act_width);
}

size_t moe_row_ids_workspace_size(int64_t n_tokens, int32_t n_used, int32_t n_experts) {
    if (check_tokens(n_tokens, n_used) || check_experts(n_experts)) return 0;
    Carve c(nullptr);
    carve_row_ids(c, n_tokens * n_used, n_experts, false, 0);
    return c.off;
}

moe_status moe_gather_rows(const void* src1, moe_dtype src1_type, int64_t src1_rows, int64_t K,
                           const int32_t* ids_src1, int64_t n, void* dst, void* stream) {
    g_err.clear();
    if (src1_type != MOE_BF16 && src1_type != MOE_F32)
        return fail(MOE_EINVAL, "gather: src1_type must be BF16 or F32");
    if (src1_rows <= 0 || K <= 0 || n < 0) return fail(MOE_EINVAL, "gather: sizes must be > 0 (n >= 0)");
    if (src1_rows > INT32_MAX) return fail(MOE_ELIMIT, "gather: src1_rows must fit in int32");
    if (n > (int64_t)INT32_MAX * 4) return fail(MOE_ELIMIT, "gather: too many rows for one launch");
    if (n == 0) return MOE_OK;
    if (!src1 || !ids_src1 || !dst) return fail(MOE_EINVAL, "NULL pointer argument");
    GatherArgs a{src1, src1_rows, K * (src1_type == MOE_BF16 ? 2 : 4), ids_src1, n, dst};
    return hip_check(launch_gather(a, (hipStream_t)stream), "gather");
}

moe_status moe_row_ids(const int32_t* ids, int64_t n_tokens, int32_t n_used, int32_t n_experts,
                       int32_t src1_rows_per_token, int32_t* ids_src1, int32_t* ids_dst,
                       int32_t* expert_bounds, void* ws, size_t ws_bytes, void* stream) {
    moe_status s;
    g_err.clear();
    if ((s = check_tokens(n_tokens, n_used))) return s;
    if ((s = check_experts(n_experts))) return s;
    if (src1_rows_per_token != 1 && src1_rows_per_token != n_used)
        return fail(MOE_EINVAL, "src1_rows_per_token must be 1 or n_used");
    if (!expert_bounds || (n_tokens > 0 && (!ids || !ids_src1 || !ids_dst)))
        return fail(MOE_EINVAL, "NULL pointer argument");
    const size_t need = moe_row_ids_workspace_size(n_tokens, n_used, n_experts);
    if (need > ws_bytes || (need && !ws)) return fail(MOE_EWORKSPACE, "workspace needs %zu bytes", need);
    Carve c(ws);
    RowIdsPlan p = carve_row_ids(c, n_tokens * n_used, n_experts, false, 0);
    p.ids_src1 = ids_src1;
    p.ids_dst = ids_dst;
    p.bounds = expert_bounds;
    const RowIdsArgs a = row_ids_args(ids, n_tokens * n_used, n_used, n_experts, src1_rows_per_token, p);
    return hip_check(launch_row_ids(a, (hipStream_t)stream, nullptr), "row ids");
}

size_t moe_ffn_fused_workspace_size(const moe_weights* gate, const moe_weights* sh_gate,
                                    moe_dtype x_type, int64_t n_tokens, int32_t n_used,
                                    const moe_options* opt) {
    if (!gate) return 0;
    FfnDims d{};
    const moe_weights up = *gate;
    moe_weights down = *gate;
    down.rows = gate->cols;
    down.cols = gate->rows;
    const moe_weights* su = nullptr;
    moe_weights sup{}, sdown{};
    if (sh_gate && sh_gate->n_mat) {
        sup = *sh_gate;
        sdown = *sh_gate;
        sdown.rows = sh_gate->cols;
        sdown.cols = sh_gate->rows;
        su = &sup;
    }
    if (validate_ffn(gate, &up, &down, (su ? sh_gate : nullptr), su, (su ? &sdown : nullptr),
                     x_type, n_tokens, n_used, &d))
        return 0;
    const int path = select_path_aq(d.T, d.k, d.E, ffn_act_width(d), gate->type, opt, d.S,
                                    ffn_min_width(d));
    if (path < 0) return 0;
    Carve c(nullptr);
    carve_ffn(c, d, path);
    return c.off;
}

moe_status moe_ffn_fused(const moe_weights* gate, const moe_weights* up, const moe_weights* down,
                         const moe_weights* sh_gate, const moe_weights* sh_up,
                         const moe_weights* sh_down, const void* x, moe_dtype x_type,
                         const int32_t* ids, const float* route_w, int64_t n_tokens, int32_t n_used,
                         float* out, const moe_options* opt, void* ws, size_t ws_bytes,
                         void* stream) {
    g_err.clear();
    FfnDims d{};
    moe_status s = validate_ffn(gate, up, down, sh_gate, sh_up, sh_down, x_type, n_tokens, n_used, &d);
    if (s) return s;
    if (n_tokens == 0) {
        g_stages = 0;
        return MOE_OK;
    }
    if (!x || !ids || !route_w || !out) return fail(MOE_EINVAL, "NULL pointer argument");
    const int path = select_path_aq(d.T, d.k, d.E, ffn_act_width(d), gate->type, opt, d.S,
                                    ffn_min_width(d));
    if (path < 0) return (moe_status)path;
    Carve sz(nullptr);
    carve_ffn(sz, d, path);
    if (sz.off > ws_bytes || !ws) return fail(MOE_EWORKSPACE, "workspace needs %zu bytes", sz.off);
    if ((path == 4 || path == 5) && (s = check_fp4_act(ws, "the workspace"))) return s;
    Carve c(ws);
    const FfnPlan p = carve_ffn(c, d, path);
    const hipStream_t st = (hipStream_t)stream;
    Timer tm(opt, st);
    const int64_t n = d.T * d.k;
    const bool shared = d.S > 0;
    bool reduced = false;

    if (path == 3) {
        // quantized activations: row ids, x -> codes, gate/up int8 GEMM (h in bf16),
        // h -> codes, down int8 GEMM, then the reduce below
        const int bm = kQ8aTileM;
        RowIdsArgs ra = row_ids_args(ids, n, d.k, d.E, 1, p.r);
        ra.tile_off[0] = p.r.tile_a;
        ra.tile_m[0] = bm;
        ra.tile_tab[0] = p.r.tile_tab;
        ra.tile_cap[0] = p.r.tile_cap;
        QuantArgs qx{};
        qx.src_bf16 = 1;
        qx.n_part = 1;
        qx.part[0] = qpart(x, d.T, d.n_embd, p.xq, p.xd);
        GemmArgs g{};
        g.mode = 1;
        g.n_prob = shared ? 2 : 1;
        GemmProblem& r = g.p[0];
        r.qs1 = (const int8_t*)gate->data;
        r.d1 = (const uint16_t*)gate->scales;
        r.qs2 = (const int8_t*)up->data;
        r.d2 = (const uint16_t*)up->scales;
        r.N = d.n_ff;
        r.K = d.n_embd;
        r.bounds = p.r.bounds;
        r.tile_off = p.r.tile_a;
        r.tile_tab = p.r.tile_tab;
        r.n_seg = d.E;
        r.m_tiles_max = (int32_t)m_tiles_bound(n, d.E, bm);
        r.Aq = p.xq;
        r.Ad = p.xd;
        r.a_rows = p.r.ids_src1;
        r.out = p.h;
        r.ldo = d.n_ff;
        if (shared) {
            GemmProblem& q = g.p[1];
            q.qs1 = (const int8_t*)sh_gate->data;
            q.d1 = (const uint16_t*)sh_gate->scales;
            q.qs2 = (const int8_t*)sh_up->data;
            q.d2 = (const uint16_t*)sh_up->scales;
            q.N = d.n_ff_sh;
            q.K = d.n_embd;
            q.n_seg = d.S;
            q.seg_len = (int32_t)d.T;
            q.m_tiles_max = (int32_t)(d.S * ((d.T + bm - 1) / bm));
            q.Aq = p.xq;
            q.Ad = p.xd;
            q.a_row_mod = (int32_t)d.T;
            q.out = p.hsh;
            q.ldo = d.n_ff_sh;
        }
        QuantArgs qh{};
        qh.src_bf16 = 1;
        qh.n_part = shared ? 2 : 1;
        qh.part[0] = qpart(p.h, n, d.n_ff, p.hq, p.hd);
        if (shared) qh.part[1] = qpart(p.hsh, (int64_t)d.S * d.T, d.n_ff_sh, p.hshq, p.hshd);
        GemmArgs g2{};
        g2.mode = 0;
        g2.n_prob = shared ? 2 : 1;
        GemmProblem& r2 = g2.p[0];
        r2.qs1 = (const int8_t*)down->data;
        r2.d1 = (const uint16_t*)down->scales;
        r2.N = d.n_embd;
        r2.K = d.n_ff;
        r2.bounds = p.r.bounds;
        r2.tile_off = p.r.tile_a;
        r2.tile_tab = p.r.tile_tab;
        r2.n_seg = d.E;
        r2.m_tiles_max = r.m_tiles_max;
        r2.Aq = p.hq;
        r2.Ad = p.hd;
        r2.out = p.y;
        r2.ldo = d.n_embd;
        r2.out_rows = p.r.ids_dst;
        if (shared) {
            GemmProblem& q = g2.p[1];
            q.qs1 = (const int8_t*)sh_down->data;
            q.d1 = (const uint16_t*)sh_down->scales;
            q.N = d.n_embd;
            q.K = d.n_ff_sh;
            q.n_seg = d.S;
            q.seg_len = (int32_t)d.T;
            q.m_tiles_max = g.p[1].m_tiles_max;
            q.Aq = p.hshq;
            q.Ad = p.hshd;
            q.out = p.ysh;
            q.ldo = d.n_embd;
        }
        if ((uintptr_t)x % 16) return fail(MOE_EINVAL, "quantized activations: x must be 16-byte aligned");
        if ((s = check_q8a_limits(g, d.T, d.n_embd, "gate/up"))) return s;
        if ((s = check_q8a_limits(g2, 0, d.n_ff, "down"))) return s;
        tm.begin();
        if ((s = hip_check(launch_row_ids(ra, st, nullptr), "row ids"))) return s;
        tm.end();
        tm.begin();
        if ((s = hip_check(launch_quant_act(qx, st), "quantize x"))) return s;
        tm.end();
        tm.begin();
        if ((s = hip_check(launch_gemm_q8a(g, st), "gate/up grouped GEMM (int8)"))) return s;
        tm.end();
        tm.begin();
        if ((s = hip_check(launch_quant_act(qh, st), "quantize h"))) return s;
        tm.end();
        tm.begin();
        if ((s = hip_check(launch_gemm_q8a(g2, st), "down grouped GEMM (int8)"))) return s;
        tm.end();
    } else if (path == 4) {
        if ((s = ffn_fp4(d, p, gate, up, down, sh_gate, sh_up, sh_down, x, ids, tm, st))) return s;
    } else if (path == 5) {
        if ((s = ffn_dec_fp4(d, p, gate, up, down, sh_gate, sh_up, sh_down, x, ids, route_w, out, tm, st))) return s;
        reduced = p.fuse;
    } else if (path == 1) {
        const int bm = gemm_tile_m(p.msub);
        RowIdsArgs ra = row_ids_args(ids, n, d.k, d.E, 1, p.r);
        ra.tile_off[0] = p.r.tile_a;
        ra.tile_m[0] = bm;
        ra.tile_tab[0] = p.r.tile_tab;
        ra.tile_cap[0] = p.r.tile_cap;

        GemmArgs g{};
        g.mode = 1;
        g.fmt = d.fmt;
        g.n_prob = shared ? 2 : 1;
        GemmProblem& r = g.p[0];
        r.qs1 = (const int8_t*)gate->data;
        r.d1 = (const uint16_t*)gate->scales;
        r.qs2 = (const int8_t*)up->data;
        r.d2 = (const uint16_t*)up->scales;
        r.N = d.n_ff;
        r.K = d.n_embd;
        r.bounds = p.r.bounds;
        r.tile_off = p.r.tile_a;
        r.tile_tab = p.r.tile_tab;
        r.n_seg = d.E;
        r.m_tiles_max = (int32_t)m_tiles_bound(n, d.E, bm);
        r.A = (const uint16_t*)x;
        r.lda = d.n_embd;
        r.a_rows = p.r.ids_src1;
        r.out = p.h;
        r.ldo = d.n_ff;
        r.w_once = n <= (int64_t)d.E * bm;   // at most one M tile per expert on average
        if (shared) {
            GemmProblem& q = g.p[1];
            q.qs1 = (const int8_t*)sh_gate->data;
            q.d1 = (const uint16_t*)sh_gate->scales;
            q.qs2 = (const int8_t*)sh_up->data;
            q.d2 = (const uint16_t*)sh_up->scales;
            q.N = d.n_ff_sh;
            q.K = d.n_embd;
            q.n_seg = d.S;
            q.seg_len = (int32_t)d.T;
            q.m_tiles_max = (int32_t)(d.S * ((d.T + bm - 1) / bm));
            q.A = (const uint16_t*)x;
            q.lda = d.n_embd;
            q.a_row_mod = (int32_t)d.T;
            q.out = p.hsh;
            q.ldo = d.n_ff_sh;
            q.w_once = d.T <= bm;
        }

        GemmArgs g2{};
        g2.mode = 0;
        g2.fmt = g.fmt;
        g2.n_prob = shared ? 2 : 1;
        GemmProblem& r2 = g2.p[0];
        r2.qs1 = (const int8_t*)down->data;
        r2.d1 = (const uint16_t*)down->scales;
        r2.N = d.n_embd;
        r2.K = d.n_ff;
        r2.bounds = p.r.bounds;
        r2.tile_off = p.r.tile_a;
        r2.tile_tab = p.r.tile_tab;
        r2.n_seg = d.E;
        r2.m_tiles_max = r.m_tiles_max;
        r2.A = (const uint16_t*)p.h;
        r2.lda = d.n_ff;
        r2.out = p.y;
        r2.ldo = d.n_embd;
        r2.out_rows = p.r.ids_dst;
        r2.w_once = r.w_once;
        if (shared) {
            GemmProblem& q = g2.p[1];
            q.qs1 = (const int8_t*)sh_down->data;
            q.d1 = (const uint16_t*)sh_down->scales;
            q.N = d.n_embd;
            q.K = d.n_ff_sh;
            q.n_seg = d.S;
            q.seg_len = (int32_t)d.T;
            q.m_tiles_max = g.p[1].m_tiles_max;
            q.A = (const uint16_t*)p.hsh;
            q.lda = d.n_ff_sh;
            q.out = p.ysh;
            q.ldo = d.n_embd;
            q.w_once = d.T <= bm;
        }
        // segment-last tiles of up to 160 rows where both GEMMs (and the shared ones they
        // launch with) run the wide kernel: the two share the row-id pass's tile table
        // MXFP4: every scale tensor at an even address; IQ4_NL: 4-byte, IQ4_XS: 8-byte aligned
        const uintptr_t smask = g.fmt == 3 ? 7 : (g.fmt == 2 ? 3 : 1);
        bool even = true;
        for (const moe_weights* w : {gate, up, down, sh_gate, sh_up, sh_down})
            if (w && ((uintptr_t)w->scales & smask)) even = false;
        int tx = gemm_tile_x(p.msub, g.fmt, d.n_embd, even);
        if (gemm_tile_x(p.msub, g.fmt, d.n_ff, even) == 0 ||
            (shared && gemm_tile_x(p.msub, g.fmt, d.n_ff_sh, even) == 0))
            tx = 0;
        if (tx) {
            gemm_set_tall(r, ra, 0);
            gemm_set_tall(r2, ra, 0);
        }
        // x is gathered through the row map; h and the shared rows are read in order
        if ((s = check_gemm_limits(g, p.msub, d.T, d.n_embd, "gate/up"))) return s;
        if ((s = check_gemm_limits(g2, p.msub, 0, d.n_ff, "down"))) return s;

        tm.begin();
        if ((s = hip_check(launch_row_ids(ra, st, nullptr), "row ids"))) return s;
        tm.end();
        tm.begin();
        if ((s = hip_check(launch_gemm_q8(g, p.msub, st), "gate/up grouped GEMM"))) return s;
        tm.end();
        tm.begin();
        if ((s = hip_check(launch_gemm_q8(g2, p.msub, st), "down grouped GEMM"))) return s;
        tm.end();
    } else {
        DecArgs a{};
        a.ids = ids;
        a.T = (int32_t)d.T;
        a.k = d.k;
        a.E = d.E;
        const int32_t fmt = d.fmt;
        a.rw = DecWeights{(const int8_t*)gate->data, (const uint16_t*)gate->scales,
                          (const int8_t*)up->data, (const uint16_t*)up->scales, d.E, d.n_ff, d.n_embd, fmt};
        if (shared)
            a.sw = DecWeights{(const int8_t*)sh_gate->data, (const uint16_t*)sh_gate->scales,
                              (const int8_t*)sh_up->data, (const uint16_t*)sh_up->scales, d.S,
                              d.n_ff_sh, d.n_embd, fmt};
        a.act = x;
        a.act_type = 1;
        a.act_B = 1;
        a.sact = x;
        a.sact_type = 1;
        a.sact_jstride = 0;
        a.out = (float*)p.h;
        a.sout = (float*)p.hsh;
        a.mode = 1;
        a.d_max = (int32_t)(n < d.E ? n : d.E);
        a.rows_per_block = 32;
        tm.begin();
        if ((s = hip_check(launch_decode(a, st), "gate/up GEMV"))) return s;
        tm.end();

        DecArgs b{};
        b.ids = ids;
        b.T = (int32_t)d.T;
        b.k = d.k;
        b.E = d.E;
        b.rw = DecWeights{(const int8_t*)down->data, (const uint16_t*)down->scales, nullptr, nullptr,
                          d.E, d.n_embd, d.n_ff, fmt};
        if (shared)
            b.sw = DecWeights{(const int8_t*)sh_down->data, (const uint16_t*)sh_down->scales, nullptr,
                              nullptr, d.S, d.n_embd, d.n_ff_sh, fmt};
        b.act = p.h;
        b.act_type = 0;
        b.act_B = d.k;
        b.sact = p.hsh;
        b.sact_type = 0;
        b.sact_jstride = d.T;
        b.out = (float*)p.y;
        b.sout = (float*)p.ysh;
        b.mode = 0;
        b.d_max = a.d_max;
        b.rows_per_block = 32;
        b.route_w = route_w;
        b.out_tok = out;
        tm.begin();
        if ((s = hip_check(launch_decode(b, st, &reduced), "down GEMV"))) return s;
        tm.end();
    }
    if (reduced) {   // the down GEMV wrote out itself
        g_stages = tm.stage;
        return MOE_OK;
    }
    ReduceArgs rd{};
    rd.ids = ids;
    rd.route_w = route_w;
    rd.T = (int32_t)d.T;
    rd.k = d.k;
    rd.E = d.E;
    rd.N = d.n_embd;
    rd.y = (const float*)p.y;
    rd.ysh = (const float*)p.ysh;
    rd.S = d.S;
    rd.out = out;
    rd.mode = 0;
    tm.begin();
    if ((s = hip_check(launch_reduce(rd, st), "reduce"))) return s;
    tm.end();
    g_stages = tm.stage;
    return MOE_OK;
}

size_t moe_mul_mat_id_workspace_size(const moe_weights* w, moe_dtype src1_type,
                                     int32_t src1_rows_per_token, int64_t n_tokens,
                                     int32_t n_used, const moe_options* opt) {
    if (validate_mmid(w, src1_type, src1_rows_per_token, n_tokens, n_used)) return 0;
    if (is_elem(w->type)) {   // the weighted call's, which is the larger
        const int path = elem_path(n_tokens, n_used, (int32_t)w->n_mat, w->cols, w->type, opt);
        if (path < 0) return 0;
        Carve c(nullptr);
        carve_elem(c, w, n_tokens, n_used, src1_rows_per_token, true, path);
        return c.off;
    }
    const bool q8 = w->type != MOE_F32;   // quantized experts
    if (!q8 && opt && ((opt->path != 0 && opt->path != 1) || opt->act_quant)) return 0;
    const int path = q8 ? select_path_aq(n_tokens, n_used, (int32_t)w->n_mat, w->cols, w->type, opt, 0, w->cols) : 1;
    if (path < 0) return 0;
    // the weighted and unweighted calls use the same plan size when weighted
    Carve c(nullptr);
    carve_mmid(c, n_tokens, n_used, (int32_t)w->n_mat, w->rows, true, q8, path, src1_rows_per_token,
               w->cols);
    return c.off;
}

moe_status moe_mul_mat_id(const moe_weights* w, const void* src1, moe_dtype src1_type,
                          int32_t src1_rows_per_token, const int32_t* ids, int64_t n_tokens,
                          int32_t n_used, const float* route_w, float* dst, const moe_options* opt,
                          void* ws, size_t ws_bytes, void* stream) {
    g_err.clear();
    moe_status s = validate_mmid(w, src1_type, src1_rows_per_token, n_tokens, n_used);
    if (s) return s;
    if (n_tokens == 0) {
        g_stages = 0;
        return MOE_OK;
    }
    if (!src1 || !ids || !dst) return fail(MOE_EINVAL, "NULL pointer argument");
    const bool q8 = w->type != MOE_F32;   // quantized experts
    const int32_t E = (int32_t)w->n_mat, N = (int32_t)w->rows, K = (int32_t)w->cols;
    const int32_t B = src1_rows_per_token, k = n_used;
    if (is_elem(w->type))
        return mul_mat_id_elem(w, src1, src1_type, B, ids, n_tokens, k, route_w, dst, opt, ws, ws_bytes, (hipStream_t)stream);
    if (!q8 && opt && opt->path != 0 && opt->path != 1)
        return fail(MOE_EINVAL, "float32 experts run the grouped fp32 product only: options.path "
                    "must be 0 or 1 (got %d)", opt->path);
    if (!q8 && opt && opt->act_quant)
        return fail(MOE_EINVAL, "quantized activations (act_quant = 1) need Q8_0 experts");
    if (!q8 && n_tokens * k * (int64_t)N >= k4GiB - 256)
        return fail(MOE_ELIMIT, "float32 mul_mat_id: n_tokens * n_used * N must be under 2^32");
    const int path = q8 ? select_path_aq(n_tokens, k, E, K, w->type, opt, 0, K) : 1;
    if (path < 0) return (moe_status)path;
    const bool weighted = route_w != nullptr;
    Carve sz(nullptr);
    carve_mmid(sz, n_tokens, k, E, N, weighted, q8, path, B, K);
    if (sz.off > ws_bytes || (sz.off && !ws)) return fail(MOE_EWORKSPACE, "workspace needs %zu bytes", sz.off);
    if ((path == 4 || path == 5) && (s = check_fp4_act(ws, "the workspace"))) return s;
    Carve c(ws);
    const MmidPlan p = carve_mmid(c, n_tokens, k, E, N, weighted, q8, path, B, K);
    const hipStream_t st = (hipStream_t)stream;
    Timer tm(opt, st);
    const int64_t n = n_tokens * k;
    float* slot_out = weighted ? (float*)p.y : dst;  // per-slot rows [T*k][N]

    if (path == 3) {
        // quantized activations: row ids, src1 -> codes, int8 grouped GEMM, then the
        // reduce / zero fix-up below
        const int bm = kQ8aTileM;
        RowIdsArgs ra = row_ids_args(ids, n, k, E, B, p.r);
        ra.tile_off[0] = p.r.tile_a;
        ra.tile_m[0] = bm;
        ra.tile_tab[0] = p.r.tile_tab;
        ra.tile_cap[0] = p.r.tile_cap;
        QuantArgs qa{};
        qa.src_bf16 = 1;
        qa.n_part = 1;
        qa.part[0] = qpart(src1, n_tokens * B, K, p.aq, p.ad);
        GemmArgs g{};
        g.mode = 0;
        g.n_prob = 1;
        GemmProblem& r = g.p[0];
        r.qs1 = (const int8_t*)w->data;
        r.d1 = (const uint16_t*)w->scales;
        r.N = N;
        r.K = K;
        r.bounds = p.r.bounds;
        r.tile_off = p.r.tile_a;
        r.tile_tab = p.r.tile_tab;
        r.n_seg = E;
        r.m_tiles_max = (int32_t)m_tiles_bound(n, E, bm);
        r.Aq = p.aq;
        r.Ad = p.ad;
        r.a_rows = p.r.ids_src1;
        r.out = slot_out;
        r.ldo = N;
        r.out_rows = p.r.ids_dst;
        if ((uintptr_t)src1 % 16) return fail(MOE_EINVAL, "quantized activations: src1 must be 16-byte aligned");
        if ((s = check_q8a_limits(g, n_tokens * B, K, "mul_mat_id"))) return s;
        if (n_tokens * B * (K / 32) >= k4GiB) return fail(MOE_ELIMIT, "mul_mat_id: too many activation blocks");
        tm.begin();
        if ((s = hip_check(launch_row_ids(ra, st, nullptr), "row ids"))) return s;
        tm.end();
        tm.begin();
        if ((s = hip_check(launch_quant_act(qa, st), "quantize src1"))) return s;
        tm.end();
        tm.begin();
        if ((s = hip_check(launch_gemm_q8a(g, st), "grouped GEMM (int8)"))) return s;
        tm.end();
    } else if (path == 4) {
        if ((s = mmid_fp4(p, w, src1, B, ids, n_tokens, k, slot_out, weighted, tm, st))) return s;
    } else if (path == 5) {
        if ((s = mmid_dec_fp4(p, w, src1, B, ids, n_tokens, k, route_w, slot_out, dst, tm, st))) return s;
    } else if (!q8 || path == 1) {
        const int bm = gemm_tile_m(p.msub);
        RowIdsArgs ra = row_ids_args(ids, n, k, E, B, p.r);
        GemmArgs g{};
        if (q8) {
            ra.tile_off[0] = p.r.tile_a;
            ra.tile_m[0] = bm;
            ra.tile_tab[0] = p.r.tile_tab;
            ra.tile_cap[0] = p.r.tile_cap;
            g.mode = 0;
            g.fmt = kernel_fmt(w->type);
            g.n_prob = 1;
            GemmProblem& r = g.p[0];
            r.qs1 = (const int8_t*)w->data;
            r.d1 = (const uint16_t*)w->scales;
            r.N = N;
            r.K = K;
            r.bounds = p.r.bounds;
            r.tile_off = p.r.tile_a;
            r.tile_tab = p.r.tile_tab;
            r.n_seg = E;
            r.m_tiles_max = (int32_t)m_tiles_bound(n, E, bm);
            r.A = (const uint16_t*)src1;
            r.lda = K;
            r.a_rows = p.r.ids_src1;
            r.out = slot_out;
            r.ldo = N;
            r.out_rows = p.r.ids_dst;
            r.w_once = n <= (int64_t)E * bm;   // at most one M tile per expert on average
            if (gemm_tile_x(p.msub, g.fmt, K, ((uintptr_t)w->scales & (g.fmt == 3 ? 7 : (g.fmt == 2 ? 3 : 1))) == 0))
                gemm_set_tall(r, ra, 0);
            if ((s = check_gemm_limits(g, p.msub, n_tokens * B, K, "mul_mat_id"))) return s;
        }
        tm.begin();
        if ((s = hip_check(launch_row_ids(ra, st, nullptr), "row ids"))) return s;
        tm.end();
        if (q8) {
            tm.begin();
            if ((s = hip_check(launch_gemm_q8(g, p.msub, st), "grouped GEMM"))) return s;
            tm.end();
        } else {
            GemmF32Args gf{};
            gf.W = (const float*)w->data;
            gf.A = (const float*)src1;
            gf.ids = ids;
            gf.ids_src1 = p.r.ids_src1;
            gf.ids_dst = p.r.ids_dst;
            gf.bounds = p.r.bounds;
            gf.n_slots = n;
            gf.E = E;
            gf.N = N;
            gf.K = K;
            gf.out = slot_out;
            tm.begin();
            if ((s = hip_check(launch_gemm_f32(gf, st), "fp32 grouped matmul"))) return s;
            tm.end();
        }
    } else {
        DecArgs a{};
        a.ids = ids;
        a.T = (int32_t)n_tokens;
        a.k = k;
        a.E = E;
        a.rw = DecWeights{(const int8_t*)w->data, (const uint16_t*)w->scales, nullptr, nullptr, E, N, K,
                          kernel_fmt(w->type)};
        a.act = src1;
        a.act_type = 1;
        a.act_B = B;
        a.out = slot_out;
        a.mode = 0;
        a.d_max = (int32_t)(n < E ? n : E);
        a.rows_per_block = 32;
        if (weighted) {
            a.route_w = route_w;
            a.out_tok = dst;
        }
        bool reduced = false;
        tm.begin();
        if ((s = hip_check(launch_decode(a, st, &reduced), "GEMV"))) return s;
        tm.end();
        if (reduced) {   // the GEMV wrote the weighted sum itself
            g_stages = tm.stage;
            return MOE_OK;
        }
    }
    if ((path == 4 || path == 5) && (p.fuse || !weighted)) {   // written in full, rows of invalid slots too
        g_stages = tm.stage;
        return MOE_OK;
    }
    ReduceArgs rd{};
    rd.ids = ids;
    rd.route_w = route_w;
    rd.T = (int32_t)n_tokens;
    rd.k = k;
    rd.E = E;
    rd.N = N;
    rd.y = slot_out;
    rd.out = dst;
    rd.mode = weighted ? 0 : 1;
    tm.begin();
    if ((s = hip_check(launch_reduce(rd, st), weighted ? "reduce" : "zero invalid slots"))) return s;
    tm.end();
    g_stages = tm.stage;
    return MOE_OK;
}

size_t moe_mul_mat_id_backward_workspace_size(const moe_weights* w, moe_dtype d_dst_type,
                                              int32_t src1_rows_per_token, int64_t n_tokens,
                                              int32_t n_used, int32_t weighted, int32_t want,
                                              const moe_options* opt) {
    if (!w || validate_grad(w, w->type, d_dst_type, src1_rows_per_token, n_tokens, n_used, weighted != 0, want, opt))
        return 0;
    Carve c(nullptr);   // room for a copy of d_dst also where its address alone asks for one, and for a float32 d_w
    carve_grad(c, w, n_tokens, n_used, src1_rows_per_token, weighted != 0, want, false, true);
    return c.off;
}

moe_status moe_mul_mat_id_backward(const moe_weights* w, const void* src1, moe_dtype src1_type,
                                   int32_t src1_rows_per_token, const int32_t* ids,
                                   int64_t n_tokens, int32_t n_used, const float* route_w,
                                   const void* d_dst, moe_dtype d_dst_type, void* d_src1, void* d_w,
                                   moe_dtype d_w_type, float* d_route_w, const moe_options* opt,
                                   void* ws, size_t ws_bytes, void* stream) {
    g_err.clear();
    moe_status s;
    const int want = (d_src1 ? kWantX : 0) | (d_w ? kWantW : 0) | (d_route_w ? kWantR : 0);
    const bool weighted = route_w != nullptr;
    const int32_t B = src1_rows_per_token, k = n_used;
    const int64_t T = n_tokens, n = T * (int64_t)k;
    if ((s = validate_grad(w, src1_type, d_dst_type, B, T, k, weighted, want, opt))) return s;
    if (d_w && d_w_type != w->type && d_w_type != MOE_F32)
        return fail(MOE_EINVAL, "d_w must be of the experts' type (%s) or F32", type_name(w->type));
    if (T == 0 && !d_w) {
        g_stages = 0;
        return MOE_OK;
    }
    if (T > 0 && (!src1 || !ids || !d_dst)) return fail(MOE_EINVAL, "NULL pointer argument");
    if ((s = check_aligned(src1, "src1")) || (s = check_aligned(d_src1, "d_src1")) || (s = check_aligned(d_w, "d_w")))
        return s;
    if (T > 0 && ((d_src1 && (d_src1 == src1 || d_src1 == d_dst || d_src1 == d_w || d_src1 == w->data)) ||
                  (d_w && (d_w == w->data || d_w == src1 || d_w == d_dst))))   // they are read again after the first writes
        return fail(MOE_EINVAL, "d_src1 and d_w must not be one of the inputs or each other");
    const int32_t E = (int32_t)w->n_mat;
    const bool as_is = d_dst_type == w->type && w->rows % 8 == 0 && (uintptr_t)d_dst % 16 == 0;
    Carve sz(nullptr);
    carve_grad(sz, w, T, k, B, weighted, want, as_is, d_w_type == MOE_F32);
    if (sz.off > ws_bytes || !ws) return fail(MOE_EWORKSPACE, "workspace needs %zu bytes", sz.off);
    if ((s = check_aligned(ws, "the workspace"))) return s;
    const int64_t stack = (int64_t)((uint64_t)w->n_mat * w->rows * w->cols), slots4 = n * 4, src_bytes = T * B * w->cols * 2;
    const Span in[] = {{src1, src_bytes}, {w->data, 2 * stack}, {ids, slots4}, {route_w, slots4},
                       {d_dst, (weighted ? T : n) * w->rows * (d_dst_type == MOE_F32 ? 4 : 2)}};
    const Span out[] = {{d_src1, src_bytes}, {d_w, stack * (d_w_type == MOE_F32 ? 4 : 2)}, {d_route_w, slots4}};
    for (const Span& o : out) {
        for (const Span& i : in)
            if (overlap(o, i)) return fail(MOE_EINVAL, "outputs must not overlap inputs");
        for (const Span& other : out)
            if (&o != &other && overlap(o, other)) return fail(MOE_EINVAL, "outputs must not overlap each other");
    }
    Carve c(ws);
    const GradPlan p = carve_grad(c, w, T, k, B, weighted, want, as_is, d_w_type == MOE_F32);
    const hipStream_t st = (hipStream_t)stream;
    const void* dy = as_is ? d_dst : p.dy;
    // positions' tokens (ids_src1 of one row a token) and slots (ids_dst)
    RowIdsArgs ra = row_ids_args(ids, n, k, E, 1, p.r);
    elem_tiles(ra, p.r, p.tile_m);
    ExpertGemm g = elem_gemm(w, p.r, p.tile_m, n);
    g.A = dy;
    g.lda = p.ld;
    g.a_rows = weighted ? p.r.ids_src1 : p.r.ids_dst;
    g.out16 = p.direct;
    g.out = p.direct ? d_src1 : (void*)p.g;
    g.out_rows = p.r.ids_dst;
    g.row_w = p.direct ? route_w : nullptr;
    g.dots = p.dots;
    g.dot_parts = p.dot_parts;
    g.x = src1;
    ExpertGradW gw{};
    gw.type = g.type;
    gw.N = g.N;
    gw.K = g.K;
    gw.E = E;
    gw.dY = weighted ? p.scaled : dy;
    gw.ldy = (int32_t)p.ld;
    gw.terms = p.terms;
    gw.term_stride = n * p.ld;
    const bool scale = p.tops && n > 0;
    float* unscale = scale ? p.tops + kGradTops : nullptr;
    gw.unscale = unscale;
    gw.X = src1;
    gw.dy_rows = p.r.ids_dst;
    gw.x_rows = B == 1 ? p.r.ids_src1 : p.r.ids_dst;
    gw.bounds = p.r.bounds;
    gw.dW = d_w;
    gw.f32 = d_w_type == MOE_F32;
    gw.splits = p.splits;
    gw.parts = p.parts;
    const bool rows_wanted = (want & (kWantX | kWantR)) && n > 0;
    const bool both = rows_wanted && d_w && expert_grads_share(g);
    const int64_t x_grid = rows_wanted ? expert_gemm_grid(g, 1) : 0, w_grid = d_w ? expert_grad_w_grid(gw) * p.splits : 0;
    if ((s = check_grid(both ? x_grid + w_grid : x_grid > w_grid ? x_grid : w_grid, "gradients"))) return s;
    Timer tm(opt, st);
    BesideRowIds beside{};   // direct rows of invalid slots: 16-bit rows of K columns are rows of K / 2 words
    if (d_src1 && n > 0 && p.direct) beside.zero = ZeroSlots{ids, (float*)d_src1, n, E, g.K / 2};
    if ((p.dy || p.scaled) && n > 0) beside.grad = GradInArgs{d_dst, d_dst_type == MOE_F32, g.type, weighted ? T : n,
                                                              w->rows, p.ld, p.dy, route_w, k, p.scaled, p.terms,
                                                              scale ? p.tops : nullptr, grad_tops(T), unscale};
    if (scale) {
        const GradTopArgs top{d_dst, d_dst_type == MOE_F32, T, w->rows, route_w, ids, k, E, p.tops};
        tm.begin();
        if ((s = hip_check(launch_grad_top(top, st), "largest scaled gradient"))) return s;
        tm.end();
    }
    tm.begin();
    if ((s = hip_check(launch_row_ids(ra, st, nullptr, &beside), "row ids"))) return s;
    tm.end();
    if (rows_wanted) {
        tm.begin();
        if ((s = hip_check(both ? launch_expert_grads(g, gw, st) : launch_expert_grad_x(g, st), "row gradients"))) return s;
        tm.end();
        if (p.dots) {
            const JoinDotsArgs jd{p.dots, ids, n, p.dot_parts, E, d_route_w};
            tm.begin();
            if ((s = hip_check(launch_join_dots(jd, st), "join d_route_w"))) return s;
            tm.end();
        }
        if (!p.direct) {
            GradRowsArgs j{};
            j.type = g.type;
            j.g = p.g;
            j.ids = ids;
            j.route_w = route_w;
            j.x = src1;
            j.rows = T;   // B = 1
            j.k = k;
            j.E = E;
            j.K = g.K;
            j.d_x = d_src1;
            j.d_route_w = d_route_w;
            tm.begin();
            if ((s = hip_check(launch_grad_rows(j, st), "join the slots' gradients"))) return s;
            tm.end();
        }
    }
    if (d_w) {
        if (!both) {
            tm.begin();
            if ((s = hip_check(launch_expert_grad_w(gw, st), "experts' gradient"))) return s;
            tm.end();
        }
        if (p.splits > 1) {
            tm.begin();
            if ((s = hip_check(launch_join_w(gw, st), "join the experts' gradient"))) return s;
            tm.end();
        }
    }
    g_stages = tm.stage;
    return MOE_OK;
}

moe_status moe_quantize_rows(const void* x, moe_dtype x_type, int64_t rows, int64_t K, int8_t* q,
                             float* d, void* stream) {
    g_err.clear();
    if (x_type != MOE_BF16 && x_type != MOE_F16 && x_type != MOE_F32)
        return fail(MOE_EINVAL, "x must be BF16, F16 or F32");
    if (rows < 0 || K <= 0) return fail(MOE_EINVAL, "rows must be >= 0 and K > 0");
    if (rows == 0) return MOE_OK;
    if (!x || !q || !d) return fail(MOE_EINVAL, "NULL pointer argument");
    if ((uintptr_t)x % (x_type == MOE_F32 ? 4 : 2) || (uintptr_t)d % 4)
        return fail(MOE_EINVAL, "x and d must be aligned to their elements");
    int64_t n, bytes;
    if (__builtin_mul_overflow(rows, K, &n) || __builtin_mul_overflow(n, 4, &bytes))
        return fail(MOE_ELIMIT, "rows * K must be under 2^61");
    const Span xs{x, x_type == MOE_F32 ? bytes : bytes / 2}, qs{q, n}, ds{d, rows * 4};
    if (overlap(xs, qs) || overlap(xs, ds) || overlap(qs, ds)) return fail(MOE_EINVAL, "x, q and d must not overlap");
    const QuantRowsArgs a{x, elem_of(x_type), rows, K, q, d};
    return hip_check(launch_quant_rows(a, (hipStream_t)stream), "quantize rows");
}

moe_status moe_quantize_act(const void* x, moe_dtype x_type, int64_t rows, int64_t K, int8_t* q,
                            float* d, void* stream) {
    g_err.clear();
    if (x_type != MOE_BF16 && x_type != MOE_F32) return fail(MOE_EINVAL, "x must be BF16 or F32");
    if (rows < 0 || K <= 0) return fail(MOE_EINVAL, "rows must be >= 0 and K > 0");
    if (K % 32) return fail(MOE_ELIMIT, "K must be a multiple of 32 (got %lld)", (long long)K);
    if (rows > 0 && (!x || !q || !d)) return fail(MOE_EINVAL, "NULL pointer argument");
    if (((uintptr_t)x | (uintptr_t)q) % 16 || (uintptr_t)d % 4)
        return fail(MOE_EINVAL, "x and q must be 16-byte aligned, d 4-byte aligned");
    if (rows > 0 && rows * (K / 32) >= k4GiB - 256)
        return fail(MOE_ELIMIT, "rows * K / 32 must be under 2^32");
    QuantArgs a{};
    a.n_part = 1;
    a.src_bf16 = x_type == MOE_BF16;
    a.part[0] = qpart(x, rows, K, q, d);
    return hip_check(launch_quant_act(a, (hipStream_t)stream), "quantize activations");
}

moe_status moe_quantize_mxfp4(const void* x, moe_dtype x_type, int64_t rows, int64_t K,
                              uint8_t* codes, uint8_t* scales, void* values, void* stream) {
    g_err.clear();
    if (x_type != MOE_BF16 && x_type != MOE_F32) return fail(MOE_EINVAL, "x must be BF16 or F32");
    if (rows < 0 || K <= 0) return fail(MOE_EINVAL, "rows must be >= 0 and K > 0");
    if (K % 32) return fail(MOE_ELIMIT, "K must be a multiple of 32 (got %lld)", (long long)K);
    if (rows == 0) return MOE_OK;
    if (!x || !codes || !scales) return fail(MOE_EINVAL, "NULL pointer argument");
    if (((uintptr_t)x | (uintptr_t)codes | (uintptr_t)values) % 16)
        return fail(MOE_EINVAL, "x, codes and values must be 16-byte aligned");
    if (rows >= kFp4MaxBlocks || K / 32 >= kFp4MaxBlocks || rows * (K / 32) >= kFp4MaxBlocks)
        return fail(MOE_ELIMIT, "rows * K / 32 must be under 2^31");
    QuantFp4Args a{};
    a.src = x;
    a.rows = rows;
    a.K = K;
    a.q = codes;
    a.s = scales;
    a.values = values;
    a.src_bf16 = x_type == MOE_BF16;
    return hip_check(launch_quant_mxfp4(a, (hipStream_t)stream), "quantize to MXFP4");
}

moe_status moe_router_scored(const void* logits, moe_dtype logits_type, const float* bias,
                             int64_t n_tokens, int32_t n_experts, int32_t n_used,
                             const moe_router_config* cfg, int32_t* ids, float* route_w,
                             float* scores, void* stream) {
    moe_status s;
    g_err.clear();
    if (logits_type != MOE_F32 && logits_type != MOE_BF16) return fail(MOE_EINVAL, "logits must be F32 or BF16");
    if ((s = check_router(cfg, n_tokens, n_experts, n_used, true))) return s;
    if (n_tokens > 0 && (!logits || !ids || !route_w)) return fail(MOE_EINVAL, "NULL pointer argument");
    if (scores && (const void*)scores == logits)   // logits are read again after the scores
        return fail(MOE_EINVAL, "scores must not be logits");
    RouterScoredArgs a{};
    a.logits = logits;
    a.bf16 = logits_type == MOE_BF16;
    a.bias = bias;
    a.T = n_tokens;
    a.E = n_experts;
    a.k = n_used;
    a.sigmoid = cfg->score == MOE_SCORE_SIGMOID;
    a.n_group = cfg->n_group;
    a.topk_group = cfg->topk_group;
    a.group_top = cfg->group_top;
    a.renorm = cfg->renorm;
    a.scale = cfg->scale;
    a.ids = ids;
    a.w = route_w;
    a.scores = scores;
    return hip_check(launch_router_scored(a, (hipStream_t)stream), "scored router");
}

moe_status moe_router_scored_backward(const void* logits, moe_dtype logits_type, const int32_t* ids,
                                      const float* d_route_w, const float* d_scores,
                                      int64_t d_scores_stride, int64_t n_tokens, int32_t n_experts,
                                      int32_t n_used, const moe_router_config* cfg, void* d_logits,
                                      void* stream) {
    moe_status s;
    g_err.clear();
    if (logits_type != MOE_F32 && logits_type != MOE_BF16) return fail(MOE_EINVAL, "logits must be F32 or BF16");
    if ((s = check_router(cfg, n_tokens, n_experts, n_used, false))) return s;
    if (d_scores && d_scores_stride != 0 && d_scores_stride < n_experts)
        return fail(MOE_EINVAL, "d_scores_stride must be 0 or at least n_experts (got %lld)",
                    (long long)d_scores_stride);
    if (n_tokens > 0 && (!logits || !ids || !d_route_w || !d_logits)) return fail(MOE_EINVAL, "NULL pointer argument");
    RouterGradArgs a{};
    a.logits = logits;
    a.bf16 = logits_type == MOE_BF16;
    a.ids = ids;
    a.dw = d_route_w;
    a.ds = d_scores;
    a.ds_stride = d_scores_stride;
    a.T = n_tokens;
    a.E = n_experts;
    a.k = n_used;
    a.sigmoid = cfg->score == MOE_SCORE_SIGMOID;
    a.renorm = cfg->renorm;
    a.scale = cfg->scale;
    a.dl = d_logits;
    return hip_check(launch_router_grad(a, (hipStream_t)stream), "scored router gradient");
}

moe_status moe_router_topk(const float* logits, int64_t n_tokens, int32_t n_experts, int32_t n_used,
                           int32_t* ids, float* route_w, void* stream) {
    moe_status s;
    g_err.clear();
    if ((s = check_tokens(n_tokens, n_used))) return s;
    if ((s = check_experts(n_experts))) return s;
    if (n_used > n_experts)
        return fail(MOE_EINVAL, "n_used (%d) must not exceed n_experts (%d) for top-k", n_used, n_experts);
    if (n_tokens > 0 && (!logits || !ids || !route_w)) return fail(MOE_EINVAL, "NULL pointer argument");
    RouterArgs a{};
    a.logits = logits;
    a.T = n_tokens;
    a.E = n_experts;
    a.k = n_used;
    a.ids = ids;
    a.w = route_w;
    return hip_check(launch_router(a, (hipStream_t)stream), "router top-k");
}

}  // extern "C"
