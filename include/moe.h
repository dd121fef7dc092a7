/*
 * moe.h -- C ABI of libmoe, the MI355X (gfx950) Mixture-of-Experts indirect
 * matrix multiplication (mul_mat_id) library.
 *
 * The operation. mul_mat_id takes stacked expert weights, activations and an
 * integer ids table; every token is multiplied only by the weight matrices of the
 * experts its ids row names ("CUDA: better MoE implementation", the ik_llama.cpp
 * PR #283 write-up, section 1.2). The deterministic fast path first turns ids into
 * three maps -- the src1 rows reordered so each expert's rows are contiguous, the
 * same reordering for dst, and each expert's bounds in that order -- and then
 * reorders and reduces by those maps with no atomic slot counters (same page,
 * sections 2 and 2.1; summary in section 6). The fused MoE FFN adds gate/up with
 * SiLU(gate) * up (section 4.2 names the fused up/gate forward) and always-on
 * shared experts computed in the same operation ("CUDA: fuse shared experts into
 * MMVQ", llama.cpp release b11370: fused shared experts, optional buffers checked
 * for null).
 *
 * Layouts (row-major, last index contiguous):
 *   weights  W[n_mat][rows][cols]; Q8_0: int8 qs[n_mat][rows][cols] plus fp16
 *            scales d[n_mat][rows][cols/32], value = d * q (32 values per scale).
 *            MXFP4 (the format the TensorSharp page lists for GPT-OSS 20B experts;
 *            defined by the OCP Microscaling v1.0 specification): uint8
 *            codes[n_mat][rows][cols/2], two FP4 E2M1 codes per byte, column 2i in
 *            bits 0-3 and column 2i+1 in bits 4-7, plus uint8 E8M0 scales
 *            x[n_mat][rows][cols/32], value = e2m1(code) * 2^(x - 127) (x = 255: NaN).
 *            IQ4_NL (the 4-bit codes of the IQ-series types the pages name: IQ2_K_R4
 *            in the PR #283 write-up, section 3.2, UD-IQ4_XS models on the TensorSharp
 *            page; defined by ggml): uint8 codes[n_mat][rows][cols/2] packed as MXFP4's,
 *            plus fp16 scales d[n_mat][rows][cols/32] as Q8_0's, value = d * level(code)
 *            with ggml's 16 IQ4_NL levels (-127 -104 -83 -65 -49 -35 -22 -10 1 13 25
 *            38 53 69 89 113).
 *            IQ4_XS (ggml's super-block form of those codes): codes as IQ4_NL's, plus one
 *            8-byte record per 256 columns, uint8 scales[n_mat][rows][cols/256][8] (8-byte
 *            aligned): fp16 d (bytes 0-1), uint16 scales_h (bytes 2-3), uint8 scales_l[4]
 *            (bytes 4-7); block j (0..7) of the 256 has the 6-bit sub-scale ls = (nibble
 *            j%2 of scales_l[j/2], low nibble first) | ((scales_h >> 2j) & 3) << 4, and
 *            value = d * (ls - 32) * level(code). cols % 256 == 0.
 *            BF16, F16 (moe_mul_mat_id and its gradients): 16-bit values as they are,
 *            cols % 8 == 0, 16-byte aligned. I8 (moe_mul_mat_id; what moe_quantize_rows
 *            makes): int8 q[n_mat][rows][cols] and float32 d[n_mat][rows], value = d * q,
 *            cols % 16 == 0, cols <= 131072, 16-byte aligned.
 *   ids      int32 [n_tokens][n_used]; route_w float32 [n_tokens][n_used].
 *   src1     [n_tokens][B][K] with B = src1_rows_per_token in {1, n_used}:
 *            slot s of token t reads row t*B + (s mod B).
 *   x        [n_tokens][n_embd]; bf16 tensors are raw 16-bit patterns.
 *
 * Ownership and ordering. Every tensor pointer is a caller-owned DEVICE pointer;
 * the library never allocates, frees or keeps one. Structs passed by pointer
 * (moe_weights, moe_options) are read before the call returns, so host memory is
 * never touched after return. Work is enqueued on `stream` (a hipStream_t; NULL =
 * the default stream) and the call returns without synchronising. The workspace
 * `ws` is caller-owned device memory of at least the size the matching
 * *_workspace_size function reports; its contents are undefined on entry and on
 * exit, and two calls in flight at once must not share one.
 *
 * Errors. Arguments are validated before anything is enqueued; on any status other
 * than MOE_OK nothing was enqueued and outputs are untouched (MOE_EHIP: a launch
 * failed; earlier launches of the same call may have run). moe_last_error()
 * returns a thread-local description of the last failure.
 *
 * Determinism. No floating-point or placement atomics are used: for identical
 * inputs, shapes, options and device, outputs are bitwise identical run to run.
 *
 * Ids outside [0, n_experts) are a caller error that does not fault: such an entry
 * joins no expert segment (expert_bounds[n_experts] counts valid entries only),
 * its per-slot output row is zero and it contributes nothing to weighted sums.
 * Duplicate ids within a token are legal; every (token, slot) is its own row.
 *
 * Limits (MOE_ELIMIT): n_tokens < 2^22 and n_used < 2^10 (the bounds the page
 * above quotes for safe 32-bit packing, section 2.1), n_tokens * n_used < 2^31,
 * n_experts <= 1024, Q8_0, MXFP4 and IQ4_NL cols % 32 == 0, IQ4_XS cols % 256 == 0, BF16 and
 * F16 cols % 8 == 0, I8 cols % 16 == 0 and <= 131072. On the grouped GEMM path the
 * activation tensor whose rows are gathered through the row map (moe_ffn_fused: x;
 * moe_mul_mat_id with quantized experts: src1) must be under 4 GiB, and each GEMM or GEMV launch must hold fewer
 * than 2^32 work-items; float32 moe_mul_mat_id needs n_tokens * n_used * N < 2^32.
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_EINVAL = -1,     /* null pointer, bad size, unsupported dtype combination */
    MOE_ELIMIT = -2,     /* a size limit above is exceeded                         */
    MOE_EWORKSPACE = -3, /* ws_bytes smaller than the required workspace           */
    MOE_EHIP = -4        /* a HIP launch failed                                    */
} moe_status;

typedef enum {
    MOE_F32 = 0, MOE_BF16 = 1, MOE_Q8_0 = 2, MOE_MXFP4 = 3, MOE_IQ4_NL = 4, MOE_IQ4_XS = 5,
    MOE_F16 = 6, /* IEEE half: activations, experts, gradients                     */
    MOE_I8 = 7   /* experts: int8 with one float32 scale per output row            */
} moe_dtype;

/* n_mat stacked matrices of rows x cols. */
typedef struct {
    moe_dtype type;     /* MOE_F32, MOE_Q8_0, MOE_MXFP4, MOE_IQ4_NL, MOE_IQ4_XS; */
                        /* moe_mul_mat_id also MOE_BF16, MOE_F16, MOE_I8         */
    const void *data;   /* F32: float[n_mat][rows][cols]; Q8_0: int8 qs[...];    */
                        /* BF16, F16: 16-bit [n_mat][rows][cols]; I8: int8 [...]; */
                        /* MXFP4, IQ4_NL, IQ4_XS: uint8 codes[n_mat][rows][cols/2] */
    const void *scales; /* Q8_0, IQ4_NL: uint16 (fp16) d[n_mat][rows][cols/32];  */
                        /* MXFP4: uint8 E8M0 x[n_mat][rows][cols/32];            */
                        /* IQ4_XS: uint8 records[n_mat][rows][cols/256][8];      */
                        /* I8: float d[n_mat][rows]; F32, BF16, F16: NULL        */
    int64_t n_mat, rows, cols;
} moe_weights;

/* Path selection (the pages' backend picks its quantized grouped path by comparing
 * the token count with a threshold times the expert count, section 2.1):
 * GEMM when n_tokens >= tau * n_experts, else the GEMV (decode) path within the
 * bounds that moe_select_path states.
 * Optional per-kernel timing: when timing_events is non-NULL it points to
 * n_timing_events hipEvent_t handles; the call records events[2i] before and
 * events[2i+1] after its i-th kernel launch on `stream` (while 2i+1 <
 * n_timing_events). Kernel order -- moe_ffn_fused GEMM path: row ids, gate/up
 * grouped GEMM, down grouped GEMM, reduce; GEMV path: gate/up GEMV, down GEMV,
 * reduce, where small batches (the distinct experts plus the shared ones fit two per
 * wave) do the reduce inside the down GEMV and time two kernels only.
 * moe_mul_mat_id GEMM path: row ids, grouped GEMM, fix-up/reduce; GEMV path: GEMV,
 * fix-up/reduce (weighted calls of small batches: the GEMV alone; BF16 and F16 experts: always; I8
 * experts: a quantize kernel before the GEMV for more than one token; the reduce only for single tokens
 * with more than 64 KB of activations as int8. Their GEMM path has no fix-up kernel; I8: a quantize kernel
 * after the row ids from 6 * 2^20 activations on).
 * moe_last_stage_count() tells how many kernels the last call timed. */
typedef struct {
    int32_t path; /* 0 auto, 1 force grouped GEMM, 2 force GEMV (decode)        */
    float tau;    /* <= 0 means the default, 1.0                                 */
    /* 1: quantized activations (the MMQ-style path; Q8_0 experts only): activation
     * rows are quantized (moe_quantize_act's format) and the grouped GEMM runs int8
     * MFMA with per-block scales, for every batch size (path must be 0 or 1). The
     * fused FFN quantizes x before gate/up and h (rounded to bf16) before down.
     * Kernel order for timing: row ids, quantize, grouped GEMM[, quantize h, down
     * grouped GEMM], reduce / fix-up. 0 (default): bf16 activations.
     * 2: MXFP4 activations (MXFP4 experts only): activation rows are quantized to MXFP4
     * (moe_quantize_mxfp4's format) and multiplied with the experts' codes by the block
     * scaled FP4 MFMA, fp32 accumulation. The fused FFN quantizes x before gate/up and the
     * float32 h before down. GEMV path: n_tokens * n_used <= 64, n_tokens * shared experts <=
     * 64, every row at least 128 columns wide; path 0 takes it there while n_tokens * n_used <=
     * 16 * n_experts; tau is not read. The two paths add the same products in different orders. x / src1,
     * the experts' codes and the workspace must be 16-byte aligned (MOE_EINVAL); cols < 2^24,
     * rows < 2^31 - 512, rows of activations * cols / 32 < 2^31 and, on the grouped GEMM,
     * src1's codes under 4 GiB (MOE_ELIMIT). Kernel order for timing: row ids with quantize and fix-up, grouped GEMM[, down
     * grouped GEMM][, reduce]; GEMV path: GEMV[, down GEMV][, reduce], the reduce only in
     * weighted calls too large to sum inside the GEMV. For the FFN of a single token this is
     * slower than bf16 activations (27 against 22 us on 4 experts of 2880 x 2880): every
     * thread block quantizes the row again. */
    int32_t act_quant;
    int32_t reserved[5];
    void *const *timing_events;
    int32_t n_timing_events;
    int32_t reserved2;
} moe_options;

/*
 * moe_row_ids -- the three maps of section 2.1 of the PR #283 write-up.
 *   ids              device int32 [n_tokens][n_used]
 *   ids_src1, ids_dst device int32 [n_tokens * n_used] (written)
 *   expert_bounds    device int32 [n_experts + 1] (written)
 * Position j enumerates experts ascending, and inside an expert its entries by
 * token then slot (a stable counting sort): ids_src1[j] = t*B + (s mod B) is the
 * src1 row entry j reads, ids_dst[j] = t*n_used + s the dst row it writes, and
 * expert e owns [expert_bounds[e], expert_bounds[e+1]). Entries with invalid ids
 * follow position expert_bounds[n_experts], in (t, s) order.
 * n_tokens = 0 is allowed (all bounds 0). Workspace: moe_row_ids_workspace_size.
 */
moe_status moe_row_ids(const int32_t *ids, int64_t n_tokens, int32_t n_used, int32_t n_experts,
                       int32_t src1_rows_per_token, int32_t *ids_src1, int32_t *ids_dst,
                       int32_t *expert_bounds, void *ws, size_t ws_bytes, void *stream);

/*
 * moe_gather_rows -- the src1 rows copied into expert order by the first map of
 * moe_row_ids (section 2.1 of the PR #283 write-up: ids_src1 names the src1 row each
 * position of the expert-grouped buffer reads; section 2 shows the atomic-slot copy
 * k_copy_src1_to_contiguous this replaces): dst[j][:] = src1[ids_src1[j]][:].
 *   src1      device BF16 or F32 [src1_rows][K]
 *   ids_src1  device int32 [n] (moe_row_ids' ids_src1 with n = n_tokens * n_used)
 *   dst       device [n][K] of src1's type (written; a position whose index is outside
 *             [0, src1_rows) gets a zero row)
 * The fused calls never need it (their grouped GEMM gathers the rows into LDS itself);
 * it is for callers that want the expert-contiguous copy. No workspace. n = 0 is a
 * no-op. MOE_ELIMIT: src1_rows >= 2^31 or n >= 2^33.
 */
moe_status moe_gather_rows(const void *src1, moe_dtype src1_type, int64_t src1_rows, int64_t K,
                           const int32_t *ids_src1, int64_t n, void *dst, void *stream);

/*
 * moe_mul_mat_id -- GGML_OP_MUL_MAT_ID (section 1.2 of the PR #283 write-up).
 *   w        n_mat = n_experts, rows = N, cols = K. Supported pairs: (Q8_0 w, BF16
 *            src1), (MXFP4, IQ4_NL or IQ4_XS w, BF16 src1) on the MFMA grouped
 *            GEMM or the GEMV path (the 4-bit types on the GEMV path: n_tokens *
 *            n_used <= 64 and K <= 4096, else the GEMM path is taken, and forcing the
 *            GEMV path is MOE_EINVAL); (F32 w, F32
 *            src1), which has one path, the fp32 grouped product: opt->path must be
 *            0 or 1 (else MOE_EINVAL); (BF16 w, BF16 src1) and (F16 w, F16 src1), products
 *            of the 16-bit values summed in float32; (I8 w; BF16, F16 or F32 src1): each row of
 *            src1 is quantized as moe_quantize_rows does and
 *              row[n] = d_row * d_w[n] * sum over the columns of q_row * q_w[n]
 *            with the sum exact in int32 (rows of src1 with an infinity or a NaN give NaN).
 *            BF16, F16 and I8: src1, w's data and the workspace 16-byte aligned
 *            (MOE_EINVAL), rows and cols < 2^30, opt->act_quant 0. Their GEMV path: n_tokens *
 *            n_used <= 64, I8 also cols <= 16384 (else forcing it is MOE_EINVAL); path 0 takes it
 *            there while n_tokens * n_used <= 4 * n_experts, or 12; tau is not read. The order in
 *            which a row's products are added goes by the path and the call's sizes.
 *   src1     device [n_tokens][B][K], B = src1_rows_per_token in {1, n_used}
 *   ids      device int32 [n_tokens][n_used]
 *   route_w  NULL: dst = float32 [n_tokens][n_used][N], dst[t][s] = W_{ids[t][s]} src1_row;
 *            else device float32 [n_tokens][n_used] and dst = float32 [n_tokens][N],
 *            dst[t] = sum over s ascending of route_w[t][s] * (slot s's row).
 * Outputs are overwritten, never accumulated into. n_tokens = 0 is a no-op.
 */
moe_status moe_mul_mat_id(const moe_weights *w, const void *src1, moe_dtype src1_type,
                          int32_t src1_rows_per_token, const int32_t *ids, int64_t n_tokens,
                          int32_t n_used, const float *route_w, float *dst, const moe_options *opt,
                          void *ws, size_t ws_bytes, void *stream);

/*
 * moe_mul_mat_id_backward -- the gradients of moe_mul_mat_id with BF16 or F16 experts. With slot
 * i = (t, s) of expert e, r = t*B + (s mod B) its src1 row, w_i = route_w[t][s] (1 without
 * route_w) and dy_i = d_dst[t][s] (with route_w: d_dst[t]):
 *   d_src1[r]    = sum over r's slots, ascending, of w_i * g_i,   g_i[k] = sum_n dy_i[n] W_e[n][k]
 *   d_w[e]       = sum over e's slots of w_i * dy_i (outer) src1[r]
 *   d_route_w[i] = sum_k g_i[k] * src1[r][k]   ( = the inner product of d_dst[t] and slot i's row)
 * Slots with invalid ids have no part in any sum: their d_route_w is 0, and with B = n_used their
 * d_src1 rows; experts without slots get a d_w of zeros, also with n_tokens = 0.
 *   w            BF16 or F16, n_mat = n_experts, rows = N, cols = K
 *   src1         device [n_tokens][B][K] of w's type; ids, route_w as in the forward call
 *   d_dst        device [n_tokens][n_used][N], with route_w [n_tokens][N]; of w's type, or F32,
 *                which is rounded once to w's type (but not for d_w with route_w)
 *   d_src1       NULL (not wanted), or device [n_tokens][B][K] of w's type (written, summed in
 *                float32 and rounded once)
 *   d_w          NULL, or device [n_experts][N][K] (written), d_w_type: w's type or F32. With route_w
 *                the rows w_i * dy_i are float32 products (of d_dst as it is given) that are multiplied
 *                as sums of two numbers of w's type, off by at most 2^-15 of them (BF16) or 2^-21
 *                (F16), for an F32 d_w of three, which hold them. F16: times a power of two that
 *                takes the call's largest finite one of a slot with an expert to [2^14, 2^15), which
 *                adds up to 2^-38 of that one. Infinities and NaN stay what they are
 *   d_route_w    NULL, or device float32 [n_tokens][n_used] (written); needs route_w
 * At least one of d_src1, d_w and d_route_w. No output may overlap an input or another output
 * (MOE_EINVAL). w's data, src1, d_src1, d_w and the workspace 16-byte aligned (MOE_EINVAL); rows and cols < 2^30.
 * opt: path must be 0 or 1, act_quant 0; kernel order for timing: [F16, d_w with route_w: the largest
 * product, ]row ids (which also round and scale d_dst's rows)[, rows of g, for small segments with the experts' gradient][, join][, experts' gradient][, join].
 */
moe_status moe_mul_mat_id_backward(const moe_weights *w, const void *src1, moe_dtype src1_type,
                                   int32_t src1_rows_per_token, const int32_t *ids,
                                   int64_t n_tokens, int32_t n_used, const float *route_w,
                                   const void *d_dst, moe_dtype d_dst_type, void *d_src1, void *d_w,
                                   moe_dtype d_w_type, float *d_route_w, const moe_options *opt,
                                   void *ws, size_t ws_bytes, void *stream);

/*
 * moe_ffn_fused -- MoE FFN layer on the indirect matmul: the gate and up projections
 * with the fused up/gate forward SiLU(gate) * up ("CUDA: better MoE implementation",
 * section 4.2), the down projection, and the deterministic reorder and fixed-order
 * reduction of the routed slots (sections 2.1 and 6), plus the always-on shared
 * experts computed in the same operation ("CUDA: fuse shared experts into MMVQ",
 * llama.cpp release b11370; optional, so checked for null):
 *   out[t] = sum_{s ascending, valid} route_w[t][s] * Wd_e (silu(Wg_e x_t) * (Wu_e x_t)),
 *            e = ids[t][s];  then + sum_{j ascending} Sd_j (silu(Sg_j x_t) * (Su_j x_t)).
 *   gate, up  Q8_0 [n_experts][n_ff][n_embd]; down Q8_0 [n_experts][n_embd][n_ff]
 *   sh_gate, sh_up Q8_0 [S][n_ff_sh][n_embd]; sh_down Q8_0 [S][n_embd][n_ff_sh];
 *             or all of them MXFP4, all IQ4_NL or all IQ4_XS (their GEMV path needs n_tokens *
 *             n_used <= 64 and n_embd, n_ff, n_ff_sh <= 4096; larger calls take the
 *             grouped GEMM);
 *             all three NULL (or n_mat == 0) = no shared experts; giving only some of
 *             them is MOE_EINVAL.
 *   x         device BF16 [n_tokens][n_embd]; ids, route_w as above.
 *   out       device float32 [n_tokens][n_embd] (overwritten).
 * silu(z) = z / (1 + exp(-z)). Intermediates: GEMM path -- bf16 weights (Q8_0: d*q
 * rounded to nearest-even; MXFP4: exact; IQ4_NL, IQ4_XS: scale*level rounded to nearest-even), bf16 activations, fp32 accumulate, bf16 SiLU*up, fp32 down
 * results; GEMV path -- weights exact, fp32 accumulate throughout.
 */
moe_status moe_ffn_fused(const moe_weights *gate, const moe_weights *up, const moe_weights *down,
                         const moe_weights *sh_gate, const moe_weights *sh_up,
                         const moe_weights *sh_down, const void *x, moe_dtype x_type,
                         const int32_t *ids, const float *route_w, int64_t n_tokens, int32_t n_used,
                         float *out, const moe_options *opt, void *ws, size_t ws_bytes,
                         void *stream);

/*
 * moe_ffn_fused_noalloc -- moe_ffn_fused for callers that cannot allocate: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc. The same
 * arguments and results as moe_ffn_fused, without ws / ws_bytes: the workspace is a
 * fixed array of MOE_NOALLOC_SCRATCH_BYTES (64 MiB) that the library holds on every
 * device it runs on, from the first call there until the process ends. Enough for a
 * DeepSeek-Lite-shaped PP512 layer and any decode batch; a call needing more
 * (moe_ffn_fused_workspace_size) is MOE_ELIMIT, with nothing enqueued. The call itself
 * allocates nothing. All calls on one device share that device's array, so calls that
 * overlap in time on one device (different streams, or different host threads) race
 * and give undefined results: serialise them, e.g. on one stream. Its contents need no
 * clearing between calls (the kernels overwrite what they read).
 */
#define MOE_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
moe_status moe_ffn_fused_noalloc(const moe_weights *gate, const moe_weights *up,
                                 const moe_weights *down, const moe_weights *sh_gate,
                                 const moe_weights *sh_up, const moe_weights *sh_down,
                                 const void *x, moe_dtype x_type, const int32_t *ids,
                                 const float *route_w, int64_t n_tokens, int32_t n_used, float *out,
                                 const moe_options *opt, void *stream);

/*
 * moe_quantize_act -- the activation format of the quantized-activation path (the
 * pages' mmq_id multiplies quantized experts with quantized activations, "CUDA: better
 * MoE implementation", section 2.1; they do not define the format, so it is a
 * reading): each row of x is cut into blocks of 32 columns; a block gets the float32
 * scale d = max|x| / 127 and int8 codes q = x / d rounded to the nearest integer, ties
 * to even (float32 division and rounding; clamped to [-127, 127]); a block of zeros has
 * d = 0 and q = 0. Value = d * q. x must be finite.
 *   x   device BF16 or F32 [rows][K], K % 32 == 0 (MOE_ELIMIT otherwise), 16-byte aligned
 *   q   device int8 [rows][K] (written, 16-byte aligned); d device float32 [rows][K/32]
 *       (written)
 * rows = 0 is a no-op. No workspace. Deterministic.
 */
moe_status moe_quantize_act(const void *x, moe_dtype x_type, int64_t rows, int64_t K, int8_t *q,
                            float *d, void *stream);

/*
 * moe_quantize_rows -- rows to int8 with one float32 scale each: the activation format of
 * moe_mul_mat_id with I8 experts, and the way to make such experts from float32 or 16-bit ones
 * (rows = n_mat * rows of the matrices). d = max|x| / 127 over the row and q = x / d rounded to the
 * nearest integer, ties to even (float32 division and rounding; clamped to [-127, 127]); d = 0 and
 * q = 0 for a row of zeros, d = NaN and q = 0 for one with an infinity or a NaN. Value = d * q.
 *   x   device BF16, F16 or F32 [rows][K], any K > 0
 *   q   device int8 [rows][K] (written); d device float32 [rows] (written)
 * The three must not overlap (MOE_EINVAL). rows = 0 is a no-op. No workspace. Deterministic.
 */
moe_status moe_quantize_rows(const void *x, moe_dtype x_type, int64_t rows, int64_t K, int8_t *q,
                             float *d, void *stream);

/*
 * moe_router_topk -- the step ahead of the op: the ids table the op consumes (section
 * 1.2 of the PR #283 write-up: ids names the experts each token uses) and routing
 * weights, from router logits.
 *   logits   device float32 [n_tokens][n_experts]
 *   ids      device int32 [n_tokens][n_used] (written): the n_used largest logits of
 *            each token in descending order, equal logits taken lower index first;
 *            NaN logits rank strictly below every number, -inf included (NaNs among
 *            themselves: lower index first)
 *   route_w  device float32 [n_tokens][n_used] (written): softmax over the picked
 *            logits only (exp(v_r - v_0) / sum_r exp(v_r - v_0)), the weighting the
 *            DeepSeek-V3-shaped configuration calls softmax renormalised over the
 *            picks. A NaN pick is weighted as -inf (weight 0). When the largest pick
 *            v_0 is +inf or -inf the softmax's limit is used: the c picks equal to v_0
 *            get 1/c each and the others 0 (a token whose picks are all -inf or NaN
 *            gets 1/n_used on every pick)
 * Requires 1 <= n_used <= n_experts <= 1024 (MOE_EINVAL / MOE_ELIMIT otherwise) and
 * n_tokens < 2^22. No workspace. Deterministic. n_tokens = 0 is a no-op.
 */
moe_status moe_router_topk(const float *logits, int64_t n_tokens, int32_t n_experts, int32_t n_used,
                           int32_t *ids, float *route_w, void *stream);

/*
 * moe_quantize_mxfp4 -- rows to MXFP4 (the weight format above, from the OCP Microscaling
 * v1.0 specification): the activation format of act_quant = 2, and the way to make MXFP4
 * experts from bf16 or float32 ones (rows = n_mat * rows of the matrices). Each row is cut
 * into blocks of 32 columns. With m = max|x| of a block, its scale byte is
 * max(floor(log2 m) - 2 + 127, 0) (0 for a block of zeros), and each element gets the E2M1
 * code nearest to x / 2^(byte - 127), ties to the even code, magnitudes over 6 taken as 6;
 * a value that rounds to zero keeps its sign. A block with an infinity or a NaN gets scale
 * byte 255 (every value NaN) and codes 0.
 *   x       device BF16 or F32 [rows][K], K % 32 == 0 (MOE_ELIMIT otherwise), 16-byte aligned
 *   codes   device uint8 [rows][K/2] (written, 16-byte aligned), column 2i in bits 0-3
 *   scales  device uint8 [rows][K/32] (written)
 *   values  NULL, or device [rows][K] of x's type (written, 16-byte aligned; may be x
 *           itself): the values the codes stand for, exactly representable in both types --
 *           what quantization-aware training puts in place of x
 * rows = 0 is a no-op. rows * K / 32 < 2^31 (MOE_ELIMIT). No workspace. Deterministic.
 */
moe_status moe_quantize_mxfp4(const void* x, moe_dtype x_type, int64_t rows, int64_t K,
                              uint8_t* codes, uint8_t* scales, void* values, void* stream);

/*
 * moe_router_scored -- routing by scores over all experts, the form of routers trained with
 * a balance bias and expert groups; moe_router_topk is the softmax over the picks alone.
 * For each token, with l its logits:
 *   score   s_e = exp(l_e) / sum_f exp(l_f) (MOE_SCORE_SOFTMAX) or 1 / (1 + exp(-l_e))
 *           (MOE_SCORE_SIGMOID)
 *   choice  c_e = s_e + bias[e] (bias NULL: the order of the logits); the bias steers the
 *           choice and enters neither scores nor weights
 *   groups  the experts form n_group groups of n_experts / n_group neighbours. A group's
 *           score is its largest choice (group_top = 1) or the sum of its two largest ones
 *           (group_top = 2; a single one counts alone); the topk_group best groups are
 *           kept, equal scores lower group first
 *   picks   the n_used largest choices in the kept groups, descending, equal choices lower
 *           expert first
 *   weight  scale * s_i, or with renorm scale * s_i / sum of the picks' s
 * Choices are compared as 64-bit values, so the picks do not depend on float32 rounding.
 * Masks: an expert whose logit is -inf or NaN, or whose bias is -inf or NaN, is never
 * picked; a logit of -inf or NaN also has score 0 and stays out of the softmax's sum.
 * Picks that find no expert (a token with every logit -inf, say padding) get id -1 and
 * weight 0, which the calls above skip. Logits of +inf take the limit: sigmoid 1, softmax
 * shared equally among them.
 *   logits   device F32 or BF16 [n_tokens][n_experts]
 *   bias     NULL or device float32 [n_experts]
 *   ids      device int32 [n_tokens][n_used] (written)
 *   route_w  device float32 [n_tokens][n_used] (written)
 *   scores   NULL or device float32 [n_tokens][n_experts] (written): s, for balance losses;
 *            not in the place of logits (MOE_EINVAL)
 * Requires 1 <= n_used <= topk_group * n_experts / n_group, n_experts <= 1024,
 * n_experts % n_group == 0, 1 <= topk_group <= n_group (MOE_EINVAL / MOE_ELIMIT
 * otherwise), a finite scale, n_tokens < 2^22. No workspace. Deterministic.
 * n_tokens = 0 is a no-op.
 */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score;
typedef struct {
    int32_t score;      /* moe_score                                              */
    int32_t n_group;    /* 1: no groups                                           */
    int32_t topk_group; /* groups kept                                            */
    int32_t group_top;  /* choices summed to a group's score: 1 or 2              */
    int32_t renorm;     /* 1: weights divided by the sum of the picks' scores     */
    float scale;        /* factor on the weights                                  */
    int32_t reserved[2];
} moe_router_config;
moe_status moe_router_scored(const void* logits, moe_dtype logits_type, const float* bias,
                             int64_t n_tokens, int32_t n_experts, int32_t n_used,
                             const moe_router_config* cfg, int32_t* ids, float* route_w,
                             float* scores, void* stream);

/*
 * moe_router_scored_backward -- the gradient of the logits through moe_router_scored's
 * weights and scores (the choice itself and the bias have none):
 *   d_logits[t][f] = sum_s d_route_w[t][s] * d route_w[t][s] / d l_f
 *                  + sum_e d_scores[t][e] * d s_e / d l_f
 *   logits     as in the forward call
 *   ids        device int32 [n_tokens][n_used], the forward call's; entries outside
 *              [0, n_experts) or naming a masked logit contribute nothing, an expert named
 *              more than once gets the sum of its entries' gradients
 *   d_route_w  device float32 [n_tokens][n_used]
 *   d_scores   NULL, or device float32: row t at d_scores + t * d_scores_stride. A stride of
 *              0 gives every token the same row (a balance loss's gradient), else the
 *              stride is at least n_experts (MOE_EINVAL)
 *   d_logits   device [n_tokens][n_experts] of the logits' type (written, computed in
 *              float32 and rounded once; masked logits get 0). It may be logits itself.
 * cfg: score, renorm and scale as in the forward call; its group fields are not read.
 * No workspace. Deterministic. n_tokens = 0 is a no-op.
 */
moe_status moe_router_scored_backward(const void* logits, moe_dtype logits_type, const int32_t* ids,
                                      const float* d_route_w, const float* d_scores,
                                      int64_t d_scores_stride, int64_t n_tokens, int32_t n_experts,
                                      int32_t n_used, const moe_router_config* cfg, void* d_logits,
                                      void* stream);

/* Workspace sizes in bytes for the calls above with the same arguments (0 if the
 * arguments are invalid; a valid call may also need 0 bytes, then ws may be NULL). */
size_t moe_row_ids_workspace_size(int64_t n_tokens, int32_t n_used, int32_t n_experts);
size_t moe_mul_mat_id_workspace_size(const moe_weights *w, moe_dtype src1_type,
                                     int32_t src1_rows_per_token, int64_t n_tokens,
                                     int32_t n_used, const moe_options *opt);
/* want: 1 d_src1, 2 d_w, 4 d_route_w, added up; weighted: route_w is given */
size_t moe_mul_mat_id_backward_workspace_size(const moe_weights *w, moe_dtype d_dst_type,
                                              int32_t src1_rows_per_token, int64_t n_tokens,
                                              int32_t n_used, int32_t weighted, int32_t want,
                                              const moe_options *opt);
size_t moe_ffn_fused_workspace_size(const moe_weights *gate, const moe_weights *sh_gate,
                                    moe_dtype x_type, int64_t n_tokens, int32_t n_used,
                                    const moe_options *opt);

/* Which path a call with these sizes takes: 1 grouped GEMM, 2 GEMV (decode), or a
 * negative moe_status for invalid arguments. act_width is the widest activation
 * row a GEMV kernel would stage (mul_mat_id: K; FFN: max(n_embd, n_ff, n_ff_sh)).
 * Auto (Q8_0): GEMV when n_tokens < tau * n_experts and either n_tokens * n_used <= 48
 * with act_width <= 4096, or n_tokens == 1 with n_used <= 256 and act_width <= 16384;
 * else GEMM. 4-bit experts: GEMV when n_tokens < tau * n_experts, n_tokens * n_used
 * <= 64 (MXFP4: 32) and act_width <= 4096. Forcing GEMV is allowed up to n_tokens * n_used <= 256
 * and act_width <= 16384 (Q8_0; 64 and 4096 for 4-bit), else MOE_EINVAL.
 * Pure host function. */
int32_t moe_select_path(int64_t n_tokens, int32_t n_used, int32_t n_experts, int64_t act_width,
                        const moe_options *opt);

/* The path moe_mul_mat_id / moe_ffn_fused take for experts of weight_type (MOE_Q8_0,
 * MOE_MXFP4, MOE_IQ4_NL or MOE_IQ4_XS; moe_mul_mat_id also MOE_BF16, MOE_F16, MOE_I8) under opt: 1 grouped GEMM, 2 GEMV, 3 the grouped
 * GEMM over quantized activations (opt->act_quant = 1, Q8_0 only), 4 the grouped GEMM or 5
 * the GEMV over MXFP4 activations (opt->act_quant = 2, MXFP4 only; act_width: the narrowest
 * row, shared experts apart), or a negative moe_status (MOE_EINVAL for other weight types,
 * or for options the call would reject).
 * Q8_0 gives the same answer as moe_select_path. Pure host function. */
int32_t moe_select_path_typed(int64_t n_tokens, int32_t n_used, int32_t n_experts, int64_t act_width,
                              moe_dtype weight_type, const moe_options *opt);

const char *moe_status_string(moe_status s);
const char *moe_last_error(void); /* thread-local detail of the last failure ("" if none) */
/* Kernels (timing-event pairs, see moe_options) enqueued by the last successful
 * moe_mul_mat_id or moe_ffn_fused call on this thread; 0 before any such call. */
int32_t moe_last_stage_count(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H */
