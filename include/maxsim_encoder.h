/*
 * maxsim_encoder.h -- C ABI of the operators around MaxSim's operands, in the
 * same library (libmaxsim.so): the embedding head that makes the token rows
 * maxsim.h scores, and the step that trains it.
 *
 *     hidden rows (+ residual) -> RMS norm, 8 bits with scales
 *       -> product in 8-bit floating point -> RMS norm, 16 bits (maxsim_fwd)
 *          or int8 with a scale per token (maxsim_fwd_i8)
 *     dQ / dD of maxsim_bwd -> RMS norm backward -> products -> AdamW
 *
 * Conventions, as in maxsim.h: data pointers are DEVICE pointers the caller
 * owns; a call only enqueues work on `stream` (NULL = the null stream) of the
 * current device and returns; the library allocates nothing; arguments are
 * checked on the host before any HIP call, and the status codes are those of
 * maxsim.h.  Differences and additions:
 *   - Matrices are row-major with a row pitch (ld*, in elements) of at least
 *     their width, so a slice of wider rows can be passed.  Elements between
 *     the width and the pitch are neither used nor written.
 *   - 16- and 32-bit rows need the alignment of one element only (16 bytes are
 *     fastest); 8-bit operands of the product need 16-byte aligned rows.
 *   - An output may be the same memory as an input of the same shape, type and
 *     pitch where a call says so.  No other overlap is allowed.
 *   - Calls keep no state.  Calls that share a workspace must be ordered on one
 *     stream; two captured graphs that share one must not run at once.
 *   - Results are bit-identical from run to run (no atomics).
 *   - NaN and infinity pass through as the formulas give them; where a block
 *     of values to be held in 8 bits has one that is not finite, the block's
 *     scale is NaN and its values are 0.
 *
 * 8-bit values.  A block of values v shares one fp32 scale and is held as
 * round(v / scale), ties to even:
 *     e4m3  scale = max|v| * c, c the fp32 value next to 1/448 (what torch's division of
 *           a tensor by 448.0 does on the device: scales and codes equal the plain form's);
 *     int8  scale = max|v| / 127, rounded to nearest in fp32.
 * v / scale is the nearest fp32 value or, in about 1 of 10^7 cases, its neighbour, before it is rounded to 8 bits.
 * A block whose largest magnitude is below 2^-100 is held as zeros with scale 1, so
 * that 1 / scale never overflows.
 * e4m3 is the OCP 8-bit format (4 exponent bits, 3 mantissa bits, largest value 448).
 */
#ifndef MAXSIM_ENCODER_H
#define MAXSIM_ENCODER_H

#include "maxsim.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Further element types, beside MAXSIM_F16 and MAXSIM_BF16. */
enum { MAXSIM_F32 = 2, MAXSIM_I8 = 3, MAXSIM_E4M3 = 4 };

/* Values that share a scale: columns of an e4m3 row, elements of an optimiser state. */
#define MAXSIM_QBLOCK 128

/*
 * Root-mean-square norm of rows, with the residual's addition before it:
 *     h = x + residual;  r = 1 / sqrt(mean(h^2) + eps);  y = h * r * weight
 *   x         [R, H] dtype (F16, BF16 or F32), pitch ldx
 *   residual  [R, H] dtype, pitch ldr, or NULL
 *   weight    [H] of weight_dtype (dtype or F32), or NULL for all ones
 *   y         [R, H] of out_dtype, pitch ldy:
 *               F16, BF16, F32: rounded to nearest;
 *               I8:   one scale per row, scale [R] -- the operand and scales of
 *                     maxsim_fwd_i8 when H = 128 (which takes finite scales only: not
 *                     a row whose values were not finite);
 *               E4M3: one scale per 128 columns, scale [R, ceil(H/128)] -- the
 *                     operand of maxsim_gemm_fp8 (ldy a multiple of 16 there).
 *   scale     fp32 out for I8 and E4M3, NULL otherwise
 *   sum       [R, H] dtype out, pitch lds: h rounded, or NULL
 *   rstd      [R] fp32 out: r, or NULL (the backward reads it)
 * The norm uses h in fp32, before it is rounded into sum.  Sums are fp32: a
 * row whose sum of squares overflows fp32 gives zeros.  x, residual, sum and a y of
 * dtype may be the same memory.  Requires R >= 0, 1 <= H <= 32768, eps >= 0.
 */
int maxsim_rmsnorm_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                       int32_t weight_dtype, int32_t R, int32_t H, int32_t dtype, float eps, int32_t out_dtype,
                       void* y, int64_t ldy, float* scale, void* sum, int64_t lds, float* rstd, void* stream);

/* Bytes of device workspace maxsim_rmsnorm_bwd needs for dweight (0 for few rows, and on bad sizes). */
size_t maxsim_rmsnorm_bwd_workspace_bytes(int32_t R, int32_t H);

/*
 * Backward of the norm (of a y not held in 8 bits, or with the rounding to 8 bits passed straight through):
 *     g = dy * weight;  xh = h * r;  dx = r * (g - xh * mean(g * xh)) + dsum
 *     dweight = sum over rows of dy * xh
 *   dy, h     [R, H] dtype: the gradient of y, and h (the forward's sum, or x without a residual)
 *   rstd      [R] fp32 from the forward;  weight as there (NULL: all ones)
 *   dsum      [R, H] dtype: the gradient that arrives at sum itself, or NULL
 *   dx        [R, H] dtype out: the gradient of x and of residual alike; may be
 *             the memory of dy, h or dsum
 *   dweight   [H] fp32 out, or NULL; rows are added in a fixed order
 *   workspace of maxsim_rmsnorm_bwd_workspace_bytes() bytes, 16-byte aligned
 *             (NULL is fine without dweight, or when that is 0).
 * Requires R >= 0 (dweight is 0 for R = 0), 1 <= H <= 32768.
 */
int maxsim_rmsnorm_bwd(const void* dy, int64_t lddy, const void* h, int64_t ldh, const float* rstd,
                       const void* weight, int32_t weight_dtype, const void* dsum, int64_t ldds, int32_t R, int32_t H,
                       int32_t dtype, void* dx, int64_t lddx, float* dweight, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * Rows in 8-bit floating point, for the operands of maxsim_gemm_fp8.
 *   x        [R, C] dtype (F16, BF16 or F32), pitch ldx
 *   block_rows 1:   q [R, C] e4m3, scale [R, ceil(C/128)]: a scale for 128 columns of a row;
 *                   qt [C, R] e4m3, scale_t [C, ceil(R/128)]: x transposed, a scale for 128 of x's rows
 *   block_rows 128: one scale for 128 x 128 values: q with scale [ceil(R/128), ceil(C/128)], and qt, scale_t
 *                   the transposes of q and scale.
 *   q (pitch ldq) with scale, qt (pitch ldqt) with scale_t: either pair may be NULL, not both.
 * One pass over x makes both.  Requires R, C >= 0 and ceil(R/128) * ceil(C/128) < 2^24.
 */
int maxsim_quant_fp8(const void* x, int64_t ldx, int32_t R, int32_t C, int32_t dtype, int32_t block_rows, void* q,
                     int64_t ldq, float* scale, void* qt, int64_t ldqt, float* scale_t, void* stream);

/* Bytes of device workspace maxsim_gemm_fp8 needs for these sizes (may be 0; 0 on bad sizes). */
size_t maxsim_gemm_fp8_workspace_bytes(int32_t M, int32_t N, int32_t K);

/*
 * Product of two matrices in 8-bit floating point with a scale for each 128 along K:
 *     c[m, n] = sum_kb a_scale[m, kb] * b_scale[n / b_block_rows, kb] * sum over k in block kb of A[m, k] * B[n, k]
 *   A        [M, K] e4m3, pitch lda;  a_scale [M, ceil(K/128)] fp32
 *   B        [N, K] e4m3, pitch ldb;  b_scale [ceil(N/b_block_rows), ceil(K/128)] fp32, b_block_rows 1 or 128
 *   c        [M, N] F16, BF16 or F32 (out_dtype), pitch ldc
 * The scaled blocks are added in fp32 and c is rounded once.  A block's products
 * are added on the matrix cores: for an F32 c in fp32; for F16 and BF16 by the
 * 8-bit instruction, which adds eight products that follow each other along K at a time, each
 * cut toward 0 to a multiple of 2^(e - 13), where e is the largest sum of two values' exponents
 * among the eight (a subnormal value counts with exponent -6).  So eight normal values
 * of one sign lose less than 7 * 2^-13 = 8.5e-4 of their sum (half a step of F16 is
 * 4.9e-4, of BF16 3.9e-3); on normally distributed values the whole product is off by
 * 1.4e-5 of its norm.  Where large products cancel, or large values meet subnormal ones of the
 * other operand (less than 7 * 2^-10), and that matters, take an F32 c.
 * The two scales are multiplied with each other or with a block's sum (up to 2.6e7) first, in fp32:
 * where that passes 3.4e38 the result is infinite or NaN.
 * A, B: 16-byte aligned, lda and ldb
 * multiples of 16, at least K rounded up to 16, and every row readable that far (what lies
 * there after K is not used).  workspace: maxsim_gemm_fp8_workspace_bytes()
 * bytes, 16-byte aligned (NULL is fine when that is 0).
 * Requires M, N, K >= 0 (K = 0 gives zeros), K, lda, ldb <= 2^22, and
 * ceil(M/128) * ceil(N/128) < 2^22.
 */
int maxsim_gemm_fp8(const void* A, int64_t lda, const float* a_scale, const void* B, int64_t ldb,
                    const float* b_scale, int32_t b_block_rows, int32_t M, int32_t N, int32_t K, int32_t out_dtype,
                    void* c, int64_t ldc, void* workspace, size_t workspace_bytes, void* stream);

/* One tensor of an AdamW step; every pointer a device pointer to n values (scales: ceil(n/128)). */
typedef struct {
    void* param;       /* param_dtype, updated */
    const void* grad;  /* grad_dtype */
    float* master;     /* fp32 weights that a 16-bit param is rounded from, or NULL; updated */
    void* m;           /* first moment: fp32, or e4m3 with m_scale; updated */
    void* v;           /* second moment: fp32, or its square root as e4m3 with v_scale; updated */
    float* m_scale;    /* e4m3 states: a scale for each 128 values, else NULL */
    float* v_scale;
    int64_t n;         /* values; 0 is allowed */
} maxsim_adamw_tensor;

/*
 * One AdamW step over many tensors:
 *     m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g^2
 *     p = p (1 - lr weight_decay) - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 *   tensors      HOST array of `count` entries, read during the call; all of them
 *                share param_dtype, grad_dtype (F16, BF16 or F32 each) and
 *                state_dtype (F32 or E4M3).  The same memory in two entries is not allowed.
 *   step         t >= 1, the number of this step; or, where step_dev is not
 *                NULL, the device int32 there holds it when the work runs (for
 *                a captured step that is replayed; a captured `step` stays what it was)
 * The moments are formed in fp32 as written here, left to right: beta m rounded, then
 * the gradient's term (g^2 rounded) added with one rounding.  (So a gradient past 1.8e19
 * makes v infinite.)  E4M3 states: the update uses the new m and v in fp32, before they are held
 * in 8 bits again; a second moment that is not 0 is never held as 0 (its root
 * is at least the smallest e4m3 value, 2^-9, times the block's scale) nor read as 0 (where that
 * value's square leaves fp32, it is read as the smallest fp32 value, 2^-149).
 * All-zero memory is a valid start for both kinds of state.
 * Up to 56 tensors go into one launch.  After MAXSIM_ERR_HIP some of the tensors may have
 * been stepped: the step is not to be made again from this state.  Requires 0 <= beta1, beta2 < 1,
 * eps >= 0, lr and weight_decay finite.  A gradient that is not finite makes its own values NaN or infinite and,
 * with E4M3 states, the moments of its whole block of 128 NaN from the next step on: where that may
 * happen, look at the gradients before the step.
 */
int maxsim_adamw(const maxsim_adamw_tensor* tensors, int32_t count, int32_t param_dtype, int32_t grad_dtype,
                 int32_t state_dtype, double lr, double beta1, double beta2, double eps, double weight_decay,
                 int32_t step, const int32_t* step_dev, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MAXSIM_ENCODER_H */
