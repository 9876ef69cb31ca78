/*
 * maxsim_layers.h -- C ABI of the operators of the encoder's attention layer and of
 * the loss that trains it, in the same library (libmaxsim.so):
 *
 *     projected rows -> rotary positions -> attention -> hidden rows (maxsim_encoder.h)
 *     MaxSim's scores, a teacher's top scores -> distillation loss, grad_scores (maxsim_bwd)
 *
 * Conventions, as in maxsim.h: data pointers are DEVICE pointers the caller owns;
 * a call only enqueues work on `stream` (NULL = the null stream) of the current
 * device and returns; the library allocates nothing; arguments are checked on the
 * host before any HIP call, and the status codes are those of maxsim.h.  What lies
 * on the device (lengths, positions, indices) is not checked: kernels clamp it, so
 * that no access leaves the memory that the sizes describe.  Further:
 *   - Inputs may be strided as each call says; an output may not overlap an input
 *     or itself except where a call says so.
 *   - Calls keep no state.  Calls that share a workspace must be ordered on one
 *     stream; two captured graphs that share one must not run at once.
 *   - Results are bit-identical from run to run (no atomics).  Sums, softmax
 *     statistics and angles are held in 32 bits or more.
 */
#ifndef MAXSIM_LAYERS_H
#define MAXSIM_LAYERS_H

#include "maxsim_encoder.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows of heads in memory: element (b, t, h, c) is data[b * batch + t * token + h * head + c] (steps in elements). */
typedef struct {
    void* data;
    int64_t batch, token, head;
} maxsim_view;

/* Which columns make a pair that is rotated. */
enum { MAXSIM_ROPE_HALF = 0 /* (i, i + rotary/2) */, MAXSIM_ROPE_INTERLEAVED = 1 /* (2i, 2i + 1) */ };

/*
 * Rotary positions: pair i of the first `rotary` columns of each head of the token at
 * position p is turned by the angle a = p * inv_freq[i] and multiplied by `scale`,
 *     (u, w) -> scale * (u cos a - w sin a, w cos a + u sin a);
 * the other columns are copied.  inverse != 0 turns by -a: the gradient of x from that of y.
 *   x, y       [B, L, H, D] dtype (F16, BF16 or F32) views; y may be x (the same view)
 *   inv_freq   [rotary / 2] fp64, radians a position.  Stretched contexts (linear, or by parts of
 *              the frequencies) are in these values and in `scale`.
 *   positions  [B, L] int32: each token's position; or NULL: offsets[b] + t, and t where that is
 *   offsets    [B] int32, or NULL.  (Not both.)
 * The angle is formed in fp64 and brought into one turn before it is rounded to fp32 (off by pi 2^-24 at most), so that far
 * positions lose nothing; sine, cosine and their products with scale are fp32, each rounded (an fp32 result is off by 5e-8 of
 * its norm, one made with fp64 factors by 4e-8).  Rows need the alignment of one element (16 bytes are fastest).
 * Requires B, L >= 0, H >= 1, 1 <= D <= 1024, rotary even, 2 <= rotary <= D, B * L < 2^25 and scale finite.
 */
int maxsim_rope(const maxsim_view* x, const maxsim_view* y, int32_t B, int32_t L, int32_t H, int32_t D, int32_t rotary,
                int32_t layout, int32_t dtype, const double* inv_freq, const int32_t* positions, const int32_t* offsets,
                float scale, int32_t inverse, void* stream);

/*
 * Attention with a sliding window and a few first tokens that stay visible.
 * Sequence b has Lq(b) queries and Lk(b) keys.  Query i stands at p = i + Lk - Lq (the
 * last query at the last key) and sees key j where
 *     j <= p + right   and   (j >= p - left or j < sinks)
 * left < 0 and right < 0: no bound on that side (right 0 is causal).  For each of Hq query
 * heads h, with the key head h / (Hq / Hk):
 *     S_ij = scale * sum_c q_ic k_jc;  P = softmax over the keys that i sees;  out_i = sum_j P_ij v_j
 * A query that sees no key gives zeros (lse -infinity, no gradient).
 *   q, out    [B, max_q, Hq, D], or, with cu_q, packed [rows_q, Hq, D] (batch step not used):
 *             sequence b is rows [cu_q[b], cu_q[b + 1]); starts may not decrease (else rows of the outputs are unspecified)
 *   k, v      [B, max_k, Hk, D], or, with cu_k, packed [rows_k, Hk, D]
 *   q_lens    [B] int32: Lq(b), without cu_q; NULL: max_q for all.  k_lens likewise.
 *   max_q, max_k  bounds of the lengths (longer ones are cut)
 *   lse       fp32 out, or NULL: log of the sum of exp(S_ij), of row and head n = (b * max_q + i) * Hq + h (packed:
 *             row * Hq + h) at lse[n * lse_step].  lse_step 1, or at least 1 + D/2: then the D values of dtype behind
 *             each hold what rounding left off out, which keeps rowsum(dO * out) of the backward exact (the backward
 *             takes of them what is half a step of out at most, so that other memory there costs no more than rounding does)
 * Rows of no sequence (past a sequence's length, before the first one, past the last one) are not read; in
 * outputs they are left as they were, or made 0 where zero_rest is not 0.  B = 0 enqueues nothing.
 * Scores, statistics and sums are fp32; P (and in the backward dS) is rounded to dtype for its product, as
 * the matrix cores take it; each output is rounded once.  Keys that no query of their sequence sees are not read and
 * may hold anything (entries dropped from a cache; their gradients are 0).  A NaN elsewhere in a
 * sequence reaches all rows that see it and may reach rows near them that do not; so does an infinity, but for a score of
 * -infinity, whose weight is 0 (a query with no other score counts as one that sees no key).  In fp16, P and dS are
 * rounded in the scale of the row's (dK, dV: the key's) largest ones, so that dO and v may be of any size that fp16 holds.
 * Requires data 16-byte aligned and steps multiples of 8, token steps of at least D and at most 2^20; D a multiple of 8 from 8 to 128;
 * Hq a multiple of Hk; 0 <= max_q * (Hq / Hk), max_k < 2^29; 2^-60 <= scale <= 2^60; sinks >= 0; and tiles of
 * 128 rows, of queries (max_q * (Hq / Hk)) or keys, of which B * Hk times one more than there are stay below 2^21.
 */
typedef struct {
    maxsim_view q, k, v, out;
    const int32_t *cu_q, *cu_k;      /* [B + 1], or NULL */
    const int32_t *q_lens, *k_lens;  /* [B], or NULL */
    int64_t rows_q, rows_k;          /* rows in memory where packed */
    int32_t B, max_q, max_k, Hq, Hk, D;
    int32_t dtype; /* F16 or BF16 */
    int32_t left, right, sinks;
    int32_t zero_rest;
    float scale;
    int32_t lse_step;
} maxsim_attn;

/* Bytes of device workspace (may be 0; 0 on bad sizes).  Sizes, type, the window and which lengths are given are looked at, no data. */
size_t maxsim_attn_fwd_workspace_bytes(const maxsim_attn* a);
size_t maxsim_attn_bwd_workspace_bytes(const maxsim_attn* a);

/* The forward: a->out and lse (or NULL).  workspace: 16-byte aligned (NULL is fine when 0 bytes are needed). */
int maxsim_attn_fwd(const maxsim_attn* a, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The backward: dq, dk, dv (views as q, k, v) from dout (a view as out), with a->out and lse of the forward.
 *     dV = P^T dO;  dS = P * (dO V^T - rowsum(dO * out));  dQ = scale dS K;  dK = scale dS^T Q
 * dK and dV of a shared head are summed over its query heads in fp32 before they are rounded.
 */
int maxsim_attn_bwd(const maxsim_attn* a, const float* lse, const maxsim_view* dout, const maxsim_view* dq,
                    const maxsim_view* dk, const maxsim_view* dv, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Distillation from a teacher's top scores, a loss of each row of scores:
 *     q_k = softmax over the row's entries of teacher_k / T;   p_v = softmax over all columns of z_v / T
 *     loss = T^2 * sum_k q_k (log q_k - log p_{index_k})
 *   scores   [N, V] dtype (F16, BF16 or F32), pitch ld: z
 *   index    [N, K] int32, teacher [N, K] fp32: the teacher's columns and scores.  An index outside
 *            [0, V) is no entry (rows with fewer than K); a column listed twice counts twice.
 *   loss     [N] fp32 out
 *   stat     [N, 4] fp32 out, for the backward: the row's largest z, log of the sum of exp((z_v - largest) / T), and
 *            the same of the teacher's entries (of none: 0 and +infinity)
 * A row without entries (or whose entries are all -infinity) gives 0 and no gradient.  Scores of -infinity are
 * columns that are not there (p = 0); one that the teacher's q > 0 asks for gives an infinite loss.
 * Requires N, V >= 0, 0 <= K <= 1024, N < 2^24, V < 2^30, 2^-60 <= T <= 2^60.
 * The workspace (rows split over workgroups): 16-byte aligned, NULL is fine when 0 bytes are needed.
 */
size_t maxsim_distill_workspace_bytes(int32_t N, int32_t V);
int maxsim_distill_fwd(const void* scores, int64_t ld, const int32_t* index, const float* teacher, int32_t N, int32_t V,
                       int32_t K, int32_t dtype, float temperature, float* loss, float* stat, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * Its gradient: dscores[n, v] = dloss[n] * T * (p_v - sum over the entries k with index_k = v of q_k)
 *   dloss [N] fp32;  stat from the forward;  dscores [N, V] dtype out, pitch ldd; may be the memory of scores
 *   (with the same pitch)
 */
int maxsim_distill_bwd(const float* dloss, const void* scores, int64_t ld, const float* stat, const int32_t* index,
                       const float* teacher, int32_t N, int32_t V, int32_t K, int32_t dtype, float temperature,
                       void* dscores, int64_t ldd, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MAXSIM_LAYERS_H */
