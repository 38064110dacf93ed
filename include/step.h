/*
 * step.h -- C ABI of the operators a serving step runs around the routed LoRA
 * delta on MI355X (gfx950): the norm in front of a projection, the shared
 * projection with every request's adapter added to it, and the log
 * probabilities of the answered tokens.  Library: libstep.so.
 *
 * Conventions, the same as lora.h's:
 *  - bf16 values travel as uint16_t bit patterns, e4m3 (OCP, no infinities,
 *    largest value 448) as uint8_t; float is IEEE binary32.
 *  - Every array pointer is a DEVICE pointer unless marked [host].
 *  - `stream` is a hipStream_t (NULL = the default stream).  A call only
 *    enqueues kernels on it: it does not allocate, free, clear, synchronize,
 *    print or abort, so every call may be captured into a graph.
 *  - The caller owns every buffer.  The library keeps no pointer and no state
 *    after a call returns.
 *  - Every check that can run on the host runs before any launch and returns
 *    an error code; nothing is enqueued then.
 *  - Workspaces must be zero-filled before their first use and may then be
 *    passed to any number of calls of the same operator, of any shape they
 *    are large enough for, one after another on one stream (or on streams
 *    joined by events).  Calls that overlap need workspaces of their own.
 *  - n == 0 is a valid call that enqueues nothing (row pointers may be null).
 */
#ifndef TENANT_STEP_H
#define TENANT_STEP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
    STEP_OK = 0,
    STEP_EINVAL = -1,       /* bad pointer, size, alignment or leading dimension */
    STEP_EUNSUPPORTED = -2, /* a shape outside the limits of the call */
    STEP_EWORKSPACE = -3,   /* workspace missing or too small */
    STEP_ELAUNCH = -4       /* the HIP runtime refused a launch */
};

/* The largest `top` of step_token_logprobs. */
#define STEP_MAX_TOP 32

/*
 * Root-mean-square norm, with the residual's addition and an 8-bit copy:
 *     s[i][j] = x[i][j] + residual[i][j]                (x alone without residual)
 *     y[i][j] = s[i][j] / sqrt(mean_j(s[i][j]^2) + eps) * weight[j]
 * computed in fp32 from the unrounded s.  Outputs, each [n][h] contiguous:
 *     residual_out  s rounded to bf16; given exactly when residual is, and
 *                   may be the same buffer (then ldr must be h)
 *     y             bf16, or null
 *     q, q_scale    y's e4m3 copy: q_scale[i] = max_j |y[i][j]| / 448 and
 *                   q[i][j] = y[i][j] / q_scale[i] from the unrounded y; both
 *                   null or both given.  A row of zeros gets scale 0 and q 0 (and
 *                   y 0, also with eps 0).
 *                   A row whose y holds a NaN or an infinity, from x, residual or
 *                   weight, gets scale NaN and q 0; one whose squares sum past
 *                   3.4e38 gets y, scale and q 0.
 * At least one of y and q is given.  Shapes: h a multiple of 8 in [8, 32768];
 * n <= 1 << 24; ldx, ldr >= h and multiples of 8; x, residual, weight,
 * residual_out and y 16-byte aligned, q 8-byte aligned; eps >= 0 and finite.
 */
int step_rms_norm(const uint16_t *x, int64_t ldx, const uint16_t *residual, int64_t ldr, const uint16_t *weight,
                  int32_t n, int32_t h, float eps, uint16_t *residual_out, uint16_t *y, uint8_t *q, float *q_scale,
                  void *stream);

/* Workspace bytes step_lora_linear needs: `out` is the sum of the slice
 * widths.  0 for a shape that the call refuses.  They serve every call of the
 * same or smaller sizes too. */
size_t step_lora_linear_workspace_bytes(int32_t n, int32_t k, int32_t out, int32_t num_slices, int32_t max_rank);

/*
 * The shared projection with every row's adapter: for s = slot[i],
 *     y[i][c] = sum_k x[i][k] w[c][k]
 *               + scale[s] * sum_r (sum_k x[i][k] a_pool[s][l][r][k]) * b_pool[s][c][r]
 * where l is the slice that holds column c; the second term is absent for
 * s < 0 and for s >= num_slots.  Sums in fp32, one rounding to bf16.  Layouts:
 *    x       [n][ldx]        bf16, k used columns
 *    w       [out][k]        bf16, out = sum(slice_sizes); with xq: e4m3
 *    a_pool  [num_slots][num_slices][max_rank][k]   bf16
 *    b_pool  [num_slots][out][max_rank]             bf16
 *    scale   [num_slots]     float
 *    slot    [n]             int32
 *    y       [n][ldy]        bf16, columns 0 .. out written
 * The 8-bit form (xq not null): the first sum reads xq [n][ldxq] (e4m3) with
 * x_scale [n] and w with w_scale [out] (float), as
 *    x_scale[i] * w_scale[c] * sum_k xq[i][k] w[c][k];
 * the adapters still read x.  Without it xq, x_scale and w_scale are null.
 * For k > 256 this sum is what the matrix cores' 8-bit product gives: of every
 * 8 consecutive products (k from a multiple of 8) each is first cut towards
 * zero to a multiple of 2^(E - 13), where E is the largest sum of two factors'
 * exponents among the 8 (-6 for a subnormal), and what is left is added in
 * fp32.  A group is so off by less than 2^-10 of its largest product (more if
 * that has a subnormal factor), and a sum by less than its rounding to bf16
 * unless large products cancel in it.  For k <= 256 nothing is cut.
 * slice_sizes is a [host] array of num_slices widths.  The products with
 * b_pool take the fp32 inner sums as two bf16 terms (16 bits of mantissa).
 * An infinity or NaN in an adapter or a row of x reaches no row but its own:
 * in b_pool[s][c] it makes y[i][c] NaN or infinite for the rows of slot s, in
 * x[i] or an inner sum it may do so for any column of that row.
 * Limits: k a multiple of 16 in [16, 1 << 18]; every slice width a multiple
 * of 8; 1 <= num_slices <= 8; out <= 1 << 24; max_rank a multiple of 8 in
 * [8, 128]; 1 <= num_slots <= 8192; n <= 1 << 18; ldx and ldy multiples of 8
 * and ldxq of 16; n * ldx < 1 << 30, n * ldxq < 1 << 31; n * out < 10^11 with
 * xq and k <= 256 (STEP_EUNSUPPORTED past the limits on k, out, max_rank,
 * num_slots, n and the products); every pointer 16-byte aligned, but scales
 * and slot 4-byte.
 */
int step_lora_linear(const uint16_t *x, int64_t ldx, int32_t n, int32_t k, const uint8_t *xq, int64_t ldxq,
                     const float *x_scale, const void *w, const float *w_scale, const uint16_t *a_pool,
                     const uint16_t *b_pool, const float *scale, int32_t num_slots, int32_t num_slices,
                     const int32_t *slice_sizes, int32_t max_rank, const int32_t *slot, uint16_t *y, int64_t ldy,
                     void *ws, size_t ws_bytes, void *stream);

/* Workspace bytes step_token_logprobs needs (0 for a shape that it refuses).
 * They serve every call of the same or smaller n, v and top too. */
size_t step_token_logprobs_workspace_bytes(int32_t n, int32_t v, int32_t top);

/*
 * Log probabilities of given tokens, with entropy and top alternatives.  Per
 * row z of logits ([n][ld], bf16, or float with fp32 != 0) with
 * logp[j] = z[j] - max z - log(sum exp(z - max z)):
 *    logprob  [n]       logp[tokens[i]]
 *    rank     [n]       1 + the number of j with z[j] > z[tokens[i]]
 *    entropy  [n]       -sum_j exp(logp[j]) logp[j]
 *    top_ids, top_logprobs  [n][top]  the `top` largest logits in descending
 *             order, of equal ones the lowest index first; -1 and -infinity
 *             where the row has no further logit above -infinity.  Both null
 *             when top == 0.
 * tokens[i] < 0 asks for no token: logprob 0 and rank 0; tokens[i] >= v gets
 * logprob NaN and rank 0.  A logit of -infinity is a masked token: it has
 * logp -infinity and adds nothing; a row without any other has entropy 0.  A
 * row that holds a NaN or +infinity has NaN log probabilities and entropy.
 * Limits: 1 <= v <= 1 << 20, 0 <= top <= 32, n <= 1 << 16, ld >= v; logits
 * aligned to their own type only.
 */
int step_token_logprobs(const void *logits, int64_t ld, int32_t fp32, int32_t n, int32_t v, const int32_t *tokens,
                        int32_t top, float *logprob, int32_t *rank, float *entropy, int32_t *top_ids,
                        float *top_logprobs, void *ws, size_t ws_bytes, void *stream);

/* A static, human-readable name for a status code. */
const char *step_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* TENANT_STEP_H */
