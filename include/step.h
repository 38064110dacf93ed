/*
 * step.h -- C ABI of the operators a serving step runs around the routed LoRA
 * delta on MI355X (gfx950): the norm in front of a projection, the shared
 * projection with every request's adapter added to it, the paged cache of keys
 * and values with the attention that reads it, and the log probabilities of the
 * answered tokens.  Library: libstep.so.
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

/*
 * The paged cache of keys and values: two arrays of the same shape [pages][page]
 * [kv_heads][dim] and the same strides (page_stride, token_stride and
 * head_stride, in elements; dim is contiguous), in bf16 or, with k_scale and
 * v_scale ([kv_heads], float, at least 0), in e4m3, a stored value times its
 * head's scale being the value.  A token's place is page number * page + place
 * in the page.  dim is a multiple of 16 in [16, 256]; heads a multiple of
 * kv_heads, at most 64 times and at most 4096; strides multiples of 8 (of 16 in
 * e4m3), at least dim, below 1 << 35, and free where the axis has length 1; both
 * arrays 16-byte aligned; pages * page < 1 << 31.
 */

/* The most tokens of a call, and the most requests and prefixes. */
#define STEP_MAX_TOKENS (1 << 20)
#define STEP_MAX_REQUESTS (1 << 16)

/*
 * Tokens' keys and values into the cache, the keys and the queries turned by
 * their positions' angles on the way.  For token t with row
 * (cos_0 .. cos_{rot/2-1}, sin_0 .. sin_{rot/2-1}) of rotation at positions[t],
 * in every head of q and k and for i < rot / 2
 *     (a, b) -> (a cos_i - b sin_i, b cos_i + a sin_i)
 * where (a, b) are the columns (i, i + rot / 2) or, with neighbours != 0,
 * (2 i, 2 i + 1); columns from rot on stay as they are.  In fp32, rounded once.
 *    q      [n][ldq], heads * dim used columns, or null with q_out
 *    k, v   [n][ldk], [n][ldv], kv_heads * dim used columns
 *    positions [n], rotation [rotation_rows][rot] (not read with rot == 0)
 *    place  [n]; a token whose place is not in the cache is not stored
 *    q_out  [n][ldo]; may be q itself (then ldo == ldq)
 * In e4m3 a value over its head's scale is rounded to nearest, and to +-448 where
 * it is larger; over a scale of 0 a 0 is stored as 0, any other as +-448.  A position outside the rotation makes the token's q NaN, and the
 * token is not stored.  Where two tokens have one place, each 16 values (8 in
 * bf16) of it are one of the two's.  Limits: n <= STEP_MAX_TOKENS; rot a multiple
 * of 16, at most dim; leading dimensions multiples of 8; q, k, v, q_out and
 * rotation 16-byte aligned.
 */
int step_kv_append(const uint16_t *q, int64_t ldq, const uint16_t *k, int64_t ldk, const uint16_t *v, int64_t ldv,
                   int32_t n, int32_t heads, int32_t kv_heads, int32_t dim, const int32_t *positions,
                   const float *rotation, int32_t rotation_rows, int32_t rot, int32_t neighbours, const int32_t *place,
                   void *k_cache, void *v_cache, int64_t page_stride, int64_t token_stride, int64_t head_stride,
                   int32_t pages, int32_t page, const float *k_scale, const float *v_scale, uint16_t *q_out,
                   int64_t ldo, void *stream);

/* Workspace bytes step_paged_attention needs (0 for a shape that it refuses).
 * They serve every call of the same heads and dim with at most n rows, with
 * prefixes only if prefixes > 0 here.  Of this workspace only the first
 * STEP_ATTENTION_ZEROED bytes need the zero fill. */
#define STEP_ATTENTION_ZEROED 4096
size_t step_paged_attention_workspace_bytes(int32_t n, int32_t heads, int32_t kv_heads, int32_t dim,
                                            int32_t prefixes);

/*
 * Attention of a batch of requests over the paged cache.  Request b has the
 * rows starts[b] .. starts[b + 1] of q (row b alone without starts) and its keys
 * 0 .. lens[b], key j in place j % page of page table[b][j / page].  For row i
 * and head h, with the keys and values of head h / (heads / kv_heads),
 *     out[i][h] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q[i][h] k_j)
 *     lse[i][h] = ln sum_j p_j                                  (if not null)
 * over the request's keys; with causal != 0 the request's rows are its last
 * tokens, so the t-th of r rows sees keys j <= lens[b] - r + t.
 * Prefixes: the requests prefix_starts[p] .. prefix_starts[p + 1] share the
 * prefix_lens[p] keys on the pages prefix_table[p], which all their rows see
 * before their own keys; requests before the first group and behind the last
 * have no prefix.  Each prefix is read once for all its requests.
 *    q [n][ldq], out [n][ldo], heads * dim used columns; lse [n][heads]
 *    starts [requests + 1] and prefix_starts [prefixes + 1] ascending
 *    table, prefix_table  rows ld_table and ld_prefix_table apart, which do not overlap
 *    max_rows   the most rows of a request; it decides only which kernel runs
 * Rows that belong to no request stay as they are.  A row without keys gets 0
 * and lse -infinity; one that sees keys whose scale is NaN or infinite gets NaN.
 * Keys on a page number that the cache does not have count as absent, lengths end
 * with the table.  A key whose score is -infinity weighs nothing, and a row all of
 * whose keys are such is one without keys; but an infinity or NaN among the values
 * of a key makes that column infinite or NaN in every row that sees the key, and in
 * no other.  Products in bf16 with fp32 sums, p rounded to bf16 before its product
 * with v, one rounding of the result; the sums of p v have to stay within fp32 with
 * p up to 2^8.  The same call on the same inputs gives the same bits.  Other sizes,
 * max_rows or widths of the tables, other lengths or values of the batch may change
 * the order of a row's sums, and so its last bits.
 * Limits: n <= STEP_MAX_TOKENS; requests, prefixes <= STEP_MAX_REQUESTS;
 * table_cols * page and prefix_cols * page <= 1 << 24; leading dimensions of q
 * and out multiples of 8; q, out and ws 16-byte aligned; scale in [1e-30, 1e30].
 */
int step_paged_attention(const uint16_t *q, int64_t ldq, int32_t n, int32_t requests, int32_t heads, int32_t kv_heads,
                         int32_t dim, const void *k_cache, const void *v_cache, int64_t page_stride,
                         int64_t token_stride, int64_t head_stride, int32_t pages, int32_t page, const float *k_scale,
                         const float *v_scale, const int32_t *table, int64_t ld_table, int32_t table_cols,
                         const int32_t *lens, const int32_t *starts, int32_t max_rows, int32_t causal, float scale,
                         int32_t prefixes, const int32_t *prefix_table, int64_t ld_prefix_table, int32_t prefix_cols,
                         const int32_t *prefix_lens, const int32_t *prefix_starts, uint16_t *out, int64_t ldo,
                         float *lse, void *ws, size_t ws_bytes, void *stream);

/* A static, human-readable name for a status code. */
const char *step_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* TENANT_STEP_H */
