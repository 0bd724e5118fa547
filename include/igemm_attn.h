/*
 * igemm_attn.h -- the attention block that stands between convolution layers,
 * on MI355X (gfx950), behind the same C ABI as igemm_conv.h: attention of a
 * map's pixels (or of decoded tokens) to an encoder's states of another
 * length, forward and backward, and the per-head norm of queries and keys
 * with the position rotation, forward and backward.
 *
 * An NHWC tensor [N, H, W, heads * D], as the convolutions write it, is the
 * query tensor [batch = N, token = H*W, head, D] of these operators without a
 * copy.
 *
 * Conventions, beyond those of igemm_conv.h (device pointers to caller-owned
 * memory, asynchronous work on the given stream, no exceptions, thread-safe):
 *   - A tensor is an igc_attn_view: a pointer and the strides of its batch,
 *     token and head axes in elements; the D values of a head are adjacent.
 *     Pointers and strides are multiples of 16 bytes (8 elements).  Strides
 *     are not negative; inputs may have stride 0 (one encoder's states shared
 *     by a whole batch), outputs may not overlap themselves.  The range from
 *     an output's first to its last element must not meet an input's.
 *   - Every entry returns 1 = handled (work enqueued, or nothing to do), 0 =
 *     declined (nothing enqueued; the _check function gives the reason, an
 *     IGC_DECLINE_* code), or -(hipError_t).
 *   - The element type is IGC_DTYPE_BF16 or IGC_DTYPE_FP16 for all tensors;
 *     products accumulate, and softmax statistics, norms and sums are held,
 *     in fp32, and each output is rounded once to nearest even.
 *   - workspace may be NULL: it is then taken stream-ordered from
 *     hipMallocAsync and released on the same stream.
 */
#ifndef IGEMM_ATTN_H
#define IGEMM_ATTN_H

#include <stddef.h>
#include <stdint.h>

#include "igemm_conv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Decline reasons of these operators, after those of igemm_conv.h. */
enum {
    IGC_DECLINE_HEAD_DIM = 15,  /* D not one of 8, 16, ... 128; for the norm an
                                   odd or too large number of rotated values */
    IGC_DECLINE_SCALE = 16      /* scale below 1e-30, or scale * log2(e) not
                                   finite in fp32; eps negative or not finite */
};

typedef struct igc_attn_view {
    void* data;
    int64_t batch, token, head;   /* strides, elements */
} igc_attn_view;

/*
 * Cross attention.  For query token i and head h of batch b, over the valid
 * keys j of head h / (q_heads / kv_heads):
 *   valid:  j < min(kv_lens[b], kv_len)  and  key_mask[b][j] != 0
 *   s_j = scale * q . k_j,   lse = log sum_j exp(s_j),   p_j = exp(s_j - lse)
 *   out = sum_j p_j v_j
 * A row without a valid key has out = 0 and lse = -inf.  The key and value
 * rows of keys that are not valid never enter a sum (they may hold NaN).
 *   q, out   [batch, q_len, q_heads, head_dim];  k, v [batch, kv_len,
 *            kv_heads, head_dim], kv_heads dividing q_heads
 *   lse      fp32 [batch, q_heads, q_len], dense, or NULL when no backward
 *            pass follows
 *   kv_lens  int32 [batch] or NULL (kv_len; a negative length is 0)
 *   key_mask bytes, rows of kv_len at key_mask_stride bytes, or NULL
 * The probabilities are rounded to the element type before their product
 * with v, which accumulates in fp32; their sum is taken before the rounding.
 * Few rows over many keys run as several workgroups per row block whose
 * partial results (fp32, in the workspace) a second launch joins in a fixed
 * order: results do not change from run to run.
 * Limits: kv_len and batch * heads below 2^31, q_len * q_heads / kv_heads
 * below 2^29; token strides of q, k, v, out (and of the gradients), and head
 * strides of q and out (dout, dq), below 2^23 elements; of these 65 token
 * strides and the strides over the heads of a group together below 2^31
 * bytes.  Batch strides, and head strides of k and v (dk, dv), below 2^40.  A
 * launch holds fewer than 2^32 threads: with at most 32 rows (q_len * q_heads
 * / kv_heads) batch * kv_heads is below 2^23; with more, batch * kv_heads times
 * the tiles of 128 rows is below 2^24 (with at most 128 keys, where workgroups
 * walk their rows, batch * kv_heads alone for large batches).
 */
typedef struct igc_cross_attn {
    int64_t batch, q_len, kv_len, q_heads, kv_heads, head_dim;
    igc_attn_view q, k, v, out;
    float* lse;
    const int32_t* kv_lens;
    const uint8_t* key_mask;
    int64_t key_mask_stride;
    double scale;
    int64_t dtype;
    void* workspace;
    size_t workspace_bytes;
} igc_cross_attn;

int32_t cross_attn_fwd(const igc_cross_attn* args, void* stream);

/* Host-only gate of cross_attn_fwd (pointers compared, never dereferenced). */
int32_t cross_attn_fwd_check(const igc_cross_attn* args);

/* Workspace of cross_attn_fwd: the partial results of calls with few rows,
 * else 0 (also for arguments that would be declined; pointers play no part). */
size_t cross_attn_fwd_workspace_bytes(const igc_cross_attn* args);

/*
 * Gradients of cross attention from dout, the gradient at out, with out and
 * lse as cross_attn_fwd left them:
 *   Delta = dout . out,  dp_j = dout . v_j,  ds_j = p_j (dp_j - Delta)
 *   dq = scale sum_j ds_j k_j,  dk_j = scale sum ds_j q,  dv_j = sum p_j dout
 * the last two summed over the query tokens and over the query heads that
 * share a key head.  Gradients of keys that are not valid are 0.  k and v
 * that several batch entries share through stride 0 still get one dk and dv
 * an entry.  dq.data may be NULL, or dk.data and dv.data both (not wanted).
 *   fwd    the forward's arguments, out and lse now inputs, and the
 *          workspace of this call
 * ds and p are rounded to the element type before their products, which
 * accumulate in fp32 (for fp16 scaled by powers of two that keep them in
 * range).  Sums are taken in a fixed order.  Limits as the forward, and batch *
 * kv_heads times the tiles of 128 keys below 2^23.  dq, dk and dv may
 * interleave in one buffer, provided no element belongs to two of them.
 */
typedef struct igc_cross_attn_grad {
    igc_cross_attn fwd;
    igc_attn_view dout, dq, dk, dv;
} igc_cross_attn_grad;

int32_t cross_attn_bwd(const igc_cross_attn_grad* args, void* stream);

/* Host-only gate of cross_attn_bwd (pointers compared, never dereferenced). */
int32_t cross_attn_bwd_check(const igc_cross_attn_grad* args);

/* Workspace of cross_attn_bwd: row statistics, and partial sums where few
 * keys or rows are split over workgroups (0 for arguments that would be
 * declined; pointers play no part). */
size_t cross_attn_bwd_workspace_bytes(const igc_cross_attn_grad* args);

/*
 * Norm of queries and keys per head with the position rotation in the same
 * pass.  Every head's D values x of every token, with w = weight (or 1):
 *   r = 1 / sqrt(mean(x^2) + eps),   n_d = x_d * r * w_d
 * and the first rot_dim = R values turn in pairs by the angles of one table
 * row, (a, b) = (i, i + R/2), or (2i, 2i + 1) when interleaved, i < R/2:
 *   y_a = n_a cos_i - n_b sin_i,   y_b = n_b cos_i + n_a sin_i
 * (y = n past R).  The table holds fp32 rows {cos_0 .. cos_{R/2-1}, sin_0 ..};
 * any angles do (one axis, or the rows and columns of a map).  Token t of
 * batch b uses row positions[b][t], or row t when positions is NULL (then
 * table_rows >= tokens); the outputs of a token whose position is outside the
 * table are NaN.  R = 0 is the norm alone (table may be NULL).
 * One call takes the queries and the keys (either may be empty: batch 0), of
 * different lengths and head counts, in one launch.
 * Backward, from grad = dy and the forward's x: out = dx and
 *   dweight[d] = sum over tokens and heads of (R^T dy)_d x_d r
 * (fp32, summed in a fixed order; NULL: not wanted; zeros for an empty part).
 * Accumulation is fp32, one rounding at the end.  out may be x (forward) or
 * grad (backward) exactly; otherwise the ranges may not meet.  With both
 * parts in place the two may interleave in one buffer, provided no element
 * belongs to both.
 * Limits: each axis below 2^31 and batch * tokens * heads below 2^40; the
 * forward launches one workgroup for every 8192 values, heads rounded up to a
 * multiple of four and D to 32, 64 or 128, and fewer than 2^24 of them.
 */
typedef struct igc_qk_part {
    int64_t batch, tokens, heads;
    igc_attn_view x, grad, out;
    const float* weight;          /* [D] or NULL */
    float* dweight;               /* [D] or NULL; backward only */
    const float* table;           /* [table_rows][R] */
    int64_t table_rows;
    const int32_t* positions;     /* [batch][tokens] or NULL */
    int64_t positions_stride;     /* elements between batches (0: shared) */
} igc_qk_part;

typedef struct igc_qk_norm {
    igc_qk_part q, k;
    int64_t head_dim, rot_dim, interleaved, dtype;
    double eps;
    void* workspace;              /* backward with a dweight */
    size_t workspace_bytes;
} igc_qk_norm;

int32_t qk_norm_rope_fwd(const igc_qk_norm* args, void* stream);
int32_t qk_norm_rope_bwd(const igc_qk_norm* args, void* stream);

/* Host-only gates (pointers compared, never dereferenced). */
int32_t qk_norm_rope_fwd_check(const igc_qk_norm* args);
int32_t qk_norm_rope_bwd_check(const igc_qk_norm* args);

/* Workspace of qk_norm_rope_bwd: the workgroups' partial weight gradients
 * (0 without a dweight, or for arguments that would be declined). */
size_t qk_norm_rope_bwd_workspace_bytes(const igc_qk_norm* args);

#ifdef __cplusplus
}
#endif

#endif /* IGEMM_ATTN_H */
