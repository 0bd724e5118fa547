/*
 * igemm_decoder.h -- the operators of a decoder block around the attention of
 * igemm_attn.h, on MI355X (gfx950), behind the same C ABI: layer norm with its
 * gradient, the product in 8-bit integers of a projection, the paged cache of
 * keys and values held in 8 bits, and the attention of new tokens over that
 * cache.
 *
 * Conventions as in igemm_attn.h (device pointers to caller-owned memory,
 * asynchronous work on the given stream, no exceptions, thread-safe; 1 =
 * handled, 0 = declined, -(hipError_t) otherwise; workspace NULL: taken
 * stream-ordered and released on the same stream).  Elements are
 * IGC_DTYPE_BF16 or IGC_DTYPE_FP16; sums and statistics are held in fp32, and
 * each output is rounded once to nearest even.
 *
 * Rows in 8 bits.  A row x of n values (a token's channels, a head of a token)
 * is held as integers q and one fp32 scale s:
 *   m = max |x|,   s = m / 127 (rounded to fp32),   q_i = round(127 x_i / m)
 * with ties to even, exactly (the quotient is never rounded first).  A row
 * whose m is below 2^-110 has s = 0 and q = 0; a row that holds an infinity
 * or a NaN has s = NaN and q = 0, so that it stays recognisable.  The value
 * held is q_i s.
 */
#ifndef IGEMM_DECODER_H
#define IGEMM_DECODER_H

#include <stddef.h>
#include <stdint.h>

#include "igemm_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Layer norm of rows of C = channels values, with w = weight (or 1) and b =
 * bias (or 0):
 *   mean = sum x / C,  r = 1 / sqrt(sum (x - mean)^2 / C + eps)
 *   xh = (x - mean) r,  y = xh w + b
 * Backward, from grad = dy and the forward's x (no statistics are kept):
 *   u = dy w,  dx = r (u - mean(u) - xh mean(u xh))
 *   dweight = sum over rows of dy xh,  dbias = sum over rows of dy
 * the last two in fp32, summed in a fixed order; NULL: not wanted; zeros
 * without rows.
 *   x, out, grad  [n0, n1, n2, C], C adjacent, any alignment of the element
 *                 type; strides not negative, inputs may have stride 0
 *   out           y, or dx; may be x (forward) or grad (backward) exactly,
 *                 otherwise the ranges may not meet
 *   weight, bias  fp32 [C] or NULL
 * Limits: C from 1 to 16384, fewer than 2^31 rows, strides below 2^40; a launch
 * holds fewer than 2^32 threads (a row takes 8 to 64 of them up to 2048
 * channels, 256 up to 6144, 512 past that).  Rows
 * whose squares overflow fp32 (magnitudes past 1e19 / sqrt(C)) give 0 or NaN.
 */
typedef struct igc_layer_norm {
    int64_t n[3], channels;
    igc_attn_view x, grad, out;   /* strides of the axes n0, n1, n2 */
    const float *weight, *bias;
    float *dweight, *dbias;       /* backward only */
    double eps;
    int64_t dtype;
    void* workspace;              /* backward with a dweight or dbias */
    size_t workspace_bytes;
} igc_layer_norm;

int32_t layer_norm_fwd(const igc_layer_norm* args, void* stream);
int32_t layer_norm_bwd(const igc_layer_norm* args, void* stream);

/* Host-only gates (pointers compared, never dereferenced). */
int32_t layer_norm_fwd_check(const igc_layer_norm* args);
int32_t layer_norm_bwd_check(const igc_layer_norm* args);

/* Workspace of layer_norm_bwd: the workgroups' partial gradients of weight
 * and bias (0 without them, or for sizes that would be declined). */
size_t layer_norm_bwd_workspace_bytes(const igc_layer_norm* args);

/*
 * Rows of x in 8 bits (the definition at the top): x [n0, n1, n2, C] as in
 * igc_layer_norm, q int8 [n0, n1, n2, C] with the strides of its view in
 * bytes, scale fp32 [n0, n1, n2], dense.
 * q's pointer and strides are multiples of 16 bytes; bytes between C and the
 * next row are not written.
 * Limits: C from 1 to 131071, fewer than 2^31 rows, launches as in
 * igc_layer_norm (past 16384 values 512 threads a row).
 */
typedef struct igc_quantize_rows {
    int64_t n[3], channels;
    igc_attn_view x, q;
    float* scale;
    int64_t dtype;               /* of x */
} igc_quantize_rows;

int32_t quantize_rows(const igc_quantize_rows* args, void* stream);
int32_t quantize_rows_check(const igc_quantize_rows* args);

/*
 * Product of rows in 8 bits: for x int8 [m][k] with a scale a row (a token) and
 * w int8 [n][k] with a scale a row (an output channel),
 *   y[i][j] = (sum_k x[i][k] w[j][k]) x_scale[i] w_scale[j] + bias[j]
 * The integer sums are exact; scales and bias enter in fp32, x_scale first: a
 * sum times x_scale that passes 2^128 is infinite, whatever w_scale is (an
 * x_scale up to 2^96, rows of values up to 2^102, never does).
 *   x, w     pointers and row pitches (bytes) are multiples of 16; a row's last
 *            16-byte piece is read whole, its bytes past k do not matter.
 *            Every int8 value is allowed, -128 too
 *   x_scale  fp32 [m], w_scale fp32 [n], bias fp32 [n] or NULL
 *   y        dtype (bf16 or fp16) [m][n], any row pitch (elements) from n on,
 *            and any alignment of the type
 * Limits: k from 0 to 131071, m and n below 2^31, pitches of x and w below 2^22
 * and of y below 2^40; a launch holds fewer than 2^32 threads (256 for
 * every 16 columns of at most 32 rows, or for a tile of 256 x 256, 128 x 128 or
 * 64 x 64, the largest that fills the card).
 */
typedef struct igc_linear_i8 {
    int64_t m, n, k;
    const int8_t* x;
    int64_t x_pitch;
    const int8_t* w;
    int64_t w_pitch;
    const float *x_scale, *w_scale, *bias;
    void* y;
    int64_t y_pitch;
    int64_t dtype;               /* of y */
} igc_linear_i8;

int32_t linear_i8(const igc_linear_i8* args, void* stream);
int32_t linear_i8_check(const igc_linear_i8* args);

/*
 * The paged cache of keys and values in 8 bits.  A pool holds `pages` pages of
 * page_tokens tokens; k and v are int8 [pages][kv_heads][page_tokens][Dp],
 * Dp = head_dim rounded up to 16, k_scale and v_scale fp32
 * [pages][kv_heads][page_tokens]: one row in 8 bits (the definition at the
 * top) a head of a token.  Sequence b's token at position p is token
 * p % page_tokens of page table[b][p / page_tokens].  Several sequences may
 * share pages.
 * Limits: page_tokens 16, 32, ... 1024 (a power of two), head_dim a multiple
 * of 8 up to 128, pools 16-byte aligned, pages and kv_heads below 2^31, at
 * most 2^40 rows.
 */
typedef struct igc_kv_cache {
    int8_t *k, *v;
    float *k_scale, *v_scale;
    int64_t pages, page_tokens, kv_heads, head_dim;
} igc_kv_cache;

/*
 * Writing and reading back.  Token i < min(lens[b], tokens) of sequence b has
 * the position start[b] + i.
 *   k, v     16-bit [batch, tokens, kv_heads, head_dim], views as in
 *            igemm_attn.h: inputs of kv_cache_write, outputs of kv_cache_read
 *   table    int32 rows of table_entries at table_stride elements
 *   start    int32 [batch];  lens int32 [batch] or NULL (tokens)
 * kv_cache_write leaves everything else of the pool as it was; tokens whose
 * position is negative or past the table, or whose page is not one of the
 * pool, are not written (a negative page number so leaves a page out).  A
 * place that one call writes twice (a page shared by sequences that both
 * write to it) holds a mix of the two rows afterwards.
 * kv_cache_read writes all of k and v: zeros at i >= lens[b], NaN where the
 * position or the page does not exist.  k and v may interleave in one buffer,
 * with the same strides, and not share an element.
 * Limits: batch, tokens below 2^31; a launch holds one group of 4 to 16 lanes
 * (head_dim / 8, rounded up to a power of two) for every four heads of a
 * token, of keys and of values, a sequence's tokens rounded up to a workgroup
 * of 256 lanes, and fewer than 2^32 threads.
 */
typedef struct igc_kv_io {
    igc_kv_cache cache;
    int64_t batch, tokens;
    igc_attn_view k, v;
    const int32_t* table;
    int64_t table_stride, table_entries;
    const int32_t *start, *lens;
    int64_t dtype;
} igc_kv_io;

int32_t kv_cache_write(const igc_kv_io* args, void* stream);
int32_t kv_cache_write_check(const igc_kv_io* args);
int32_t kv_cache_read(const igc_kv_io* args, void* stream);
int32_t kv_cache_read_check(const igc_kv_io* args);

/*
 * Attention of new tokens over the cache.  q, out [batch, q_len, q_heads,
 * head_dim], kv_heads dividing q_heads; lens int32 [batch]: the tokens that a
 * sequence holds, at positions 0 .. lens[b] - 1 (a negative length is 0;
 * positions past the table are not attended to).  With causal != 0 the new
 * tokens are the last q_len of the lens[b]: token i attends to positions below
 * lens[b] - (q_len - 1 - i).  With the values held, k_j and v_j, and as in
 * cross_attn_fwd:
 *   s_j = scale * q . k_j,  lse = log sum_j exp(s_j),  out = sum_j p_j v_j
 * A row that attends to nothing has out = 0 and lse = -inf; one that attends
 * to a page outside the pool is NaN, and so is one whose scores are all -inf.
 * Positions that a row does not attend to never enter its sums, whatever the
 * pool holds there.
 *   lse  fp32 [batch, q_heads, q_len], dense, or NULL
 * The integers enter the matrix products as they are; p_j times the value's
 * scale is held in 16 significant bits, sums in fp32.  Scores, q . K_j of the
 * integers (queries up to 2^113) and sums of p_j v_j (values up to 2^119 /
 * lens[b]) have to stay within fp32's range; past it rows are infinite or NaN.
 * Sequences of more than 640 tokens (by the table's capacity) may be read by
 * several workgroups, whose results (fp32, in the workspace) a second launch
 * joins in a fixed order: results do not change from run to run.
 * Limits: as cross_attn_fwd for q and out; the table's capacity below
 * 2^31 - 4096, batch * q_heads below 2^31, batch * kv_heads times the tiles of
 * 32 rows (q_len * q_heads / kv_heads) below 2^23.
 */
typedef struct igc_cache_attn {
    igc_kv_cache cache;
    int64_t batch, q_len, q_heads;
    igc_attn_view q, out;
    float* lse;
    const int32_t* table;
    int64_t table_stride, table_entries;
    const int32_t* lens;
    int64_t causal;
    double scale;
    int64_t dtype;
    void* workspace;
    size_t workspace_bytes;
} igc_cache_attn;

int32_t cache_attn_fwd(const igc_cache_attn* args, void* stream);
int32_t cache_attn_fwd_check(const igc_cache_attn* args);
size_t cache_attn_fwd_workspace_bytes(const igc_cache_attn* args);

#ifdef __cplusplus
}
#endif

#endif /* IGEMM_DECODER_H */
