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
 * holds fewer than 2^32 threads (a row takes 8 to 512: C / 8, rounded up to a
 * power of two, 64 for C from 264 to 2048, 256 to 8192).  Rows
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

#ifdef __cplusplus
}
#endif

#endif /* IGEMM_DECODER_H */
