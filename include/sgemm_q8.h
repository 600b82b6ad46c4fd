/*
 * sgemm_q8.h -- around the feed-forward block: the root-mean-square norm before
 * it, with the residual's addition and its gradient, and products of 8-bit
 * integers for serving it with many rows, whose operands the norm, the gate and
 * the weights are brought into 8 bits for.
 *
 * Conventions are those of sgemm_ffn.h, its workspace of a device and stream among them
 * (of sgemm_rms_norm_backward with dweight and of sgemm_q8_matmul here; a call's first use on a
 * stream may allocate, so run it once before capturing it; graphs captured on one
 * stream share its workspace and run one after the other, not at once).  Element types and
 * activations are the constants declared there.  All results are bitwise reproducible.
 *
 * Rows in 8 bits: a row a[0..n) has one scale and n codes,
 *
 *     top = max(max |a[i]|, 2^-96),  q[i] = round(127 a[i] / top),  a[i] ~ q[i] top / 127
 *
 * round() is to nearest, ties to even; codes lie in -127 .. 127.  The codes are
 * those of exact arithmetic: an element too near a border between two codes for
 * 32 bits, or not finite in them, is decided with about 48 or 53 bits.  A row with an
 * infinity, a NaN or an element (in the norm: of h too) beyond FP32 has the scale NaN and
 * codes of zero.
 */
#ifndef GB300_SGEMM_Q8_H
#define GB300_SGEMM_Q8_H

#include <stddef.h>
#include <stdint.h>

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * sgemm_rms_norm -- per row of x (T x D)
 *
 *     h = x + residual,  y = h * weight / sqrt(mean(h^2) + eps)
 *
 * x, residual, h, y: T x D of `type`, leading dimensions at least D.  residual:
 * NULL, then h = x.  h: NULL, or receives the sum, rounded to `type`; the norm
 * is taken of the sum in 32 bits, before that rounding.  h may be x or residual
 * itself, and so may y (same address and leading dimension), but not both.
 * weight: D elements of weight_type, which is `type` or SGEMM_TYPE_F32.
 * Squares are summed in FP32: where their sum passes its range, y is zero.  eps counts as
 * rounded to FP32.
 * T == 0 or D == 0: nothing is done.
 * Returns SGEMM_ERR_INVALID_ARG for a negative size, a leading dimension below
 * D, a NULL or misaligned pointer, an unknown type, another weight_type or an
 * eps that is negative or NaN; SGEMM_ERR_UNSUPPORTED for a T above 2^31 - 1 or a D above
 * 2^26.
 */
SGEMM_API sgemm_status_t sgemm_rms_norm(int64_t T, int64_t D, int type, const void *x, int64_t ldx,
                                        const void *residual, int64_t ldr, const void *weight,
                                        int weight_type, double eps, void *h, int64_t ldh, void *y,
                                        int64_t ldy, void *stream);

/*
 * sgemm_rms_norm_q8 -- the same with y in 8 bits: q (T x D, ldq >= D) and
 * scales (T floats).  The row that is coded is a = h * weight, whose codes do
 * not depend on the norm; its scale is top / 127 / sqrt(mean(h^2) + eps).  h is
 * added in more bits where a code needs them.  q overlaps no other argument.
 * D == 0: the scales are 2^-96 / 127.
 */
SGEMM_API sgemm_status_t sgemm_rms_norm_q8(int64_t T, int64_t D, int type, const void *x,
                                           int64_t ldx, const void *residual, int64_t ldr,
                                           const void *weight, int weight_type, double eps, void *h,
                                           int64_t ldh, int8_t *q, int64_t ldq, float *scales,
                                           void *stream);

/*
 * sgemm_rms_norm_backward -- gradients of y = h * weight / sqrt(mean(h^2) + eps),
 * h = x + residual
 *
 *     r = 1 / sqrt(mean(h^2) + eps),  n = dy * weight
 *     dx = r (n - h r^2 mean(n h)) + dh,  dweight = sum over rows of dy h r
 *
 * x and residual: as in the forward call, for the gradients at the sum in 32 bits;
 * or x the sum that it stored and residual NULL, which reads less, for the gradients
 * at the rounded sum.  dh: NULL, or the gradient that reaches h otherwise (the
 * residual stream's own).  dx: T x D of `type`, the gradient of x and of the
 * residual alike; it may be dy or dh itself (same address and leading dimension).  dweight: D elements
 * of weight_type.  One of dx and dweight may be NULL.  T == 0: dweight is zero.
 * Sums are held in 32 bits, in an order that depends on sizes and alignment alone:
 * where the squares' passes FP32's range, r counts as zero (dx is dh there, and the row
 * adds nothing to dweight); where that of n h does, dx is not finite.
 * Errors as for the forward call.
 */
SGEMM_API sgemm_status_t sgemm_rms_norm_backward(int64_t T, int64_t D, int type, const void *x,
                                                 int64_t ldx, const void *residual, int64_t ldr,
                                                 const void *weight, int weight_type, double eps,
                                                 const void *dy, int64_t lddy, const void *dh,
                                                 int64_t lddh, void *dx, int64_t lddx,
                                                 void *dweight, void *stream);

/*
 * sgemm_q8_gate -- act(g) * u in 8 bits: what the down product reads.
 * g, u: T x F of `type` (they may be halves of one T x 2F matrix); q: T x F,
 * ldq >= F; scales: T floats.  u NULL: the rows of g itself are coded, and
 * `activation` is not looked at.
 * T == 0: nothing is done.  F == 0: the scales are 2^-96 / 127.
 */
SGEMM_API sgemm_status_t sgemm_q8_gate(int64_t T, int64_t F, int type, int activation,
                                       const void *g, int64_t ldg, const void *u, int64_t ldu,
                                       int8_t *q, int64_t ldq, float *scales, void *stream);

/*
 * sgemm_q8_quantize -- a K x N matrix W of `type` (ldw >= N) in 8 bits, channel
 * by channel: q: N x K, row n the codes of column n of W (ldq >= K); scales: N
 * floats.
 */
SGEMM_API sgemm_status_t sgemm_q8_quantize(int64_t N, int64_t K, int type, const void *W,
                                           int64_t ldw, int8_t *q, int64_t ldq, float *scales,
                                           void *stream);

/*
 * sgemm_q8_matmul -- y = (x Wq^T) scaled for each token and channel
 *
 *     y[m][n] = x_scales[m] * w_scales[n] * sum over k of x[m][k] * w[n][k]
 *
 * x: M x K (ldx >= K), w: N x K (ldw >= K), 8-bit integers, all 256 values of them;
 * x_scales: M floats; w_scales: N floats; y: M x N of `type` (ldy >= N).  The
 * sum is exact, and is rounded to FP32 once; its two scalings (x's first, in FP32) and y's
 * rounding follow.  16-byte aligned w whose rows lie a multiple of 16 bytes apart is read in
 * place, other w through a copy made by every call.
 * M == 0 or N == 0: nothing is done.  K == 0: y = 0.
 * Returns SGEMM_ERR_INVALID_ARG for a negative size, a leading dimension below
 * its row length, a NULL or misaligned pointer or an unknown type;
 * SGEMM_ERR_UNSUPPORTED for a K above 131071 (beyond it a sum could pass 32 bits) or
 * an M or N above 2^26.
 */
SGEMM_API sgemm_status_t sgemm_q8_matmul(int64_t M, int64_t N, int64_t K, int type, const int8_t *x,
                                         int64_t ldx, const float *x_scales, const int8_t *w,
                                         int64_t ldw, const float *w_scales, void *y, int64_t ldy,
                                         void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GB300_SGEMM_Q8_H */
