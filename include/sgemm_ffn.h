/*
 * sgemm_ffn.h -- the feed-forward block of a language model on top of the
 * GEMM library: the gated block with its backward pass, products with 4-bit
 * weights for serving it token by token, and the AdamW step that trains it.
 * (The pages behind sgemm.h have no counterpart; "GEMM from Scratch", end of
 * Module 08, "When to just call the library", names fusing what follows a
 * product into it as the reason to write one's own.)
 *
 * Conventions are those of sgemm.h: row-major matrices with a leading
 * dimension in elements, device pointers owned by the caller, work queued on
 * `stream` without host synchronisation, workspace kept per (device, stream)
 * until sgemm_release_workspace() (what a captured graph holds of it too, when
 * a larger call outgrows it), errors returned before any work is queued, a bounded device wait that gave up reported by
 * sgemm_device_status().  A pointer has to be aligned to its element's size;
 * 16-byte aligned pointers whose rows lie a multiple of 16 bytes apart take
 * the fastest path.  For given sizes, leading dimensions and alignment the
 * results are bitwise reproducible.
 */
#ifndef GB300_SGEMM_FFN_H
#define GB300_SGEMM_FFN_H

#include <stddef.h>
#include <stdint.h>

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
enum {
    SGEMM_TYPE_F32 = 0,
    SGEMM_TYPE_F16 = 1,
    SGEMM_TYPE_BF16 = 2
};

/* The gate's activation. */
enum {
    SGEMM_GATE_SILU = 0, /* g / (1 + exp(-g))                                          */
    SGEMM_GATE_GELU = 1, /* g/2 * (1 + tanh(sqrt(2/pi) * (g + 0.044715 g^3)))           */
    SGEMM_GATE_RELU = 2  /* g > 0 ? g : 0; its derivative at 0 is 0                     */
};

/*
 * sgemm_ffn_forward -- the gated feed-forward block
 *
 *     g = x Wg,  u = x Wu,  h = act(g) * u,  y = h Wd
 *
 * x: T x D (ldx >= D); Wg, Wu: D x F (ldg, ldu >= F; they may be the halves of
 * one D x 2F matrix); Wd: F x D (ldd >= D); y: T x D (ldy >= D), not
 * overlapping any input.  All matrices are of `type` (SGEMM_TYPE_*); sums are
 * held in 32 bits.  With FP32 nothing is rounded below 24 bits.  With 16-bit
 * types h is rounded to the type between the two products, as the second one's
 * operand: an FP16 h above 65504 becomes infinite there, and its row of y with it.
 * Only the form for few rows keeps h in 32 bits; calls without `saved` take it
 * up to T = 24 with FP32, and with 16-bit types up to T = 4 where D F > 6 * 2^20
 * and the three weights lie in 16-byte aligned rows, else up to T = 8.
 * Infinities and NaN in x reach their own rows of y alone.  With FP32 on the tensor
 * cores (above T = 24, with `saved`, and in the backward pass) an infinite element
 * is NaN in every sum that it enters: values are taken in parts there, and
 * infinity times the zero part of another value is NaN.
 * saved: NULL, or a device buffer (16-byte aligned) of sgemm_ffn_saved_floats(T, F,
 * type) floats for sgemm_ffn_backward: it receives u act'(g) and act(g) in 32
 * bits and h, in a layout of the library's own.
 * T == 0 or D == 0: nothing is done.  F == 0: y = 0.
 * Returns SGEMM_ERR_INVALID_ARG for a negative size, a leading dimension below
 * its row length, a NULL or misaligned pointer, an unknown type or activation;
 * SGEMM_ERR_UNSUPPORTED for a T, D or F above 2^26.
 */
SGEMM_API sgemm_status_t sgemm_ffn_forward(int64_t T, int64_t D, int64_t F, int type, int activation,
                                           const void *x, int64_t ldx, const void *Wg, int64_t ldg,
                                           const void *Wu, int64_t ldu, const void *Wd, int64_t ldd,
                                           void *y, int64_t ldy, float *saved, void *stream);

/* Floats of the `saved` buffer for T rows of F columns (0 for invalid sizes or
 * an unknown type).  FP32 needs the most. */
SGEMM_API int64_t sgemm_ffn_saved_floats(int64_t T, int64_t F, int type);

/*
 * sgemm_ffn_backward -- gradients of the block for dy (T x D, lddy >= D):
 *
 *     dh = dy Wd^T,  dg = dh * u * act'(g),  du = dh * act(g)
 *     dx = dg Wg^T + du Wu^T,  dWg = x^T dg,  dWu = x^T du,  dWd = h^T dy
 *
 * The first arguments are those of the forward call.  saved: the buffer the
 * forward call filled from the same x, Wg and Wu, or NULL: then its contents
 * are computed again.  dx: T x D, dWg and dWu: D x F, dWd: F x D, written whole.
 * dx may be NULL (no gradient of the input), and so may dWg, dWu and dWd, all
 * three together (frozen weights).  With 16-bit types h, dg and du are
 * rounded to the type before they enter the products.  In FP16 they are infinite
 * above 65504, lose bits below 2^-14 and are zero below 2^-25, whatever the sizes
 * of the gradients that they add up to: with small dy, scale dy up by a power of
 * two and the gradients down again (loss scaling; the AdamW step's grad_scale).
 * T == 0: the weight gradients are zero.  Errors as for the forward call.
 */
SGEMM_API sgemm_status_t sgemm_ffn_backward(int64_t T, int64_t D, int64_t F, int type,
                                            int activation, const void *x, int64_t ldx,
                                            const void *Wg, int64_t ldg, const void *Wu,
                                            int64_t ldu, const void *Wd, int64_t ldd,
                                            const void *dy, int64_t lddy, const float *saved,
                                            void *dx, int64_t lddx, void *dWg, int64_t lddg,
                                            void *dWu, int64_t lddu, void *dWd, int64_t lddd,
                                            void *stream);

/*
 * sgemm_w4_matvec -- y = x W with 4-bit weights, for a few rows of x
 *
 *     W[k][n] = scales[k / group][n] * (q[k][n] - z[k / group][n])
 *
 * x: M x K, y: M x N, scales: ceil(K / group) x N, all of `type`.  qweight:
 * ceil(K / 8) x N 32-bit words (ldq >= N); bits 4i to 4i + 3 of word (r, n)
 * are q[8 r + i][n]; what the last row of words holds beyond K is ignored.
 * zeros: NULL (every z is 8), or ceil(K / group) x N bytes of which the low
 * four bits are read (ldz >= N).  group: a multiple of 32.
 * x enters with all its bits; sums are held in 32 bits, and each group's sum is
 * scaled in 32 bits.  With FP32 x the products are those of x and q - z.  With
 * 16-bit x they are those of x and q (FP16) or 128 + q (BF16), and the offset's
 * part comes off at the end of a group: at most two (FP16) or five (BF16) of the
 * 24 bits of a group's sum go with it, an infinity in x gives NaN where its
 * q - z would give an infinity, and in BF16 143 times the group's sum of |x| has
 * to stay within FP32.  Weights are read once per 16 rows of x (8 with FP32).
 * M == 0 or N == 0: nothing is done.  K == 0: y = 0.
 * Returns SGEMM_ERR_INVALID_ARG for a negative size, a group that is not a
 * positive multiple of 32, a leading dimension below its row length, a NULL or
 * misaligned pointer or an unknown type; SGEMM_ERR_UNSUPPORTED for an N or K
 * above 2^30 or M above 2^20.
 */
SGEMM_API sgemm_status_t sgemm_w4_matvec(int64_t M, int64_t N, int64_t K, int64_t group, int type,
                                         const void *x, int64_t ldx, const uint32_t *qweight,
                                         int64_t ldq, const void *scales, int64_t lds,
                                         const uint8_t *zeros, int64_t ldz, void *y, int64_t ldy,
                                         void *stream);

/*
 * sgemm_w4_quantize -- 4-bit weights of a K x N matrix W of `type`, group by
 * group of a column, in the layout of sgemm_w4_matvec.
 *
 * zeros != NULL: lo = min(w, 0), hi = max(w, 0) over the group,
 *   scale = (hi - lo) / 15, z = round(-lo / scale), q = clamp(round(w / scale) + z, 0, 15).
 * zeros == NULL: scale = max |w| / 7, q = clamp(round(w / scale) + 8, 0, 15).
 * The scale is rounded to `type` before it divides.  A group of zeros has
 * scale 0 and q = z (8 without zeros).  round() is to nearest, ties to even.
 * An infinity or NaN in a group makes its scale NaN, and so its weights.
 * Arguments and errors as for sgemm_w4_matvec.
 */
SGEMM_API sgemm_status_t sgemm_w4_quantize(int64_t N, int64_t K, int64_t group, int type,
                                           const void *W, int64_t ldw, uint32_t *qweight,
                                           int64_t ldq, void *scales, int64_t lds, uint8_t *zeros,
                                           int64_t ldz, void *stream);

/* Values of one tensor that share a scale of its 8-bit states. */
#define SGEMM_ADAMW_BLOCK 256

/* One tensor of sgemm_adamw_step (contiguous, numel elements). */
typedef struct {
    void *param;       /* of param_type, updated in place                              */
    const void *grad;  /* of grad_type                                                 */
    void *m, *v;       /* 32-bit states: floats; 8-bit states: one byte per element    */
    float *m_scale;    /* 8-bit states: ceil(numel / SGEMM_ADAMW_BLOCK) floats each,   */
    float *v_scale;    /* else ignored                                                 */
    void *copy;        /* NULL, or of copy_type: receives the updated parameter        */
    int64_t numel;
} sgemm_adamw_tensor_t;

/*
 * sgemm_adamw_step -- one AdamW step over `count` tensors
 *
 *     g <- grad_scale * g
 *     m <- beta1 m + (1 - beta1) g,   v <- beta2 v + (1 - beta2) g^2
 *     p <- p (1 - lr weight_decay) - lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 *
 * in 32-bit arithmetic (the constants are formed in 64 bits on the host).
 * tensors: a host array, read during the call.  param_type, grad_type and
 * copy_type: SGEMM_TYPE_*, the same for all tensors.  Regions must not
 * overlap.  A 16-bit parameter is rounded to nearest after the update.
 * state_bits 32: m and v are floats.  state_bits 8: in blocks of
 * SGEMM_ADAMW_BLOCK consecutive elements, m is held as e4m3 codes in units of
 * m_scale / 448 and sqrt(v) as e4m3 codes in units of v_scale / 448, where the
 * scales are the block's largest |m| and sqrt(v), at least 2^-96; codes are
 * rounded to nearest even, and a sqrt(v) above zero takes at least the
 * smallest code above zero.  The update uses the values before rounding.
 * All-zero codes with any finite scale are the initial state.  A block that meets an
 * infinity or NaN keeps NaN in its state.
 * Returns SGEMM_ERR_INVALID_ARG for a negative count or numel, a NULL or
 * misaligned pointer, an unknown type, state_bits other than 8 or 32,
 * step < 1, betas outside [0, 1) or a negative eps; SGEMM_ERR_UNSUPPORTED for
 * a numel above 2^42.
 */
SGEMM_API sgemm_status_t sgemm_adamw_step(const sgemm_adamw_tensor_t *tensors, int64_t count,
                                          int param_type, int grad_type, int copy_type,
                                          int state_bits, double lr, double beta1, double beta2,
                                          double eps, double weight_decay, int64_t step,
                                          double grad_scale, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GB300_SGEMM_FFN_H */
