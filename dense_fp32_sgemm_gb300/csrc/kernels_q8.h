// Parameter blocks and launch wrappers of the norm's kernels and of those that
// work in 8 bits (include/sgemm_q8.h).  Host-visible only.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels_ffn.h"

namespace sgemm {

// ---------------------------------------------------------------------------
// Rows in one pass: the norm, and rows that leave in 8 bits.
// ---------------------------------------------------------------------------

struct RowParams {
    long long rows;
    int cols;
    const void *a, *b;       // x or g; residual or u (null: none)
    long long lda, ldb;
    const void *w;           // the norm's weight
    int w_f32;               // it is FP32 whatever the type
    float eps, inv_cols;
    int act;
    void *h;                 // null, or receives a + b
    long long ldh;
    int h_last;              // it lies over a or b: they are read until the codes are done
    void *y;
    long long ldy;
    int8_t *q;
    long long ldq;
    int q_vec;               // its rows start on 8 bytes (FP32: 4)
    float *scales;
    int device;
    int stages;              // (set by the launch) rows on their way
};
// y = norm(a + b) * w, or with q8 its codes; codes of act(a) * b, or of a where b is
// null.  vec: rows of every matrix (and the weight) start on 16 bytes, those of q as above.
cudaError_t launch_norm(const RowParams &p, int type, bool q8, bool vec, int num_sms,
                        cudaStream_t stream);
cudaError_t launch_gate_q8(const RowParams &p, int type, bool vec, int num_sms, cudaStream_t stream);

struct NormGradParams {
    long long rows;
    int cols;
    const void *x, *r, *dy, *dh;  // h is x, or x + r; dh: null, or added to dx
    long long ldx, ldr, lddy, lddh;
    const void *w;
    int w_f32;
    float eps;
    void *dx;                 // null: not wanted
    long long lddx;
    void *dw;                 // null: not wanted
    float *partials;          // parts x cols, sums of some rows each
    float *stats;             // rows: r, where rows do not fit registers
    int parts;
    int device;
    int stages;               // (set by the launch) rows on their way
};
// What a gradient with dw needs beside its operands (one without: nothing): partial rows of dw,
// and whether the rows' statistics are kept.
struct NormGradSpace {
    int parts;
    bool stats;
};
NormGradSpace norm_grad_space(const NormGradParams &p, int type, bool vec, int num_sms);
cudaError_t launch_norm_grad(const NormGradParams &p, int type, bool vec, int num_sms,
                             cudaStream_t stream);

struct Q8QuantParams {
    int N, K, type;
    const void *W;
    long long ldw;
    int8_t *q;
    long long ldq;
    float *scales;
};
cudaError_t launch_q8_quantize(const Q8QuantParams &p, cudaStream_t stream);

// ---------------------------------------------------------------------------
// Products of 8-bit integers.
// ---------------------------------------------------------------------------
// A few rows of x, on the integer dot product.
constexpr int kQ8StreamRows = 8;
constexpr int kQ8StreamBytes = 96 * 1024;  // of x that a CTA stages at once

struct Q8StreamParams {
    int M, N, K;
    const int8_t *x;
    long long ldx;
    const float *x_scales;
    const int8_t *w;
    long long ldw;
    const float *w_scales;
    void *y;
    long long ldy;
    int x_vec;   // rows of x start on 16 bytes
};
cudaError_t launch_q8_stream(const Q8StreamParams &p, int type, int num_sms, cudaStream_t stream);

// Many rows, on the tensor cores: tiles of 128 channels (256 by pairs of CTAs)
// by up to 96 (192) tokens.
constexpr int kQ8Channels = 128;      // of a CTA's tile
constexpr int kQ8Tokens = 96;         // most tokens that a CTA brings in
constexpr int kQ8StageK = 128;        // k of a stage: one 128-byte row of w
constexpr int kQ8SlotK = 64;          // k of a slot of converted weights in tensor memory
constexpr int kQ8ExactK = 1024;       // k after which an FP32 accumulator is taken out

struct Q8GemmParams {
    int M, N, K;
    int tokens;                       // of a tile
    int tiles_n, tiles_m;
    int stages_k;                     // ceil(K / kQ8StageK)
    // Workers (CTAs or pairs) take full_tiles each, round-robin; the tail_tiles left over are
    // cut along k into `pieces` of a worker each.
    int workers, full_tiles, tail_tiles, pieces;
    int *counters;                    // CTAs of the tail's tiles x 8, zero at rest
    int *meet;                        // as many accumulators of q8_tile_ints(), zero at rest
    const float *x_scales, *w_scales;
    void *y;
    long long ldy;
    int y_vec;                        // its rows start on 16 bytes
    int device;
    int *err;
    unsigned long long timeout_ns;
    int skip_loads_from;
};
constexpr int q8_tile_ints() { return kQ8Channels * kQ8Tokens * 2; }  // of a CTA
// w: boxes of 128 channels x 128 bytes; x: fp16, boxes of two stretches of tokens x 64
// (128-byte swizzles).
cudaError_t launch_q8_gemm(const CUtensorMap &w, const CUtensorMap &x, const Q8GemmParams &p,
                           int type, bool pair, cudaStream_t stream);

// x in fp16 (M x ldo, zeros from K on), and w in aligned rows.
cudaError_t launch_q8_widen(const int8_t *x, long long ldx, int M, int K, uint16_t *out,
                            long long ldo, int num_sms, cudaStream_t stream);
cudaError_t launch_q8_align(const int8_t *w, long long ldw, int N, int K, int8_t *out,
                            long long ldo, int num_sms, cudaStream_t stream);

}  // namespace sgemm
