// Parameter blocks and launch wrappers of the feed-forward operators' kernels
// (the gated block, products with 4-bit weights, the AdamW step).
// Host-visible only.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace sgemm {

// Element types and gate activations, as in include/sgemm_ffn.h.
enum : int { kTypeF32 = 0, kTypeF16 = 1, kTypeBF16 = 2 };
enum : int { kGateSilu = 0, kGateGelu = 1, kGateRelu = 2 };

inline int type_bytes(int type) { return type == kTypeF32 ? 4 : 2; }

// ---------------------------------------------------------------------------
// Products with 4-bit weights.
// ---------------------------------------------------------------------------
constexpr int kW4Cols = 64;      // columns of W per warp
constexpr int kW4Warps = 4;      // computing warps of a CTA, along the columns and along K
constexpr int kW4UnitK = 128;    // k of a unit
constexpr int kW4Stages = 3;     // units a warp has under way
constexpr int kW4BoxCols = 32, kW4BoxRows = kW4UnitK / 8;  // TMA box of words
constexpr int kW4MaxCluster = 8;

struct W4Params {
    int M, N, K;
    int group, group_shift;  // group_shift: log2 of group, or -1
    const void *x;
    long long ldx;
    const uint32_t *q;
    long long ldq;
    const void *scales;
    long long lds;
    const uint8_t *zeros;  // nullptr: every zero point is 8
    long long ldz;
    void *y;
    long long ldy;
    int x_vec;         // 8 elements of x may be loaded at once
    int units;         // ceil(K / kW4UnitK)
    int cta_units;     // units of one CTA
    int chunk_units;   // units whose x is staged at once
    int warps_n;       // warps side by side along the columns (1, 2 or 4)
    int safe_rows;     // of q, at either end, from whose inside a piece may reach outside
    int device;
    int *err;
    unsigned long long timeout_ns;
};

// vec: rows of q, scales and zeros start on 16 bytes, N % 16 == 0; q through
// `map` (boxes of kW4BoxRows x kW4BoxCols words, 128-byte swizzle).
cudaError_t launch_w4(const CUtensorMap &map, const W4Params &p, int type, bool vec, int cluster, cudaStream_t stream);
// Rows of x one launch takes (FP32 rows take three of the instruction's each).
int w4_max_rows(int type);
// Bytes of shared memory a unit of staged x takes, and the limit for all of them.
int w4_unit_bytes(int type, int M);
constexpr int kW4StageBytes = 64 * 1024;
// CTAs that an SM holds with x of `units` units staged.
int w4_ctas_per_sm(int type, int M, int group, int units);

struct W4QuantParams {
    int N, K, group, type;
    const void *W;
    long long ldw;
    uint32_t *q;
    long long ldq;
    void *scales;
    long long lds;
    uint8_t *zeros;
    long long ldz;
};
cudaError_t launch_w4_quantize(const W4QuantParams &p, cudaStream_t stream);

// ---------------------------------------------------------------------------
// AdamW.
// ---------------------------------------------------------------------------
constexpr int kAdamBlock = 256;   // elements that share a scale of the 8-bit states
constexpr int kAdamMinChunk = 2048, kAdamChunk = 16384;  // elements of one tensor a CTA takes
constexpr int kAdamTensors = 400; // tensors of one launch

struct AdamTensor {
    void *p;
    const void *g;
    void *m, *v;
    float *ms, *vs;
    void *copy;
    unsigned chunk0;  // first chunk of this tensor in the launch
    unsigned vec;     // every array allows its widest loads
    long long numel;
};

struct AdamHyper {
    float beta1, omb1, beta2, omb2;  // omb: one minus beta
    float decay;                     // 1 - lr * weight_decay
    float step_size;                 // lr / (1 - beta1^step)
    float inv_sqrt_bc2;              // 1 / sqrt(1 - beta2^step)
    float eps;
    float grad_scale;
    int p_type, g_type, c_type;
    int chunk;  // elements of one tensor a CTA takes
};

// `tensors` (count <= kAdamTensors) with chunk0 filled in; `chunks` in all.
cudaError_t launch_adamw(const AdamTensor *tensors, int count, unsigned chunks, int state_bits,
                         const AdamHyper &h, int device, cudaStream_t stream);

// ---------------------------------------------------------------------------
// The gated block's products on the tensor cores (kernel_ffn.cu).
// ---------------------------------------------------------------------------
// An operand in memory: `planes` matrices of rows x cols 16-bit values, rows
// ld elements apart (16-byte aligned), planes plane_rows rows apart.  16-bit
// types have one plane; FP32 values are held as three bf16 planes that add up
// to them.
struct FfnOperand {
    const void *p;
    int64_t rows, cols, ld, plane_stride;  // plane_stride in elements
    int planes;
};

enum : int {
    kFfnStore = 0,     // C = A B, or A B + A2 B2
    kFfnGate = 1,      // g = A B, u = A B2; h = act(g) u; u act'(g) and act(g) kept when asked
    kFfnGateGrad = 2,  // dh = A B; dg = dh u act'(g) and du = dh act(g) from the kept values
};

constexpr int kFfnBM = 128;      // rows of a CTA's tile
// Columns of B that each CTA brings in per k block.
constexpr int ffn_b_cols(bool f32, bool pair) { return f32 && pair ? 64 : 128; }
constexpr int kFfnBK = 64;       // k per stage: one 128-byte swizzled row
constexpr int kFfnThreads = 384; // 4 warps of roles, 8 of epilogue

constexpr int kFfnProblems = 4;  // products of one launch (kFfnStore)
constexpr int kFfnMaps = 10;     // operands of one launch

// One product of a launch.  Its operands are maps a, a + 1 (second product of a
// sum) and b, b + 1.
struct FfnProblem {
    int M, N;
    int a, b;
    int segs;            // products added up (2: A B + A2 B2)
    int a_mn, b_mn;      // operand is MN-major: its rows run along k
    uint32_t a_bytes;    // of A per CTA and stage: rows of `a` boxes, 128 bytes each
    int kblocks;         // ceil(K / kFfnBK)
    int tiles_m, tiles_n, tile0;  // tiles, and the first one's number in the launch
    // kFfnStore: C[0], `type`.  kFfnGate: C[0] = h.  kFfnGateGrad: C[0] = dg,
    // C[1] = du.  h, dg and du are 16-bit operands for the next product: one
    // plane of `type`, or three bf16 planes.
    void *C[2];
    long long ldc, c_plane;
    int c_vec;           // 16-byte stores allowed
};

struct FfnGemmParams {
    int mode;
    int type;            // of the user's matrices
    int act;
    int count;           // products, those with the longest tiles first
    FfnProblem prob[kFfnProblems];
    int tiles;           // of all products
    // Workers (CTAs or pairs) take whole tiles round-robin: first the long_tiles
    // of the products with the longest tiles, where there are two lengths; then
    // those that got one long tile fewer take `extra` of the others; then all
    // take full_tiles each.  The tail_tiles left over are cut along k into
    // tail_workers equal shares (tail_workers 0: taken whole).
    int workers, long_tiles, extra, full_tiles, tail_tiles, tail_workers;
    float *partials;     // 2 slots per worker of ffn_slot_floats() per CTA (tail)
    int *counters;       // tail_tiles x CTAs of a worker x 8, zero at rest
    int device;
    // u act'(g) and act(g), or null: blocks of 32 x 32 values, block (i, j) at
    // (i * keep_cols + j) * 1024, in it element (row r, column c) at
    // (c / 4 * 32 + r) * 4 + c % 4: as a warp holds them.
    float *keep[2];
    int keep_cols;
    int *err;
    unsigned long long timeout_ns;
    int skip_loads_from;
};

// Floats of a CTA's accumulator; a worker's partial tile has one per CTA.
inline int ffn_slot_floats(bool f32, bool pair) {
    return kFfnBM * ffn_b_cols(f32, pair) * (pair ? 2 : 1);
}

// The operands' TMA descriptors: boxes of 64 along the contiguous dimension.
struct FfnMaps {
    CUtensorMap m[kFfnMaps];
};
// pair: 256-row tiles by pairs of CTAs.
cudaError_t launch_ffn_gemm(const FfnMaps &maps, const FfnGemmParams &p, bool pair,
                            cudaStream_t stream);

// Copies that make operands of the user's matrices: FP32 split into three
// bf16 planes, or 16-bit values moved to aligned rows.
struct FfnPrepJob {
    const void *src;
    int64_t ld_src;
    int rows, cols;
    void *dst;
    int64_t ld_dst, plane_stride;
};
constexpr int kFfnPrepJobs = 5;
cudaError_t launch_ffn_prep(const FfnPrepJob *jobs, int count, int type, int num_sms,
                            cudaStream_t stream);

// ---------------------------------------------------------------------------
// The gated block for a few rows (kernel_ffn_stream.cu).
// ---------------------------------------------------------------------------
constexpr int kFfnStreamRows = 8;  // most rows it takes

struct FfnStreamParams {
    int T, N, K;
    int act;
    const void *x;        // T x K: of the weights' type (gate) or FP32 (down)
    long long ldx;
    const void *W, *W2;   // K x N; W2 of the gate's two
    long long ldw, ldw2;
    void *y;              // T x N: FP32 (gate: h) or of the weights' type
    long long ldy;
    int device;
    // set by launch_ffn_stream
    int lanes_per_row, cta_rows, chunk_rows;
    int safe_rows;           // see ffn_stream_kernel
    const void *end, *end2;  // of W and W2
};
// vec: 16 bytes of a row's columns may be loaded at once (N a multiple too).
cudaError_t launch_ffn_stream(const FfnStreamParams &p, int type, bool gate, bool vec, int num_sms,
                              cudaStream_t stream);

}  // namespace sgemm
