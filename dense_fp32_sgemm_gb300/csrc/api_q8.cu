// C ABI of the norm and of the operators in 8 bits (declared in
// include/sgemm_q8.h): argument checks, workspace and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "../../include/sgemm_ffn.h"
#include "../../include/sgemm_q8.h"
#include "kernels_q8.h"
#include "ops_internal.h"

namespace sgemm {
namespace {

constexpr int64_t kMaxRows = INT32_MAX, kMaxSize = int64_t(1) << 26, kMaxQ8K = 131071;

bool aligned(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool type_ok(int type) {
    return type == SGEMM_TYPE_F32 || type == SGEMM_TYPE_F16 || type == SGEMM_TYPE_BF16;
}
bool present(const void *p, int type) { return p && aligned(p, type_bytes(type)); }
int64_t at_least_one(int64_t v) { return v > 1 ? v : 1; }
sgemm_status_t status(cudaError_t e) { return e == cudaSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH; }
int64_t up(int64_t v, int64_t unit) { return (v + unit - 1) / unit * unit; }

// A matrix whose rows all start on 16 bytes (or that is not there).
bool rows16(const void *p, int64_t ld, int64_t rows, int type) {
    return !p || (aligned(p, 16) && (rows <= 1 || ld * type_bytes(type) % 16 == 0));
}
// A matrix of codes whose rows all start where a thread's piece is stored at once.
bool codes_vec(const int8_t *q, int64_t ld, int64_t rows, int type) {
    const int64_t piece = type == kTypeF32 ? 4 : 8;
    return aligned(q, piece) && (rows <= 1 || ld % piece == 0);
}

struct NormArgs {
    int64_t T, D;
    int type;
    const void *x;
    int64_t ldx;
    const void *residual;
    int64_t ldr;
    const void *weight;
    int weight_type;
    double eps;
    void *h;
    int64_t ldh;
};

sgemm_status_t check_norm(const NormArgs &a) {
    if (a.T < 0 || a.D < 0 || !type_ok(a.type) || !(a.eps >= 0.0) ||
        (a.weight_type != a.type && a.weight_type != SGEMM_TYPE_F32))
        return SGEMM_ERR_INVALID_ARG;
    const int64_t least = at_least_one(a.D);
    if (a.ldx < least || (a.residual && a.ldr < least) || (a.h && a.ldh < least))
        return SGEMM_ERR_INVALID_ARG;
    if (a.T > kMaxRows || a.D > kMaxSize) return SGEMM_ERR_UNSUPPORTED;
    if (a.D > 0 && (!present(a.weight, a.weight_type) ||
                    (a.T > 0 && (!present(a.x, a.type) || !aligned(a.residual, type_bytes(a.type)) ||
                                 !aligned(a.h, type_bytes(a.type))))))
        return SGEMM_ERR_INVALID_ARG;
    return SGEMM_OK;
}

RowParams row_params(const NormArgs &a) {
    RowParams p = {};
    p.rows = a.T;
    p.cols = (int)a.D;
    p.a = a.x; p.lda = a.ldx;
    p.b = a.residual; p.ldb = a.ldr;
    p.w = a.weight;
    p.w_f32 = a.weight_type == SGEMM_TYPE_F32;
    p.eps = (float)a.eps;
    p.inv_cols = 1.0f / (float)a.D;
    p.h = a.h; p.ldh = a.ldh;
    return p;
}
bool norm_vec(const NormArgs &a) {
    return rows16(a.x, a.ldx, a.T, a.type) && rows16(a.residual, a.ldr, a.T, a.type) &&
           rows16(a.h, a.ldh, a.T, a.type) && aligned(a.weight, 16);
}

// Single CTAs or pairs, tokens of a tile, and how the tiles left over after whole rounds
// are cut along k: the least of a model of SM clocks, fitted to GB300 times.  A stage (128 k)
// takes 4 for each token of a pair's tile (single CTAs 4 too: half the products, but
// operands that pass through shared memory twice as often), at least 700, which its
// weights take to be widened and to come from HBM.  A tile takes 3000 more for its results, one
// cut in pieces 5000 for those to meet, and 600 for each.  (Even shares of the tail for
// all workers, as the gated block has them, touch two tiles each and meet twice:
// 96 x 4096 x 4096 26 us.)
bool q8_plan(Q8GemmParams &p, bool &pair, int num_sms) {
    double least = -1.0;
    p.stages_k = (p.K + kQ8StageK - 1) / kQ8StageK;
    for (int two = 0; two < 2; ++two) {
        const int64_t most = kQ8Tokens * (two + 1), channels = kQ8Channels * (two + 1);
        const int64_t tiles_n = (p.N + channels - 1) / channels, rows = (p.M + most - 1) / most;
        const int workers = num_sms / (two + 1);
        for (int64_t m = rows; m < rows + 4; ++m) {
            const int tokens = (int)up((p.M + m - 1) / m, 32);
            const int64_t tiles_m = (p.M + tokens - 1) / tokens, tiles = tiles_m * tiles_n;
            if (tiles > INT32_MAX / 2) continue;
            const double stage = std::max(700.0, 4.0 * tokens);
            const int full = (int)(tiles / workers), tail = (int)(tiles % workers);
            const double whole = full * (p.stages_k * stage + 3000.0);
            for (int n = 1; n == 1 || (n * tail <= workers && n <= p.stages_k); ++n) {
                const int per_piece = (p.stages_k + n - 1) / n;
                const double cost = whole + (tail ? per_piece * stage + 3000.0 : 0.0) +
                                    (n > 1 ? 5000.0 + 600.0 * n * tokens / most : 0.0);
                if (least < 0.0 || cost < least) {
                    least = cost;
                    pair = two != 0;
                    p.tokens = tokens;
                    p.tiles_m = (int)tiles_m;
                    p.tiles_n = (int)tiles_n;
                    p.workers = workers;
                    p.full_tiles = full;
                    p.tail_tiles = tail;
                    p.pieces = n;
                }
                if (tail == 0) break;
            }
        }
    }
    return least >= 0.0;
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

// (No exception leaves an entry point.  There is one, of a host without memory for the library's own
// state, which is made before anything is queued.)
extern "C" {

sgemm_status_t sgemm_rms_norm(int64_t T, int64_t D, int type, const void *x, int64_t ldx,
                              const void *residual, int64_t ldr, const void *weight, int weight_type,
                              double eps, void *h, int64_t ldh, void *y, int64_t ldy, void *stream) try {
    const NormArgs a{T, D, type, x, ldx, residual, ldr, weight, weight_type, eps, h, ldh};
    sgemm_status_t s = check_norm(a);
    if (s != SGEMM_OK) return s;
    if (ldy < at_least_one(D)) return SGEMM_ERR_INVALID_ARG;
    if (T == 0 || D == 0) return SGEMM_OK;
    if (!present(y, type)) return SGEMM_ERR_INVALID_ARG;
    std::lock_guard<std::mutex> lock(api_mutex());
    OpDevice dev;
    s = op_device(&dev);
    if (s != SGEMM_OK) return s;
    RowParams p = row_params(a);
    p.device = dev.index;
    p.y = y; p.ldy = ldy;
    return status(launch_norm(p, type, false, norm_vec(a) && rows16(y, ldy, T, type), dev.num_sms,
                              static_cast<cudaStream_t>(stream)));
} catch (...) {
    return SGEMM_ERR_ALLOC;
}

sgemm_status_t sgemm_rms_norm_q8(int64_t T, int64_t D, int type, const void *x, int64_t ldx,
                                 const void *residual, int64_t ldr, const void *weight,
                                 int weight_type, double eps, void *h, int64_t ldh, int8_t *q,
                                 int64_t ldq, float *scales, void *stream) try {
    const NormArgs a{T, D, type, x, ldx, residual, ldr, weight, weight_type, eps, h, ldh};
    sgemm_status_t s = check_norm(a);
    if (s != SGEMM_OK) return s;
    if (ldq < at_least_one(D)) return SGEMM_ERR_INVALID_ARG;
    if (T == 0) return SGEMM_OK;
    // (rows of nothing have the scale of rows of zeros)
    if (D == 0) return sgemm_q8_gate(T, 0, type, 0, nullptr, 1, nullptr, 1, q, ldq, scales, stream);
    if (!q || !scales || !aligned(scales, 4)) return SGEMM_ERR_INVALID_ARG;
    std::lock_guard<std::mutex> lock(api_mutex());
    OpDevice dev;
    s = op_device(&dev);
    if (s != SGEMM_OK) return s;
    RowParams p = row_params(a);
    p.device = dev.index;
    p.h_last = h && (h == x || h == residual);
    p.q = q; p.ldq = ldq;
    p.q_vec = codes_vec(q, ldq, T, type);
    p.scales = scales;
    return status(launch_norm(p, type, true, norm_vec(a) && p.q_vec,
                              dev.num_sms, static_cast<cudaStream_t>(stream)));
} catch (...) {
    return SGEMM_ERR_ALLOC;
}

sgemm_status_t sgemm_rms_norm_backward(int64_t T, int64_t D, int type, const void *x, int64_t ldx,
                                       const void *residual, int64_t ldr, const void *weight, int weight_type, double eps,
                                       const void *dy, int64_t lddy, const void *dh, int64_t lddh,
                                       void *dx, int64_t lddx, void *dweight, void *stream) try {
    const NormArgs a{T, D, type, x, ldx, residual, ldr, weight, weight_type, eps, nullptr, 0};
    sgemm_status_t s = check_norm(a);
    if (s != SGEMM_OK) return s;
    const int64_t least = at_least_one(D);
    const int e = type_bytes(type), we = type_bytes(weight_type);
    if (lddy < least || (dh && lddh < least) || (dx && lddx < least) || !aligned(dh, e) ||
        !aligned(dx, e) || !aligned(dweight, we))
        return SGEMM_ERR_INVALID_ARG;
    if (D == 0 || (!dx && !dweight)) return SGEMM_OK;
    if (T > 0 && !present(dy, type)) return SGEMM_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    std::lock_guard<std::mutex> lock(api_mutex());
    OpDevice dev;
    s = op_device(&dev);
    if (s != SGEMM_OK) return s;
    if (T == 0)
        return dweight ? status(cudaMemsetAsync(dweight, 0, (size_t)D * we, st)) : SGEMM_OK;
    const bool vec = norm_vec(a) && rows16(dy, lddy, T, type) && rows16(dh, lddh, T, type) &&
                     rows16(dx, lddx, T, type);
    NormGradParams p = {};
    p.rows = T;
    p.cols = (int)D;
    p.x = x; p.ldx = ldx;
    p.r = residual; p.ldr = ldr;
    p.dy = dy; p.lddy = lddy;
    p.dh = dh; p.lddh = lddh;
    p.w = weight;
    p.w_f32 = weight_type == SGEMM_TYPE_F32;
    p.eps = (float)eps;
    p.dx = dx; p.lddx = lddx;
    p.dw = dweight;
    p.device = dev.index;
    const NormGradSpace space = norm_grad_space(p, type, vec, dev.num_sms);
    p.parts = space.parts;
    if (dweight) {
        void *w = nullptr;
        const size_t stats = space.stats ? up(T * (int64_t)sizeof(float), 256) : 0;
        s = op_workspace(st, stats + (size_t)p.parts * D * sizeof(float), &w);
        if (s != SGEMM_OK) return s;
        p.stats = space.stats ? static_cast<float *>(w) : nullptr;
        p.partials = reinterpret_cast<float *>(static_cast<char *>(w) + stats);
    }
    return status(launch_norm_grad(p, type, vec, dev.num_sms, st));
} catch (...) {
    return SGEMM_ERR_ALLOC;
}

sgemm_status_t sgemm_q8_gate(int64_t T, int64_t F, int type, int activation, const void *g,
                             int64_t ldg, const void *u, int64_t ldu, int8_t *q, int64_t ldq,
                             float *scales, void *stream) try {
    if (T < 0 || F < 0 || !type_ok(type)) return SGEMM_ERR_INVALID_ARG;
    if (u && activation != SGEMM_GATE_SILU && activation != SGEMM_GATE_GELU &&
        activation != SGEMM_GATE_RELU)
        return SGEMM_ERR_INVALID_ARG;
    const int64_t least = at_least_one(F);
    if (ldg < least || (u && ldu < least) || ldq < least) return SGEMM_ERR_INVALID_ARG;
    if (T > kMaxRows || F > kMaxSize) return SGEMM_ERR_UNSUPPORTED;
    if (T == 0) return SGEMM_OK;
    if (!scales || !aligned(scales, 4)) return SGEMM_ERR_INVALID_ARG;
    if (F > 0 && (!present(g, type) || !aligned(u, type_bytes(type)) || !q)) return SGEMM_ERR_INVALID_ARG;
    std::lock_guard<std::mutex> lock(api_mutex());
    OpDevice dev;
    const sgemm_status_t s = op_device(&dev);
    if (s != SGEMM_OK) return s;
    RowParams p = {};
    p.rows = T;
    p.cols = (int)F;
    p.a = g; p.lda = ldg;
    p.b = u; p.ldb = ldu;
    p.act = activation;
    p.device = dev.index;
    p.q = q; p.ldq = ldq;
    p.q_vec = codes_vec(q, ldq, T, type);
    p.scales = scales;
    const bool vec = rows16(g, ldg, T, type) && rows16(u, ldu, T, type) && p.q_vec;
    return status(launch_gate_q8(p, type, vec, dev.num_sms, static_cast<cudaStream_t>(stream)));
} catch (...) {
    return SGEMM_ERR_ALLOC;
}

sgemm_status_t sgemm_q8_quantize(int64_t N, int64_t K, int type, const void *W, int64_t ldw, int8_t *q,
                                 int64_t ldq, float *scales, void *stream) try {
    if (N < 0 || K < 0 || !type_ok(type)) return SGEMM_ERR_INVALID_ARG;
    if (ldw < at_least_one(N) || ldq < at_least_one(K)) return SGEMM_ERR_INVALID_ARG;
    if (N > kMaxSize || K > kMaxSize) return SGEMM_ERR_UNSUPPORTED;
    if (N == 0) return SGEMM_OK;
    if (!scales || !aligned(scales, 4) || (K > 0 && (!present(W, type) || !q))) return SGEMM_ERR_INVALID_ARG;
    std::lock_guard<std::mutex> lock(api_mutex());
    OpDevice dev;
    const sgemm_status_t s = op_device(&dev);
    if (s != SGEMM_OK) return s;
    Q8QuantParams p;
    p.N = (int)N; p.K = (int)K;
    p.type = type;
    p.W = W; p.ldw = ldw;
    p.q = q; p.ldq = ldq;
    p.scales = scales;
    return status(launch_q8_quantize(p, static_cast<cudaStream_t>(stream)));
} catch (...) {
    return SGEMM_ERR_ALLOC;
}

sgemm_status_t sgemm_q8_matmul(int64_t M, int64_t N, int64_t K, int type, const int8_t *x, int64_t ldx,
                               const float *x_scales, const int8_t *w, int64_t ldw,
                               const float *w_scales, void *y, int64_t ldy, void *stream) try {
    if (M < 0 || N < 0 || K < 0 || !type_ok(type)) return SGEMM_ERR_INVALID_ARG;
    if (ldx < at_least_one(K) || ldw < at_least_one(K) || ldy < at_least_one(N)) return SGEMM_ERR_INVALID_ARG;
    if (M > kMaxSize || N > kMaxSize || K > kMaxQ8K) return SGEMM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (!present(y, type)) return SGEMM_ERR_INVALID_ARG;
    if (K > 0 && (!x || !w || !present(x_scales, kTypeF32) || !present(w_scales, kTypeF32)))
        return SGEMM_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    std::lock_guard<std::mutex> lock(api_mutex());
    OpDevice dev;
    sgemm_status_t s = op_device(&dev);
    if (s != SGEMM_OK) return s;
    if (K == 0) {
        const size_t e = type_bytes(type);
        return status(cudaMemset2DAsync(y, ldy * e, 0, N * e, M, st));
    }
    // From five rows on a pass over a large matrix costs the streaming kernel more in
    // multiplications than the tensor cores in their second launch (us, streaming and tensor
    // cores, 5 to 8 rows: 4096 x 4096 14.5 and 14.6, 4096 x 8192 18.6 and 16.7,
    // 12288 x 4096 22.9 and 18.6, 8192 x 28672 64 and 53; 3 rows of the last 48 and 53).
    const bool stream_form = M <= 4 || (M <= kQ8StreamRows && N * K <= 24LL << 20);
    const bool in_place = aligned(w, 16) && (N == 1 || ldw % 16 == 0);

    // Workspace: aligned weights, x in FP16, partial tiles.
    size_t bytes = 0;
    auto take = [&](size_t n) {
        const size_t at = bytes;
        bytes += (n + 255) / 256 * 256;
        return at;
    };
    const int64_t ld_w = in_place ? ldw : up(K, 16), ld_x = up(K, 64);
    const size_t w_at = in_place ? 0 : take((size_t)(N * ld_w));
    const size_t x_at = stream_form ? 0 : take((size_t)(M * ld_x) * 2);
    char *base = nullptr;
    if (bytes) {
        void *p = nullptr;
        s = op_workspace(st, bytes, &p);
        if (s != SGEMM_OK) return s;
        base = static_cast<char *>(p);
    }
    if (!in_place) {
        int8_t *copy = reinterpret_cast<int8_t *>(base + w_at);
        if (launch_q8_align(w, ldw, (int)N, (int)K, copy, ld_w, dev.num_sms, st) != cudaSuccess)
            return SGEMM_ERR_LAUNCH;
        w = copy;
    }
    if (stream_form) {
        Q8StreamParams p = {};
        p.M = (int)M; p.N = (int)N; p.K = (int)K;
        p.x = x; p.ldx = ldx;
        p.x_scales = x_scales;
        p.w = w; p.ldw = ld_w;
        p.w_scales = w_scales;
        p.y = y; p.ldy = ldy;
        p.x_vec = aligned(x, 16) && (M == 1 || ldx % 16 == 0);
        return status(launch_q8_stream(p, type, dev.num_sms, st));
    }

    Q8GemmParams p = {};
    p.M = (int)M; p.N = (int)N; p.K = (int)K;
    bool pair = false;
    if (!q8_plan(p, pair, dev.num_sms)) return SGEMM_ERR_UNSUPPORTED;
    // (15 MB whatever the sizes, so that the first call on a stream is the one that allocates)
    s = op_counters(st, (size_t)dev.num_sms * (8 + q8_tile_ints()), &p.counters);
    if (s != SGEMM_OK) return s;
    p.meet = p.counters + (size_t)dev.num_sms * 8;
    uint16_t *wide = reinterpret_cast<uint16_t *>(base + x_at);
    p.x_scales = x_scales;
    p.w_scales = w_scales;
    p.y = y; p.ldy = ldy;
    p.y_vec = rows16(y, ldy, M, type);
    p.device = dev.index;
    p.err = dev.err;
    p.timeout_ns = dev.timeout_ns;
    p.skip_loads_from = dev.skip_loads_from;
    CUtensorMap map_w, map_x;
    s = op_encode_bytes(&map_w, w, N, K, ld_w, kQ8Channels);
    // x as its stretches of 64 k, two of which are a stage's.
    if (s == SGEMM_OK)
        s = op_encode_16(&map_x, false, wide, M, 64, ld_x, ld_x / 64, 64, p.tokens / (pair ? 2 : 1), 2);
    if (s != SGEMM_OK) return s;
    if (launch_q8_widen(x, ldx, (int)M, (int)K, wide, ld_x, dev.num_sms, st) != cudaSuccess)
        return SGEMM_ERR_LAUNCH;
    return status(launch_q8_gemm(map_w, map_x, p, type, pair, st));
} catch (...) {
    return SGEMM_ERR_ALLOC;
}

}  // extern "C"
