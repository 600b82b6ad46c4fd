// C ABI of the feed-forward operators (declared in include/sgemm_ffn.h):
// argument checks, workspace and the sequence of kernels of each call.
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <vector>

#include "../../include/sgemm_ffn.h"
#include "kernels_ffn.h"
#include "ops_internal.h"

namespace sgemm {
namespace {

constexpr int64_t kMaxFfnSize = int64_t(1) << 26;

bool aligned(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

bool type_ok(int type) {
    return type == SGEMM_TYPE_F32 || type == SGEMM_TYPE_F16 || type == SGEMM_TYPE_BF16;
}

// A matrix the call has to read or write: present, aligned to its elements.
bool matrix_ok(const void *p, int type) { return p && aligned(p, type_bytes(type)); }

int64_t at_least_one(int64_t v) { return v > 1 ? v : 1; }

sgemm_status_t status(cudaError_t e) { return e == cudaSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH; }

struct FfnArgs {
    int64_t T, D, F;
    int type, act;
    const void *x;
    int64_t ldx;
    const void *Wg;
    int64_t ldg;
    const void *Wu;
    int64_t ldu;
    const void *Wd;
    int64_t ldd;
};

sgemm_status_t check_ffn(const FfnArgs &a) {
    if (a.T < 0 || a.D < 0 || a.F < 0 || !type_ok(a.type)) return SGEMM_ERR_INVALID_ARG;
    if (a.act != SGEMM_GATE_SILU && a.act != SGEMM_GATE_GELU && a.act != SGEMM_GATE_RELU)
        return SGEMM_ERR_INVALID_ARG;
    if (a.ldx < at_least_one(a.D) || a.ldg < at_least_one(a.F) || a.ldu < at_least_one(a.F) ||
        a.ldd < at_least_one(a.D))
        return SGEMM_ERR_INVALID_ARG;
    if (a.T > kMaxFfnSize || a.D > kMaxFfnSize || a.F > kMaxFfnSize) return SGEMM_ERR_UNSUPPORTED;
    if (a.T > 0 && a.D > 0 && !matrix_ok(a.x, a.type)) return SGEMM_ERR_INVALID_ARG;
    if (a.D > 0 && a.F > 0 &&
        (!matrix_ok(a.Wg, a.type) || !matrix_ok(a.Wu, a.type) || !matrix_ok(a.Wd, a.type)))
        return SGEMM_ERR_INVALID_ARG;
    return SGEMM_OK;
}

int64_t saved_ld(int64_t F) { return (F + 3) / 4 * 4; }

FfnView view(const void *p, int type, int64_t ld) { return FfnView{p, type, ld, 1}; }
FfnView transposed(const FfnView &v) { return FfnView{v.p, v.type, v.cs, v.rs}; }

// h (null: not wanted) and g, u (null: not kept) of the block's first half.
sgemm_status_t run_gate(const FfnArgs &a, float *h, float *gu, cudaStream_t st) {
    FfnProduct p = {};
    p.mode = kFfnGate;
    p.M = (int)a.T; p.N = (int)a.F; p.K = (int)a.D;
    p.act = a.act;
    p.A = p.A2 = view(a.x, a.type, a.ldx);
    p.B = view(a.Wg, a.type, a.ldg);
    p.B2 = view(a.Wu, a.type, a.ldu);
    p.C = view(h, kTypeF32, a.F);
    p.ldgu = saved_ld(a.F);
    p.g = gu;
    p.u = gu ? gu + a.T * p.ldgu : nullptr;
    return status(launch_ffn_product(p, st));
}

sgemm_status_t run_product(int64_t M, int64_t N, int64_t K, const FfnView &A, const FfnView &B,
                           const FfnView &C, cudaStream_t st, FfnView A2 = {}, FfnView B2 = {}) {
    FfnProduct p = {};
    p.mode = kFfnStore;
    p.M = (int)M; p.N = (int)N; p.K = (int)K;
    p.A = A; p.B = B; p.A2 = A2; p.B2 = B2; p.C = C;
    return status(launch_ffn_product(p, st));
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" {

int64_t sgemm_ffn_saved_floats(int64_t T, int64_t F) {
    if (T < 0 || F < 0 || T > kMaxFfnSize || F > kMaxFfnSize) return 0;
    return 2 * T * saved_ld(F);
}

sgemm_status_t sgemm_ffn_forward(int64_t T, int64_t D, int64_t F, int type, int activation,
                                 const void *x, int64_t ldx, const void *Wg, int64_t ldg,
                                 const void *Wu, int64_t ldu, const void *Wd, int64_t ldd, void *y,
                                 int64_t ldy, float *saved, void *stream) {
    const FfnArgs a{T, D, F, type, activation, x, ldx, Wg, ldg, Wu, ldu, Wd, ldd};
    sgemm_status_t s = check_ffn(a);
    if (s != SGEMM_OK) return s;
    if (ldy < at_least_one(D) || !aligned(saved, 16)) return SGEMM_ERR_INVALID_ARG;
    if (T == 0 || D == 0) return SGEMM_OK;
    if (!matrix_ok(y, type)) return SGEMM_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    std::lock_guard<std::mutex> lock(api_mutex());
    OpDevice dev;
    s = op_device(&dev);
    if (s != SGEMM_OK) return s;
    void *w = nullptr;
    s = op_workspace(st, std::max<size_t>((size_t)(T * F) * 4, 16), &w);
    if (s != SGEMM_OK) return s;
    float *h = static_cast<float *>(w);
    s = run_gate(a, h, saved, st);
    if (s != SGEMM_OK) return s;
    return run_product(T, D, F, view(h, kTypeF32, F), view(Wd, type, ldd), view(y, type, ldy), st);
}

sgemm_status_t sgemm_ffn_backward(int64_t T, int64_t D, int64_t F, int type, int activation,
                                  const void *x, int64_t ldx, const void *Wg, int64_t ldg,
                                  const void *Wu, int64_t ldu, const void *Wd, int64_t ldd,
                                  const void *dy, int64_t lddy, const float *saved, void *dx,
                                  int64_t lddx, void *dWg, int64_t lddg, void *dWu, int64_t lddu,
                                  void *dWd, int64_t lddd, void *stream) {
    const FfnArgs a{T, D, F, type, activation, x, ldx, Wg, ldg, Wu, ldu, Wd, ldd};
    sgemm_status_t s = check_ffn(a);
    if (s != SGEMM_OK) return s;
    if (lddy < at_least_one(D) || !aligned(saved, 16)) return SGEMM_ERR_INVALID_ARG;
    const bool weights = dWg || dWu || dWd;
    if (dx && (lddx < at_least_one(D) || !aligned(dx, type_bytes(type)))) return SGEMM_ERR_INVALID_ARG;
    if (weights && (lddg < at_least_one(F) || lddu < at_least_one(F) || lddd < at_least_one(D) ||
                    !matrix_ok(dWg, type) || !matrix_ok(dWu, type) || !matrix_ok(dWd, type)))
        return SGEMM_ERR_INVALID_ARG;
    if (D == 0 || (T == 0 && F == 0) || (!dx && !weights)) return SGEMM_OK;
    if (T > 0 && !matrix_ok(dy, type)) return SGEMM_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    std::lock_guard<std::mutex> lock(api_mutex());
    OpDevice dev;
    s = op_device(&dev);
    if (s != SGEMM_OK) return s;
    const size_t tf = (size_t)(T * F), gu_floats = saved ? 0 : (size_t)(2 * T * saved_ld(F));
    void *w = nullptr;
    s = op_workspace(st, std::max<size_t>((3 * tf + gu_floats) * 4, 16), &w);
    if (s != SGEMM_OK) return s;
    float *gu = static_cast<float *>(w);
    float *dg = gu + gu_floats, *du = dg + tf, *h = du + tf;
    if (!saved) {
        s = run_gate(a, nullptr, gu, st);
        if (s != SGEMM_OK) return s;
    }
    const float *kept = saved ? saved : gu;
    const FfnView vx = view(x, type, ldx), vdy = view(dy, type, lddy);
    const FfnView vdg = view(dg, kTypeF32, F), vdu = view(du, kTypeF32, F), vh = view(h, kTypeF32, F);
    FfnProduct p = {};
    p.mode = kFfnGateGrad;
    p.M = (int)T; p.N = (int)F; p.K = (int)D;
    p.act = activation;
    p.A = vdy;
    p.B = transposed(view(Wd, type, ldd));
    p.C = vh; p.dg = vdg; p.du = vdu;
    p.ldgu = saved_ld(F);
    p.g = const_cast<float *>(kept);
    p.u = p.g + T * p.ldgu;
    s = status(launch_ffn_product(p, st));
    if (s == SGEMM_OK && dx)
        s = run_product(T, D, F, vdg, transposed(view(Wg, type, ldg)), view(dx, type, lddx), st, vdu,
                        transposed(view(Wu, type, ldu)));
    if (!weights) return s;
    if (s == SGEMM_OK) s = run_product(D, F, T, transposed(vx), vdg, view(dWg, type, lddg), st);
    if (s == SGEMM_OK) s = run_product(D, F, T, transposed(vx), vdu, view(dWu, type, lddu), st);
    if (s == SGEMM_OK) s = run_product(F, D, T, transposed(vh), vdy, view(dWd, type, lddd), st);
    return s;
}

sgemm_status_t sgemm_w4_matvec(int64_t M, int64_t N, int64_t K, int64_t group, int type,
                               const void *x, int64_t ldx, const uint32_t *qweight, int64_t ldq,
                               const void *scales, int64_t lds, const uint8_t *zeros, int64_t ldz,
                               void *y, int64_t ldy, void *stream) {
    if (M < 0 || N < 0 || K < 0 || !type_ok(type) || group < 32 || group % 32 != 0)
        return SGEMM_ERR_INVALID_ARG;
    if (ldx < at_least_one(K) || ldq < at_least_one(N) || lds < at_least_one(N) ||
        ldy < at_least_one(N) || (zeros && ldz < at_least_one(N)))
        return SGEMM_ERR_INVALID_ARG;
    if (N > (int64_t(1) << 30) || K > (int64_t(1) << 30) || M > (int64_t(1) << 20))
        return SGEMM_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (!matrix_ok(y, type)) return SGEMM_ERR_INVALID_ARG;
    if (K > 0 && (!matrix_ok(x, type) || !matrix_ok(scales, type) || !qweight || !aligned(qweight, 4)))
        return SGEMM_ERR_INVALID_ARG;
    std::lock_guard<std::mutex> lock(api_mutex());
    OpDevice dev;
    const sgemm_status_t s = op_device(&dev);
    if (s != SGEMM_OK) return s;
    const size_t e = type_bytes(type);
    W4Params p = {};
    p.N = (int)N; p.K = (int)K;
    p.group = (int)std::min<int64_t>(group, int64_t(1) << 30);
    p.q = qweight; p.ldq = ldq;
    p.scales = scales; p.lds = lds;
    p.zeros = zeros; p.ldz = ldz;
    p.ldx = ldx; p.ldy = ldy;
    p.x_vec = aligned(x, 16) && ldx % (16 / (int64_t)e) == 0;
    p.units = (int)((K + kW4UnitK - 1) / kW4UnitK);
    const bool vec = N % 4 == 0 && aligned(qweight, 16) && ldq % 4 == 0 && aligned(scales, 4 * e) &&
                     lds % 4 == 0 && (!zeros || (aligned(zeros, 4) && ldz % 4 == 0));
    // A cluster shares K where the columns alone leave SMs without work: at
    // least two CTAs per SM, as long as every warp keeps a unit.
    const int64_t tiles = (N + kW4Cols - 1) / kW4Cols;
    int cluster = 1;
    while (cluster < kW4MaxCluster && tiles * cluster < 2 * dev.num_sms &&
           p.units >= 2 * cluster * kW4Warps)
        cluster *= 2;
    p.cta_units = (p.units + cluster - 1) / cluster;
    const int max_rows = w4_max_rows(type);
    for (int64_t m0 = 0; m0 < M; m0 += max_rows) {
        p.M = (int)std::min<int64_t>(M - m0, max_rows);
        p.x = static_cast<const char *>(x) + m0 * ldx * e;
        p.y = static_cast<char *>(y) + m0 * ldy * e;
        p.chunk_units = std::max(1, std::min(p.cta_units, kW4StageBytes / w4_unit_bytes(type, p.M)));
        const cudaError_t err = launch_w4(p, type, vec, cluster, static_cast<cudaStream_t>(stream));
        if (err != cudaSuccess) return SGEMM_ERR_LAUNCH;
    }
    return SGEMM_OK;
}

sgemm_status_t sgemm_w4_quantize(int64_t N, int64_t K, int64_t group, int type, const void *W,
                                 int64_t ldw, uint32_t *qweight, int64_t ldq, void *scales,
                                 int64_t lds, uint8_t *zeros, int64_t ldz, void *stream) {
    if (N < 0 || K < 0 || !type_ok(type) || group < 32 || group % 32 != 0)
        return SGEMM_ERR_INVALID_ARG;
    if (ldw < at_least_one(N) || ldq < at_least_one(N) || lds < at_least_one(N) ||
        (zeros && ldz < at_least_one(N)))
        return SGEMM_ERR_INVALID_ARG;
    if (N > (int64_t(1) << 30) || K > (int64_t(1) << 30)) return SGEMM_ERR_UNSUPPORTED;
    if (N == 0 || K == 0) return SGEMM_OK;
    if (!matrix_ok(W, type) || !matrix_ok(scales, type) || !qweight || !aligned(qweight, 4))
        return SGEMM_ERR_INVALID_ARG;
    std::lock_guard<std::mutex> lock(api_mutex());
    OpDevice dev;
    const sgemm_status_t s = op_device(&dev);
    if (s != SGEMM_OK) return s;
    W4QuantParams p;
    p.N = (int)N; p.K = (int)K;
    p.group = (int)std::min<int64_t>(group, int64_t(1) << 30);
    p.type = type;
    p.W = W; p.ldw = ldw; p.q = qweight; p.ldq = ldq; p.scales = scales; p.lds = lds;
    p.zeros = zeros; p.ldz = ldz;
    return status(launch_w4_quantize(p, static_cast<cudaStream_t>(stream)));
}

sgemm_status_t sgemm_adamw_step(const sgemm_adamw_tensor_t *tensors, int64_t count, int param_type,
                                int grad_type, int copy_type, int state_bits, double lr,
                                double beta1, double beta2, double eps, double weight_decay,
                                int64_t step, double grad_scale, void *stream) {
    if (count < 0 || (count > 0 && !tensors) || !type_ok(param_type) || !type_ok(grad_type) ||
        !type_ok(copy_type) || (state_bits != 8 && state_bits != 32) || step < 1 ||
        !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0))
        return SGEMM_ERR_INVALID_ARG;
    const size_t state = state_bits == 8 ? 1 : 4;
    for (int64_t i = 0; i < count; ++i) {
        const sgemm_adamw_tensor_t &t = tensors[i];
        if (t.numel < 0) return SGEMM_ERR_INVALID_ARG;
        if (t.numel > (int64_t(1) << 42)) return SGEMM_ERR_UNSUPPORTED;
        if (t.numel == 0) continue;
        if (!matrix_ok(t.param, param_type) || !matrix_ok(t.grad, grad_type) || !t.m || !t.v ||
            !aligned(t.m, state) || !aligned(t.v, state) ||
            (t.copy && !aligned(t.copy, type_bytes(copy_type))))
            return SGEMM_ERR_INVALID_ARG;
        if (state_bits == 8 &&
            (!t.m_scale || !t.v_scale || !aligned(t.m_scale, 4) || !aligned(t.v_scale, 4)))
            return SGEMM_ERR_INVALID_ARG;
    }
    if (count == 0) return SGEMM_OK;
    std::lock_guard<std::mutex> lock(api_mutex());
    OpDevice dev;
    const sgemm_status_t s = op_device(&dev);
    if (s != SGEMM_OK) return s;
    const double bc1 = 1.0 - pow(beta1, (double)step), bc2 = 1.0 - pow(beta2, (double)step);
    AdamHyper h;
    h.beta1 = (float)beta1; h.omb1 = (float)(1.0 - beta1);
    h.beta2 = (float)beta2; h.omb2 = (float)(1.0 - beta2);
    h.decay = (float)(1.0 - lr * weight_decay);
    h.step_size = (float)(lr / bc1);
    h.inv_sqrt_bc2 = (float)(1.0 / sqrt(bc2));
    h.eps = (float)eps;
    h.grad_scale = (float)grad_scale;
    h.p_type = param_type; h.g_type = grad_type; h.c_type = copy_type;
    const size_t state_vec = state_bits == 8 ? 8 : 16;
    AdamTensor batch[kAdamTensors];
    int n = 0;
    uint64_t chunks = 0;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    for (int64_t i = 0; i < count; ++i) {
        const sgemm_adamw_tensor_t &t = tensors[i];
        if (t.numel == 0) continue;
        const uint64_t need = (uint64_t)((t.numel + kAdamChunk - 1) / kAdamChunk);
        if (n == kAdamTensors || (n > 0 && chunks + need > INT32_MAX)) {
            if (launch_adamw(batch, n, (unsigned)chunks, state_bits, h, st) != cudaSuccess)
                return SGEMM_ERR_LAUNCH;
            n = 0;
            chunks = 0;
        }
        AdamTensor &b = batch[n++];
        b.p = t.param; b.g = t.grad; b.m = t.m; b.v = t.v;
        b.ms = t.m_scale; b.vs = t.v_scale; b.copy = t.copy;
        b.numel = t.numel;
        b.chunk0 = (unsigned)chunks;
        b.vec = aligned(t.param, 16) && aligned(t.grad, 16) && aligned(t.m, state_vec) &&
                aligned(t.v, state_vec) && (!t.copy || aligned(t.copy, 16));
        chunks += need;
    }
    return status(n ? launch_adamw(batch, n, (unsigned)chunks, state_bits, h, st) : cudaSuccess);
}

}  // extern "C"
