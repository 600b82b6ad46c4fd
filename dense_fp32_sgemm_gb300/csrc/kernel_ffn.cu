// The gated block's products, in the form that takes any type, stride and
// alignment: 64 x 64 tiles, 16-deep slices of bounds-checked loads, FP32
// multiply-adds on the SIMT pipe.
#include "ops_common.cuh"

namespace sgemm {
namespace {

constexpr int BM = 64, BN = 64, BK = 16;

__device__ __forceinline__ float gate_act(float g, int act) {
    if (act == kGateSilu) return g / (1.0f + expf(-g));
    if (act == kGateGelu) {
        const float t = tanhf(0.7978845608028654f * (g + 0.044715f * g * g * g));
        return 0.5f * g * (1.0f + t);
    }
    return g > 0.0f ? g : 0.0f;
}

__device__ __forceinline__ float gate_slope(float g, int act) {
    if (act == kGateSilu) {
        const float s = 1.0f / (1.0f + expf(-g));
        return s * (1.0f + g * (1.0f - s));
    }
    if (act == kGateGelu) {
        const float t = tanhf(0.7978845608028654f * (g + 0.044715f * g * g * g));
        return 0.5f * (1.0f + t) +
               0.5f * g * (1.0f - t * t) * 0.7978845608028654f * (1.0f + 0.134145f * g * g);
    }
    return g > 0.0f ? 1.0f : 0.0f;
}

__device__ __forceinline__ float at(const FfnView &v, long long i, long long j) {
    return load_as_float(v.p, v.type, i * v.rs + j * v.cs);
}
__device__ __forceinline__ void put(const FfnView &v, long long i, long long j, float x) {
    store_from_float(const_cast<void *>(v.p), v.type, i * v.rs + j * v.cs, x);
}

// acc += A B over this CTA's tile.
__device__ __forceinline__ void product(const FfnView &A, const FfnView &B, const FfnProduct &p,
                                        int m0, int n0, float (*sa)[BM], float (*sb)[BN],
                                        float (&acc)[4][4]) {
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    for (int k0 = 0; k0 < p.K; k0 += BK) {
        for (int i = tid; i < BM * BK; i += 256) {
            const int k = i % BK, m = i / BK;
            sa[k][m] = (m0 + m < p.M && k0 + k < p.K) ? at(A, m0 + m, k0 + k) : 0.0f;
        }
        for (int i = tid; i < BN * BK; i += 256) {
            const int n = i % BN, k = i / BN;
            sb[k][n] = (n0 + n < p.N && k0 + k < p.K) ? at(B, k0 + k, n0 + n) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < BK; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], acc[i][j]);
        __syncthreads();
    }
}

__global__ void __launch_bounds__(256) ffn_simple_kernel(const FfnProduct p) {
    __shared__ float sa[BK][BM], sb[BK][BN];
    const int tiles_n = (p.N + BN - 1) / BN;
    const int m0 = (int)(blockIdx.x / tiles_n) * BM, n0 = (int)(blockIdx.x % tiles_n) * BN;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {}, acc2[4][4] = {};
    product(p.A, p.B, p, m0, n0, sa, sb, acc);
    if (p.B2.p) {
        if (p.mode == kFfnGate)
            product(p.A2, p.B2, p, m0, n0, sa, sb, acc2);
        else
            product(p.A2, p.B2, p, m0, n0, sa, sb, acc);
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (m >= p.M || n >= p.N) continue;
            if (p.mode == kFfnStore) {
                put(p.C, m, n, acc[i][j]);
                continue;
            }
            const long long gu = m * p.ldgu + n;
            if (p.mode == kFfnGate) {
                if (p.g) {
                    p.g[gu] = acc[i][j];
                    p.u[gu] = acc2[i][j];
                }
                if (p.C.p) put(p.C, m, n, gate_act(acc[i][j], p.act) * acc2[i][j]);
            } else {
                const float g = p.g[gu], u = p.u[gu], a = gate_act(g, p.act);
                put(p.dg, m, n, acc[i][j] * u * gate_slope(g, p.act));
                put(p.du, m, n, acc[i][j] * a);
                put(p.C, m, n, a * u);
            }
        }
}

}  // namespace

cudaError_t launch_ffn_product(const FfnProduct &p, cudaStream_t stream) {
    const long long tiles = (long long)((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
    if (tiles == 0) return cudaSuccess;
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    ffn_simple_kernel<<<(unsigned)tiles, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace sgemm
