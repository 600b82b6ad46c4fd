// One AdamW step over many tensors in one launch, with 32-bit or 8-bit states.
//
//   m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g^2
//   p <- p (1 - lr wd) - lr / bc1 * m / (sqrt(v) / sqrt(bc2) + eps)
//
// Bound: HBM.  Per element p is read and written, g read, m and v read and
// written (28 bytes with everything in FP32; 14 with a bf16 gradient and 8-bit
// states).  So each element is touched once, in registers from its loads to
// its stores, and all tensors share a launch: a CTA takes one chunk of
// kAdamChunk elements and finds its tensor by bisection over the tensors'
// first chunks, which travel with the pointers in the kernel's parameters
// (no table to upload, nothing kept on the device between steps).
//
// 8-bit states: a warp owns a block of 256 elements, eight per lane, so that
// the block's largest |m| and sqrt(v) are one warp reduction each.  The
// reduction compares the values' bit patterns as integers, which orders
// non-negative floats and puts NaN above everything, so a NaN reaches the
// scale.  Every operation that decides a code is a single correctly rounded
// FP32 one (no contraction), so the codes are reproducible from the formula.
#include "ops_common.cuh"

namespace sgemm {
namespace {

constexpr int kThreads = 256;
constexpr float kTiny = 1.2621774483536189e-29f;  // 2^-96: the least scale
constexpr float kLeast = 0.001953125f;            // 2^-9: the least e4m3 value above zero

struct AdamTable {
    int count;
    AdamTensor t[kAdamTensors];
};

// Eight consecutive elements from i (vec: all of them exist and may be loaded
// at once).
__device__ __forceinline__ void load8(const void *p, int type, long long i, int n, bool vec,
                                      float (&x)[8]) {
    if (!vec) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = j < n ? load_as_float(p, type, i + j) : 0.0f;
    } else if (type == kTypeF32) {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        const float4 a = __ldcs(q), b = __ldcs(q + 1);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        const uint4 a =
            __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = type == kTypeF16 ? unpack16<kTypeF16>(w[j]) : unpack16<kTypeBF16>(w[j]);
            x[2 * j] = f.x;
            x[2 * j + 1] = f.y;
        }
    }
}

__device__ __forceinline__ void store8(void *p, int type, long long i, int n, bool vec,
                                       const float (&x)[8]) {
    if (!vec) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) store_from_float(p, type, i + j, x[j]);
    } else if (type == kTypeF32) {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        __stcs(q, make_float4(x[0], x[1], x[2], x[3]));
        __stcs(q + 1, make_float4(x[4], x[5], x[6], x[7]));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = type == kTypeF16 ? pack16<kTypeF16>(x[2 * j], x[2 * j + 1])
                                    : pack16<kTypeBF16>(x[2 * j], x[2 * j + 1]);
        __stcs(reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i),
               make_uint4(w[0], w[1], w[2], w[3]));
    }
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
    uint32_t h;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(h) : "r"(two));
    return unpack16<kTypeF16>(h);
}

__device__ __forceinline__ uint32_t float2_to_e4m3x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\tcvt.rn.satfinite.e4m3x2.f32 c, %1, %2;\n\tcvt.u32.u16 %0, c;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}

// Eight codes times `unit`.
__device__ __forceinline__ void load_codes(const void *p, long long i, int n, bool vec, float unit,
                                           float (&x)[8]) {
    uint32_t w[2] = {0, 0};
    const uint8_t *q = static_cast<const uint8_t *>(p) + i;
    if (vec) {
        const uint2 a = __ldcs(reinterpret_cast<const uint2 *>(q));
        w[0] = a.x;
        w[1] = a.y;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) w[j / 4] |= (uint32_t)q[j] << (8 * (j % 4));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = e4m3x2_to_float2((w[j / 2] >> (16 * (j % 2))) & 0xFFFFu);
        x[2 * j] = __fmul_rn(f.x, unit);
        x[2 * j + 1] = __fmul_rn(f.y, unit);
    }
}

__device__ __forceinline__ void store_codes(void *p, long long i, int n, bool vec,
                                            const float (&x)[8]) {
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
        w[j] = float2_to_e4m3x2(x[4 * j], x[4 * j + 1]) |
               float2_to_e4m3x2(x[4 * j + 2], x[4 * j + 3]) << 16;
    uint8_t *q = static_cast<uint8_t *>(p) + i;
    if (vec) {
        __stcs(reinterpret_cast<uint2 *>(q), make_uint2(w[0], w[1]));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) q[j] = (uint8_t)(w[j / 4] >> (8 * (j % 4)));
    }
}

// The largest of a warp's non-negative values (or NaN).
__device__ __forceinline__ float warp_max_abs(float x) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x) & 0x7FFFFFFFu));
}

template <int BITS>
__global__ void __launch_bounds__(kThreads)
    adamw_kernel(const __grid_constant__ AdamTable table, const AdamHyper h) {
    // The last tensor whose first chunk is not behind this one.
    int lo = 0, hi = table.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (table.t[mid].chunk0 <= blockIdx.x)
            lo = mid;
        else
            hi = mid;
    }
    const AdamTensor &t = table.t[lo];
    const long long first = (long long)(blockIdx.x - t.chunk0) * kAdamChunk;
    const long long left = t.numel - first;

    for (int k = 0; k < kAdamChunk / (8 * kThreads); ++k) {
        const int at = (k * kThreads + (int)threadIdx.x) * 8;
        // A warp's 32 x 8 elements are one block, so its lanes leave together.
        if ((at & ~(kAdamBlock - 1)) >= left) break;
        const long long rest = left - at;
        const int n = rest >= 8 ? 8 : rest > 0 ? (int)rest : 0;
        const bool vec = t.vec && n == 8;
        const long long i = first + at;
        float p[8], g[8], m[8], v[8];
        load8(t.p, h.p_type, i, n, vec, p);
        load8(t.g, h.g_type, i, n, vec, g);
        if constexpr (BITS == 32) {
            load8(t.m, kTypeF32, i, n, vec, m);
            load8(t.v, kTypeF32, i, n, vec, v);
        } else {
            const long long b = i / kAdamBlock;
            load_codes(t.m, i, n, vec, __fdiv_rn(t.ms[b], 448.0f), m);
            load_codes(t.v, i, n, vec, __fdiv_rn(t.vs[b], 448.0f), v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], v[j]);
        }
        float r[8];
        float top_m = 0.0f, top_r = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float gj = __fmul_rn(g[j], h.grad_scale);
            m[j] = __fadd_rn(__fmul_rn(m[j], h.beta1), __fmul_rn(gj, h.omb1));
            v[j] = __fadd_rn(__fmul_rn(v[j], h.beta2), __fmul_rn(__fmul_rn(gj, gj), h.omb2));
            r[j] = __fsqrt_rn(v[j]);
            p[j] = p[j] * h.decay - h.step_size * __fdiv_rn(m[j], r[j] * h.inv_sqrt_bc2 + h.eps);
        }
        store8(t.p, h.p_type, i, n, vec, p);
        if (t.copy) store8(t.copy, h.c_type, i, n, vec, p);
        if constexpr (BITS == 32) {
            store8(t.m, kTypeF32, i, n, vec, m);
            store8(t.v, kTypeF32, i, n, vec, v);
        } else {
            uint32_t um = 0, ur = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j < n) {
                    um = max(um, __float_as_uint(m[j]) & 0x7FFFFFFFu);
                    ur = max(ur, __float_as_uint(r[j]) & 0x7FFFFFFFu);
                }
            }
            top_m = warp_max_abs(__uint_as_float(um));
            top_r = warp_max_abs(__uint_as_float(ur));
            if (top_m < kTiny) top_m = kTiny;
            if (top_r < kTiny) top_r = kTiny;
            const float km = __fdiv_rn(448.0f, top_m), kr = __fdiv_rn(448.0f, top_r);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                m[j] = __fmul_rn(m[j], km);
                const float q = __fmul_rn(r[j], kr);
                r[j] = (r[j] > 0.0f && q < kLeast) ? kLeast : q;
            }
            store_codes(t.m, i, n, vec, m);
            store_codes(t.v, i, n, vec, r);
            if ((threadIdx.x & 31) == 0) {
                t.ms[i / kAdamBlock] = top_m;
                t.vs[i / kAdamBlock] = top_r;
            }
        }
    }
}

}  // namespace

cudaError_t launch_adamw(const AdamTensor *tensors, int count, unsigned chunks, int state_bits,
                         const AdamHyper &h, cudaStream_t stream) {
    if (chunks == 0) return cudaSuccess;
    AdamTable table;
    table.count = count;
    for (int i = 0; i < count; ++i) table.t[i] = tensors[i];
    if (state_bits == 8)
        adamw_kernel<8><<<chunks, kThreads, 0, stream>>>(table, h);
    else
        adamw_kernel<32><<<chunks, kThreads, 0, stream>>>(table, h);
    return cudaGetLastError();
}

}  // namespace sgemm
