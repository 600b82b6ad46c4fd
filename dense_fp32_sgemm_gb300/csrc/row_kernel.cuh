// Rows in one pass: the root-mean-square norm with the residual's addition, and
// rows that leave in 8 bits (the norm, the gate act(g) u, plain rows).
//
// A group of threads takes a row into registers with one round of 16-byte loads,
// reduces it (sum of squares and largest magnitude together), and writes it out:
// every byte moves once.  Rows that are too long for registers are read a second
// time.
#pragma once

#include <algorithm>

#include "kernels_q8.h"
#include "row_codes.cuh"
#include "row_io.cuh"

namespace sgemm {
namespace {

// ---- the gate in FP32 and in 48 bits --------------------------------------------

constexpr double kGeluC2 = 2.0 * 0.79788456080286535588;  // 2 sqrt(2 / pi)

// What gate_value() gathers over a thread's elements.
struct GateSpread {
    float mass = 0.0f;             // of the exponent's rounding (GELU)
    float lowest = 0.0f;           // z
    float largest = 0.0f;          // |g u|
    // Beyond z = -80 the exponential leaves FP32.  An element there matters from |g u| =
    // 100 on: below, its magnitude is under 2^-108 and its code zero whatever it is.
    __device__ __forceinline__ bool far() const { return lowest < -80.0f && largest >= 100.0f; }
};

// act(g) u with act(g) = g / (1 + exp(-z)), off by at most 2^-20.5 of itself and 2^-21 of
// `mass` (GELU's z is a rounded value: what it is off by counts as far as the
// exponential does).
template <int ACT>
__device__ __forceinline__ float gate_value(float g, float u, GateSpread &s) {
    if constexpr (ACT == kGateRelu) return (g > 0.0f ? g : (g != g ? g : 0.0f)) * u;
    const float gu = g * u;
    const float z = ACT == kGateSilu ? g : (float)kGeluC2 * fmaf(0.044715f * g * g, g, g);
    const float x = fminf(fmaxf(z, -80.0f), 100.0f);
    // exp(-x) = 2^t 2^c: c is what t lost in rounding.
    constexpr float kL = 1.4426950408889634f;
    constexpr float kLRest = (float)(1.4426950408889634074 - (double)kL);
    const float t = -x * kL;
    const float c = fmaf(-x, kLRest, fmaf(-x, kL, -t));
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    e = fmaf(e, 0.6931471805599453f * c, e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    const float a = gu * r;
    s.lowest = fminf(s.lowest, z);
    s.largest = fmaxf(s.largest, fabsf(gu));
    if constexpr (ACT == kGateGelu) s.mass = fmaxf(s.mass, fabsf(a * x) * (e * r));
    return a;
}
template <int ACT>
__device__ __noinline__ double gate_exact(float g, float u) {
    if (ACT == kGateRelu) return g > 0.0f ? (double)g * u : 0.0;
    Two z = {g, 0.0f};
    if (ACT == kGateGelu) {
        constexpr double k = 0.044715;
        const Two g2 = two_prod(g, g);
        z = g2 * Two{(float)k, (float)(k - (float)k)} + Two{1.0f, 0.0f};
        z = z * Two{g, 0.0f} * Two{(float)kGeluC2, (float)(kGeluC2 - (float)kGeluC2)};
    }
    const bool neg = z.hi < 0.0f;
    if (neg) z = Two{-z.hi, -z.lo};
    if (!(z.hi <= 60.0f))  // (beyond, the second float of the exponential loses bits)
        return (double)g * (double)u * (neg ? exp(-((double)z.hi + (double)z.lo)) : 1.0);
    const Two e = two_exp_neg(z), one = {1.0f, 0.0f};
    const Two s = (neg ? e : one) / (one + e);
    return ((double)s.hi + (double)s.lo) * ((double)g * (double)u);
}

// ---- the kernel -----------------------------------------------------------------

enum : int { kRowNorm, kRowNormQ8, kRowGateQ8 };  // what a row becomes

constexpr int kRowThreads = 1024;  // most of a row
constexpr int kRowPieces = 2;      // most of a thread (with four the registers leave too few warps)

// The larger; NaN where one is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// A positive double of FP32's range, cut to FP32 (a conversion would go through the
// FP64 pipe, for every thread).
__device__ __forceinline__ float cut_to_float(unsigned long long bits) {
    return __uint_as_float((unsigned)(bits >> 29) - ((1023u - 127u) << 23));
}

// NP: pieces of a thread, a row in registers.  KEEP false: a row has more than
// that, and is read again.  ACT: the gate's, or -1: plain rows.
template <int TYPE, int OP, int ACT, int NP, bool KEEP, bool ALIGNED>
__global__ void __launch_bounds__(kRowThreads, 1) row_kernel(const RowParams p) {
    constexpr int V = piece_elements(TYPE), E = 16 / V;
    constexpr bool kGate = OP == kRowGateQ8 && ACT >= 0, kPlain = OP == kRowGateQ8 && ACT < 0;
    constexpr bool kStores = OP != kRowGateQ8;  // matrices of TYPE
    __shared__ float s_sum[kRowThreads / 32];
    __shared__ unsigned s_max[kRowThreads / 32];
    __shared__ unsigned long long s_top[kRowThreads / 32];
    __shared__ uint4 s_stage[ALIGNED || !kStores ? 1 : kRowThreads / 32 * kStageWords / 4];
    const int tid = threadIdx.x, lane = tid & 31;
    const int group = threadIdx.y, warps = blockDim.x >> 5;
    uint32_t *stage = reinterpret_cast<uint32_t *>(s_stage) +
                      (ALIGNED || !kStores ? 0 : (group * warps + (tid >> 5)) * kStageWords);
    const long long row = (long long)blockIdx.x * blockDim.y + group;
    const bool live = row < p.rows;
    const int step = blockDim.x * V, cols = live ? p.cols : 0;
    const bool two = kGate || (!kPlain && p.b != nullptr);
    // Rows that are neither the first nor the last may be read in pieces that reach
    // over their ends.
    const bool inside = row > 0 && row + 1 < p.rows;
    const RowSource A = row_source(p.a, row, p.cols, p.lda, E, inside);
    const RowSource B = row_source(p.b, row, p.cols, p.ldb, E, inside);
    const RowSource W = row_source(p.w, 0, p.cols, 0, p.w_f32 ? 4 : E, false);

    if (tid == 0) s_top[group] = 0;
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");

    // Of the thread's elements: h of the norm; what is coded.
    float keep[NP][V];
    float sum = 0.0f, largest = 0.0f;  // of squares; |what is coded|, NaN where one is
    GateSpread spread;

    auto exact = [&](int c) -> double {
        const float a = load_as_float(A.row, TYPE, c);
        if constexpr (kPlain) {
            return a;
        } else if constexpr (kGate) {
            return gate_exact<ACT>(a, load_as_float(B.row, TYPE, c));
        } else {
            const double h = two ? (double)a + (double)load_as_float(B.row, TYPE, c) : (double)a;
            return h * (double)load_as_float(p.w, p.w_f32 ? kTypeF32 : TYPE, c);
        }
    };
    // A piece (n > 0 elements from c on) as it comes from memory; what of it is kept.
    auto fetch = [&](int c, int n, uint4 &x, uint4 &y) {
        x = load_piece<TYPE, ALIGNED>(A, c * E, n);
        if (two) y = load_piece<TYPE, ALIGNED>(B, c * E, n);
    };
    auto take = [&](uint4 x, uint4 y, float (&v)[V]) {
        unpack_piece<TYPE>(x, v);
        if (two) {
            float w[V];
            unpack_piece<TYPE>(y, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if constexpr (kGate)
                    v[j] = gate_value<ACT>(v[j], w[j], spread);
                else
                    v[j] += w[j];
            }
        }
    };
    auto weigh = [&](int c, int n, float (&v)[V]) {
        float w[V];
        load_weight<TYPE, ALIGNED>(W, p.w_f32, c, n, w);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] *= w[j];
    };
    // (Elements that the row does not have are zeros.)
    auto square = [&](const float (&v)[V]) {
#pragma unroll
        for (int j = 0; j < V; ++j) sum = fmaf(v[j], v[j], sum);
    };
    auto compare = [&](const float (&v)[V]) {
#pragma unroll
        for (int j = 0; j < V; ++j) largest = max_nan(largest, fabsf(v[j]));
    };
    auto put = [&](void *to, long long ld, int c, int n, const float (&v)[V]) {
        // The address of lane 0's piece.
        char *at = static_cast<char *>(to) + (row * ld + c - lane * V) * E;
        store_piece<TYPE, ALIGNED>(at, n, pack_piece<TYPE>(v), stage);
    };
    // h over x or the residual would take from exact() what it reads: then it is stored last.
    const bool early = KEEP && !p.h_last;

    if constexpr (KEEP) {
        uint4 x[NP], y[NP];
        // All loads before the first use.
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int c = tid * V + i * step, n = cols - c;
            x[i] = y[i] = make_uint4(0, 0, 0, 0);
            if (n > 0) fetch(c, n, x[i], y[i]);
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int c = tid * V + i * step, n = cols - c;
            if (c - lane * V < cols) {  // (the whole warp, for put())
                take(x[i], y[i], keep[i]);
                if constexpr (kStores) {
                    square(keep[i]);
                    if (p.h && early) put(p.h, p.ldh, c, n, keep[i]);
                }
                if (OP == kRowNormQ8 && n > 0) weigh(c, n, keep[i]);
                if constexpr (OP != kRowNorm) compare(keep[i]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) keep[i][j] = 0.0f;
            }
        }
    } else {
        for (int c = tid * V; c < cols; c += step) {
            uint4 x, y = make_uint4(0, 0, 0, 0);
            fetch(c, cols - c, x, y);
            take(x, y, keep[0]);
            if constexpr (kStores) square(keep[0]);
            if constexpr (OP == kRowNormQ8) weigh(c, cols - c, keep[0]);
            if constexpr (OP != kRowNorm) compare(keep[0]);
        }
    }
    static_assert(NP * V <= 32, "");
    // The column of the thread's i-th element in registers.
    auto element = [&](int i) { return tid * V + i / V * step + i % V; };
    // Calls f(c) for each of the thread's elements.
    auto each = [&](auto &&f) {
        for (int c = tid * V; c < cols; c += step)
            for (int j = 0; j < min(V, cols - c); ++j) f(c + j);
    };
    const bool far = kGate && spread.far();
    if constexpr (kGate) {
        if (far && largest == largest) {
            largest = 0.0f;
            each([&](int c) { largest = max_nan(largest, (float)fabs(exact(c))); });
        }
    }

    // Over the row's threads.
    unsigned most = __float_as_uint(largest);  // (above infinity's bits where it is NaN)
    if constexpr (kStores) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if constexpr (OP != kRowNorm) most = __reduce_max_sync(0xffffffffu, most);
    if (OP != kRowNorm || warps > 1) {
        const int slot = group * warps;
        if (lane == 0) {
            s_sum[slot + (tid >> 5)] = sum;
            s_max[slot + (tid >> 5)] = most;
        }
        __syncthreads();
        if constexpr (kStores) {
            sum = lane < warps ? s_sum[slot + lane] : 0.0f;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        if constexpr (OP != kRowNorm)
            most = __reduce_max_sync(0xffffffffu, lane < warps ? s_max[slot + lane] : 0u);
    }
    if constexpr (kStores) sum = __shfl_sync(0xffffffffu, sum, 0);
    const float rstd = kStores ? 1.0f / sqrtf(sum / (float)p.cols + p.eps) : 1.0f;

    // Calls f(c, n, values, number) for each piece of the row, with the whole warp.
    auto pieces = [&](auto &&f) {
        if constexpr (KEEP) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int c = tid * V + i * step;
                if (c - lane * V < cols) f(c, cols - c, keep[i], i);
            }
        } else {
            for (int c = tid * V; c - lane * V < cols; c += step) {
                uint4 x = make_uint4(0, 0, 0, 0), y = x;
                if (c < cols) fetch(c, cols - c, x, y);
                take(x, y, keep[0]);
                if (OP == kRowNormQ8 && c < cols) weigh(c, cols - c, keep[0]);
                f(c, cols - c, keep[0], 0);
            }
        }
    };

    if constexpr (OP == kRowNorm) {
        pieces([&](int c, int n, float (&v)[V], int) {
            float w[V], y[V];
            if (n > 0) load_weight<TYPE, ALIGNED>(W, p.w_f32, c, n, w);
#pragma unroll
            for (int j = 0; j < V; ++j) y[j] = n > 0 ? v[j] * rstd * w[j] : 0.0f;
            if (p.h && !early) put(p.h, p.ldh, c, n, v);
            put(p.y, p.ldy, c, n, y);
        });
    } else {
        const bool bad = most >= 0x7F800000u;
        const float top32 = fmaxf(__uint_as_float(most), kRowTiny);
        // The largest magnitude in more bits, among those that FP32 cannot tell
        // from it (plain rows are exact as they are).
        float top = top32;
        if constexpr (!kPlain) {
            const float limit = top32 * (1.0f - 0x1p-12f);
            if (!bad && largest >= limit) {
                auto raise = [&](int c) {
                    atomicMax(&s_top[group], (unsigned long long)__double_as_longlong(fabs(exact(c))));
                };
                if (far) {
                    each(raise);
                } else if constexpr (KEEP) {
                    unsigned mask = 0;
#pragma unroll
                    for (int i = 0; i < NP; ++i)
#pragma unroll
                        for (int j = 0; j < V; ++j)
                            mask |= (unsigned)(fabsf(keep[i][j]) >= limit) << (i * V + j);
                    for (; mask; mask &= mask - 1) raise(element(__ffs(mask) - 1));
                } else {
                    for (int c = tid * V; c < cols; c += step) {
                        uint4 x, y = make_uint4(0, 0, 0, 0);
                        fetch(c, cols - c, x, y);
                        take(x, y, keep[0]);
                        if constexpr (OP == kRowNormQ8) weigh(c, cols - c, keep[0]);
#pragma unroll
                        for (int j = 0; j < V; ++j)
                            if (fabsf(keep[0][j]) >= limit) raise(c + j);
                    }
                }
            }
            __syncthreads();
            const unsigned long long bits = s_top[group];
            if (bits > (unsigned long long)(1023 - 96) << 52) top = cut_to_float(bits);
        }
        auto exact_top = [&]() {
            return kPlain ? (double)top
                          : fmax(__longlong_as_double((long long)s_top[group]), (double)kRowTiny);
        };
        const float inv = bad ? 0.0f : 127.0f / top;
        // Nearer than this to the middle between two codes FP32 does not decide.
        float border = 0.5f - 127.0f * 0x1p-20f;
        if constexpr (kGate) border -= fminf(spread.mass * inv, 1e4f) * 0x1p-21f;
        unsigned doubt = 0;  // of the thread's elements
        auto decide = [&](int c) {
            p.q[row * p.ldq + c] = (int8_t)row_code_exact(exact(c), exact_top(), inv);
        };
        pieces([&](int c, int n, float (&v)[V], int number) {
            if (n <= 0) return;
            // v inv + 1.5 2^23 is rounded to a whole number, ties to even, whose low byte is
            // the code's.
            constexpr float kWhole = 12582912.0f;
            uint32_t r[V], word[V / 4];
            float widest = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float q = fmaf(v[j], inv, kWhole);
                r[j] = __float_as_uint(q);
                widest = fmaxf(widest, fabsf(fmaf(v[j], inv, kWhole - q)));
            }
#pragma unroll
            for (int k = 0; k < V / 4; ++k)
                word[k] = bad ? 0u
                              : __byte_perm(__byte_perm(r[4 * k], r[4 * k + 1], 0x0040),
                                            __byte_perm(r[4 * k + 2], r[4 * k + 3], 0x0040), 0x5410);
            int8_t *out = p.q + row * p.ldq + c;
            if (n >= V && (ALIGNED || p.q_vec)) {
                if constexpr (V == 8)
                    *reinterpret_cast<uint2 *>(out) = make_uint2(word[0], word[V / 4 - 1]);
                else
                    *reinterpret_cast<uint32_t *>(out) = word[0];
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (j < n) out[j] = (int8_t)(word[j / 4] >> (8 * (j % 4)));
            }
            if (widest > border && !bad && !far) {
                unsigned mask = 0;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float q = fmaf(v[j], inv, kWhole);
                    mask |= (unsigned)(j < n && fabsf(fmaf(v[j], inv, kWhole - q)) > border) << j;
                }
                if constexpr (KEEP)
                    doubt |= mask << (number * V);
                else
                    for (; mask; mask &= mask - 1) decide(c + __ffs(mask) - 1);
            }
        });
        for (; doubt; doubt &= doubt - 1) decide(element(__ffs(doubt) - 1));
        if (far && !bad) each([&](int c) { decide(c); });
        if (OP == kRowNormQ8 && p.h && !early)
            for (int c = tid * V; c - lane * V < cols; c += step) {
                uint4 x = make_uint4(0, 0, 0, 0), y = x;
                float v[V];
                if (c < cols) fetch(c, cols - c, x, y);
                take(x, y, v);
                put(p.h, p.ldh, c, cols - c, v);
            }
        if (tid == 0 && live)
            p.scales[row] = bad ? __int_as_float(0x7FC00000) : (float)exact_top() * rstd / 127.0f;
    }
}

template <int TYPE, int OP, int ACT, bool ALIGNED>
cudaError_t launch_op(const RowParams &p, int num_sms, cudaStream_t stream) {
    constexpr int V = piece_elements(TYPE), kDeep = kRowPieces;
    // Threads of a row: with few rows as many as leave each one piece, else as many as
    // hold the row in two pieces each.
    const long long most = (p.cols + V - 1) / V;  // pieces
    const bool few = p.rows <= 2 * num_sms && most <= kRowThreads;
    const long long want = few ? most : (most + kDeep - 1) / kDeep;
    int threads = 32;
    while (threads < want && threads < 128) threads *= 2;
    if (threads < want) threads = (int)std::min<long long>((want + 31) / 32 * 32, kRowThreads);
    const int groups = threads >= 128 ? 1 : 128 / threads;
    const bool fits = (long long)threads * (few ? 1 : kDeep) >= most;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.rows + groups - 1) / groups));
    cfg.blockDim = dim3(threads, groups);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (!fits) return cudaLaunchKernelEx(&cfg, row_kernel<TYPE, OP, ACT, 1, false, ALIGNED>, p);
    if (few) return cudaLaunchKernelEx(&cfg, row_kernel<TYPE, OP, ACT, 1, true, ALIGNED>, p);
    return cudaLaunchKernelEx(&cfg, row_kernel<TYPE, OP, ACT, kDeep, true, ALIGNED>, p);
}

// For one of the library's types and alignments.
template <int OP, int ACT>
cudaError_t launch_rows_of(const RowParams &p, int type, bool vec, int num_sms, cudaStream_t stream) {
    switch (type) {
        case kTypeF32:
            return vec ? launch_op<kTypeF32, OP, ACT, true>(p, num_sms, stream)
                       : launch_op<kTypeF32, OP, ACT, false>(p, num_sms, stream);
        case kTypeF16:
            return vec ? launch_op<kTypeF16, OP, ACT, true>(p, num_sms, stream)
                       : launch_op<kTypeF16, OP, ACT, false>(p, num_sms, stream);
        default:
            return vec ? launch_op<kTypeBF16, OP, ACT, true>(p, num_sms, stream)
                       : launch_op<kTypeBF16, OP, ACT, false>(p, num_sms, stream);
    }
}

}  // namespace
}  // namespace sgemm
