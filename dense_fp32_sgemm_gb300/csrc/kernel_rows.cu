// Rows in one pass: the root-mean-square norm with the residual's addition, and
// rows that leave in 8 bits (the norm, the gate act(g) u, plain rows).
//
// A group of threads takes a row into registers with one round of 16-byte loads,
// reduces it (sum of squares and largest magnitude together), and writes it out:
// every byte moves once.  Rows that are too long for registers are read a second
// time.
#include <algorithm>

#include "kernels_q8.h"
#include "row_codes.cuh"
#include "row_io.cuh"

namespace sgemm {
namespace {

// ---- the gate in FP32 and in 48 bits --------------------------------------------

constexpr double kGeluC2 = 2.0 * 0.79788456080286535588;  // 2 sqrt(2 / pi)

// act(g) u, off by at most 2^-20 of itself and 2^-21 of `mass` (GELU's exponent is a
// rounded value: what it is off by counts as far as the exponential does).  Beyond
// |z| = 80 the exponential may be flushed to zero: `far` says that it matters (below
// 2^-108 the element's code is zero whatever it is).
__device__ __forceinline__ float gate_value(float g, float u, int act, float &mass, bool &far) {
    far = false;
    if (act == kGateRelu) {
        mass = 0.0f;
        return (g > 0.0f ? g : (g != g ? g : 0.0f)) * u;
    }
    // act(g) = g / (1 + exp(-z))
    const float z = act == kGateSilu ? g : (float)kGeluC2 * fmaf(0.044715f * g * g, g, g);
    const float x = fabsf(z);
    // exp(-x) = 2^t 2^c: c is what t lost in rounding.
    constexpr float kL = 1.4426950408889634f;
    constexpr float kLRest = (float)(1.4426950408889634074 - (double)kL);
    const float t = -x * kL;
    const float c = fmaf(-x, kLRest, fmaf(-x, kL, -t));
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    e = fmaf(e, 0.6931471805599453f * c, e);
    if (x > 160.0f) e = 0.0f;  // (c is NaN for an infinite x)
    const float s = __fdividef(1.0f, 1.0f + e), r = e * s;
    // z NaN stays NaN; at -infinity g times 0 is NaN, as in the formula.
    const float a = (z < 0.0f ? g * r : g * s) * u;
    mass = act == kGateSilu ? 0.0f : fabsf(a) * x * (z < 0.0f ? s : r);
    far = z < -80.0f && !(fabsf(g * u) < 100.0f);
    return a;
}
__device__ __noinline__ double gate_exact(float g, float u, int act) {
    if (act == kGateRelu) return g > 0.0f ? (double)g * u : 0.0;
    Two z = {g, 0.0f};
    if (act == kGateGelu) {
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

constexpr int kRowThreads = 512;  // most of a row
constexpr int kRowPieces = 4;     // most of a thread

// NP: pieces of a thread, a row in registers.  KEEP false: a row has more than
// that, and is read again.
template <int TYPE, int OP, int NP, bool KEEP, bool ALIGNED>
__global__ void __launch_bounds__(kRowThreads, 1) row_kernel(const RowParams p) {
    constexpr int V = piece_elements(TYPE), E = 16 / V;
    __shared__ float s_sum[kRowThreads / 32];
    __shared__ unsigned s_max[kRowThreads / 32];
    __shared__ unsigned long long s_top[kRowThreads / 32];
    __shared__ uint4 s_stage[ALIGNED || OP == kRowGateQ8 ? 1 : kRowThreads / 32 * kStageWords / 4];
    const int tid = threadIdx.x, lane = tid & 31;
    const int group = threadIdx.y, warps = blockDim.x >> 5;
    uint32_t *stage = reinterpret_cast<uint32_t *>(s_stage) +
                      (ALIGNED || OP == kRowGateQ8 ? 0 : (group * warps + (tid >> 5)) * kStageWords);
    const long long row = (long long)blockIdx.x * blockDim.y + group;
    const bool live = row < p.rows;
    const int step = blockDim.x * V, cols = live ? p.cols : 0;
    const bool two = p.b != nullptr;
    const Matrix A = matrix(p.a, p.rows, p.cols, p.lda, E), B = matrix(p.b, p.rows, p.cols, p.ldb, E);
    const Matrix W = matrix(p.w, 1, p.cols, 0, p.w_f32 ? 4 : E);
    const char *row_a = A.begin + row * A.ld, *row_b = B.begin + row * B.ld;

    if (tid == 0) s_top[group] = 0;
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");

    // Of the thread's elements: h of the norm; what is coded.
    float keep[NP][V];
    float sum = 0.0f, mass = 0.0f;
    unsigned most = 0;  // bits of the largest |a|; above those of infinity where one is NaN
    bool far = false;   // FP32 does not do for some of them

    auto exact = [&](int c) -> double {
        const float a = load_as_float(row_a, TYPE, c);
        if constexpr (OP == kRowGateQ8) {
            if (!two) return a;
            return gate_exact(a, load_as_float(row_b, TYPE, c), p.act);
        } else {
            const double h = two ? (double)a + (double)load_as_float(row_b, TYPE, c) : (double)a;
            return h * (double)load_as_float(p.w, p.w_f32 ? kTypeF32 : TYPE, c);
        }
    };
    // A piece (n > 0 elements from c on) as it comes from memory; and what of it is kept,
    // with its part in the row's statistics.
    auto fetch = [&](int c, int n, uint4 &x, uint4 &y) {
        x = load_piece<TYPE, ALIGNED>(row_a + (long long)c * E, n, A);
        if (two) y = load_piece<TYPE, ALIGNED>(row_b + (long long)c * E, n, B);
    };
    auto take = [&](int c, int n, uint4 x, uint4 y, float (&v)[V], bool first) {
        unpack_piece<TYPE>(x, v);
        float w[V];
        if (two) unpack_piece<TYPE>(y, w);
        if constexpr (OP == kRowGateQ8) {
            if (two) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float m;
                    bool f;
                    v[j] = gate_value(v[j], w[j], p.act, m, f);
                    mass = fmaxf(mass, m);
                    if (f) {
                        far = true;
                        if (first) most = max(most, __float_as_uint((float)fabs(exact(c + j))));
                    }
                }
            }
        } else {
            if (two) {
#pragma unroll
                for (int j = 0; j < V; ++j) v[j] += w[j];
            }
            if (first) {
#pragma unroll
                for (int j = 0; j < V; ++j) sum = fmaf(v[j], v[j], sum);
            }
        }
    };
    // Elements that the row does not have are zeros (a gate of 0 is 0 too).
    auto code = [&](int c, int n, float (&v)[V], bool first) {
        if constexpr (OP == kRowNormQ8) {
            float w[V];
            load_weight<TYPE, ALIGNED>(W, p.w_f32, c, n, w);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] *= w[j];
        }
        if (OP != kRowNorm && first) {
#pragma unroll
            for (int j = 0; j < V; ++j) most = max(most, __float_as_uint(v[j]) & 0x7FFFFFFFu);
        }
    };
    auto put = [&](void *to, long long ld, int c, int n, const float (&v)[V]) {
        // The address of lane 0's piece.
        char *at = static_cast<char *>(to) + (row * ld + c - lane * V) * E;
        store_piece<TYPE, ALIGNED>(at, n, pack_piece<TYPE>(v), stage);
    };
    // h over x or the residual would take from exact() what it reads: then it is stored last.
    const bool early = !p.h_last;

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
                take(c, n, x[i], y[i], keep[i], true);
                if (OP != kRowGateQ8 && p.h && early) put(p.h, p.ldh, c, n, keep[i]);
                if (n > 0) code(c, n, keep[i], true);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) keep[i][j] = 0.0f;
            }
        }
    } else {
        for (int c = tid * V; c < cols; c += step) {
            uint4 x, y = make_uint4(0, 0, 0, 0);
            fetch(c, cols - c, x, y);
            take(c, cols - c, x, y, keep[0], true);
            code(c, cols - c, keep[0], true);
        }
    }
    const unsigned mine = most;

    // Over the row's threads.
    if constexpr (OP != kRowGateQ8) {
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
        sum = lane < warps ? s_sum[slot + lane] : 0.0f;
        most = lane < warps ? s_max[slot + lane] : 0u;
        if constexpr (OP != kRowGateQ8) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        if constexpr (OP != kRowNorm) most = __reduce_max_sync(0xffffffffu, most);
    }
    const float rstd = OP == kRowGateQ8 ? 1.0f : 1.0f / sqrtf(sum / (float)p.cols + p.eps);

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
                take(c, cols - c, x, y, keep[0], false);
                if (OP == kRowNormQ8 && c < cols) code(c, cols - c, keep[0], false);
                f(c, cols - c, keep[0], 0);
            }
        }
    };
    auto store_h = [&](int c, int n) {
        uint4 x = make_uint4(0, 0, 0, 0), y = x;
        float v[V];
        if (n > 0) fetch(c, n, x, y);
        take(c, n, x, y, v, false);
        put(p.h, p.ldh, c, n, v);
    };

    if constexpr (OP == kRowNorm) {
        pieces([&](int c, int n, float (&v)[V], int) {
            float w[V], y[V];
            if (n > 0) load_weight<TYPE, ALIGNED>(W, p.w_f32, c, n, w);
#pragma unroll
            for (int j = 0; j < V; ++j) y[j] = n > 0 ? v[j] * rstd * w[j] : 0.0f;
            if (!KEEP && p.h) put(p.h, p.ldh, c, n, v);
            put(p.y, p.ldy, c, n, y);
        });
    } else {
        const bool bad = most >= 0x7F800000u;
        const float top32 = fmaxf(__uint_as_float(most), kRowTiny);
        // The largest magnitude in more bits, among those that FP32 cannot tell
        // from it (plain rows are exact as they are).
        double top = top32;
        if (OP != kRowGateQ8 || two) {
            const float limit = top32 * (1.0f - 0x1p-12f);
            if (!bad && (far || __uint_as_float(mine) >= limit)) {
                for (int c = tid * V, i = 0; c < cols; c += step, ++i) {
                    unsigned mask = 0;
                    if (far || !KEEP) {
                        mask = (1u << min(V, cols - c)) - 1;
                    } else if constexpr (KEEP) {
#pragma unroll
                        for (int k = 0; k < NP; ++k)
#pragma unroll
                            for (int j = 0; j < V; ++j)
                                mask |= (unsigned)(k == i && fabsf(keep[k][j]) >= limit) << j;
                    }
                    for (; mask; mask &= mask - 1)
                        atomicMax(&s_top[group], (unsigned long long)__double_as_longlong(
                                                     fabs(exact(c + __ffs(mask) - 1))));
                }
            }
            __syncthreads();
            top = fmax(__longlong_as_double((long long)s_top[group]), (double)kRowTiny);
        }
        const float inv = bad ? 0.0f : 127.0f / (float)top;
        // Nearer than this to the middle between two codes FP32 does not decide.
        const float border = 0.5f - (127.0f * 0x1p-20f + fminf(mass * inv, 1e4f) * 0x1p-21f);
        static_assert(NP * V <= 32, "");
        unsigned doubt = 0;  // of the thread's elements
        auto decide = [&](unsigned mask, int c) {
            for (; mask; mask &= mask - 1) {
                const int at = c + __ffs(mask) - 1;
                p.q[row * p.ldq + at] = (int8_t)row_code_exact(exact(at), top, inv);
            }
        };
        pieces([&](int c, int n, float (&v)[V], int number) {
            if (n <= 0) return;
            // v inv + 1.5 2^23 is rounded to a whole number, ties to even, whose low byte is
            // the code's.
            uint32_t r[V];
            float widest = 0.0f;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float q = fmaf(v[j], inv, 12582912.0f);
                r[j] = bad ? 0u : __float_as_uint(q);
                widest = fmaxf(widest, fabsf(fmaf(v[j], inv, -(q - 12582912.0f))));
            }
            uint32_t word[V / 4];
#pragma unroll
            for (int k = 0; k < V / 4; ++k)
                word[k] = __byte_perm(__byte_perm(r[4 * k], r[4 * k + 1], 0x0040),
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
            if ((widest > border || far) && !bad) {
                unsigned mask = 0;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float q = fmaf(v[j], inv, 12582912.0f) - 12582912.0f;
                    mask |= (unsigned)(j < n && (far || fabsf(fmaf(v[j], inv, -q)) > border)) << j;
                }
                if constexpr (KEEP)
                    doubt |= mask << (number * V);
                else
                    decide(mask, c);
            }
        });
        if constexpr (KEEP) {
            for (; doubt; doubt &= doubt - 1) {
                const int at = __ffs(doubt) - 1;
                decide(1u, tid * V + at / V * step + at % V);
            }
        }
        if (OP == kRowNormQ8 && p.h && !(KEEP && early))
            for (int c = tid * V; c - lane * V < cols; c += step) store_h(c, cols - c);
        if (tid == 0 && live)
            p.scales[row] = bad ? __int_as_float(0x7FC00000) : (float)top * rstd / 127.0f;
    }
}

template <int TYPE, int OP, bool ALIGNED>
cudaError_t launch_op(const RowParams &p, int num_sms, cudaStream_t stream) {
    constexpr int V = piece_elements(TYPE), kDeep = kRowPieces;
    // Threads of a row: with few rows as many as leave each one piece, else as many as
    // hold the row in four pieces each.
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
    if (!fits) return cudaLaunchKernelEx(&cfg, row_kernel<TYPE, OP, 1, false, ALIGNED>, p);
    if (few) return cudaLaunchKernelEx(&cfg, row_kernel<TYPE, OP, 1, true, ALIGNED>, p);
    return cudaLaunchKernelEx(&cfg, row_kernel<TYPE, OP, kDeep, true, ALIGNED>, p);
}

template <int TYPE>
cudaError_t launch_type(const RowParams &p, int op, bool vec, int num_sms, cudaStream_t stream) {
    switch (op) {
        case kRowNorm:
            return vec ? launch_op<TYPE, kRowNorm, true>(p, num_sms, stream)
                       : launch_op<TYPE, kRowNorm, false>(p, num_sms, stream);
        case kRowNormQ8:
            return vec ? launch_op<TYPE, kRowNormQ8, true>(p, num_sms, stream)
                       : launch_op<TYPE, kRowNormQ8, false>(p, num_sms, stream);
        default:
            return vec ? launch_op<TYPE, kRowGateQ8, true>(p, num_sms, stream)
                       : launch_op<TYPE, kRowGateQ8, false>(p, num_sms, stream);
    }
}

}  // namespace

cudaError_t launch_rows(const RowParams &p, int type, int op, bool vec, int num_sms,
                        cudaStream_t stream) {
    if (type == kTypeF32) return launch_type<kTypeF32>(p, op, vec, num_sms, stream);
    if (type == kTypeF16) return launch_type<kTypeF16>(p, op, vec, num_sms, stream);
    return launch_type<kTypeBF16>(p, op, vec, num_sms, stream);
}

}  // namespace sgemm
