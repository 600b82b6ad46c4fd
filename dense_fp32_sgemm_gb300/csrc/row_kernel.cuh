// Rows in one pass: the root-mean-square norm with the residual's addition, and
// rows that leave in 8 bits (the norm, the gate act(g) u, plain rows).
//
// A group of threads takes a row into registers, reduces it (sum of squares and
// largest magnitude together), and writes it out: every byte moves once.  CTAs
// stay and take rows in turn; the pieces of their next rows are on their way to shared
// memory meanwhile.  Rows that are too long for registers are read a second time.
//
// Measured, and the time of the bytes: norm of 8192 x 2048 BF16 with its residual 24 us (20); in
// 8 bits of 4096 x 4096 BF16 with its residual 31 us (17.6, 3.8 TB/s); gate of 4096 x 12288 BF16
// 72 us (37.7, 3.5 TB/s).  Bound: instructions, 39 and 37 an element: the issue slots are 65
// to 70 % used with what registers leave of warps (35 to 46 % of the SM's).
#pragma once

#include <algorithm>
#include <atomic>
#include <limits>

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
    float lowest = 0.0f;           // z; beyond -80 the exponential leaves FP32
};

// act(g) u with act(g) = g / (1 + exp(-z)), off by at most 2^-20.5 of itself and 2^-21 of
// `mass` (GELU's z is a rounded value: what it is off by counts as far as the
// exponential does).  Where FP32 does not hold g u, z or its multiple below, the result is not
// finite, whatever act(g) u is; gate_exact() has it then.
template <int ACT>
__device__ __forceinline__ float gate_z(float g) {
    return ACT == kGateSilu ? g : (float)kGeluC2 * fmaf(0.044715f * g * g, g, g);
}
template <int ACT>
__device__ __forceinline__ float gate_value(float g, float u, GateSpread &s) {
    if constexpr (ACT == kGateRelu) return (g > 0.0f ? g : (g != g ? g : 0.0f)) * u;
    const float gu = g * u;
    const float z = gate_z<ACT>(g);
    const float x = fmaxf(z, -80.0f);
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
    if constexpr (ACT == kGateGelu) s.mass = fmaxf(s.mass, fabsf(a * x) * (e * r));
    return a;
}
template <int ACT>
__device__ __forceinline__ double gate_exact(float g, float u) {
    if (ACT == kGateRelu) return g > 0.0f ? (double)g * u : 0.0;
    Two z = {g, 0.0f};
    if (ACT == kGateGelu) {
        // (beyond +-100 the exponential is 0 or beyond 64 bits; two floats do not hold the cube of
        // 10^13)
        const float c = fminf(fmaxf(g, -100.0f), 100.0f);
        constexpr double k = 0.044715;
        const Two g2 = two_prod(c, c);
        z = g2 * Two{(float)k, (float)(k - (float)k)} + Two{1.0f, 0.0f};
        z = z * Two{c, 0.0f} * Two{(float)kGeluC2, (float)(kGeluC2 - (float)kGeluC2)};
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

// A thread's pieces of a row and its registers.  The norm takes two pieces (of 8192 x 8192
// FP16 55 us, with four 64: fewer warps; 8192 x 2048 BF16 with its residual 24 and 28); what leaves in 8 bits, whose threads have more to
// do for every row, four (the gate of 4096 x 12288 96 us, with two, which leave one CTA of
// 768 threads an SM, 132).
constexpr int row_pieces(int op) { return op == kRowNorm ? 2 : 4; }
constexpr int row_threads(int op) { return op == kRowNorm ? 1024 : 512; }  // most of a row
constexpr int row_regs(int op, int act, bool aligned) {
    return op == kRowNorm ? 64 : act >= 0 && !aligned ? 88 : 80;
}
constexpr int kMaxDevices = 64;
constexpr int kRingBytes = 192 * 1024;  // of an SM, for rows on their way

// The larger; NaN where one is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// NP: pieces of a thread, a row in registers.  KEEP false: a row has more than
// that, and is read again.  ACT: the gate's, or -1: plain rows.
template <int TYPE, int OP, int ACT, int NP, bool KEEP, bool ALIGNED>
__global__ void __maxnreg__(row_regs(OP, ACT, ALIGNED)) row_kernel(const RowParams p) {
    constexpr int V = piece_elements(TYPE), E = 16 / V;
    constexpr bool kGate = OP == kRowGateQ8 && ACT >= 0, kPlain = OP == kRowGateQ8 && ACT < 0;
    constexpr bool kStores = OP != kRowGateQ8;  // matrices of TYPE
    // Alternating from row to row, so that a row's readers are done when they are written again.
    constexpr int kWarps = row_threads(OP) / 32;
    __shared__ float s_sum[2][kWarps];
    __shared__ unsigned s_max[2][kWarps], s_mass[2][kWarps];
    __shared__ unsigned long long s_top[3][kWarps];
    __shared__ float s_root[3][kWarps];  // what the scale is multiplied by
    const int tid = threadIdx.x, lane = tid & 31;
    const int group = threadIdx.y, warps = blockDim.x >> 5;
    // The ring below, and before it what store_piece() needs of each warp.
    extern __shared__ uint4 s_dynamic[];
    constexpr int kStage = kStores && !ALIGNED ? kStageWords / 4 : 0;
    const int pitch = blockDim.x * blockDim.y;
    uint32_t *stage = reinterpret_cast<uint32_t *>(s_dynamic + (group * warps + (tid >> 5)) * kStage);
    uint4 *const s_ring = s_dynamic + (pitch >> 5) * kStage;
    const int step = blockDim.x * V;
    const bool two = kGate || (!kPlain && p.b != nullptr);
    const RowSource W = row_source(p.w, 0, p.cols, 0, p.w_f32 ? 4 : E, 1);
    const unsigned rows = (unsigned)p.rows, stride = gridDim.x * blockDim.y;
    unsigned row = blockIdx.x * blockDim.y + group;  // at work on
    int cols = 0;  // of it: none behind the last row
    // (made anew where they are used: they would hold registers all along)
    auto A = [&](unsigned r) { return row_source(p.a, r, p.cols, p.lda, E, p.rows); };
    auto B = [&](unsigned r) { return row_source(p.b, r, p.cols, p.ldb, E, p.rows); };

    if (tid == 0) s_top[0][group] = s_top[1][group] = 0;
    // (The kernel behind this one may start when this one's CTAs end: its own, started earlier, took
    // their places from rows still to be done, 85 us for a training step that takes 73.)
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // Of the thread's elements: h of the norm; what is coded.
    float keep[NP][V];
    float sum, largest;  // of squares; |what is coded|, NaN where one is
    GateSpread spread;

    auto exact = [&](int c) -> double {
        const float a = load_as_float(A(row).row, TYPE, c);
        if constexpr (kPlain) {
            return a;
        } else if constexpr (kGate) {
            return gate_exact<ACT>(a, load_as_float(B(row).row, TYPE, c));
        } else {
            const double h = two ? (double)a + (double)load_as_float(B(row).row, TYPE, c) : (double)a;
            return h * (double)load_as_float(p.w, p.w_f32 ? kTypeF32 : TYPE, c);
        }
    };
    // A piece (n > 0 elements from c on) as it comes from memory; what of it is kept.
    auto fetch = [&](int c, int n, uint4 &x, uint4 &y) {
        x = load_piece<TYPE, ALIGNED>(A(row), c * E, n);
        if (two) y = load_piece<TYPE, ALIGNED>(B(row), c * E, n);
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
        char *first = static_cast<char *>(to) + ((long long)row * ld + c - lane * V) * E;
        store_piece<TYPE, ALIGNED>(first, n, pack_piece<TYPE>(v), stage);
    };
    // h over x or the residual would take from exact() what it reads: then it is stored last.
    const bool early = KEEP && (OP == kRowNorm || !p.h_last);

    // In registers: the pieces of the next rows are on their way, a thread's own into its own
    // places of a ring, so that nobody has to wait for another's.
    constexpr int kSlots = piece_slots(ALIGNED);
    const int arrays = two ? 2 : 1;
    auto slot = [&](int stage_of, int array, int i) {
        return s_ring + (((stage_of * arrays + array) * NP + i) * kSlots) * pitch + group * blockDim.x + tid;
    };
    auto start = [&](unsigned r, int stage_of) {
        if (r < rows) {
            const RowSource a = A(r), b = B(r);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int c = tid * V + i * step;
                if (c < p.cols) {
                    start_piece<ALIGNED>(slot(stage_of, 0, i), pitch, a, c * E);
                    if (two) start_piece<ALIGNED>(slot(stage_of, 1, i), pitch, b, c * E);
                }
            }
        }
        cp_async_commit();
    };
    int ring = 0;
    if constexpr (KEEP)
        for (int s = 0; s < p.stages; ++s) start(row + s * stride, s);
    static_assert(NP * V <= 32, "");
    // The column of the thread's i-th element in registers.
    auto element = [&](int i) { return tid * V + i / V * step + i % V; };
    // Calls f(c) for each of the thread's elements.
    auto each = [&](auto &&f) {
        for (int c = tid * V; c < p.cols; c += step)
            for (int j = 0; j < min(V, p.cols - c); ++j) f(c + j);
    };
    // What is left to do for a row whose codes are stored: those in doubt (of the thread's
    // elements in registers; `all`: every element) and the scale.
    unsigned doubt = 0;
    bool all = false;
    auto decide = [&](int c, int turn_of) {
        const double top = fmax(__longlong_as_double((long long)s_top[turn_of][group]), (double)kRowTiny);
        p.q[(long long)row * p.ldq + c] = (int8_t)row_code_exact(exact(c), top, 127.0f / (float)top);
    };
    auto finish = [&](int turn_of) {  // of `row`
        for (; doubt; doubt &= doubt - 1) decide(element(__ffs(doubt) - 1), turn_of);
        if (all) each([&](int c) { decide(c, turn_of); });
        all = false;
        // (Rounded to FP32 before the division: in 64 bits, rounded once, it would be off by 2.8e-8 of
        // itself where it is by 3.8e-8, and rows of 233 BF16 would take 25.4 us for 22.8.)
        if (tid == 0 && row < rows)
            p.scales[row] = fmaxf((float)__longlong_as_double((long long)s_top[turn_of][group]), kRowTiny) /
                            127.0f * s_root[turn_of][group];
    };
    auto finish_last = [&](int turn_of) {  // of the row before
        if (doubt || all || tid == 0) {
            row -= stride;
            finish(turn_of);
            row += stride;
        }
    };
    int turn = 0;
    bool flip = false, begun = false;
    for (; row - group < rows; row += stride, flip = !flip) {
        cols = row < rows ? p.cols : 0;
        sum = largest = 0.0f;
        spread = GateSpread();
        if constexpr (KEEP) {
            // All but the last stages - 1 rows' copies have landed.
            if (p.stages == 1) cp_async_wait<0>();
            else if (p.stages == 2) cp_async_wait<1>();
            else cp_async_wait<2>();
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const int c = tid * V + i * step, n = cols - c;
                if (c - lane * V < cols) {  // (the whole warp, for put())
                    uint4 x = make_uint4(0, 0, 0, 0), y = x;
                    if (n > 0) {
                        x = take_piece<TYPE, ALIGNED>(slot(ring, 0, i), pitch, A(row), c * E);
                        if (two) y = take_piece<TYPE, ALIGNED>(slot(ring, 1, i), pitch, B(row), c * E);
                    }
                    take(x, y, keep[i]);
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
            start(row + p.stages * stride, ring);
            if (++ring == p.stages) ring = 0;
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
        bool far = false;
        if constexpr (kGate && ACT != kGateRelu) {
            // An element beyond z = -80 matters from |g u| = 100 on: below, its magnitude is under
            // 2^-108 and its code zero whatever it is.  One that is not finite in FP32 may be in 64 bits.
            constexpr float kInf = std::numeric_limits<float>::infinity();
            if (spread.lowest < -80.0f || largest >= kInf || largest != largest) {
                each([&](int c) {
                    const float g = load_as_float(A(row).row, TYPE, c), u = load_as_float(B(row).row, TYPE, c);
                    far = far || (gate_z<ACT>(g) < -80.0f && !(fabsf(g * u) < 100.0f)) || !(largest < kInf);
                });
                if (far) {
                    largest = 0.0f;
                    each([&](int c) { largest = max_nan(largest, (float)fabs(exact(c))); });
                }
            }
        }

        // Over the row's threads.
        unsigned most = __float_as_uint(largest);  // (above infinity's bits where it is NaN)
        if constexpr (kStores) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        if constexpr (OP != kRowNorm) most = __reduce_max_sync(0xffffffffu, most);
        unsigned mass = __float_as_uint(spread.mass);
        if constexpr (ACT == kGateGelu) mass = __reduce_max_sync(0xffffffffu, mass);
        if (OP != kRowNorm || warps > 1) {
            const int slot = group * warps;
            if (lane == 0) {
                s_sum[flip][slot + (tid >> 5)] = sum;
                s_max[flip][slot + (tid >> 5)] = most;
                if constexpr (ACT == kGateGelu) s_mass[flip][slot + (tid >> 5)] = mass;
            }
            __syncthreads();
            if constexpr (kStores) {
                sum = lane < warps ? s_sum[flip][slot + lane] : 0.0f;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            }
            if constexpr (OP != kRowNorm)
                most = __reduce_max_sync(0xffffffffu, lane < warps ? s_max[flip][slot + lane] : 0u);
            if constexpr (ACT == kGateGelu)
                mass = __reduce_max_sync(0xffffffffu, lane < warps ? s_mass[flip][slot + lane] : 0u);
        }
        const float rstd = kStores ? rsqrtf(fmaf(sum, p.inv_cols, p.eps)) : 1.0f;

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
                if (!KEEP && p.h) put(p.h, p.ldh, c, n, v);
                put(p.y, p.ldy, c, n, y);
            });
        } else {
            // Nobody reads what the row before the last one left any more.
            const int next_turn = turn == 2 ? 0 : turn + 1;
            if (tid == 0) s_top[next_turn][group] = 0;
            const bool later = KEEP && !p.h_last;  // what is left of a row is done with the next one
            if (later && begun) finish_last(turn == 0 ? 2 : turn - 1);
            begun = true;
            const bool bad = most >= 0x7F800000u;
            const float top = fmaxf(__uint_as_float(most), kRowTiny);
            const float inv = bad ? 0.0f : 127.0f / top;
            all = far && !bad;
            if (tid == 0) s_root[turn][group] = bad ? __int_as_float(0x7FC00000) : rstd;
            // The largest magnitude in more bits, among those that FP32 cannot tell from it.
            const float limit = top * (1.0f - 0x1p-12f);
            auto refine = [&]() {
                if (bad || !(largest >= limit)) return;
                auto raise = [&](int c) {
                    atomicMax(&s_top[turn][group],
                              (unsigned long long)__double_as_longlong(fabs(exact(c))));
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
            };
            if constexpr (!KEEP) {
                refine();
                __syncthreads();
            }
            // What FP32 does not decide: a quotient nearer to the middle between two codes than it
            // is off itself, kOff of it for a and top (in the gate 2^-20.5 each, two roundings
            // each in the norm) and, in GELU, twice what the exponents are off.
            constexpr float kOff = kGate ? 0x1p-19f : 0x1p-21f;
            float border = 0.5f - 0x1p-19f;
            if constexpr (ACT == kGateGelu) border -= fminf(__uint_as_float(mass) * inv, 1e4f) * 0x1p-20f;
            pieces([&](int c, int n, float (&v)[V], int number) {
                if (n <= 0) return;
                // v inv + 1.5 2^23 is rounded to a whole number, ties to even, whose low byte is
                // the code's.
                constexpr float kWhole = 12582912.0f;
                uint32_t r[V], word[V / 4];
                float widest = 0.0f;
                auto doubt_of = [&](int j, uint32_t &bits) {
                    const float q = fmaf(v[j], inv, kWhole), k = kWhole - q;
                    bits = __float_as_uint(q);
                    return fmaf(fabsf(k), kOff, fabsf(fmaf(v[j], inv, k)));
                };
#pragma unroll
                for (int j = 0; j < V; ++j) widest = fmaxf(widest, doubt_of(j, r[j]));
#pragma unroll
                for (int k = 0; k < V / 4; ++k)
                    word[k] = bad ? 0u
                                  : __byte_perm(__byte_perm(r[4 * k], r[4 * k + 1], 0x0040),
                                                __byte_perm(r[4 * k + 2], r[4 * k + 3], 0x0040), 0x5410);
                int8_t *out = p.q + (long long)row * p.ldq + c;
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
                        uint32_t bits;
                        mask |= (unsigned)(j < n && doubt_of(j, bits) > border) << j;
                    }
                    if constexpr (KEEP)
                        doubt |= mask << (number * V);
                    else
                        for (; mask; mask &= mask - 1) decide(c + __ffs(mask) - 1, turn);
                }
            });
            if constexpr (KEEP) refine();
            // Decided when all of the row's threads have refined its largest magnitude: after the
            // next row's barrier, or (h over what decide() reads) one of its own.
            if (!later) {
                if constexpr (KEEP) __syncthreads();
                finish(turn);
                if (OP == kRowNormQ8 && p.h)
                    for (int c = tid * V; c - lane * V < cols; c += step) {
                        uint4 x = make_uint4(0, 0, 0, 0), y = x;
                        float v[V];
                        if (c < cols) fetch(c, cols - c, x, y);
                        take(x, y, v);
                        put(p.h, p.ldh, c, cols - c, v);
                    }
            }
            turn = next_turn;
        }
    }
    if (OP != kRowNorm && KEEP && !p.h_last) {
        __syncthreads();
        if (begun) finish_last(turn == 0 ? 2 : turn - 1);
    }
}

// So few rows that each thread has one piece of one.
template <int TYPE, int OP>
bool few_rows(const RowParams &p, int num_sms) {
    constexpr int V = piece_elements(TYPE);
    return p.rows <= 2 * num_sms && (p.cols + V - 1) / V <= row_threads(OP);
}

template <int TYPE, int OP, int ACT, bool ALIGNED>
cudaError_t launch_op(const RowParams &p, int num_sms, cudaStream_t stream) {
    constexpr int V = piece_elements(TYPE), kDeep = row_pieces(OP);
    // Threads of a row: with few rows as many as leave each one piece, else as many as
    // hold the row in registers.
    const long long most = (p.cols + V - 1) / V;  // pieces
    const bool few = few_rows<TYPE, OP>(p, num_sms);
    const long long want = few ? most : (most + kDeep - 1) / kDeep;
    int threads = 32;
    while (threads < want && threads < 128) threads *= 2;
    if (threads < want) threads = (int)std::min<long long>((want + 31) / 32 * 32, row_threads(OP));
    const int groups = threads >= 128 ? 1 : 128 / threads;
    const bool fits = (long long)threads * (few ? 1 : kDeep) >= most;
    cudaLaunchConfig_t cfg = {};
    // As many CTAs as the SMs hold at once, each taking rows in turn.
    const int per_sm = std::max(1, 65536 / row_regs(OP, ACT, ALIGNED) / (threads * groups));
    cfg.gridDim = dim3((unsigned)std::min<long long>((p.rows + groups - 1) / groups, (long long)num_sms * per_sm));
    cfg.blockDim = dim3(threads, groups);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // A ring of up to three rows' pieces in what shared memory the SM has for so many threads.
    RowParams q = p;
    const int bytes = (OP == kRowGateQ8 ? (ACT >= 0 ? 2 : 1) : p.b ? 2 : 1) * (few ? 1 : kDeep) *
                      piece_slots(ALIGNED) * 16 * threads * groups;
    q.stages = std::max(1, std::min(3, kRingBytes / (bytes * per_sm)));
    constexpr int kStageBytes = OP != kRowGateQ8 && !ALIGNED ? kStageWords * 4 : 0;  // of a warp
    cfg.dynamicSmemBytes = (size_t)threads * groups / 32 * kStageBytes;
    // (Many rows off 16 bytes have a kernel of their own in the norm.)
    constexpr bool kFewOnly = OP == kRowNorm && !ALIGNED;
    if (!fits || (kFewOnly && !few))
        return cudaLaunchKernelEx(&cfg, row_kernel<TYPE, OP, ACT, 1, false, ALIGNED>, q);
    cfg.dynamicSmemBytes += (size_t)bytes * q.stages;
    const auto kernel = few ? row_kernel<TYPE, OP, ACT, 1, true, ALIGNED>
                            : row_kernel<TYPE, OP, ACT, kFewOnly ? 1 : kDeep, true, ALIGNED>;
    static std::atomic<bool> configured[kMaxDevices][2];
    if (p.device >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!configured[p.device][few].load()) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kRingBytes + row_threads(OP) / 32 * kStageBytes);
        if (e != cudaSuccess) return e;
        configured[p.device][few].store(true);
    }
    return cudaLaunchKernelEx(&cfg, kernel, q);
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
