// Gradients of the root-mean-square norm.
//
//   r = 1 / sqrt(mean(h^2) + eps), n = dy w
//   dx = r n - (h r) (r^2 mean(n h)) + dh,  dw = sum over rows of dy (h r)
//
// A group of threads holds a row of h and dy in registers (its next rows are on their way to
// shared memory), reduces both sums at once, and writes dx; it owns the same columns in every
// row that it takes, so the weight's gradient gathers in its registers and leaves once, a
// CTA's groups added up, as one of `parts` partial rows, which a second kernel adds up in order.  Every input is read once and
// every output written once (plus the partial rows).  Rows that are too long for
// registers are read again (norm_grad_wide_kernel).  16-bit rows of more than 8192 columns
// keep the weight's gradient in shared memory, and dy and dh stay there until they are used
// (calls from Python with cold inputs and dh, and in two readings: 1388 x 10504 BF16 63 us, 88;
// 2048 x 16384 101, 182; 1388 x 10504 off 16 bytes 89, 159).
//
// 8192 x 2048 BF16 with residual and dh: 39 us and 5 for the partial rows (its bytes take 25).  Bound:
// latency, one CTA of 512 threads an SM, which the weight's gradient leaves no registers beside
// (three of 256 with it in shared memory took 1 us more, 4096 x 4096 5).
// Rows off 16 bytes: 1023 x 1025 FP32 12 and 5 us.
#include <algorithm>
#include <atomic>

#include "kernels_q8.h"
#include "row_io.cuh"

namespace sgemm {
namespace {

constexpr int kMostThreads = 512;
constexpr int kMaxDevices = 64;
constexpr int kRingBytes = 192 * 1024;  // of an SM, for rows on their way
constexpr int kLateBytes = 214 * 1024;  // and the weight's gradient beside them
// Whether a thread of so many pieces has registers for a row's h alone.
constexpr bool is_late(int type, int np) { return piece_elements(type) * np > 16; }
// Matrices whose pieces are on their way, of those that there are.
constexpr int ring_arrays(int type, int np, bool r, bool dh) { return 2 + r + (dh && (np <= 2 || is_late(type, np))); }

__device__ __forceinline__ float2 warp_sum2(float2 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    return v;
}
// Over the `warps` warps of each group, which wait for one another alone; `buf` alternates,
// so that one barrier is enough.
__device__ __forceinline__ float2 group_sum2(float2 v, float2 (*buf)[32], int group, int warps) {
    v = warp_sum2(v);
    if (warps == 1) return v;
    const int tid = threadIdx.x, lane = tid & 31;
    if (lane == 0) (*buf)[group * warps + (tid >> 5)] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"((int)blockDim.x) : "memory");
    v = lane < warps ? (*buf)[group * warps + lane] : make_float2(0.0f, 0.0f);
    return warp_sum2(v);
}
// r, and r^2 mean(n h), from the sums of h^2 and n h.  (h r is of size one and this of dx's: a
// factor r^3 would leave FP32 for rows of 10^13, and of 10^-13 without eps.)
__device__ __forceinline__ float2 row_stats(float2 sums, int cols, float eps) {
    const float r = rsqrtf(sums.x / (float)cols + eps);
    return make_float2(r, sums.y / (float)cols * r * r);
}

// A piece of a row as it comes from memory; zeros where it has no elements.
struct Raw {
    uint4 x, r, dy, dh;
};
template <int TYPE, bool ALIGNED>
__device__ __forceinline__ Raw fetch(const NormGradParams &p, long long row, int c, int n, bool with_dh) {
    constexpr int E = 16 / piece_elements(TYPE);
    Raw v;
    v.x = v.r = v.dy = v.dh = make_uint4(0, 0, 0, 0);
    if (n <= 0) return v;
    v.x = load_piece<TYPE, ALIGNED>(row_source(p.x, row, p.cols, p.ldx, E, p.rows), c * E, n);
    v.dy = load_piece<TYPE, ALIGNED>(row_source(p.dy, row, p.cols, p.lddy, E, p.rows), c * E, n);
    if (p.r) v.r = load_piece<TYPE, ALIGNED>(row_source(p.r, row, p.cols, p.ldr, E, p.rows), c * E, n);
    if (with_dh) v.dh = load_piece<TYPE, ALIGNED>(row_source(p.dh, row, p.cols, p.lddh, E, p.rows), c * E, n);
    return v;
}
// h: the sum of its parts in FP32.
template <int TYPE>
__device__ __forceinline__ void sum_h(const Raw &v, bool two, float (&h)[piece_elements(TYPE)]) {
    unpack_piece<TYPE>(v.x, h);
    if (two) {
        float r[piece_elements(TYPE)];
        unpack_piece<TYPE>(v.r, r);
#pragma unroll
        for (int j = 0; j < piece_elements(TYPE); ++j) h[j] += r[j];
    }
}
// dx of a piece, from h r.
template <int TYPE>
__device__ __forceinline__ uint4 make_dx(const float (&hr)[piece_elements(TYPE)], const float (&w)[piece_elements(TYPE)],
                                         const float (&dy)[piece_elements(TYPE)], uint4 dh_raw, float2 st) {
    constexpr int V = piece_elements(TYPE);
    float dx[V];
    unpack_piece<TYPE>(dh_raw, dx);
#pragma unroll
    for (int j = 0; j < V; ++j) dx[j] = fmaf(-hr[j], st.y, fmaf(dy[j] * w[j], st.x, dx[j]));
    return pack_piece<TYPE>(dx);
}

// NP: pieces of a thread.
template <int TYPE, int NP, bool ALIGNED>
__global__ void __launch_bounds__(kMostThreads, 1) norm_grad_kernel(const NormGradParams p) {
    constexpr int V = piece_elements(TYPE), E = 16 / V, kSlots = piece_slots(ALIGNED);
    __shared__ float2 s_sum[2][32];
    __shared__ uint4 s_stage[ALIGNED ? 1 : kMostThreads / 32 * kStageWords / 4];
    extern __shared__ uint4 s_ring[];  // pieces of the next rows, a thread's own in its own places
    const int tid = threadIdx.x, lane = tid & 31, group = threadIdx.y, groups = blockDim.y;
    const int warps = blockDim.x >> 5, step = blockDim.x * V, pitch = blockDim.x * groups;
    uint32_t *stage = reinterpret_cast<uint32_t *>(s_stage) +
                      (ALIGNED ? 0 : (group * warps + (tid >> 5)) * kStageWords);
    const RowSource W = row_source(p.w, 0, p.cols, 0, p.w_f32 ? 4 : E, 1);
    // kLate: dy, dh and dw lie in shared memory.  Else (with three pieces or four) dh is loaded
    // where it is used: it would not fit the registers.
    constexpr bool kLate = is_late(TYPE, NP), kAhead = NP <= 2;
    const int arrays = ring_arrays(TYPE, NP, p.r, p.dh);
    float4 *const s_dw = reinterpret_cast<float4 *>(s_ring + p.stages * arrays * NP * kSlots * pitch) + tid;  // (kLate)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float dw[kLate ? 1 : NP][V];
#pragma unroll
    for (int i = 0; i < (kLate ? 1 : NP); ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) dw[i][j] = 0.0f;
    if (kLate)
        for (int i = 0; i < NP * V / 4; ++i) s_dw[i * pitch] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);

    auto slot = [&](int ring, int array, int i) {
        return s_ring + (((ring * arrays + array) * NP + i) * kSlots) * pitch + group * blockDim.x + tid;
    };
    // In this order in a stage: x, dy, r, dh.
    auto source = [&](int array, unsigned row) {
        if (array == 2 && !p.r) array = 3;
        return array == 0   ? row_source(p.x, row, p.cols, p.ldx, E, p.rows)
               : array == 1 ? row_source(p.dy, row, p.cols, p.lddy, E, p.rows)
               : array == 2 ? row_source(p.r, row, p.cols, p.ldr, E, p.rows)
                            : row_source(p.dh, row, p.cols, p.lddh, E, p.rows);
    };
    auto start = [&](unsigned row, int ring) {
        if (row < p.rows) {
#pragma unroll
            for (int a = 0; a < 4; ++a)
                if (a < arrays) {
                    const RowSource m = source(a, row);
#pragma unroll
                    for (int i = 0; i < NP; ++i)
                        if (tid * V + i * step < p.cols)
                            start_piece<ALIGNED>(slot(ring, a, i), pitch, m, (tid * V + i * step) * E);
                }
        }
        cp_async_commit();
    };
    auto take = [&](int ring, int array, int i, unsigned row) {
        return take_piece<TYPE, ALIGNED>(slot(ring, array, i), pitch, source(array, row), (tid * V + i * step) * E);
    };
    const unsigned first = blockIdx.x * groups + group, stride = gridDim.x * groups;
    for (int s = 0; s < p.stages; ++s) start(first + s * stride, s);
    int flip = 0, ring = 0;
    for (unsigned row = first; row < p.rows; row += stride, flip ^= 1) {
        // All but the last stages - 1 rows' copies have landed.
        if (p.stages == 1) cp_async_wait<0>();
        else if (p.stages == 2) cp_async_wait<1>();
        else cp_async_wait<2>();
        float h[NP][V];
        uint4 dy_raw[kLate ? 1 : NP], dh_raw[kLate ? 1 : NP];
        float2 sums = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int c = tid * V + i * step;
            if (c < p.cols) {
                float w[V], dy[V];
                unpack_piece<TYPE>(take(ring, 0, i, row), h[i]);
                if (p.r) {
                    unpack_piece<TYPE>(take(ring, 2, i, row), w);
#pragma unroll
                    for (int j = 0; j < V; ++j) h[i][j] += w[j];
                }
                const uint4 raw = take(ring, 1, i, row);
                if (!kLate) dy_raw[i] = raw;
                if (kAhead) dh_raw[i] = p.dh ? take(ring, arrays - 1, i, row) : make_uint4(0, 0, 0, 0);
                load_weight<TYPE, ALIGNED>(W, p.w_f32, c, p.cols - c, w);
                unpack_piece<TYPE>(raw, dy);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    sums.x = fmaf(h[i][j], h[i][j], sums.x);
                    sums.y = fmaf(dy[j] * w[j], h[i][j], sums.y);
                }
            }
        }
        if (!kLate) start(row + p.stages * stride, ring);
        const float2 st = row_stats(group_sum2(sums, &s_sum[flip], group, warps), p.cols, p.eps);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int c = tid * V + i * step, n = p.cols - c;
            float dy[V];
            uint4 dh = make_uint4(0, 0, 0, 0);
            if (n > 0) {
#pragma unroll
                for (int j = 0; j < V; ++j) h[i][j] *= st.x;
                if constexpr (kLate) {
                    unpack_piece<TYPE>(take(ring, 1, i, row), dy);
                    if (p.dh) dh = take(ring, arrays - 1, i, row);
#pragma unroll
                    for (int k = 0; k < V / 4; ++k) {
                        float4 *at = s_dw + (i * (V / 4) + k) * pitch, d = *at;
                        d.x = fmaf(dy[4 * k], h[i][4 * k], d.x);
                        d.y = fmaf(dy[4 * k + 1], h[i][4 * k + 1], d.y);
                        d.z = fmaf(dy[4 * k + 2], h[i][4 * k + 2], d.z);
                        d.w = fmaf(dy[4 * k + 3], h[i][4 * k + 3], d.w);
                        *at = d;
                    }
                } else {
                    unpack_piece<TYPE>(dy_raw[i], dy);
#pragma unroll
                    for (int j = 0; j < V; ++j) dw[i][j] = fmaf(dy[j], h[i][j], dw[i][j]);
                    if (kAhead) dh = dh_raw[i];
                }
            }
            if (p.dx && c - lane * V < p.cols) {  // (the whole warp)
                float w[V];
                if (n > 0) {
                    load_weight<TYPE, ALIGNED>(W, p.w_f32, c, n, w);
                    if (!kAhead && !kLate && p.dh) dh = load_piece<TYPE, ALIGNED>(source(3, row), c * E, n);
                }
                store_piece<TYPE, ALIGNED>(static_cast<char *>(p.dx) + ((long long)row * p.lddx + c - lane * V) * E, n,
                                           make_dx<TYPE>(h[i], w, dy, dh, st), stage);
            }
        }
        if (kLate) start(row + p.stages * stride, ring);
        if (++ring == p.stages) ring = 0;
    }
    if (!p.dw) return;
    if constexpr (kLate) {  // (one group)
        for (int i = 0; i < NP * V / 4; ++i) {
            const float4 d = s_dw[i * pitch];
            const int c = tid * V + i / (V / 4) * step + i % (V / 4) * 4;
            float *out = p.partials + (long long)blockIdx.x * p.cols + c;
            if (c < p.cols) __stcg(out, d.x);
            if (c + 1 < p.cols) __stcg(out + 1, d.y);
            if (c + 2 < p.cols) __stcg(out + 2, d.z);
            if (c + 3 < p.cols) __stcg(out + 3, d.w);
        }
        return;
    }
    // The groups' sums, added up in order: one partial row of a CTA.
    cp_async_wait<0>();
    __syncthreads();
    float *all = reinterpret_cast<float *>(s_ring);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int c = tid * V + i * step;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (c + j < p.cols) all[group * p.cols + c + j] = dw[i][j];
    }
    __syncthreads();
    for (int c = group * blockDim.x + tid; c < p.cols; c += pitch) {
        float sum = all[c];
        for (int g = 1; g < groups; ++g) sum += all[g * p.cols + c];
        __stcg(p.partials + (long long)blockIdx.x * p.cols + c, sum);
    }
}

// A CTA a row: both sums, then dx from a second reading; the row's statistics go
// to the kernel below.
template <int TYPE, bool ALIGNED>
__global__ void __launch_bounds__(kMostThreads, 1) norm_grad_wide_kernel(const NormGradParams p) {
    constexpr int V = piece_elements(TYPE), E = 16 / V;
    __shared__ float2 s_sum[32];
    __shared__ uint4 s_stage[ALIGNED ? 1 : kMostThreads / 32 * kStageWords / 4];
    const int tid = threadIdx.x, lane = tid & 31, step = blockDim.x * V;
    uint32_t *stage = reinterpret_cast<uint32_t *>(s_stage) + (ALIGNED ? 0 : (tid >> 5) * kStageWords);
    const long long row = blockIdx.x;
    const RowSource W = row_source(p.w, 0, p.cols, 0, p.w_f32 ? 4 : E, 1);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float2 sums = make_float2(0.0f, 0.0f);
    float h[V], dy[V], w[V];
    for (int c = tid * V; c < p.cols; c += step) {
        const Raw raw = fetch<TYPE, ALIGNED>(p, row, c, p.cols - c, false);
        sum_h<TYPE>(raw, p.r, h);
        unpack_piece<TYPE>(raw.dy, dy);
        load_weight<TYPE, ALIGNED>(W, p.w_f32, c, p.cols - c, w);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            sums.x = fmaf(h[j], h[j], sums.x);
            sums.y = fmaf(dy[j] * w[j], h[j], sums.y);
        }
    }
    const float2 st = row_stats(group_sum2(sums, &s_sum, 0, blockDim.x >> 5), p.cols, p.eps);
    if (tid == 0 && p.stats) p.stats[row] = st.x;
    if (!p.dx) return;
    for (int c = tid * V; c - lane * V < p.cols; c += step) {
        const int n = p.cols - c;
        const Raw raw = fetch<TYPE, ALIGNED>(p, row, c, n, p.dh);
        sum_h<TYPE>(raw, p.r, h);
        unpack_piece<TYPE>(raw.dy, dy);
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] *= st.x;
        if (n > 0) load_weight<TYPE, ALIGNED>(W, p.w_f32, c, n, w);
        store_piece<TYPE, ALIGNED>(static_cast<char *>(p.dx) + (row * p.lddx + c - lane * V) * E, n,
                                   make_dx<TYPE>(h, w, dy, raw.dh, st), stage);
    }
}

// Partial rows of dw where rows do not fit registers: a thread a column, a CTA
// every parts-th row.
template <int TYPE>
__global__ void __launch_bounds__(256) norm_grad_columns_kernel(const NormGradParams p) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (c >= p.cols) return;
    float sum = 0.0f;
#pragma unroll 4
    for (long long row = blockIdx.y; row < p.rows; row += p.parts) {
        float h = load_as_float(p.x, TYPE, row * p.ldx + c);
        if (p.r) h += load_as_float(p.r, TYPE, row * p.ldr + c);
        sum = fmaf(load_as_float(p.dy, TYPE, row * p.lddy + c), h * p.stats[row], sum);
    }
    p.partials[(long long)blockIdx.y * p.cols + c] = sum;
}

// dw: the partial rows added up, eight columns a CTA (a thread adds few of them, so
// that its loads are under way at once).
__global__ void __launch_bounds__(1024) norm_grad_reduce_kernel(const NormGradParams p, int type) {
    __shared__ float s[32][9];
    const int c = blockIdx.x * 8 + threadIdx.x, y = threadIdx.y;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float sum = 0.0f;
    if (c < p.cols) {
#pragma unroll 8
        for (int q = y; q < p.parts; q += 128) sum += __ldcg(p.partials + (long long)q * p.cols + c);
    }
    // A warp has four values of each column.
    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
    if (y % 4 == 0) s[y / 4][threadIdx.x] = sum;
    __syncthreads();
    if (y >= 32) return;
    // Eight warps, a column each.
    const int lane = (y * 8 + threadIdx.x) & 31, column = (y * 8 + threadIdx.x) >> 5;
    sum = s[lane][column];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const int out = blockIdx.x * 8 + column;
    if (lane == 0 && out < p.cols) store_from_float(p.dw, p.w_f32 ? kTypeF32 : type, out, sum);
}

// Most pieces of a thread that fit its registers.
constexpr int grad_depth(int type, bool aligned) { return type != kTypeF32 ? 2 : aligned ? 4 : 3; }

// 16-bit rows of more columns: pieces of a thread, bytes of a stage of the ring, and of dw.
constexpr int kLatePieces = 4;
int stage_bytes(int type, int np, bool vec, bool r, bool dh, int threads) {
    return ring_arrays(type, np, r, dh) * np * piece_slots(vec) * 16 * threads;
}
int late_bytes(int threads) { return kLatePieces * 8 * 4 * threads; }

// How a row lies over threads: pieces of a thread (0: too many for registers),
// threads of a row, rows that a CTA has at once, CTAs (one on an SM).
struct Shape {
    int depth, threads, groups, ctas;
};
Shape shape(long long rows, int cols, int type, bool vec, bool r, int num_sms) {
    const int most = grad_depth(type, vec);
    Shape s;
    const int pieces = (cols + piece_elements(type) - 1) / piece_elements(type);
    s.depth = pieces <= kMostThreads && rows <= num_sms ? 1 : pieces <= 2 * kMostThreads ? 2
              : pieces <= most * kMostThreads ? most : 0;
    if (s.depth == 0 && type != kTypeF32 && pieces <= kLatePieces * kMostThreads) {
        // As many threads as there is shared memory for, with dh or without (dw's order is the same).
        for (int each = (pieces + kMostThreads - 1) / kMostThreads; each <= kLatePieces && s.depth == 0; ++each) {
            s.threads = (pieces + 32 * each - 1) / (32 * each) * 32;
            if (stage_bytes(type, kLatePieces, vec, r, true, s.threads) + late_bytes(s.threads) > kLateBytes) continue;
            s.depth = kLatePieces;
            s.groups = 1;
            s.ctas = (int)std::min<long long>(rows, num_sms);
        }
        return s;
    }
    if (s.depth == 0) return s;
    s.threads = std::max(1, (pieces + 32 * s.depth - 1) / (32 * s.depth)) * 32;
    // Few rows are spread over the SMs first.
    s.groups = (int)std::max<long long>(1, std::min<long long>({kMostThreads / s.threads, 15, rows / num_sms}));
    s.ctas = (int)std::min<long long>((rows + s.groups - 1) / s.groups, num_sms);
    return s;
}
constexpr int kWideParts = 64;

template <class... Params, class... Args>
cudaError_t launch(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                   Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int TYPE, int NP, bool ALIGNED>
cudaError_t launch_depth(const NormGradParams &p, const Shape &s, cudaStream_t stream) {
    const auto kernel = norm_grad_kernel<TYPE, NP, ALIGNED>;
    constexpr bool kLate = is_late(TYPE, NP);
    static std::atomic<bool> configured[kMaxDevices];
    if (p.device >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!configured[p.device].load()) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kLate ? kLateBytes : kRingBytes);
        if (e != cudaSuccess) return e;
        configured[p.device].store(true);
    }
    NormGradParams q = p;
    const int bytes = stage_bytes(TYPE, NP, ALIGNED, p.r, p.dh, s.threads) * s.groups;
    const int beside = kLate ? late_bytes(s.threads) : 0;
    q.stages = std::max(1, std::min(3, ((kLate ? kLateBytes : kRingBytes) - beside) / bytes));
    const size_t all = kLate ? 0 : (size_t)s.groups * p.cols * sizeof(float);  // the groups' sums
    const size_t smem = std::max<size_t>((size_t)bytes * q.stages + beside, all);
    return launch(kernel, dim3(s.ctas), dim3(s.threads, s.groups), smem, stream, q);
}

template <int TYPE, bool ALIGNED>
cudaError_t launch_form(const NormGradParams &p, int num_sms, cudaStream_t stream) {
    const Shape s = shape(p.rows, p.cols, TYPE, ALIGNED, p.r, num_sms);
    cudaError_t e;
    if (s.depth) {
        constexpr int kMost = TYPE == kTypeF32 ? grad_depth(TYPE, ALIGNED) : kLatePieces;
        e = s.depth == 1   ? launch_depth<TYPE, 1, ALIGNED>(p, s, stream)
            : s.depth == 2 ? launch_depth<TYPE, 2, ALIGNED>(p, s, stream)
                           : launch_depth<TYPE, kMost, ALIGNED>(p, s, stream);
    } else {
        // dx may lie over dy: the statistics first, then dw, then dx.
        NormGradParams q = p;
        e = cudaSuccess;
        if (p.dw) {
            q.dx = nullptr;
            e = launch(norm_grad_wide_kernel<TYPE, ALIGNED>, dim3((unsigned)p.rows), dim3(kMostThreads), 0, stream, q);
            if (e == cudaSuccess)
                e = launch(norm_grad_columns_kernel<TYPE>, dim3((p.cols + 255) / 256, p.parts), dim3(256), 0,
                           stream, p);
        }
        if (e == cudaSuccess && p.dx)
            e = launch(norm_grad_wide_kernel<TYPE, ALIGNED>, dim3((unsigned)p.rows), dim3(kMostThreads), 0, stream, p);
    }
    if (e != cudaSuccess || !p.dw) return e;
    return launch(norm_grad_reduce_kernel, dim3((p.cols + 7) / 8), dim3(8, 128), 0, stream, p, TYPE);
}

}  // namespace

NormGradSpace norm_grad_space(const NormGradParams &p, int type, bool vec, int num_sms) {
    if (!p.dw) return {0, false};
    const Shape s = shape(p.rows, p.cols, type, vec, p.r, num_sms);
    return {s.depth ? s.ctas : (int)std::min<long long>(p.rows, kWideParts), s.depth == 0};
}

cudaError_t launch_norm_grad(const NormGradParams &p, int type, bool vec, int num_sms,
                             cudaStream_t stream) {
    switch (type) {
        case kTypeF32:
            return vec ? launch_form<kTypeF32, true>(p, num_sms, stream)
                       : launch_form<kTypeF32, false>(p, num_sms, stream);
        case kTypeF16:
            return vec ? launch_form<kTypeF16, true>(p, num_sms, stream)
                       : launch_form<kTypeF16, false>(p, num_sms, stream);
        default:
            return vec ? launch_form<kTypeBF16, true>(p, num_sms, stream)
                       : launch_form<kTypeBF16, false>(p, num_sms, stream);
    }
}

}  // namespace sgemm
