// Gradients of the root-mean-square norm.
//
//   r = 1 / sqrt(mean(h^2) + eps), n = dy w
//   dx = r (n - h r^2 mean(n h)) + dh,  dw = sum over rows of dy h r
//
// A group of threads holds a row of h and dy in registers, reduces both sums at
// once, and writes dx; it owns the same columns in every row that it takes, so the
// weight's gradient gathers in its registers and leaves once, as one of `parts` partial
// rows, which a second kernel adds up in order.  Every input is read once and
// every output written once (plus the partial rows).  Rows that are too long for
// registers are read again (norm_grad_wide_kernel).
#include <algorithm>

#include "kernels_q8.h"
#include "row_io.cuh"

namespace sgemm {
namespace {

constexpr int kMostThreads = 512;

__device__ __forceinline__ float2 warp_sum2(float2 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    return v;
}
// Over the `warps` warps of each group; `buf` alternates, so that one barrier is enough.
__device__ __forceinline__ float2 group_sum2(float2 v, float2 (*buf)[32], int group, int warps) {
    v = warp_sum2(v);
    if (warps == 1) return v;
    const int tid = threadIdx.x, lane = tid & 31;
    if (lane == 0) (*buf)[group * warps + (tid >> 5)] = v;
    __syncthreads();
    v = lane < warps ? (*buf)[group * warps + lane] : make_float2(0.0f, 0.0f);
    return warp_sum2(v);
}
// r, and r^3 mean(n h), from the sums of h^2 and n h.
__device__ __forceinline__ float2 row_stats(float2 sums, int cols, float eps) {
    const float r = 1.0f / sqrtf(sums.x / (float)cols + eps);
    return make_float2(r, r * r * r * (sums.y / (float)cols));
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
template <int TYPE>
__device__ __forceinline__ uint4 make_dx(const float (&h)[piece_elements(TYPE)], const float (&w)[piece_elements(TYPE)],
                                         uint4 dy_raw, uint4 dh_raw, float2 st) {
    constexpr int V = piece_elements(TYPE);
    float dy[V], dh[V], dx[V];
    unpack_piece<TYPE>(dy_raw, dy);
    unpack_piece<TYPE>(dh_raw, dh);
#pragma unroll
    for (int j = 0; j < V; ++j) dx[j] = fmaf(-h[j], st.y, dy[j] * w[j] * st.x) + dh[j];
    return pack_piece<TYPE>(dx);
}

// NP: pieces of a thread.  With up to two, the next row is under way while one is worked on.
template <int TYPE, int NP, bool ALIGNED>
__global__ void __launch_bounds__(kMostThreads, 1) norm_grad_kernel(const NormGradParams p) {
    constexpr int V = piece_elements(TYPE), E = 16 / V;
    constexpr bool kAhead = NP <= 2;
    __shared__ float2 s_sum[2][32];
    __shared__ uint4 s_stage[ALIGNED ? 1 : kMostThreads / 32 * kStageWords / 4];
    const int tid = threadIdx.x, lane = tid & 31, group = threadIdx.y, groups = blockDim.y;
    const int warps = blockDim.x >> 5, step = blockDim.x * V;
    uint32_t *stage = reinterpret_cast<uint32_t *>(s_stage) +
                      (ALIGNED ? 0 : (group * warps + (tid >> 5)) * kStageWords);
    const RowSource W = row_source(p.w, 0, p.cols, 0, p.w_f32 ? 4 : E, 1);
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
    float dw[NP][V];
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) dw[i][j] = 0.0f;

    Raw raw[NP];
    auto load = [&](long long row) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int c = tid * V + i * step;
            raw[i] = fetch<TYPE, ALIGNED>(p, row, c, row < p.rows ? p.cols - c : 0, p.dh && kAhead);
        }
    };
    const long long first = (long long)blockIdx.x * groups + group, stride = (long long)gridDim.x * groups;
    if (kAhead) load(first);
    int flip = 0;
    for (long long row = first; row - group < p.rows; row += stride, flip ^= 1) {
        const bool live = row < p.rows;
        if (!kAhead) load(row);
        float h[NP][V];
        uint4 dy_raw[NP], dh_raw[NP];
        float2 sums = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int c = tid * V + i * step;
            sum_h<TYPE>(raw[i], p.r, h[i]);
            dy_raw[i] = raw[i].dy;
            dh_raw[i] = raw[i].dh;
            if (c < p.cols) {
                float w[V], dy[V];
                load_weight<TYPE, ALIGNED>(W, p.w_f32, c, p.cols - c, w);
                unpack_piece<TYPE>(dy_raw[i], dy);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    sums.x = fmaf(h[i][j], h[i][j], sums.x);
                    sums.y = fmaf(dy[j] * w[j], h[i][j], sums.y);
                }
            }
        }
        if (kAhead) load(row + stride);
        const float2 st = row_stats(group_sum2(sums, &s_sum[flip], group, warps), p.cols, p.eps);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int c = tid * V + i * step, n = live ? p.cols - c : 0;
            float dy[V];
            unpack_piece<TYPE>(dy_raw[i], dy);  // (zeros where there are no elements)
#pragma unroll
            for (int j = 0; j < V; ++j) dw[i][j] = fmaf(dy[j] * st.x, h[i][j], dw[i][j]);
            if (p.dx && live && c - lane * V < p.cols) {  // (the whole warp)
                float w[V];
                if (n > 0) {
                    load_weight<TYPE, ALIGNED>(W, p.w_f32, c, n, w);
                    if (!kAhead && p.dh)
                        dh_raw[i] = load_piece<TYPE, ALIGNED>(
                            row_source(p.dh, row, p.cols, p.lddh, E, p.rows), c * E, n);
                }
                store_piece<TYPE, ALIGNED>(static_cast<char *>(p.dx) + (row * p.lddx + c - lane * V) * E, n,
                                           make_dx<TYPE>(h[i], w, dy_raw[i], dh_raw[i], st), stage);
            }
        }
    }
    if (!p.dw) return;
    float *part = p.partials + ((long long)blockIdx.x * groups + group) * p.cols;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const int c = tid * V + i * step;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (c + j < p.cols) __stcg(part + c + j, dw[i][j]);
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
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
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
    if (tid == 0) p.stats[row] = st;
    if (!p.dx) return;
    for (int c = tid * V; c - lane * V < p.cols; c += step) {
        const int n = p.cols - c;
        const Raw raw = fetch<TYPE, ALIGNED>(p, row, c, n, p.dh);
        sum_h<TYPE>(raw, p.r, h);
        if (n > 0) load_weight<TYPE, ALIGNED>(W, p.w_f32, c, n, w);
        store_piece<TYPE, ALIGNED>(static_cast<char *>(p.dx) + (row * p.lddx + c - lane * V) * E, n,
                                   make_dx<TYPE>(h, w, raw.dy, raw.dh, st), stage);
    }
}

// Partial rows of dw where rows do not fit registers: a thread a column, a CTA
// every parts-th row.
template <int TYPE>
__global__ void __launch_bounds__(256) norm_grad_columns_kernel(const NormGradParams p) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
    if (c >= p.cols) return;
    float sum = 0.0f;
#pragma unroll 4
    for (long long row = blockIdx.y; row < p.rows; row += p.parts) {
        float h = load_as_float(p.x, TYPE, row * p.ldx + c);
        if (p.r) h += load_as_float(p.r, TYPE, row * p.ldr + c);
        sum = fmaf(load_as_float(p.dy, TYPE, row * p.lddy + c) * p.stats[row].x, h, sum);
    }
    p.partials[(long long)blockIdx.y * p.cols + c] = sum;
}

// dw: the partial rows added up, eight columns a CTA (a thread adds few of them, so
// that its loads are under way at once).
__global__ void __launch_bounds__(1024) norm_grad_reduce_kernel(const NormGradParams p, int type) {
    __shared__ float s[32][9];
    const int c = blockIdx.x * 8 + threadIdx.x, y = threadIdx.y;
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
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

// How a row lies over threads: pieces of a thread (0: too many for registers),
// threads of a row, rows that a CTA has at once, CTAs.
struct Shape {
    int depth, threads, groups, ctas;
};
Shape shape(long long rows, int cols, int type, bool vec, int num_sms) {
    const int most = vec ? 4 : 3;  // (shifting takes registers)
    Shape s;
    const int pieces = (cols + piece_elements(type) - 1) / piece_elements(type);
    s.depth = pieces <= kMostThreads && rows <= num_sms ? 1 : pieces <= 2 * kMostThreads ? 2
              : pieces <= most * kMostThreads ? most : 0;
    if (s.depth == 0) return s;
    s.threads = std::max(1, (pieces + 32 * s.depth - 1) / (32 * s.depth)) * 32;
    s.groups = s.threads >= 128 ? 1 : 128 / s.threads;
    const int per_sm = std::max(1, kMostThreads / (s.threads * s.groups));
    s.ctas = (int)std::min<long long>((rows + s.groups - 1) / s.groups, (long long)num_sms * per_sm);
    return s;
}
constexpr int kWideParts = 64;

template <class... Params, class... Args>
cudaError_t launch(void (*kernel)(Params...), dim3 grid, dim3 block, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int TYPE, bool ALIGNED>
cudaError_t launch_form(const NormGradParams &p, int num_sms, cudaStream_t stream) {
    const Shape s = shape(p.rows, p.cols, TYPE, ALIGNED, num_sms);
    cudaError_t e;
    if (s.depth) {
        const auto kernel = s.depth == 1   ? norm_grad_kernel<TYPE, 1, ALIGNED>
                            : s.depth == 2 ? norm_grad_kernel<TYPE, 2, ALIGNED>
                                           : norm_grad_kernel<TYPE, ALIGNED ? 4 : 3, ALIGNED>;
        e = launch(kernel, dim3(s.ctas), dim3(s.threads, s.groups), stream, p);
    } else {
        // dx may lie over dy: the statistics first, then dw, then dx.
        NormGradParams q = p;
        e = cudaSuccess;
        if (p.dw) {
            q.dx = nullptr;
            e = launch(norm_grad_wide_kernel<TYPE, ALIGNED>, dim3((unsigned)p.rows), dim3(kMostThreads), stream, q);
            if (e == cudaSuccess)
                e = launch(norm_grad_columns_kernel<TYPE>, dim3((p.cols + 255) / 256, p.parts), dim3(256),
                           stream, p);
        }
        if (e == cudaSuccess && p.dx)
            e = launch(norm_grad_wide_kernel<TYPE, ALIGNED>, dim3((unsigned)p.rows), dim3(kMostThreads), stream, p);
    }
    if (e != cudaSuccess || !p.dw) return e;
    return launch(norm_grad_reduce_kernel, dim3((p.cols + 7) / 8), dim3(8, 128), stream, p, TYPE);
}

}  // namespace

int norm_grad_parts(long long rows, int cols, int type, bool vec, int num_sms) {
    const Shape s = shape(rows, cols, type, vec, num_sms);
    return s.depth ? s.ctas * s.groups : (int)std::min<long long>(rows, kWideParts);
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
