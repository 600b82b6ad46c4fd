// The gated block for up to eight rows (decoding): one pass over the weights.
//
//   gate   g = x Wg, u = x Wu, h = act(g) u   (h stays FP32, T x F)
//   down   y = h Wd
//
// Bound: HBM; every weight is read once and meets T multiply-adds, so with 16-bit
// weights a lane spends about (1 + T / 2) instructions on each (two multiply-adds
// an instruction, packed FP32).  The weights are row-major with k along the rows,
// so a warp reads whole stretches of a row and needs no transposition: lane l
// owns eight or four neighbouring columns of both matrices and
// keeps their sums for all T rows in registers.  Its loads go through a ring in
// shared memory, up to 64 KB of weights a CTA under way at a time: in registers
// there was room for a quarter of it with eight rows of x.
//
// Split.  A CTA owns a stretch of columns and a range of K; its lanes' rows go
// round robin over warps (and over parts of a warp, where the stretch is narrower
// than a warp).  A cluster of CTAs shares K.  Sums are added warp by warp through
// shared memory and CTA by CTA through distributed shared memory, in order: no
// atomics, no workspace.  The down product's launch is a programmatic dependent
// of the gate's: its CTAs start on the SMs that come free and ask for their first
// weights before they wait for h.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "ffn_gate.cuh"

namespace cg = cooperative_groups;

namespace sgemm {
namespace {

constexpr int kMaxDevices = 64;
constexpr int kThreads = 256, kWarps = kThreads / 32;

// A lane's columns of one row: VEC, 16 (or 8) consecutive bytes; else every step-th
// element.  fetch brings them to the lane's own place in shared memory by
// asynchronous copies, take reads them from there; 16-bit elements one by one
// (which those copies cannot do) go straight to registers.
template <int TYPE, int COLS, bool VEC>
struct Columns {
    static constexpr int kCols = COLS;
    static constexpr int kBytes = COLS * (TYPE == kTypeF32 ? 4 : 2);  // 16 or 8
    static constexpr bool kAsync = VEC || TYPE == kTypeF32;
    uint32_t w[4];

    // left: columns from the lane's first to the matrix's end (0: no such row).
    static __device__ __forceinline__ void fetch(uint32_t to, const unsigned char *row, int step,
                                                 int left) {
        if constexpr (VEC) {
            if (left > 0) {
                if constexpr (kBytes == 16)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(row)
                                 : "memory");
                else
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(row)
                                 : "memory");
            }
        } else if constexpr (TYPE == kTypeF32) {
#pragma unroll
            for (int j = 0; j < kCols; ++j)
                if (j * step < left)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + 4 * j),
                                 "l"(row + 4 * j * step)
                                 : "memory");
        }
    }
    __device__ __forceinline__ void take(const unsigned char *from) {
        const uint4 v = *reinterpret_cast<const uint4 *>(from);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    }
    __device__ __forceinline__ void load(const unsigned char *row, int step, int left) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = 0;
#pragma unroll
        for (int j = 0; j < kCols; ++j)
            if (j * step < left)
                w[j / 2] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(row) + j * step)
                            << (16 * (j % 2));
    }
    // Columns 2 i and 2 i + 1.
    __device__ __forceinline__ float2 pair(int i) const {
        if constexpr (TYPE == kTypeF32)
            return make_float2(__uint_as_float(w[2 * i % 4]), __uint_as_float(w[(2 * i + 1) % 4]));
        else
            return unpack16<TYPE>(w[i]);
    }
};

// A lane's columns: eight rows of x with eight columns would leave room for one
// CTA an SM only (195 us for the block of 8 x 4096 x 12288 bf16).
constexpr int cols_of(int type, int t) { return type == kTypeF32 || t == 8 ? 4 : 8; }
// A stage of a warp's ring: round_of rows of each matrix for every lane.
constexpr int round_of(bool gate) { return gate ? 2 : 4; }
constexpr int kStages = 4;
constexpr int kCtasPerSm = 2;
constexpr int kStageBytes = 4 * 512;  // of a warp

template <int TYPE, int T, bool GATE, bool VEC>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) ffn_stream_kernel(const FfnStreamParams p) {
    using C = Columns<TYPE, cols_of(TYPE, T), VEC>;
    constexpr int kMats = GATE ? 2 : 1, kPairs = C::kCols / 2;
    constexpr int kElem = TYPE == kTypeF32 ? 4 : 2;
    constexpr int kRound = round_of(GATE);
    extern __shared__ __align__(16) float smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int lpr = p.lanes_per_row, rpw = 32 / lpr;  // rows of a warp's load
    const int cols = lpr * C::kCols, groups = kWarps * rpw;
    const int c0 = (int)(blockIdx.x / ranks) * cols;
    const int group = warp * rpw + lane / lpr, lane_col = lane % lpr;
    const int step = VEC ? 1 : lpr;
    const int col = c0 + (VEC ? lane_col * C::kCols : lane_col);
    const int k0 = rank * p.cta_rows, k1 = min(p.K, k0 + p.cta_rows);
    const int left = p.N - col;
    float *const xs = smem + kWarps * kStages * kStageBytes / 4;  // x of a chunk, k by k

    if constexpr (GATE) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    float2 acc[kMats][T][kPairs];
#pragma unroll
    for (int a = 0; a < kMats; ++a)
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int i = 0; i < kPairs; ++i) acc[a][t][i] = make_float2(0.0f, 0.0f);

    // The lane's next rows: pointers and number.
    const unsigned char *base[kMats];
    long long row_bytes[kMats], round_bytes[kMats];
    base[0] = static_cast<const unsigned char *>(p.W) + ((k0 + group) * p.ldw + col) * kElem;
    row_bytes[0] = groups * p.ldw * kElem;
    if constexpr (GATE) {
        base[kMats - 1] = static_cast<const unsigned char *>(p.W2) + ((k0 + group) * p.ldw2 + col) * kElem;
        row_bytes[kMats - 1] = groups * p.ldw2 * kElem;
    }
#pragma unroll
    for (int m = 0; m < kMats; ++m) round_bytes[m] = kRound * row_bytes[m];
    int next = k0 + group;
    unsigned char *const ring = reinterpret_cast<unsigned char *>(smem) + warp * (kStages * kStageBytes) + lane * 16;
    const uint32_t ring_addr = (uint32_t)__cvta_generic_to_shared(ring);
    auto fetch = [&](int stage) {
        if constexpr (C::kAsync) {
#pragma unroll
            for (int m = 0; m < kMats; ++m) {
#pragma unroll
                for (int r = 0; r < kRound; ++r)
                    C::fetch(ring_addr + stage * kStageBytes + (m * kRound + r) * 512,
                             base[m] + r * row_bytes[m], step, next + r * groups < k1 ? left : 0);
                base[m] += round_bytes[m];
            }
            next += kRound * groups;
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
    };
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) fetch(i);
    if constexpr (!GATE) asm volatile("griddepcontrol.wait;" ::: "memory");

    int stage = 0;
    for (int a = k0; a < k1; a += p.chunk_rows) {
        const int b = min(k1, a + p.chunk_rows);
        // x of the chunk, k by k, T values each.
        __syncthreads();
#pragma unroll 2
        for (int k = tid; k < b - a; k += kThreads) {
            float v[T];
#pragma unroll
            for (int t = 0; t < T; ++t) {
                v[t] = 0.0f;
                if (t < p.T)
                    v[t] = GATE ? load_as_float(p.x, TYPE, t * p.ldx + a + k)
                                : __ldcg(static_cast<const float *>(p.x) + t * p.ldx + a + k);
            }
            if constexpr (T >= 4) {
#pragma unroll
                for (int t = 0; t < T; t += 4)
                    *reinterpret_cast<float4 *>(xs + k * T + t) =
                        make_float4(v[t], v[t + 1], v[t + 2], v[t + 3]);
            } else {
#pragma unroll
                for (int t = 0; t < T; ++t) xs[k * T + t] = v[t];
            }
        }
        __syncthreads();
        // chunk_rows is a multiple of a round's rows, so rounds do not
        // straddle chunks.
#pragma unroll 1
        for (int k = a + group; k - group < b; k += kRound * groups) {
            if constexpr (C::kAsync)
                asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            C w[kMats][kRound];
#pragma unroll
            for (int m = 0; m < kMats; ++m)
#pragma unroll
                for (int r = 0; r < kRound; ++r) {
                    if constexpr (C::kAsync) {
                        w[m][r].take(ring + stage * kStageBytes + (m * kRound + r) * 512);
                    } else {
                        w[m][r].load(base[m] + r * row_bytes[m], step, k + r * groups < k1 ? left : 0);
                    }
                }
            if constexpr (C::kAsync) {
                fetch(stage);
                stage = stage + 1 == kStages ? 0 : stage + 1;
            } else {
#pragma unroll
                for (int m = 0; m < kMats; ++m) base[m] += round_bytes[m];
            }
#pragma unroll
            for (int r = 0; r < kRound; ++r) {
                const int row = k + r * groups;
                if (row >= b) break;
                float x[T];
                const float *xr = xs + (row - a) * T;
                if constexpr (T >= 4) {
#pragma unroll
                    for (int t = 0; t < T; t += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(xr + t);
                        x[t] = f.x; x[t + 1] = f.y; x[t + 2] = f.z; x[t + 3] = f.w;
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < T; ++t) x[t] = xr[t];
                }
#pragma unroll
                for (int m = 0; m < kMats; ++m)
#pragma unroll
                    for (int i = 0; i < kPairs; ++i) {
                        const float2 wp = w[m][r].pair(i);
#pragma unroll
                        for (int t = 0; t < T; ++t)
                            acc[m][t][i] = __ffma2_rn(make_float2(x[t], x[t]), wp, acc[m][t][i]);
                    }
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");

    // [group][matrix][row of x][column], then their sums, then the cluster's.
    __syncthreads();
    const int per_group = kMats * T * cols;
#pragma unroll
    for (int m = 0; m < kMats; ++m)
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                float *to = smem + group * per_group + (m * T + t) * cols;
                if constexpr (VEC) {
                    *reinterpret_cast<float2 *>(to + lane_col * C::kCols + 2 * i) = acc[m][t][i];
                } else {
                    to[2 * i * step + lane_col] = acc[m][t][i].x;
                    to[(2 * i + 1) * step + lane_col] = acc[m][t][i].y;
                }
            }
    __syncthreads();
    float *mine = smem + groups * per_group;
    for (int i = tid; i < per_group; i += kThreads) {
        float v = 0.0f;
        for (int g = 0; g < groups; ++g) v += smem[g * per_group + i];
        mine[i] = v;
    }
    cluster.sync();
    const int outs = T * cols, shift = 31 - __clz(cols);
    for (int i = rank * kThreads + tid; i < outs; i += ranks * kThreads) {
        const int t = i >> shift, n = c0 + (i & (cols - 1));
        float v = 0.0f, v2 = 0.0f;
        for (int r = 0; r < ranks; ++r) {
            const float *theirs = cluster.map_shared_rank(mine, r);
            v += theirs[i];
            if constexpr (GATE) v2 += theirs[outs + i];
        }
        if (t < p.T && n < p.N) {
            if constexpr (GATE)
                static_cast<float *>(p.y)[t * p.ldy + n] = gate_act<TYPE == kTypeF32>(v, p.act) * v2;
            else
                store_from_float(p.y, TYPE, t * p.ldy + n, v);
        }
    }
    cluster.sync();  // no CTA leaves while another reads its sums
}

template <int TYPE, int T, bool GATE, bool VEC>
cudaError_t launch_one(FfnStreamParams p, int num_sms, cudaStream_t stream) {
    constexpr int kMats = GATE ? 2 : 1, kCols = cols_of(TYPE, T);
    constexpr int kRound = round_of(GATE);
    // The widest stretch of columns and the cluster with which the CTAs fill
    // the SMs' places best (in whole waves), as long as a lane keeps two
    // rounds of rows.  (1 x 4096 x 12288 bf16: 6 CTAs a cluster, 288 in all,
    // against 8 and 384: 1.3 waves.)
    const int places = num_sms * kCtasPerSm;
    int cluster = 1;
    double best = -1.0;
    for (int lpr = 32; lpr >= 8; lpr /= 2) {
        const long long tiles = (p.N + lpr * kCols - 1) / (lpr * kCols);
        const int rows = kRound * kWarps * 32 / lpr;
        for (int c = 1; c <= 8 && (c == 1 || p.K >= 2 * rows * c); ++c) {
            const long long ctas = tiles * c, waves = (ctas + places - 1) / places;
            const double fill = (double)ctas / (double)(waves * places);
            if (fill > best + 0.03) {
                best = fill;
                cluster = c;
                p.lanes_per_row = lpr;
            }
        }
    }
    const int groups = kWarps * 32 / p.lanes_per_row, round = kRound * groups;
    const int tiles = (p.N + p.lanes_per_row * kCols - 1) / (p.lanes_per_row * kCols);
    p.cta_rows = (p.K + cluster - 1) / cluster;
    p.chunk_rows = std::max(1, 40 * 1024 / (T * 4 * round)) * round;
    const int cols = p.lanes_per_row * kCols;
    const size_t x = (size_t)std::min(p.chunk_rows, p.cta_rows) * T * sizeof(float) +
                     kWarps * kStages * kStageBytes;
    const size_t reduce = (size_t)(groups + 1) * kMats * T * cols * sizeof(float);
    const auto kernel = ffn_stream_kernel<TYPE, T, GATE, VEC>;
    static std::atomic<bool> configured[kMaxDevices];
    if (p.device >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!configured[p.device].load()) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
        if (e != cudaSuccess) return e;
        configured[p.device].store(true);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)tiles * cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = std::max(x, reduce);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = GATE ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int TYPE, bool GATE, bool VEC>
cudaError_t launch_rows(const FfnStreamParams &p, int num_sms, cudaStream_t stream) {
    if (p.T <= 1) return launch_one<TYPE, 1, GATE, VEC>(p, num_sms, stream);
    if (p.T <= 2) return launch_one<TYPE, 2, GATE, VEC>(p, num_sms, stream);
    if (p.T <= 4) return launch_one<TYPE, 4, GATE, VEC>(p, num_sms, stream);
    return launch_one<TYPE, 8, GATE, VEC>(p, num_sms, stream);
}

template <int TYPE>
cudaError_t launch_type(const FfnStreamParams &p, bool gate, bool vec, int num_sms,
                        cudaStream_t stream) {
    if (gate)
        return vec ? launch_rows<TYPE, true, true>(p, num_sms, stream)
                   : launch_rows<TYPE, true, false>(p, num_sms, stream);
    return vec ? launch_rows<TYPE, false, true>(p, num_sms, stream)
               : launch_rows<TYPE, false, false>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_ffn_stream(const FfnStreamParams &p, int type, bool gate, bool vec, int num_sms,
                              cudaStream_t stream) {
    if (type == kTypeF32) return launch_type<kTypeF32>(p, gate, vec, num_sms, stream);
    if (type == kTypeF16) return launch_type<kTypeF16>(p, gate, vec, num_sms, stream);
    return launch_type<kTypeBF16>(p, gate, vec, num_sms, stream);
}

}  // namespace sgemm
