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
// there was room for a quarter of it with eight rows of x.  Rows that start
// anywhere are brought in by the aligned 16-byte pieces that cover them (element by
// element FP32 1 x 2047 x 5461 took 53 us, so 35; BF16 4 x 2047 x 5461 57 and 37).
//
// Measured: 1 x 4096 x 12288 bf16 53-57 us (5.3-5.6 TB/s), 4 x 4096 x 12288 58 us,
// 4 x 2047 x 5461 34-37 us (rows off 16 bytes), 8 x 2048 x 5464 FP32 34 us (4.0 TB/s),
// 5 x 2047 x 5461 45-47 us, 24 x 2048 x 8192 150 us (three passes).
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
#include <mutex>

#include "device_common.cuh"
#include "ffn_gate.cuh"

namespace cg = cooperative_groups;

namespace sgemm {
namespace {

constexpr int kMaxDevices = 64;
constexpr int kThreads = 256, kWarps = kThreads / 32;

// A lane's columns of one row.  VEC: 16 (or 8) consecutive bytes, which the lane
// copies to a place of its own in shared memory and takes from there.  Else the
// warp copies the aligned 16-byte pieces that cover the row's stretch, and the
// lane takes every step-th element, wherever the stretch starts in them.
template <int TYPE, int COLS, bool VEC>
struct Columns {
    static constexpr int kCols = COLS;
    static constexpr int kElem = TYPE == kTypeF32 ? 4 : 2;
    static constexpr int kBytes = COLS * kElem;  // 16 or 8
    uint32_t w[4];

    static __device__ __forceinline__ void fetch(uint32_t to, const unsigned char *from) {
        if constexpr (kBytes == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
    }
    // The piece `off` bytes behind the one that holds the first byte of a row's
    // stretch of `width` bytes, as far as it lies inside the matrix [first, end).
    static __device__ __forceinline__ void fetch_piece(unsigned char *to, const unsigned char *row,
                                                       int off, int width, const unsigned char *first,
                                                       const unsigned char *end) {
        off -= (int)(reinterpret_cast<uintptr_t>(row) & 15);
        if (off >= width) return;
        const unsigned char *piece = row + off;
        const long long left = end - piece;
        if (piece >= first && (left >= 16 || left % 4 == 0)) {
            cp_async16(reinterpret_cast<float *>(to), reinterpret_cast<const float *>(piece),
                       left >= 16 ? 16 : (uint32_t)left);
        } else {
#pragma unroll 1
            for (int i = 0; i < 16 && i < left; i += kElem) {
                if (piece + i < first) continue;
                if constexpr (kElem == 4)
                    *reinterpret_cast<uint32_t *>(to + i) = __ldg(reinterpret_cast<const uint32_t *>(piece + i));
                else
                    *reinterpret_cast<uint16_t *>(to + i) = __ldg(reinterpret_cast<const uint16_t *>(piece + i));
            }
        }
    }
    __device__ __forceinline__ void take(const unsigned char *from, int step) {
        if constexpr (VEC) {
            const uint4 v = *reinterpret_cast<const uint4 *>(from);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else if constexpr (TYPE == kTypeF32) {
#pragma unroll
            for (int j = 0; j < kCols; ++j) w[j] = *reinterpret_cast<const uint32_t *>(from + 4 * j * step);
        } else {
#pragma unroll
            for (int j = 0; j < kCols; j += 2)
                w[j / 2] = *reinterpret_cast<const uint16_t *>(from + 2 * j * step) |
                           (uint32_t)*reinterpret_cast<const uint16_t *>(from + 2 * (j + 1) * step) << 16;
        }
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
// Of a warp: the lanes' places for four loads, or pieces with one more for each
// of up to four rows of a load.
constexpr int slot_bytes(bool vec) { return vec ? 512 : 512 + 64; }
constexpr int stage_bytes(bool vec) { return 4 * slot_bytes(vec); }

template <int TYPE, int T, bool GATE, bool VEC>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) ffn_stream_kernel(const FfnStreamParams p) {
    using C = Columns<TYPE, cols_of(TYPE, T), VEC>;
    constexpr int kMats = GATE ? 2 : 1, kPairs = C::kCols / 2;
    constexpr int kElem = TYPE == kTypeF32 ? 4 : 2;
    constexpr int kRound = round_of(GATE);
    constexpr int kSlot = slot_bytes(VEC), kStageBytes = stage_bytes(VEC);
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

    // The lane's next row; VEC: pointers to its columns there.
    const int sub = lane / lpr;
    int next = k0 + group;
    const unsigned char *base[kMats];
    long long row_bytes[kMats];
    if constexpr (VEC) {
        base[0] = static_cast<const unsigned char *>(p.W) + ((k0 + group) * p.ldw + col) * kElem;
        row_bytes[0] = groups * p.ldw * kElem;
        if constexpr (GATE) {
            base[kMats - 1] =
                static_cast<const unsigned char *>(p.W2) + ((k0 + group) * p.ldw2 + col) * kElem;
            row_bytes[kMats - 1] = groups * p.ldw2 * kElem;
        }
    }
    unsigned char *const warp_ring = reinterpret_cast<unsigned char *>(smem) + warp * (kStages * kStageBytes);
    const uint32_t ring_addr = (uint32_t)__cvta_generic_to_shared(warp_ring + lane * 16);
    // Pieces: a row's stretch and its place in a slot.  The row's last lane brings
    // the piece behind its own as well.
    const int stretch = lpr * C::kBytes, in_slot = sub * (stretch + 16);
    // First byte of a row's stretch (formed anew each time, for the registers'
    // sake), and where it lies in its first piece.
    auto row_start = [&](int m, int row) {
        return static_cast<const unsigned char *>(m ? p.W2 : p.W) + (row * (m ? p.ldw2 : p.ldw) + c0) * kElem;
    };
    auto row_shift = [&](int m, int row) {
        return ((uint32_t)reinterpret_cast<uintptr_t>(m ? p.W2 : p.W) +
                ((uint32_t)row * (uint32_t)(m ? p.ldw2 : p.ldw) + (uint32_t)c0) * kElem) & 15u;
    };
    auto piece = [&](unsigned char *to, const unsigned char *row, int off, bool second) {
        C::fetch_piece(to, row, off, min(p.N - c0, cols) * kElem,
                       static_cast<const unsigned char *>(second ? p.W2 : p.W),
                       static_cast<const unsigned char *>(second ? p.end2 : p.end));
    };
    // safe: all rows' pieces lie inside the matrices, wherever the columns are.
    auto fetch = [&](int stage) {
        const int first = next - sub, last = first + rpw - 1 + (kRound - 1) * groups;
        const bool safe = first >= p.safe_rows && last < min(k1, p.K - p.safe_rows);
#pragma unroll
        for (int m = 0; m < kMats; ++m) {
            const int at = stage * kStageBytes + m * kRound * kSlot;
            if constexpr (VEC) {
#pragma unroll
                for (int r = 0; r < kRound; ++r)
                    if (next + r * groups < k1 && left > 0)
                        C::fetch(ring_addr + at + r * kSlot, base[m] + r * row_bytes[m]);
            } else {
                const int off = lane_col * C::kBytes;
                unsigned char *to = warp_ring + at + in_slot;
                if (safe) {
#pragma unroll
                    for (int r = 0; r < kRound; ++r) {
                        const unsigned char *row = row_start(m, next + r * groups);
                        const float *from = reinterpret_cast<const float *>(
                            row + (off - (int)(reinterpret_cast<uintptr_t>(row) & 15)));
                        if (off % 16 == 0) cp_async16(reinterpret_cast<float *>(to + r * kSlot + off), from, 16);
                        if (lane_col == lpr - 1)
                            cp_async16(reinterpret_cast<float *>(to + r * kSlot + stretch),
                                       from + (stretch - off) / 4, 16);
                    }
                } else {
#pragma unroll 1
                    for (int r = 0; r < kRound && next + r * groups < k1; ++r) {
                        const unsigned char *row = row_start(m, next + r * groups);
                        if (off % 16 == 0) piece(to + r * kSlot + off, row, off, m == 1);
                        if (lane_col == lpr - 1) piece(to + r * kSlot + stretch, row, stretch, m == 1);
                    }
                }
            }
            if constexpr (VEC) base[m] += kRound * row_bytes[m];
        }
        next += kRound * groups;
        cp_async_commit();
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
            cp_async_wait<kStages - 1>();
            if constexpr (!VEC) __syncwarp();  // other lanes' pieces
            // VEC: the next stage is asked for as soon as the lane has its columns
            // of this one; else the rows are taken one by one (registers).
            C w[kMats][kRound];
            auto take = [&](int r) {
#pragma unroll
                for (int m = 0; m < kMats; ++m) {
                    const unsigned char *from = warp_ring + stage * kStageBytes + (m * kRound + r) * kSlot;
                    if constexpr (VEC)
                        from += lane * 16;
                    else
                        from += in_slot + row_shift(m, k + r * groups) + lane_col * kElem;
                    w[m][VEC ? r : 0].take(from, step);
                }
            };
            if constexpr (VEC) {
#pragma unroll
                for (int r = 0; r < kRound; ++r) take(r);
                fetch(stage);
                stage = stage + 1 == kStages ? 0 : stage + 1;
            }
#pragma unroll
            for (int r = 0; r < kRound; ++r) {
                const int row = k + r * groups;
                if (row >= b) break;
                if constexpr (!VEC) take(r);
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
                        const float2 wp = w[m][VEC ? r : 0].pair(i);
#pragma unroll
                        for (int t = 0; t < T; ++t)
                            acc[m][t][i] = __ffma2_rn(make_float2(x[t], x[t]), wp, acc[m][t][i]);
                    }
            }
            if constexpr (!VEC) {
                __syncwarp();
                fetch(stage);
                stage = stage + 1 == kStages ? 0 : stage + 1;
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

constexpr int kXBytes = 32 * 1024;  // of x in shared memory, about
constexpr int kMostCluster = 8;

// Clusters of each size that the card runs at once: fewer than its SMs would
// hold, as a cluster stays inside a group of SMs (38 of seven CTAs, not 43).
template <class Kernel>
cudaError_t active_clusters(Kernel kernel, size_t smem, int num_sms, int (&active)[kMostCluster + 1]) {
    for (int c = 1; c <= kMostCluster; ++c) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(num_sms * kCtasPerSm / c * c));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = c;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&active[c], kernel, &cfg);
        if (e != cudaSuccess) return e;
        active[c] = std::max(1, active[c]);
    }
    return cudaSuccess;
}

template <int TYPE, int T, bool GATE, bool VEC>
cudaError_t launch_one(FfnStreamParams p, int num_sms, cudaStream_t stream) {
    constexpr int kMats = GATE ? 2 : 1, kCols = cols_of(TYPE, T);
    constexpr int kRound = round_of(GATE);
    const auto kernel = ffn_stream_kernel<TYPE, T, GATE, VEC>;
    // Set up once per device.
    static int active[kMaxDevices][kMostCluster + 1];
    static std::once_flag once[kMaxDevices];
    static cudaError_t failed[kMaxDevices];
    if (p.device >= kMaxDevices) return cudaErrorInvalidDevice;
    std::call_once(once[p.device], [&] {
        cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
        if (e == cudaSuccess)
            e = active_clusters(kernel, kWarps * kStages * stage_bytes(VEC) + kXBytes, num_sms,
                                active[p.device]);
        failed[p.device] = e;
    });
    if (failed[p.device] != cudaSuccess) return failed[p.device];
    // Pieces reach 16 bytes before a row and 32 behind the widest stretch.
    const long long elem = TYPE == kTypeF32 ? 4 : 2;
    p.safe_rows = (int)(560 / std::max<long long>(1, std::min(p.ldw, GATE ? p.ldw2 : p.ldw) * elem) + 1);
    p.end = static_cast<const char *>(p.W) + ((p.K - 1) * p.ldw + p.N) * elem;
    if (GATE) p.end2 = static_cast<const char *>(p.W2) + ((p.K - 1) * p.ldw2 + p.N) * elem;
    // Stretch and cluster of the least time, in rows of 512 bytes a warp: a CTA's
    // rows, twice where an SM has two CTAs (one alone is 15 % faster than half of
    // two), for every wave, and 200 for each further wave's start.  FP32 5 x 2047 x
    // 5461, gate of 43 whole stretches: clusters of 3, 4, 5, 6, 7, 8 (which need
    // 1, 2, 2, 2, and 2 and 1 CTAs an SM) give a block of 51, 65, 53, 49, 57, 53 us.
    int cluster = 1;
    double least = -1.0;
    for (int lpr = 32; lpr >= 8; lpr /= 2) {
        const long long tiles = (p.N + lpr * kCols - 1) / (lpr * kCols);
        const int rows = kRound * kWarps * 32 / lpr;
        for (int c = 1; c <= kMostCluster && (c == 1 || p.K >= 2 * rows * c); ++c) {
            const long long fit = active[p.device][c], waves = (tiles + fit - 1) / fit;
            auto per_sm = [&](long long clusters) { return clusters * c > num_sms ? 2.0 : 1.15; };
            const double cost = ((waves - 1) * per_sm(fit) + per_sm(tiles - (waves - 1) * fit)) *
                                    ((p.K + c - 1) / c) * lpr / 32 + 200.0 * (waves - 1);
            if (least < 0.0 || cost < 0.98 * least) {
                least = cost;
                cluster = c;
                p.lanes_per_row = lpr;
            }
        }
    }
    const int groups = kWarps * 32 / p.lanes_per_row, round = kRound * groups;
    const int tiles = (p.N + p.lanes_per_row * kCols - 1) / (p.lanes_per_row * kCols);
    p.cta_rows = (p.K + cluster - 1) / cluster;
    p.chunk_rows = std::max(1, kXBytes / (T * 4 * round)) * round;
    const int cols = p.lanes_per_row * kCols;
    const size_t x = (size_t)std::min(p.chunk_rows, p.cta_rows) * T * sizeof(float) +
                     kWarps * kStages * stage_bytes(VEC);
    const size_t reduce = (size_t)(groups + 1) * kMats * T * cols * sizeof(float);
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
