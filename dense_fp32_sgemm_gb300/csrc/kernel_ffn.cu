// The gated block's products on the fifth-generation tensor cores.
//
// One persistent kernel serves all of them (C = A B with FP32 accumulators in
// tensor memory); what differs is which way round the operands lie and what
// happens to the accumulators:
//   gate       g = x Wg and u = x Wu into the two halves of one accumulator,
//              h = act(g) * u stored (and g, u kept in FP32 when asked for)
//   down       y = h Wd
//   gate grad  dh = dy Wd^T; dg = dh u act'(g), du = dh act(g), h stored
//   dx         dg Wg^T + du Wu^T, both products into one accumulator
//   dW         x^T dg and x^T du (two outputs of one launch), h^T dy
//
// Types.  16-bit operands enter as they are.  FP32 operands are three bf16
// planes (kernel below) whose sum they are to 24 bits; six of the nine plane
// products are taken, smallest first, the three left out are below 2^-24 of
// the product.  The tensor core adds without rounding to nearest, so an
// accumulator that runs over all of K would drift by some 10^-5; FP32 sums
// are therefore taken out of tensor memory after every k block and added up
// in registers in FP32.
//
// Structure, 384 threads a CTA, one CTA per SM:
//   warp 0       one thread issues the TMA loads of 64-deep operand blocks
//                (128-byte swizzle) into a ring of 32 KB stages
//   warp 1       one thread issues tcgen05.mma and releases stages by commit
//   warp 2       allocates and frees tensor memory
//   warps 4-11   epilogue, from one of two accumulators while the other fills
// CG = 2: a pair of CTAs on one 256 x 256 tile, each holding half of A's rows
// and half of B's columns; the first CTA's thread issues for both.
// Every wait is bounded; a role that gives up flags the error word, the others
// run out in turn, and the CTA lets its copies land before it leaves.
#include <algorithm>

#include "ffn_gate.cuh"
#include "tc_common.cuh"

namespace sgemm {
namespace {

constexpr uint32_t kABytes = kFfnBM * kFfnBK * 2;
constexpr uint32_t kBBytes = kFfnBN * kFfnBK * 2;
constexpr uint32_t kStageBytes = kABytes + kBBytes;
constexpr size_t kSmemBytes = (size_t)kFfnStages * kStageBytes + 1024;
constexpr int kEpiWarps = 8;
constexpr uint32_t kBlockBytes = 64 * kFfnBK * 2;  // 64 of m or n by 64 k

// FP32: which planes of A and B the six products take, smallest first.
__constant__ const int kPlaneA[6] = {2, 0, 1, 1, 0, 0};
__constant__ const int kPlaneB[6] = {0, 2, 1, 0, 1, 0};

struct TileAt {
    int out, m, n;  // output, tile row, tile column
};

// Tiles in groups of eight tile rows, column by column inside a group, so
// that the CTAs at work share rows of A and columns of B in L2.
__device__ __forceinline__ TileAt tile_at(const FfnGemmParams &p, int t) {
    constexpr int kGroup = 8;
    TileAt r;
    const int per_out = p.tiles_m * p.tiles_n;
    r.out = t / per_out;
    t -= r.out * per_out;
    const int per_group = kGroup * p.tiles_n;
    const int first = t / per_group * kGroup;
    const int rows = min(kGroup, p.tiles_m - first);
    t -= first * p.tiles_n;
    r.m = first + t % rows;
    r.n = t / rows;
    return r;
}

// 32 consecutive FP32 values of a row to a matrix of TYPE, from column n on
// (columns up to N).
template <int TYPE>
__device__ __forceinline__ void store_row(void *base, long long at, bool vec, int left,
                                          const float (&v)[32]) {
    if constexpr (TYPE == kTypeF32) {
        float *c = static_cast<float *>(base) + at;
        if (vec && left >= 32) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                reinterpret_cast<float4 *>(c)[i] =
                    make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < left) c[i] = v[i];
        }
    } else {
        uint16_t *c = static_cast<uint16_t *>(base) + at;
        if (vec && left >= 32) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                reinterpret_cast<uint4 *>(c)[i] =
                    make_uint4(pack16<TYPE>(v[8 * i], v[8 * i + 1]),
                               pack16<TYPE>(v[8 * i + 2], v[8 * i + 3]),
                               pack16<TYPE>(v[8 * i + 4], v[8 * i + 5]),
                               pack16<TYPE>(v[8 * i + 6], v[8 * i + 7]));
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < left) c[i] = (uint16_t)(pack16<TYPE>(v[i], 0.0f) & 0xFFFFu);
        }
    }
}

// An intermediate matrix: 16-bit values, or FP32 values as three planes.
template <int TYPE>
__device__ __forceinline__ void store_planes(void *base, long long at, long long plane, bool vec,
                                             int left, const float (&v)[32]) {
    if constexpr (TYPE != kTypeF32) {
        store_row<TYPE>(base, at, vec, left, v);
    } else {
        float rest[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) rest[i] = v[i];
#pragma unroll 1
        for (int q = 0; q < 3; ++q) {
            float part[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                float s[3];
                split3(rest[i], s);
                part[i] = s[0];
                rest[i] = isfinite(s[0]) ? rest[i] - s[0] : 0.0f;
            }
            store_row<kTypeBF16>(base, at + q * plane, vec, left, part);
        }
    }
}

__device__ __forceinline__ void load_row(const float *c, int left, float (&v)[32]) {
    if (left >= 32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 f = __ldg(reinterpret_cast<const float4 *>(c) + i);
            v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = i < left ? __ldg(c + i) : 0.0f;
    }
}

template <int TYPE, int MODE, int CG>
__global__ void __launch_bounds__(kFfnThreads, 1)
    ffn_gemm_kernel(const __grid_constant__ FfnMaps maps, const FfnGemmParams p) {
    constexpr bool kSplit = TYPE == kTypeF32;         // three planes, sums in registers
    constexpr int kProducts = kSplit ? 6 : 1;
    constexpr int kAccCols = 128 * CG;                // tensor-memory columns of an accumulator
    constexpr int kTileN = MODE == kFfnGate ? 64 * CG : 128 * CG;
    constexpr int kParts = 2 * CG;                    // groups of 32 columns of an epilogue warp
    extern __shared__ unsigned char ffn_smem_raw[];
    __shared__ uint64_t full[kFfnStages], empty[kFfnStages], acc_full[2], acc_empty[2];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int s_abort;

    const uint32_t raw = smem_addr(ffn_smem_raw);
    unsigned char *smem = ffn_smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const int worker = (int)blockIdx.x / CG, workers = (int)gridDim.x / CG;

    if (tid == 0) {
        for (int s = 0; s < kFfnStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], kEpiWarps * CG);
        }
        s_abort = 0;
        fence_barrier_init();
    }
    if (warp == 2) tc_alloc<CG, 2 * kAccCols>(&tmem_slot);
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (CG == 2) cluster_barrier();
    tc_fence_after_sync();
    const uint32_t tmem = tmem_slot;

    const int iters = p.kblocks * p.segs * kProducts;  // stages of a tile
    // Stages that one accumulator takes before the epilogue reads it.
    const int phase_iters = kSplit ? kProducts : iters;
    const int phases = iters / phase_iters;

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;  // stages so far, over all tiles
            bool ok = true;
            for (int t = worker; ok && t < p.tiles; t += workers) {
                const TileAt at = tile_at(p, t);
                const int m0 = at.m * (kFfnBM * CG) + (int)rank * kFfnBM;
                const int n0 = at.n * kTileN;
                for (int i = 0; i < iters; ++i, ++it) {
                    if (p.skip_loads_from >= 0 && it >= p.skip_loads_from) {
                        ok = false;
                        break;
                    }
                    const int s = it % kFfnStages, use = it / kFfnStages;
                    if (use > 0 && !mbar_wait_bounded(&empty[s], (use - 1) & 1, p.timeout_ns)) {
                        atomicOr(p.err, kErrWaitTimeout);
                        s_abort = 1;
                        ok = false;
                        break;
                    }
                    const int prod = i % kProducts, kb = (i / kProducts) % p.kblocks;
                    const int seg = i / (kProducts * p.kblocks);
                    const int pa = kSplit ? kPlaneA[prod] : 0, pb = kSplit ? kPlaneB[prod] : 0;
                    const int k = kb * kFfnBK;
                    unsigned char *a = smem + (size_t)s * kStageBytes, *b = a + kABytes;
                    // The pair's loads all complete on the first CTA's barrier.
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], kStageBytes * CG);
                    const uint32_t bar = CG == 2 ? cluster_addr(&full[s], 0) : smem_addr(&full[s]);
                    const CUtensorMap *ma = &maps.a[seg];
                    if (p.a_mn) {
                        tc_load_3d<CG>(a, ma, bar, m0, k, pa);
                        tc_load_3d<CG>(a + kBlockBytes, ma, bar, m0 + 64, k, pa);
                    } else {
                        tc_load_3d<CG>(a, ma, bar, k, m0, pa);
                    }
                    if constexpr (MODE == kFfnGate) {
                        // One CTA: 64 columns of each matrix.  A pair: the
                        // first CTA brings 128 of Wg, the second of Wu.
                        const CUtensorMap *m1 = CG == 2 ? &maps.b[rank] : &maps.b[0];
                        const CUtensorMap *m2 = CG == 2 ? m1 : &maps.b[1];
                        tc_load_3d<CG>(b, m1, bar, n0, k, pb);
                        tc_load_3d<CG>(b + kBlockBytes, m2, bar, CG == 2 ? n0 + 64 : n0, k, pb);
                    } else {
                        const CUtensorMap *mb = &maps.b[seg + at.out];
                        const int n = n0 + (int)rank * kFfnBN;
                        if (p.b_mn) {
                            tc_load_3d<CG>(b, mb, bar, n, k, pb);
                            tc_load_3d<CG>(b + kBlockBytes, mb, bar, n + 64, k, pb);
                        } else {
                            tc_load_3d<CG>(b, mb, bar, k, n, pb);
                        }
                    }
                }
            }
            // The last releases of the stages have to arrive before the CTA
            // leaves.
            for (int i = max(0, it - kFfnStages); ok && i < it; ++i)
                if (!mbar_wait_bounded(&empty[i % kFfnStages], (i / kFfnStages) & 1, p.timeout_ns)) {
                    atomicOr(p.err, kErrDrainTimeout);
                    s_abort = 1;
                    ok = false;
                }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            const uint32_t idesc =
                tc_idesc(kFfnBM * CG, kFfnBN * CG, TYPE != kTypeF16, p.a_mn != 0, p.b_mn != 0);
            // Per 16 k: two groups of eight rows (MN-major) or 32 bytes along
            // the swizzled row (K-major).
            const uint32_t a_step = p.a_mn ? 2048 : 32, b_step = p.b_mn ? 2048 : 32;
            int it = 0, ph = 0;
            bool ok = true;
            for (int t = worker; ok && t < p.tiles; t += workers) {
                for (int q = 0; ok && q < phases; ++q, ++ph) {
                    const int buf = ph & 1, use = ph >> 1;
                    if (use > 0 && !mbar_wait_bounded(&acc_empty[buf], (use - 1) & 1, p.timeout_ns)) {
                        atomicOr(p.err, kErrWaitTimeout);
                        s_abort = 1;
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t d = tmem + buf * kAccCols;
                    for (int i = 0; i < phase_iters; ++i, ++it) {
                        const int s = it % kFfnStages;
                        if (!mbar_wait_bounded(&full[s], (it / kFfnStages) & 1, p.timeout_ns)) {
                            atomicOr(p.err, kErrWaitTimeout);
                            s_abort = 1;
                            ok = false;
                            break;
                        }
                        tc_fence_after_sync();
                        const uint32_t a = sbase + s * kStageBytes, b = a + kABytes;
#pragma unroll
                        for (int kk = 0; kk < kFfnBK / 16; ++kk)
                            tc_mma<CG>(d, tc_desc(a + kk * a_step, kBlockBytes),
                                       tc_desc(b + kk * b_step, kBlockBytes), idesc, (i | kk) != 0);
                        tc_commit<CG>(&empty[s]);
                    }
                    if (ok) tc_commit<CG>(&acc_full[buf]);
                }
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        const int quad = warp & 3, half = (warp - 4) >> 2;
        const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
        int ph = 0;
        bool ok = true;
        for (int t = worker; ok && t < p.tiles; t += workers) {
            const TileAt at = tile_at(p, t);
            const int row = at.m * (kFfnBM * CG) + (int)rank * kFfnBM + quad * 32 + lane;
            const int n_tile = at.n * kTileN;
            const bool row_ok = row < p.M;
            // Part j is 32 accumulator columns; in the gate's product parts
            // come in twos, the same columns of g and u.
            auto part_col = [&](int j) {
                return MODE == kFfnGate ? (j & 1) * 64 * CG + half * 32 * CG + 32 * (j >> 1)
                                        : half * 64 * CG + 32 * j;
            };
            auto emit = [&](int j, const float (&v)[32], const float (&v2)[32]) {
                const int n = n_tile + part_col(j & (MODE == kFfnGate ? ~1 : ~0));
                const int left = p.N - n;
                if (!row_ok || left <= 0) return;
                const long long c_at = (long long)row * p.ldc[MODE == kFfnStore ? at.out : 0] + n;
                if constexpr (MODE == kFfnStore) {
                    store_row<TYPE>(p.C[at.out], c_at, p.c_vec, left, v);
                } else if constexpr (MODE == kFfnGate) {
                    const long long gu = (long long)row * p.ldgu + n;
                    if (p.g) {
                        store_row<kTypeF32>(p.g, gu, true, left, v);
                        store_row<kTypeF32>(p.u, gu, true, left, v2);
                    }
                    if (p.C[0]) {
                        float h[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) h[i] = gate_act<kSplit>(v[i], p.act) * v2[i];
                        store_planes<TYPE>(p.C[0], c_at, p.c_plane, p.c_vec, left, h);
                    }
                } else {
                    const long long gu = (long long)row * p.ldgu + n;
                    float g[32], u[32];
                    load_row(p.g + gu, left, g);
                    load_row(p.u + gu, left, u);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float a, slope;
                        gate_act_slope<kSplit>(g[i], p.act, a, slope);
                        const float ui = u[i];
                        g[i] = v[i] * ui * slope;  // dg
                        u[i] = v[i] * a;           // du
                    }
                    store_planes<TYPE>(p.C[1], c_at, p.c_plane, p.c_vec, left, g);
                    store_planes<TYPE>(p.C[2], c_at, p.c_plane, p.c_vec, left, u);
                    load_row(p.g + gu, left, g);
                    load_row(p.u + gu, left, u);
#pragma unroll
                    for (int i = 0; i < 32; ++i) g[i] = gate_act<kSplit>(g[i], p.act) * u[i];
                    store_planes<TYPE>(p.C[0], c_at, p.c_plane, p.c_vec, left, g);
                }
            };
            float sum[kSplit ? kParts : 1][32];
            if constexpr (kSplit) {
#pragma unroll
                for (int j = 0; j < kParts; ++j)
#pragma unroll
                    for (int i = 0; i < 32; ++i) sum[j][i] = 0.0f;
            }
            for (int q = 0; q < phases; ++q, ++ph) {
                const int buf = ph & 1;
                int got = 1;
                if (lane == 0) {
                    got = mbar_wait_bounded(&acc_full[buf], (ph >> 1) & 1, p.timeout_ns) ? 1 : 0;
                    if (!got) {
                        atomicOr(p.err, kErrWaitTimeout);
                        s_abort = 1;
                    }
                }
                got = __shfl_sync(0xffffffffu, got, 0);
                if (!got) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t d = t_lane + buf * kAccCols;
                if constexpr (kSplit) {
#pragma unroll
                    for (int j = 0; j < kParts; ++j) {
                        uint32_t r[32];
                        tc_ld32(d + part_col(j), r);
                        tc_wait_ld(r);
#pragma unroll
                        for (int i = 0; i < 32; ++i) sum[j][i] += __uint_as_float(r[i]);
                    }
                } else {
#pragma unroll 1
                    for (int j = 0; j < kParts; j += MODE == kFfnGate ? 2 : 1) {
                        uint32_t r[32], r2[32];
                        float v[32], v2[32];
                        tc_ld32(d + part_col(j), r);
                        if constexpr (MODE == kFfnGate) {
                            tc_ld32(d + part_col(j + 1), r2);
                            tc_wait_ld(r2);
                        }
                        tc_wait_ld(r);
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            v[i] = __uint_as_float(r[i]);
                            v2[i] = MODE == kFfnGate ? __uint_as_float(r2[i]) : 0.0f;
                        }
                        emit(j, v, v2);
                    }
                }
                // The accumulator may be overwritten.
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 2)
                        cluster_arrive(cluster_addr(&acc_empty[buf], 0));
                    else
                        mbar_arrive(&acc_empty[buf]);
                }
            }
            if constexpr (kSplit) {
                if (ok) {
#pragma unroll
                    for (int j = 0; j < kParts; j += MODE == kFfnGate ? 2 : 1)
                        emit(j, sum[j], sum[MODE == kFfnGate ? j + 1 : j]);
                }
            }
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (tid == 0 && (s_abort || p.skip_loads_from >= 0)) {
        // A role gave up: loads and products may still be in flight.  They
        // take microseconds; nothing here signals their end any more.
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 2000000ull) {
        }
    }
    __syncthreads();
    // No CTA of a pair leaves, or frees its tensor memory, while the other's
    // loads and products may still reach it.
    if constexpr (CG == 2) cluster_barrier();
    if (warp == 2) {
        tc_fence_after_sync();
        tc_dealloc<CG, 2 * kAccCols>(tmem);
    }
}

// ---------------------------------------------------------------------------
// Operand copies: FP32 -> three bf16 planes (4 bytes read, 6 written per
// element), or 16-bit values to aligned rows.  Bound by HBM.  A thread takes
// eight elements of a row, so stores are 16 bytes.
// ---------------------------------------------------------------------------
struct PrepTable {
    int count;
    FfnPrepJob job[kFfnPrepJobs];
};

template <bool SPLIT>
__global__ void __launch_bounds__(256) ffn_prep_kernel(const PrepTable t) {
    for (int q = 0; q < t.count; ++q) {
        const FfnPrepJob &j = t.job[q];
        const int octets = (j.cols + 7) / 8;
        const long long total = (long long)j.rows * octets;
        for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += gridDim.x * 256LL) {
            const long long row = i / octets;
            const int c = (int)(i % octets) * 8;
            const long long from = row * j.ld_src + c, to = row * j.ld_dst + c;
            if constexpr (SPLIT) {
                const float *src = static_cast<const float *>(j.src) + from;
                float part[8][3];
#pragma unroll
                for (int e = 0; e < 8; ++e) split3(c + e < j.cols ? __ldg(src + e) : 0.0f, part[e]);
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(j.dst) + k * j.plane_stride + to) =
                        make_uint4(pack16<kTypeBF16>(part[0][k], part[1][k]),
                                   pack16<kTypeBF16>(part[2][k], part[3][k]),
                                   pack16<kTypeBF16>(part[4][k], part[5][k]),
                                   pack16<kTypeBF16>(part[6][k], part[7][k]));
            } else {
                const uint16_t *src = static_cast<const uint16_t *>(j.src) + from;
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t a = c + 2 * e < j.cols ? __ldg(src + 2 * e) : 0u;
                    const uint32_t b = c + 2 * e + 1 < j.cols ? __ldg(src + 2 * e + 1) : 0u;
                    w[e] = a | b << 16;
                }
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(j.dst) + to) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

template <int TYPE, int MODE, int CG>
cudaError_t launch_one(const FfnMaps &maps, const FfnGemmParams &p, int num_sms,
                       cudaStream_t stream) {
    const auto kernel = ffn_gemm_kernel<TYPE, MODE, CG>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CG * std::min(p.tiles, num_sms / CG));
    cfg.blockDim = dim3(kFfnThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, maps, p);
}

template <int TYPE, int CG>
cudaError_t launch_mode(const FfnMaps &maps, const FfnGemmParams &p, int num_sms,
                        cudaStream_t stream) {
    switch (p.mode) {
        case kFfnStore: return launch_one<TYPE, kFfnStore, CG>(maps, p, num_sms, stream);
        case kFfnGate: return launch_one<TYPE, kFfnGate, CG>(maps, p, num_sms, stream);
        default: return launch_one<TYPE, kFfnGateGrad, CG>(maps, p, num_sms, stream);
    }
}

}  // namespace

cudaError_t launch_ffn_gemm(const FfnMaps &maps, const FfnGemmParams &p, bool pair, int num_sms,
                            cudaStream_t stream) {
    if (p.type == kTypeF32) return launch_mode<kTypeF32, 1>(maps, p, num_sms, stream);
    if (p.type == kTypeF16)
        return pair ? launch_mode<kTypeF16, 2>(maps, p, num_sms, stream)
                    : launch_mode<kTypeF16, 1>(maps, p, num_sms, stream);
    return pair ? launch_mode<kTypeBF16, 2>(maps, p, num_sms, stream)
                : launch_mode<kTypeBF16, 1>(maps, p, num_sms, stream);
}

cudaError_t launch_ffn_prep(const FfnPrepJob *jobs, int count, int type, int num_sms,
                            cudaStream_t stream) {
    if (count == 0) return cudaSuccess;
    PrepTable t;
    t.count = count;
    for (int i = 0; i < count; ++i) t.job[i] = jobs[i];
    if (type == kTypeF32)
        ffn_prep_kernel<true><<<num_sms * 8, 256, 0, stream>>>(t);
    else
        ffn_prep_kernel<false><<<num_sms * 8, 256, 0, stream>>>(t);
    return cudaGetLastError();
}

}  // namespace sgemm
