// The gated block's products on the fifth-generation tensor cores.
//
// One persistent kernel serves all of them (C = A B with FP32 accumulators in
// tensor memory); what differs is which way round the operands lie and what
// happens to the accumulators:
//   gate       g = x Wg and u = x Wu into the two halves of one accumulator,
//              h = act(g) u stored (and u act'(g), act(g) kept in FP32 when
//              asked for, in the order in which a warp holds them)
//   down       y = h Wd
//   gate grad  dh = dy Wd^T; dg = dh u act'(g), du = dh act(g)
//   dx         dg Wg^T + du Wu^T, both products into one accumulator
//   dW         x^T dg, x^T du and h^T dy
// Products that do not wait for one another share a launch (dx and the three of dW).
//
// Types.  16-bit operands enter as they are.  FP32 operands are three bf16
// planes (kernel below) whose sum they are to 24 bits; six of the nine plane
// products are taken, smallest first, the three left out are below 2^-24 of
// the product.  The tensor core adds without rounding to nearest, so an
// accumulator that runs over all of K would drift by some 10^-5; FP32 sums
// are therefore taken out of tensor memory after every k block and added
// up in registers in FP32.
//
// Structure, 384 threads a CTA, one CTA per SM:
//   warp 0       one elected thread issues the TMA loads of 64-deep operand blocks
//                (128-byte swizzle) into a ring of 32 KB (FP32 pairs: 24 KB) stages
//   warp 1       one elected thread issues tcgen05.mma and releases stages by commit
//   warp 2       allocates and frees tensor memory
//   warps 4-11   epilogue, from one of two accumulators while the other fills
// CG = 2: a pair of CTAs on one 256 x 256 tile (FP32: 256 x 128, as a thread
// holds its sums in registers), each holding half of A's rows and half of B's
// columns; the first CTA's thread issues for both.  A launch may start while the
// one before it on the stream drains (programmatic dependent launch).
// Bound: the tensor pipe where tiles are many (85 to 95 % busy, then the card's
// power), shared memory in single CTAs and FP32.  Measured in a long run, which sits at
// the power limit, and for calls apart from one another: 4096 x 4096 x 12288 bf16
// 729-744 us (1.7 PFLOP/s), apart 619-648; the training step 8192 x 2048 x 8192 bf16
// 1569-1618 us (1.5), apart 1345-1461; the step 2048 x 2048 x 8192 FP32 2364 us (262
// TFLOP/s, 1.6 PFLOP/s of plane products), apart 2130-2178; 333 x 2000 x 5336 fp16
// 47-53 us either way.
// Every wait is bounded; a role that gives up flags the error word, the others
// run out in turn, and the CTA lets its copies land before it leaves.
#include <algorithm>
#include <atomic>

#include "ffn_gate.cuh"
#include "tc_common.cuh"

namespace sgemm {
namespace {

constexpr uint32_t kABytes = kFfnBM * kFfnBK * 2;
constexpr int kMaxDevices = 64;
constexpr int kEpiWarps = 8;
constexpr uint32_t kEpiBytes = 32 * 128;  // an epilogue warp's staging: 32 rows of 32 values

// Sizes of a form: type and CTAs to a tile.
template <int TYPE, int CG>
struct Form {
    static constexpr int kBCols = ffn_b_cols(TYPE == kTypeF32, CG == 2);  // of B per CTA
    static constexpr uint32_t kBBytes = kBCols * kFfnBK * 2;
    static constexpr uint32_t kStageBytes = kABytes + kBBytes;
    static constexpr int kStages = 192 * 1024 / kStageBytes;
    static constexpr int kAccCols = kBCols * CG;  // tensor-memory columns of an accumulator
    static constexpr int kParts = kAccCols / 64;  // groups of 32 columns of an epilogue warp
    static constexpr size_t kSmem = (size_t)kStages * kStageBytes + kEpiWarps * kEpiBytes + 1024;
};
constexpr uint32_t kBlockBytes = 64 * kFfnBK * 2;  // 64 of m or n by 64 k

// FP32: the planes of a k block in the order in which they are brought in (and
// then used), each with A's and B's in one stage of the ring.
constexpr int kPlanes = 3;
__device__ __forceinline__ int plane_at(int i) { return i == 0 ? 0 : 3 - i; }  // 0, 2, 1

// A stretch of one tile's k steps (a step: one k block, with all its plane
// products) that a worker computes.
struct Unit {
    int prob, m, n;     // product, tile row and column
    int s0, s1;         // steps [s0, s1)
    int pieces, piece;  // the tile's stretches, and which this is
    int first;          // the worker of piece 0
    int tail;           // the tile's number in the tail (cut tiles)
};

// Tiles of a product in groups of eight tile rows, column by column inside a
// group, so that the CTAs at work share rows of A and columns of B in L2.
__device__ __forceinline__ void locate(const FfnGemmParams &p, int t, Unit &r) {
    constexpr int kGroup = 8;
    r.prob = 0;
#pragma unroll
    for (int i = 1; i < kFfnProblems; ++i)
        if (i < p.count && t >= p.prob[i].tile0) r.prob = i;
    const FfnProblem &q = p.prob[r.prob];
    t -= q.tile0;
    const int per_group = kGroup * q.tiles_n;
    const int first = t / per_group * kGroup;
    const int rows = min(kGroup, q.tiles_m - first);
    t -= first * q.tiles_n;
    r.m = first + t % rows;
    r.n = t / rows;
}

// The worker's u-th unit; false when there is none.  The tail's steps are
// shared out evenly, so a worker's share touches at most two tiles.
__device__ __forceinline__ bool unit_at(const FfnGemmParams &p, int worker, int u, Unit &r) {
    const int longs = p.long_tiles > worker ? (p.long_tiles - worker - 1) / p.workers + 1 : 0;
    const int more = p.long_tiles % p.workers, fewer = p.workers - more;  // one long tile more, fewer
    const int extra = worker >= more ? p.extra : 0;
    const int base = p.long_tiles + p.extra * fewer;
    const int v = u - longs - extra;  // of the tiles that all share
    if (v < p.full_tiles || p.tail_workers == 0) {
        const int t = u < longs ? worker + u * p.workers
                      : v < 0   ? p.long_tiles + (u - longs) * fewer + worker - more
                                : base + worker + v * p.workers;
        if (t >= p.tiles) return false;
        locate(p, t, r);
        r.s0 = 0;
        r.s1 = p.prob[r.prob].kblocks * p.prob[r.prob].segs;
        r.pieces = 1;
        r.piece = r.tail = 0;
        r.first = worker;
        return true;
    }
    if (worker >= p.tail_workers) return false;
    const FfnProblem &last = p.prob[p.count - 1];
    const int steps = last.kblocks * last.segs;
    const long long all = (long long)p.tail_tiles * steps;
    long long a = worker * all / p.tail_workers;
    const long long e = (worker + 1) * all / p.tail_workers;
    long long end = min(e, (a / steps + 1) * steps);
    if (v > p.full_tiles) {
        if (v > p.full_tiles + 1) return false;
        a = end;
        end = e;
    }
    if (a >= end) return false;
    const int t = (int)(a / steps);
    // Worker w starts at floor(w all / n), so step x is worker
    // floor(((x + 1) n - 1) / all)'s.
    const long long x0 = (long long)t * steps, n = p.tail_workers;
    locate(p, base + p.full_tiles * p.workers + t, r);
    r.tail = t;
    r.s0 = (int)(a - x0);
    r.s1 = (int)(end - x0);
    r.first = (int)(((x0 + 1) * n - 1) / all);
    r.pieces = (int)(((x0 + steps) * n - 1) / all) - r.first + 1;
    r.piece = worker - r.first;
    return true;
}

// Slot of piece q: a worker's first slot holds a piece that starts inside its
// tile, the second one that starts with it.
__device__ __forceinline__ int piece_slot(const Unit &u, int q) {
    return 2 * (u.first + q) + (q == 0 ? 1 : 0);
}

// 32 values of each of a warp's lanes, as they lie in registers: 512
// consecutive bytes per instruction.
__device__ __forceinline__ void put_lanes(float *base, int lane, const float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        __stcg(reinterpret_cast<float4 *>(base) + i * 32 + lane,
               make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
}
__device__ __forceinline__ void get_lanes(const float *base, int lane, float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float4 f = __ldcg(reinterpret_cast<const float4 *>(base) + i * 32 + lane);
        v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
    }
}

// A warp's 32 x 32 block (lane = row, 32 columns each) to a row-major matrix
// of TYPE: through shared memory, so that a row's 64 or 128 bytes are stored
// by neighbouring lanes.  The 16-byte chunks of a row are permuted by its
// number so that neither side has bank conflicts.  rows and cols are what is
// left of the matrix from (row0, n) on.  v(i), called once for each i in order, is
// the lane's value in column i.
template <int TYPE, class Values>
__device__ __forceinline__ void store_block(unsigned char *stage, int lane, void *base, long long ld,
                                            long long row0, int n, int rows, int cols, bool vec,
                                            Values &&v) {
    constexpr int kElem = TYPE == kTypeF32 ? 4 : 2;
    constexpr int kChunks = 32 * kElem / 16;  // of a row
    constexpr int kPer = 16 / kElem;          // elements of a chunk
    auto place = [&](int r, int c) {
        return reinterpret_cast<uint4 *>(
            stage + r * (16 * kChunks) + ((TYPE == kTypeF32 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4));
    };
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        uint4 w;
        float e[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) e[i] = v(kPer * c + i);
        if constexpr (TYPE == kTypeF32)
            w = make_uint4(__float_as_uint(e[0]), __float_as_uint(e[1]), __float_as_uint(e[2]),
                           __float_as_uint(e[3]));
        else
            w = make_uint4(pack16<TYPE>(e[0], e[1]), pack16<TYPE>(e[2], e[3]),
                           pack16<TYPE>(e[4 % kPer], e[5 % kPer]), pack16<TYPE>(e[6 % kPer], e[7 % kPer]));
        *place(lane, c) = w;
    }
    __syncwarp();
    const int c = lane % kChunks, left = cols - c * kPer;
    unsigned char *out = static_cast<unsigned char *>(base) +
                         ((row0 + lane / kChunks) * ld + n + c * kPer) * kElem;
    const long long step = (long long)(32 / kChunks) * ld * kElem;
#pragma unroll
    for (int i = 0; i < kChunks; ++i, out += step) {
        const int r = i * (32 / kChunks) + lane / kChunks;
        const uint4 w = *place(r, c);
        if (r < rows && left > 0) {
            if (vec && left >= kPer) {
                *reinterpret_cast<uint4 *>(out) = w;
            } else {
                const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (j < left) {
                        if constexpr (TYPE == kTypeF32)
                            reinterpret_cast<uint32_t *>(out)[j] = e[j];
                        else
                            reinterpret_cast<uint16_t *>(out)[j] = (uint16_t)(e[j / 2] >> (16 * (j % 2)));
                    }
            }
        }
    }
    __syncwarp();
}

// The same to an intermediate matrix: 16-bit values, or FP32 values as three
// planes.
template <int TYPE>
__device__ __forceinline__ void store_planes(unsigned char *stage, int lane, void *base, long long ld,
                                             long long plane, long long row0, int n, int rows,
                                             int cols, float (&v)[32]) {
    if constexpr (TYPE != kTypeF32) {
        store_block<TYPE>(stage, lane, base, ld, row0, n, rows, cols, true, [&](int i) { return v[i]; });
    } else {
        // v becomes what is left of it.
#pragma unroll 1
        for (int q = 0; q < 3; ++q)
            store_block<kTypeBF16>(stage, lane, static_cast<uint16_t *>(base) + q * plane, ld, row0, n,
                                   rows, cols, true, [&](int i) {
                                       const float part = bf16_part(v[i]);
                                       v[i] = bf16_rest(v[i], part);
                                       return part;
                                   });
    }
}

template <int TYPE, int MODE, int CG>
__global__ void __launch_bounds__(kFfnThreads, 1)
    ffn_gemm_kernel(const __grid_constant__ FfnMaps maps, const FfnGemmParams p) {
    constexpr bool kSplit = TYPE == kTypeF32;         // three planes, sums in registers
    constexpr int kLoads = kSplit ? kPlanes : 1;      // stages of a step
    using Fm = Form<TYPE, CG>;
    constexpr int kAccCols = Fm::kAccCols, kStages = Fm::kStages, kParts = Fm::kParts;
    constexpr uint32_t kStageBytes = Fm::kStageBytes;
    constexpr int kTileN = MODE == kFfnGate ? kAccCols / 2 : kAccCols;
    extern __shared__ unsigned char ffn_smem_raw[];
    __shared__ uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int s_abort;

    const uint32_t raw = smem_addr(ffn_smem_raw);
    unsigned char *smem = ffn_smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const int worker = (int)blockIdx.x / CG;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
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
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 2) tc_alloc<CG, 2 * kAccCols>(&tmem_slot);
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (CG == 2) cluster_barrier();
    tc_fence_after_sync();
    const uint32_t tmem = tmem_slot;
    // Up to here nothing touched memory that the kernel before this one on the
    // stream reads or writes; its results are complete after this.
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp == 0) {
        // The whole warp runs the loop, as in the next branch, and one elected
        // lane issues: alone in the loop, a lane took some 700 clocks to issue
        // a stage's loads.
        // Stages so far over all tiles, the next one's place in the ring
        // and the parity its release is waited for with (1: still new).
        int it = 0, s = 0;
        uint32_t parity = 1;
        bool ok = true;
        const uint32_t bar0 = CG == 2 ? cluster_addr(&full[0], 0) : smem_addr(&full[0]);
        Unit unit;
        for (int u = 0; ok && unit_at(p, worker, u, unit); ++u) {
            const FfnProblem &pr = p.prob[MODE == kFfnStore ? unit.prob : 0];
            const int m0 = unit.m * (kFfnBM * CG) + (int)rank * kFfnBM;
            const int n0 = unit.n * kTileN, k_end = pr.kblocks * kFfnBK;
            const bool a_mn = pr.a_mn, b_mn = pr.b_mn;
            const uint32_t bytes = (pr.a_bytes + Fm::kBBytes) * CG;
            int seg = unit.s0 >= pr.kblocks ? 1 : 0;
            int k = unit.s0 * kFfnBK - seg * k_end;
            for (int step = unit.s0; ok && step < unit.s1; ++step, k += kFfnBK) {
                if (k >= k_end) {
                    k = 0;
                    seg = 1;
                }
                const CUtensorMap *ma = &maps.m[pr.a + seg], *mb = &maps.m[pr.b + seg];
#pragma unroll 1
                for (int load = 0; load < kLoads; ++load, ++it) {
                    if (p.skip_loads_from >= 0 && it >= p.skip_loads_from) {
                        ok = false;
                        break;
                    }
                    ok = tc_wait_warp(&empty[s], parity, p.timeout_ns);
                    if (!ok) {
                        if (lane == 0) {
                            atomicOr(p.err, kErrWaitTimeout);
                            s_abort = 1;
                        }
                        break;
                    }
                    if (tc_elect()) {
                        const int plane = kSplit ? plane_at(load) : 0;
                        const uint32_t a = sbase + s * kStageBytes, b = a + kABytes;
                        // The pair's loads all complete on the first CTA's barrier.
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
                        const uint32_t bar = bar0 + s * 8;
                        if (a_mn) {
                            tc_load_3d<CG>(a, ma, bar, m0, k, plane);
                            tc_load_3d<CG>(a + kBlockBytes, ma, bar, m0 + 64, k, plane);
                        } else {
                            tc_load_3d<CG>(a, ma, bar, k, m0, plane);
                        }
                        if constexpr (MODE == kFfnGate) {
                            // One CTA: 64 columns of each matrix.  A pair: the
                            // first CTA brings Wg's columns, the second Wu's.
                            const CUtensorMap *m1 = CG == 2 ? mb + rank : mb;
                            const CUtensorMap *m2 = CG == 2 ? m1 : mb + 1;
                            tc_load_3d<CG>(b, m1, bar, n0, k, plane);
                            if constexpr (Fm::kBCols == 128)
                                tc_load_3d<CG>(b + kBlockBytes, m2, bar, CG == 2 ? n0 + 64 : n0, k, plane);
                        } else {
                            const int n = n0 + (int)rank * Fm::kBCols;
                            if (b_mn) {
                                tc_load_3d<CG>(b, mb, bar, n, k, plane);
                                if constexpr (Fm::kBCols == 128)
                                    tc_load_3d<CG>(b + kBlockBytes, mb, bar, n + 64, k, plane);
                            } else {
                                tc_load_3d<CG>(b, mb, bar, k, n, plane);
                            }
                        }
                    }
                    __syncwarp();
                    if (++s == kStages) {
                        s = 0;
                        parity ^= 1;
                    }
                }
            }
        }
        // The last releases of the stages have to arrive before the CTA
        // leaves.
        for (int i = max(0, it - kStages); ok && i < it; ++i) {
            ok = tc_wait_warp(&empty[i % kStages], (i / kStages) & 1, p.timeout_ns);
            if (!ok && lane == 0) {
                atomicOr(p.err, kErrDrainTimeout);
                s_abort = 1;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // The whole warp runs the loop, one elected lane issues: a loop of one
        // lane alone keeps its descriptors in vector registers and spent some
        // 650 clocks on a stage whose products take 512.
        if (rank == 0) {
            // Descriptors of the first stage; the others and the steps along
            // k differ in the start address alone.
            const uint64_t desc_a = tc_desc(sbase, kBlockBytes);
            const uint64_t desc_b = tc_desc(sbase + kABytes, kBlockBytes);
            int s = 0, buf = 0;
            uint32_t parity = 0, acc_parity = 1;
            bool ok = true;
            Unit unit;
            for (int u = 0; ok && unit_at(p, worker, u, unit); ++u) {
                const FfnProblem &pr = p.prob[MODE == kFfnStore ? unit.prob : 0];
                const uint32_t idesc = tc_idesc(kFfnBM * CG, kAccCols, TYPE != kTypeF16, pr.a_mn != 0,
                                                pr.b_mn != 0);
                // Per 16 k: two groups of eight rows (MN-major) or 32 bytes
                // along the swizzled row (K-major); units of 16 bytes.
                const uint32_t a_step = (pr.a_mn ? 2048 : 32) >> 4, b_step = (pr.b_mn ? 2048 : 32) >> 4;
                // Waits for the next stage and returns its number.
                auto take = [&]() {
                    const int at = s;
                    ok = ok && tc_wait_warp(&full[s], parity, p.timeout_ns);
                    if (++s == kStages) {
                        s = 0;
                        parity ^= 1;
                    }
                    return at;
                };
                // A of stage i times B of stage j into accumulator d.
                auto product = [&](uint32_t d, int i, int j, bool first) {
                    const uint64_t a = desc_a + i * (kStageBytes >> 4);
                    const uint64_t b = desc_b + j * (kStageBytes >> 4);
#pragma unroll
                    for (int kk = 0; kk < kFfnBK / 16; ++kk)
                        tc_mma<CG>(d, a + kk * a_step, b + kk * b_step, idesc, !first || kk != 0);
                };
                ok = tc_wait_warp(&acc_empty[buf], acc_parity, p.timeout_ns);
                if constexpr (kSplit) {
                    // An accumulator takes one step: six products of the
                    // planes, smallest first; a stage is released after its
                    // last use.  What the next step starts with is waited for
                    // while the last products stand in the tensor core's queue
                    // (of about four MMAs).
                    int s0 = take(), s2 = take();
                    for (int step = unit.s0; ok; ++step) {
                        tc_fence_after_sync();
                        const uint32_t d = tmem + buf * kAccCols;
                        if (tc_elect()) {
                            product(d, s2, s0, true);
                            product(d, s0, s2, false);
                            tc_commit<CG>(&empty[s2]);
                        }
                        __syncwarp();
                        const int s1 = take();
                        if (!ok) break;
                        tc_fence_after_sync();
                        if (tc_elect()) {
                            product(d, s1, s1, false);
                            product(d, s1, s0, false);
                            product(d, s0, s1, false);
                            tc_commit<CG>(&empty[s1]);
                            product(d, s0, s0, false);
                            tc_commit<CG>(&empty[s0]);
                            tc_commit<CG>(&acc_full[buf]);
                        }
                        __syncwarp();
                        buf ^= 1;
                        acc_parity ^= buf ^ 1;
                        if (step + 1 == unit.s1) break;
                        ok = tc_wait_warp(&acc_empty[buf], acc_parity, p.timeout_ns);
                        s0 = take();
                        s2 = take();
                    }
                } else {
                    const uint32_t d = tmem + buf * kAccCols;
                    for (int step = unit.s0; ok && step < unit.s1; ++step) {
                        const int at = take();
                        if (!ok) break;
                        tc_fence_after_sync();
                        if (tc_elect()) {
                            product(d, at, at, step == unit.s0);
                            tc_commit<CG>(&empty[at]);
                            if (step + 1 == unit.s1) tc_commit<CG>(&acc_full[buf]);
                        }
                        __syncwarp();
                    }
                    buf ^= 1;
                    acc_parity ^= buf ^ 1;
                }
            }
            if (!ok && lane == 0) {
                atomicOr(p.err, kErrWaitTimeout);
                s_abort = 1;
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        const int quad = warp & 3, half = (warp - 4) >> 2;
        const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
        unsigned char *stage = smem + kStages * kStageBytes + (warp - 4) * kEpiBytes;
        // Part j is 32 accumulator columns; in the gate's product parts come
        // in twos, the same columns of g and u.
        constexpr int kTwo = MODE == kFfnGate ? 2 : 1;
        auto part_col = [&](int j) {
            return MODE == kFfnGate ? (j & 1) * (kAccCols / 2) + half * (kAccCols / 4) + 32 * (j >> 1)
                                    : half * (kAccCols / 2) + 32 * j;
        };
        int buf = 0;
        uint32_t parity = 0;
        bool ok = true;
        Unit unit;
        for (int u = 0; ok && unit_at(p, worker, u, unit); ++u) {
            const FfnProblem &pr = p.prob[MODE == kFfnStore ? unit.prob : 0];
            const int row0 = unit.m * (kFfnBM * CG) + (int)rank * kFfnBM + quad * 32;
            const int n_tile = unit.n * kTileN, rows = pr.M - row0;
            float sum[kSplit ? kParts : 1][32];
            uint32_t d = t_lane;
            if constexpr (kSplit) {
#pragma unroll
                for (int j = 0; j < kParts; ++j)
#pragma unroll
                    for (int i = 0; i < 32; ++i) sum[j][i] = 0.0f;
                for (int q = unit.s0; q < unit.s1; ++q) {
                    ok = tc_wait_warp(&acc_full[buf], parity, p.timeout_ns);
                    if (!ok) break;
                    tc_fence_after_sync();
#pragma unroll
                    for (int j = 0; j < kParts; ++j) {
                        uint32_t r[32];
                        tc_ld32(t_lane + buf * kAccCols + part_col(j), r);
                        tc_wait_ld(r);
#pragma unroll
                        for (int i = 0; i < 32; ++i) sum[j][i] += __uint_as_float(r[i]);
                    }
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) cluster_arrive(cluster_addr(&acc_empty[buf], 0));
                    buf ^= 1;
                    parity ^= buf ^ 1;
                }
            } else {
                ok = tc_wait_warp(&acc_full[buf], parity, p.timeout_ns);
                tc_fence_after_sync();
                d = t_lane + buf * kAccCols;
            }
            if (!ok) break;
            // This warp's part of the accumulator.
            auto own = [&](int j, float (&v)[32]) {
                if constexpr (kSplit) {
                    // Chosen by value: unrolled over the parts, the code below
                    // is so long that fetching it takes longer than running it.
                    static_assert(kParts == 2, "");
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = j ? sum[kParts - 1][i] : sum[0][i];
                } else {
                    uint32_t r[32];
                    tc_ld32(d + part_col(j), r);
                    tc_wait_ld(r);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
                }
            };
            // Where piece q of this tile keeps this warp's parts.
            auto slot = [&](int q) {
                return p.partials + (size_t)(piece_slot(unit, q) * CG + (int)rank) *
                                        (kEpiWarps * kParts * 1024) +
                       (warp - 4) * (kParts * 1024);
            };
            bool emit = rows > 0;
            if (unit.pieces > 1 && rows > 0) {
                float *mine = slot(unit.piece);
#pragma unroll 1
                for (int j = 0; j < kParts; ++j) {
                    float v[32];
                    own(j, v);
                    put_lanes(mine + j * 1024, lane, v);
                }
                __threadfence();
                __syncwarp();
                int *counter = p.counters + (unit.tail * CG + (int)rank) * kEpiWarps + (warp - 4);
                int arrived = 0;
                if (lane == 0) {
                    arrived = atomicAdd(counter, 1);
                    if (arrived == unit.pieces - 1) *counter = 0;
                }
                emit = __shfl_sync(0xffffffffu, arrived, 0) == unit.pieces - 1;
                __threadfence();
            }
            // The last to arrive adds the pieces (its own among them) in the
            // order of k.
            auto value = [&](int j, float (&v)[32]) {
                if (unit.pieces == 1) {
                    own(j, v);
                    return;
                }
                // (with FP32 half the columns at a time, for the registers' sake)
                constexpr int kAtOnce = kSplit ? 4 : 8;
#pragma unroll
                for (int i0 = 0; i0 < 8; i0 += kAtOnce) {
#pragma unroll
                    for (int i = 4 * i0; i < 4 * (i0 + kAtOnce); ++i) v[i] = 0.0f;
#pragma unroll 1
                    for (int q = 0; q < unit.pieces; ++q) {
                        const float4 *from = reinterpret_cast<const float4 *>(slot(q) + j * 1024) + lane;
                        float4 w[kAtOnce];
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i) w[i] = __ldcg(from + (i0 + i) * 32);
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i) {
                            v[4 * (i0 + i)] += w[i].x;
                            v[4 * (i0 + i) + 1] += w[i].y;
                            v[4 * (i0 + i) + 2] += w[i].z;
                            v[4 * (i0 + i) + 3] += w[i].w;
                        }
                    }
                }
            };
            if (emit) {
#pragma unroll 1
                for (int j = 0; j < kParts; j += kTwo) {
                    const int n = n_tile + (MODE == kFfnGate ? half * (kAccCols / 4) + 16 * j : part_col(j));
                    const int cols = pr.N - n;
                    if (cols <= 0) break;
                    const long long kept =
                        ((long long)(row0 >> 5) * p.keep_cols + (n >> 5)) * 1024;
                    float v[32];
                    if constexpr (MODE == kFfnStore) {
                        value(j, v);
                        store_block<TYPE>(stage, lane, pr.C[0], pr.ldc, row0, n, rows, cols, pr.c_vec,
                                          [&](int i) { return v[i]; });
                    } else if constexpr (MODE == kFfnGate) {
                        float w[32];
                        value(j, v);
                        value(j + 1, w);
                        if (p.keep[0]) {
                            // Four columns at a time, as put_lanes would lay
                            // them: 32 more values would not fit the registers.
                            float4 *k0 = reinterpret_cast<float4 *>(p.keep[0] + kept) + lane;
                            float4 *k1 = reinterpret_cast<float4 *>(p.keep[1] + kept) + lane;
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                float a[4], t[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    float slope;
                                    gate_act_slope<kSplit>(v[4 * i + e], p.act, a[e], slope);
                                    t[e] = w[4 * i + e] * slope;
                                    w[4 * i + e] *= a[e];
                                }
                                __stcg(k0 + i * 32, make_float4(t[0], t[1], t[2], t[3]));
                                __stcg(k1 + i * 32, make_float4(a[0], a[1], a[2], a[3]));
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) w[i] *= gate_act<kSplit>(v[i], p.act);
                        }
                        store_planes<TYPE>(stage, lane, pr.C[0], pr.ldc, pr.c_plane, row0, n, rows,
                                           cols, w);
                    } else {
                        value(j, v);
#pragma unroll 1
                        for (int w = 0; w < 2; ++w) {
                            float t[32];
                            get_lanes(p.keep[w] + kept, lane, t);
#pragma unroll
                            for (int i = 0; i < 32; ++i) t[i] *= v[i];
                            store_planes<TYPE>(stage, lane, pr.C[w], pr.ldc, pr.c_plane, row0, n, rows,
                                               cols, t);
                        }
                    }
                }
            }
            if constexpr (!kSplit) {
                // The accumulator may be overwritten.
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) cluster_arrive(cluster_addr(&acc_empty[buf], 0));
                buf ^= 1;
                parity ^= buf ^ 1;
            }
        }
        if (!ok && lane == 0) {
            atomicOr(p.err, kErrWaitTimeout);
            s_abort = 1;
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (tid == 0 && (s_abort || p.skip_loads_from >= 0)) {
        // A role gave up: loads and products may still be in flight.  They
        // take microseconds; nothing here signals their end any more.
        const long long t0 = clock64();
        while (clock64() - t0 < 4000000) {
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
// element), or 16-bit values to aligned rows.  A thread takes eight elements of a
// row, so stores are 16 bytes; FP32 rows that start anywhere are read as the aligned
// 16-byte pieces that cover the eight.  The element's row is kept up by addition,
// not by a 64-bit division for each.  Bound: instructions and HBM; 8.4 M weights and
// 1 M activations of FP32 take 17 us cold (5.6 us of reading).
// ---------------------------------------------------------------------------
constexpr int kPrepCtas = 6;  // of an SM
struct PrepTable {
    int count;
    FfnPrepJob job[kFfnPrepJobs];
};

template <bool SPLIT>
__global__ void __launch_bounds__(256, kPrepCtas) ffn_prep_kernel(const PrepTable t) {
    for (int q = 0; q < t.count; ++q) {
        const FfnPrepJob &j = t.job[q];
        const int octets = (j.cols + 7) / 8;
        const long long step = gridDim.x * 256LL, start = blockIdx.x * 256LL + threadIdx.x;
        const long long step_rows = step / octets;
        const int step_octets = (int)(step - step_rows * octets);
        long long row = start / octets;
        int octet = (int)(start - row * octets);
        for (; row < j.rows; row += step_rows, octet += step_octets) {
            if (octet >= octets) {
                octet -= octets;
                if (++row >= j.rows) break;
            }
            const int c = octet * 8;
            const long long from = row * j.ld_src + c, to = row * j.ld_dst + c;
            if constexpr (SPLIT) {
                const float *src = static_cast<const float *>(j.src) + from;
                const int shift = (int)(reinterpret_cast<uintptr_t>(src) & 15) / 4;
                const float *piece = src - shift;
                const float *first = static_cast<const float *>(j.src);
                float v[8];
                if (c + 8 <= j.cols && piece >= first &&
                    piece + 12 <= first + (j.rows - 1) * j.ld_src + j.cols) {
                    float4 w[3];
                    w[0] = __ldg(reinterpret_cast<const float4 *>(piece));
                    w[1] = __ldg(reinterpret_cast<const float4 *>(piece) + 1);
                    w[2] = shift ? __ldg(reinterpret_cast<const float4 *>(piece) + 2) : w[1];
                    const float f[12] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y,
                                         w[1].z, w[1].w, w[2].x, w[2].y, w[2].z, w[2].w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float even = shift & 2 ? f[e + 2] : f[e], odd = shift & 2 ? f[e + 3] : f[e + 1];
                        v[e] = shift & 1 ? odd : even;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = c + e < j.cols ? __ldg(src + e) : 0.0f;
                }
                float part[8][3];
#pragma unroll
                for (int e = 0; e < 8; ++e) split3(v[e], part[e]);
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
cudaError_t launch_one(const FfnMaps &maps, const FfnGemmParams &p, cudaStream_t stream) {
    const auto kernel = ffn_gemm_kernel<TYPE, MODE, CG>;
    static std::atomic<bool> configured[kMaxDevices];
    if (p.device >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!configured[p.device].load()) {
        const cudaError_t e = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Form<TYPE, CG>::kSmem);
        if (e != cudaSuccess) return e;
        configured[p.device].store(true);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CG * (p.full_tiles + p.long_tiles > 0 ? p.workers
                             : p.tail_workers ? p.tail_workers : p.tail_tiles));
    cfg.blockDim = dim3(kFfnThreads);
    cfg.dynamicSmemBytes = Form<TYPE, CG>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, maps, p);
}

template <int TYPE, int CG>
cudaError_t launch_mode(const FfnMaps &maps, const FfnGemmParams &p, cudaStream_t stream) {
    switch (p.mode) {
        case kFfnStore: return launch_one<TYPE, kFfnStore, CG>(maps, p, stream);
        case kFfnGate: return launch_one<TYPE, kFfnGate, CG>(maps, p, stream);
        default: return launch_one<TYPE, kFfnGateGrad, CG>(maps, p, stream);
    }
}

}  // namespace

cudaError_t launch_ffn_gemm(const FfnMaps &maps, const FfnGemmParams &p, bool pair,
                            cudaStream_t stream) {
    if (p.type == kTypeF32)
        return pair ? launch_mode<kTypeF32, 2>(maps, p, stream)
                    : launch_mode<kTypeF32, 1>(maps, p, stream);
    if (p.type == kTypeF16)
        return pair ? launch_mode<kTypeF16, 2>(maps, p, stream)
                    : launch_mode<kTypeF16, 1>(maps, p, stream);
    return pair ? launch_mode<kTypeBF16, 2>(maps, p, stream)
                : launch_mode<kTypeBF16, 1>(maps, p, stream);
}

cudaError_t launch_ffn_prep(const FfnPrepJob *jobs, int count, int type, int num_sms,
                            cudaStream_t stream) {
    if (count == 0) return cudaSuccess;
    PrepTable t;
    t.count = count;
    for (int i = 0; i < count; ++i) t.job[i] = jobs[i];
    if (type == kTypeF32)
        ffn_prep_kernel<true><<<num_sms * kPrepCtas, 256, 0, stream>>>(t);
    else
        ffn_prep_kernel<false><<<num_sms * kPrepCtas, 256, 0, stream>>>(t);
    return cudaGetLastError();
}

}  // namespace sgemm
