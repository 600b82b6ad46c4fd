// Products of 8-bit integers on the fifth-generation tensor cores.
//
// The integer rate of this chip's tensor cores is a small part of its 16-bit rate, so the
// integers go through as FP16, which holds each of them exactly.  A product is
// below 2^14 in magnitude (or equal to it) and 1024 of them add up to 2^24 at most: an
// FP32 accumulator is exact that far.  It is taken out of tensor memory after every
// 1024 k and added up in 32-bit integers, so that y's sum is exact for every K,
// and neither the tiles nor the way that K is shared out changes a bit of it.
//
// y^T = w x^T: a tile is 128 channels (256 by a pair of CTAs) by up to 96 (192)
// tokens.  The weights stay 8 bits wide up to the SM: they are widened by eight
// warps from shared memory into tensor memory, from where the tensor core reads its
// first operand, so that shared memory carries them once in 8 bits and not again in
// 16.  x, read by every channel tile, is widened by a kernel of its own first.
//
// 640 threads a CTA, one CTA per SM, registers moved to where the sums are
// (setmaxnreg; the launch has 96 a thread):
//   warps 0, 3   TMA loads: w 16 KB and x up to 24 KB per stage of 128 k
//   warp 1       tcgen05.mma, one elected thread
//   warp 2       allocates tensor memory
//   warps 4-11   widen: a warp 64 k of 32 rows of a stage (128-byte swizzle), into 32 of
//                the 64 tensor-memory columns of a slot
//   warps 12-19  epilogue: accumulators to integers, scales, stores
// Tensor memory: two accumulators of 192 columns, two slots of 64.
// Widening takes a stage's warps some 700 clocks, the products of 192 tokens by a pair
// 768: from there on the tensor pipe is the bound (90 % busy at 4096 x 4096 x 12288, 204 us,
// 2.0 PFLOP/s; with the widening of x 12 us more; in a long run 233 to 242, at the power
// limit).  With fewer tokens it is the weights' way (64 x 12288 x 4096, pieces of 64 tiles:
// 20 us where HBM would take 7.7): widening, a pipeline of stages that fills once a tile, and
// the pieces' meeting, 2 to 3 us.
//
// Every wait is bounded; a role that gives up flags the error word, the others
// run out in turn, and the CTA lets its copies land before it leaves.
#include <algorithm>
#include <atomic>

#include "kernels_q8.h"
#include "ops_common.cuh"
#include "tc_common.cuh"

namespace sgemm {
namespace {

constexpr int kThreads = 640;
constexpr int kRegsRoles = 40, kRegsWiden = 80, kRegsEpilogue = 136;
static_assert(128 * kRegsRoles + 256 * (kRegsWiden + kRegsEpilogue) <= 96 * kThreads, "");
constexpr int kStages = 5, kSlots = 2;
constexpr uint32_t kWBytes = kQ8Channels * kQ8StageK;
constexpr uint32_t kStageBytes = kWBytes + kQ8Tokens * kQ8StageK * 2;
constexpr int kEpiWarps = 8;
constexpr uint32_t kEpiBytes = 16 * 32 * 4;  // an epilogue warp's staging: 16 tokens of 32 channels
constexpr size_t kSmem = (size_t)kStages * kStageBytes + kEpiWarps * kEpiBytes + 1024;
constexpr int kAccCols = 2 * kQ8Tokens, kSlotCol = 2 * kAccCols;  // tensor-memory columns
constexpr int kTmemCols = 512;
constexpr int kSlotCols = kQ8StageK / 2;
static_assert(kSlotCol + kSlots * kSlotCols == kTmemCols, "");
constexpr int kWidenWarps = 8;
constexpr int kFirstWiden = 4, kFirstEpi = 12;
constexpr int kParts = kQ8Tokens / 16;                // of 16 columns, an epilogue warp's
constexpr int kChunk = kQ8ExactK / kQ8StageK;         // stages of an accumulator
constexpr int kMaxDevices = 64;

// A stretch of one tile's stages that a worker computes.
struct Unit {
    int m, n;           // tile along the tokens, along the channels
    int s0, s1;         // stages [s0, s1)
    int pieces;         // the tile's stretches
    int tail;           // the tile's number in the tail
};

// Tiles in groups of eight channel tiles, token tile by token tile inside a
// group, so that the CTAs at work share weights and tokens in L2.
__device__ __forceinline__ void locate(const Q8GemmParams &p, int t, Unit &u) {
    constexpr int kGroup = 8;
    const int per_group = kGroup * p.tiles_m;
    const int first = t / per_group * kGroup;
    const int rows = min(kGroup, p.tiles_n - first);
    t -= first * p.tiles_m;
    u.n = first + t % rows;
    u.m = t / rows;
}

// The worker's i-th unit; false when there is none.  A tail tile's stages are shared out
// evenly over as many workers as it has pieces.
__device__ __forceinline__ bool unit_at(const Q8GemmParams &p, int worker, int i, Unit &u) {
    u.s0 = 0;
    u.s1 = p.stages_k;
    u.pieces = 1;
    u.tail = 0;
    int t = worker + i * p.workers;
    if (i >= p.full_tiles && p.pieces > 1) {
        if (i > p.full_tiles || worker >= p.tail_tiles * p.pieces) return false;
        u.pieces = p.pieces;
        u.tail = worker / p.pieces;
        const int piece = worker - u.tail * p.pieces;
        u.s0 = piece * p.stages_k / p.pieces;
        u.s1 = (piece + 1) * p.stages_k / p.pieces;
        t = p.full_tiles * p.workers + u.tail;
    }
    if (t >= p.tiles_m * p.tiles_n) return false;
    locate(p, t, u);
    return true;
}

// Four signed bytes to four FP16 values: with the sign bit flipped a byte is x +
// 128, and 0x6400 | (x + 128) is 1024 + 128 + x.
__device__ __forceinline__ void widen(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t v = w ^ 0x80808080u;
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    const uint32_t a = __byte_perm(v, 0x64646464u, 0x4140), b = __byte_perm(v, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), off);
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
}

// 32 consecutive columns of this warp's 32 lanes from registers.
__device__ __forceinline__ void tc_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
        "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),
        "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tc_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// 16 consecutive columns of this warp's 32 lanes.
__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tc_wait_ld16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// First operand from tensor memory.
template <int CG>
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
            "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
            "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}

// A whole warpgroup gives registers back, or takes what others gave back.
template <int N>
__device__ __forceinline__ void set_fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <int TYPE, int CG>
__global__ void __launch_bounds__(kThreads, 1)
    q8_gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                   const Q8GemmParams p) {
    extern __shared__ unsigned char q8_smem_raw[];
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ uint64_t a_full[kSlots], a_empty[kSlots], acc_full[2], acc_empty[2];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int s_abort;

    const uint32_t raw = smem_addr(q8_smem_raw);
    unsigned char *smem = q8_smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    const uint32_t sbase = smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const int worker = (int)blockIdx.x / CG;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 2);
            mbar_init(&empty[s], 1);
        }
        for (int j = 0; j < kSlots; ++j) {
            mbar_init(&a_full[j], kWidenWarps * CG);
            mbar_init(&a_empty[j], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], kEpiWarps * CG);
        }
        s_abort = 0;
        fence_barrier_init();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 2) tc_alloc<CG, kTmemCols>(&tmem_slot);
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (CG == 2) cluster_barrier();
    tc_fence_after_sync();
    const uint32_t tmem = tmem_slot;
    // Up to here nothing touched memory that the kernel before this one on the
    // stream reads or writes; its results are complete after this.
    asm volatile("griddepcontrol.wait;" ::: "memory");

    auto give_up = [&](int error) {
        if (lane == 0) {
            atomicOr(p.err, error);
            s_abort = 1;
        }
    };
    bool ok = true;
    Unit unit;

    if (warp < kFirstWiden) {
        set_fewer_registers<kRegsRoles>();
        if (warp == 0 || warp == 3) {
            // One warp brings the weights, the other the tokens: a stage's loads take one
            // some 600 clocks to issue.
            const int tokens = p.tokens / CG;  // that this CTA brings in
            const uint32_t bytes = warp == 0 ? kWBytes : (uint32_t)tokens * 256;
            int it = 0, s = 0;
            uint32_t parity = 1;
            for (int u = 0; ok && unit_at(p, worker, u, unit); ++u) {
                const int n0 = (unit.n * CG + (int)rank) * kQ8Channels;
                const int m0 = unit.m * p.tokens + (int)rank * tokens;
                for (int st = unit.s0; st < unit.s1; ++st, ++it) {
                    if (p.skip_loads_from >= 0 && it >= p.skip_loads_from) {
                        ok = false;
                        break;
                    }
                    // (products done: the weights were widened before them)
                    ok = tc_wait_warp(&empty[s], parity, p.timeout_ns);
                    if (!ok) {
                        give_up(kErrWaitTimeout);
                        break;
                    }
                    if (tc_elect()) {
                        mbar_arrive_expect_tx(&full[s], bytes);
                        if (warp == 0)
                            tma_load_2d(smem + s * kStageBytes, &map_w, &full[s], st * kQ8StageK, n0);
                        else
                            tc_load_3d<1>(sbase + s * kStageBytes + kWBytes, &map_x, smem_addr(&full[s]), 0,
                                          m0, st * 2);
                    }
                    __syncwarp();
                    if (++s == kStages) {
                        s = 0;
                        parity ^= 1;
                    }
                }
            }
            // The last releases of the stages have to arrive before the CTA leaves.
            for (int i = max(0, it - kStages); ok && i < it; ++i) {
                ok = tc_wait_warp(&empty[i % kStages], (i / kStages) & 1, p.timeout_ns);
                if (!ok) give_up(kErrDrainTimeout);
            }
            __syncwarp();
        } else if (warp == 1) {
            if (rank == 0) {
                const uint64_t desc = tc_desc(sbase + kWBytes, 0);
                const uint32_t second = (uint32_t)(p.tokens / CG) * 128 >> 4;  // from 64 k to the next
                const uint32_t idesc = tc_idesc(kQ8Channels * CG, p.tokens, false, false, false);
                int s = 0, slot = 0, buf = 0;
                uint32_t slot_parity = 0, acc_parity = 1;
                for (int u = 0; ok && unit_at(p, worker, u, unit); ++u) {
                    for (int st = unit.s0; st < unit.s1; ++st) {
                        const int at = (st - unit.s0) % kChunk;
                        const bool last = at == kChunk - 1 || st + 1 == unit.s1;
                        // The slots' warps, of both CTAs, waited for the tokens too.
                        ok = (at != 0 || tc_wait_warp(&acc_empty[buf], acc_parity, p.timeout_ns)) &&
                             tc_wait_warp(&a_full[slot], slot_parity, p.timeout_ns);
                        if (!ok) break;
                        tc_fence_after_sync();
                        if (tc_elect()) {
                            const uint64_t b = desc + ((s * kStageBytes) >> 4);
                            const uint32_t a = tmem + kSlotCol + slot * kSlotCols, d = tmem + buf * kAccCols;
#pragma unroll
                            for (int kk = 0; kk < kQ8StageK / 16; ++kk)
                                tc_mma_ts<CG>(d, a + kk * 8,
                                              b + (kk / 4) * second + (kk % 4) * 2, idesc,
                                              at != 0 || kk != 0);
                            tc_commit<CG>(&a_empty[slot]);
                            tc_commit<CG>(&empty[s]);
                            if (last) tc_commit<CG>(&acc_full[buf]);
                        }
                        __syncwarp();
                        if (last) {
                            buf ^= 1;
                            acc_parity ^= buf ^ 1;
                        }
                        if (++slot == kSlots) {
                            slot = 0;
                            slot_parity ^= 1;
                        }
                        if (++s == kStages) s = 0;
                    }
                }
                if (!ok) give_up(kErrWaitTimeout);
            }
            __syncwarp();
        }
    } else if (warp < kFirstEpi) {
        set_fewer_registers<kRegsWiden>();
        const int quad = warp & 3, half = (warp - kFirstWiden) >> 2;
        const int row = quad * 32 + lane;
        const uint32_t t_lane = tmem + kSlotCol + half * (kQ8SlotK / 2) + ((uint32_t)(quad * 32) << 16);
        const uint32_t bar0 = cluster_addr(&a_full[0], 0);
        int s = 0, slot = 0, done = 0;
        uint32_t parity = 0, slot_parity = 1;
        int total = 0;
        for (int u = 0; unit_at(p, worker, u, unit); ++u) total += unit.s1 - unit.s0;
        uint4 w[4];
        auto bring = [&]() {
            ok = tc_wait_warp(&full[s], parity, p.timeout_ns);
            const unsigned char *from = smem + s * kStageBytes + row * 128;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                w[c] = *reinterpret_cast<const uint4 *>(from + (((half * 4 + c) ^ (row & 7)) << 4));
            if (++s == kStages) {
                s = 0;
                parity ^= 1;
            }
        };
        if (total) bring();
        for (int left = total; ok && left > 0; --left) {
            uint32_t r[32];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                widen(w[c].x, r[8 * c], r[8 * c + 1]);
                widen(w[c].y, r[8 * c + 2], r[8 * c + 3]);
                widen(w[c].z, r[8 * c + 4], r[8 * c + 5]);
                widen(w[c].w, r[8 * c + 6], r[8 * c + 7]);
            }
            if (left > 1) bring();
            if (!ok) break;
            ok = tc_wait_warp(&a_empty[slot], slot_parity, p.timeout_ns);
            if (!ok) break;
            tc_fence_after_sync();
            tc_st32(t_lane + slot * kSlotCols, r);
            tc_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) cluster_arrive(bar0 + slot * 8);
            ++done;
            if (++slot == kSlots) {
                slot = 0;
                slot_parity ^= 1;
            }
        }
        if (!ok) give_up(kErrWaitTimeout);
        // The last releases of the slots have to arrive before the CTA leaves.
        for (int i = max(0, done - kSlots); ok && i < done; ++i) {
            ok = tc_wait_warp(&a_empty[i % kSlots], (i / kSlots) & 1, p.timeout_ns);
            if (!ok) give_up(kErrDrainTimeout);
        }
    } else {
        set_more_registers<kRegsEpilogue>();
        const int quad = warp & 3, half = (warp - kFirstEpi) >> 2;
        const int mine = p.tokens / 2;  // columns of this warp's half
        const int parts = (mine + 15) / 16;
        const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16) + half * mine;
        unsigned char *stage = smem + kStages * kStageBytes + (warp - kFirstEpi) * kEpiBytes;
        int buf = 0;
        uint32_t parity = 0;
        for (int u = 0; ok && unit_at(p, worker, u, unit); ++u) {
            const int n = (unit.n * CG + (int)rank) * kQ8Channels + quad * 32 + lane;
            const int m0 = unit.m * p.tokens + half * mine;
            const int left = min(mine, p.M - m0);
            // The tile's scales, before they are waited for: of 96 tokens, three a lane.
            float xs[kQ8Tokens / 32];
#pragma unroll
            for (int j = 0; j < kQ8Tokens / 32; ++j)
                xs[j] = j * 32 + lane < left ? __ldg(p.x_scales + m0 + j * 32 + lane) : 0.0f;
            const float ws = n < p.N ? __ldg(p.w_scales + n) : 0.0f;
            int sum[kParts][16];
#pragma unroll
            for (int j = 0; j < kParts; ++j)
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[j][i] = 0;
            for (int st = unit.s0; st < unit.s1; st += kChunk) {
                ok = tc_wait_warp(&acc_full[buf], parity, p.timeout_ns);
                if (!ok) break;
                tc_fence_after_sync();
#pragma unroll
                for (int j = 0; j < kParts; ++j)
                    if (j < parts) {
                        uint32_t r[16];
                        tc_ld16(t_lane + buf * kAccCols + j * 16, r);
                        tc_wait_ld16(r);
#pragma unroll
                        for (int i = 0; i < 16; ++i) sum[j][i] += __float2int_rn(__uint_as_float(r[i]));
                    }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) cluster_arrive(cluster_addr(&acc_empty[buf], 0));
                buf ^= 1;
                parity ^= buf ^ 1;
            }
            if (!ok) break;
            bool emit = true;
            if (unit.pieces > 1) {
                // The pieces are added up in L2 (whole numbers: in any order), where all is zero
                // before and, when the last to arrive has read it, again.
                int *meet = p.meet + ((size_t)(unit.tail * CG + (int)rank) * kEpiWarps + (warp - kFirstEpi)) *
                                         (kParts * 16 * 32) + lane;
#pragma unroll
                for (int j = 0; j < kParts; ++j)
                    if (j < parts) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) atomicAdd(meet + (j * 16 + i) * 32, sum[j][i]);
                    }
                __threadfence();
                __syncwarp();
                int *counter = p.counters + (unit.tail * CG + (int)rank) * kEpiWarps + (warp - kFirstEpi);
                int arrived = 0;
                if (lane == 0) {
                    arrived = atomicAdd(counter, 1);
                    if (arrived == unit.pieces - 1) *counter = 0;
                }
                emit = __shfl_sync(0xffffffffu, arrived, 0) == unit.pieces - 1;
                __threadfence();
                if (emit) {
#pragma unroll
                    for (int j = 0; j < kParts; ++j)
                        if (j < parts) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) sum[j][i] = __ldcg(meet + (j * 16 + i) * 32);
                        }
#pragma unroll
                    for (int j = 0; j < kParts; ++j)
                        if (j < parts) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) __stcg(meet + (j * 16 + i) * 32, 0);
                        }
                }
            }
            if (emit) {
                // 16 tokens at a time through shared memory, from a lane a channel to 16 bytes
                // of a token a lane.  (Stored as they lie in registers, 2 bytes a lane, a
                // tile took 16000 clocks, more than half of its products.)
                const int channels = p.N - (n - lane);  // of the warp's 32 that exist
#pragma unroll
                for (int j = 0; j < kParts; ++j)
                    if (j * 16 < left) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int t = j * 16 + i;
                            const float v =
                                (float)sum[j][i] * __shfl_sync(0xffffffffu, xs[t / 32], t % 32) * ws;
                            store_from_float(stage, TYPE, i * 32 + lane, v);
                        }
                        __syncwarp();
                        constexpr int kElem = TYPE == kTypeF32 ? 4 : 2, kPer = 16 / kElem;
                        constexpr int kRow = 32 / kPer;  // lanes of a token
                        unsigned char *out = static_cast<unsigned char *>(p.y) +
                                             ((m0 + j * 16) * p.ldy + (n - lane)) * kElem;
                        const int tokens = min(16, left - j * 16);
                        if (p.y_vec && channels >= 32) {
                            const int c = lane % kRow * 16;
#pragma unroll
                            for (int token = lane / kRow; token < 16; token += 32 / kRow)
                                if (token < tokens)
                                    *reinterpret_cast<uint4 *>(out + token * p.ldy * kElem + c) =
                                        *reinterpret_cast<const uint4 *>(stage + token * 32 * kElem + c);
                        } else if (lane < channels) {
#pragma unroll 4
                            for (int token = 0; token < tokens; ++token) {
                                unsigned char *to = out + (token * p.ldy + lane) * kElem;
                                const unsigned char *from = stage + (token * 32 + lane) * kElem;
                                if constexpr (kElem == 4)
                                    *reinterpret_cast<uint32_t *>(to) = *reinterpret_cast<const uint32_t *>(from);
                                else
                                    *reinterpret_cast<uint16_t *>(to) = *reinterpret_cast<const uint16_t *>(from);
                            }
                        }
                        __syncwarp();
                    }
            }
        }
        if (!ok) give_up(kErrWaitTimeout);
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
        tc_dealloc<CG, kTmemCols>(tmem);
    }
}

template <int TYPE, int CG>
cudaError_t launch_one(const CUtensorMap &w, const CUtensorMap &x, const Q8GemmParams &p,
                       cudaStream_t stream) {
    const auto kernel = q8_gemm_kernel<TYPE, CG>;
    static std::atomic<bool> configured[kMaxDevices];
    if (p.device >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!configured[p.device].load()) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        if (e != cudaSuccess) return e;
        configured[p.device].store(true);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CG * (p.full_tiles > 0 ? p.workers : p.tail_tiles * p.pieces));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, w, x, p);
}

// Bytes to FP16 in rows of ldo (a multiple of 8) values, eight at a time, zeros
// from K on.
__global__ void __launch_bounds__(256) q8_widen_kernel(const int8_t *x, long long ldx, int M, int K,
                                                       uint16_t *out, long long ldo, bool vec) {
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
    const int octets = (int)(ldo / 8);
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < (long long)M * octets; i += gridDim.x * 256LL) {
        const long long row = i / octets;
        const int k = (int)(i - row * octets) * 8;
        const int8_t *from = x + row * ldx + k;
        uint32_t w[2] = {0, 0};
        if (vec && k + 8 <= K) {
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(from));
            w[0] = v.x;
            w[1] = v.y;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (k + j < K) w[j / 4] |= (uint32_t)(uint8_t)__ldg(from + j) << (8 * (j % 4));
        }
        uint4 o;
        widen(w[0], o.x, o.y);
        widen(w[1], o.z, o.w);
        *reinterpret_cast<uint4 *>(out + row * ldo + k) = o;
    }
}

// Rows of bytes to rows of ldo (a multiple of 16) bytes, zeros from K on.
__global__ void __launch_bounds__(256) q8_align_kernel(const int8_t *w, long long ldw, int N, int K,
                                                       int8_t *out, long long ldo) {
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
    const long long words = ldo / 4;
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < N * words; i += gridDim.x * 256LL) {
        const long long row = i / words;
        const int k = (int)(i - row * words) * 4;
        uint32_t v = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (k + j < K) v |= (uint32_t)(uint8_t)__ldg(w + row * ldw + k + j) << (8 * j);
        *reinterpret_cast<uint32_t *>(out + row * ldo + k) = v;
    }
}

template <class... Params, class... Args>
cudaError_t launch_flat(void (*kernel)(Params...), long long items, int num_sms, cudaStream_t stream,
                        Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<long long>((items + 255) / 256, 8LL * num_sms));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_q8_gemm(const CUtensorMap &w, const CUtensorMap &x, const Q8GemmParams &p,
                           int type, bool pair, cudaStream_t stream) {
    if (type == kTypeF32)
        return pair ? launch_one<kTypeF32, 2>(w, x, p, stream) : launch_one<kTypeF32, 1>(w, x, p, stream);
    if (type == kTypeF16)
        return pair ? launch_one<kTypeF16, 2>(w, x, p, stream) : launch_one<kTypeF16, 1>(w, x, p, stream);
    return pair ? launch_one<kTypeBF16, 2>(w, x, p, stream) : launch_one<kTypeBF16, 1>(w, x, p, stream);
}

cudaError_t launch_q8_widen(const int8_t *x, long long ldx, int M, int K, uint16_t *out,
                            long long ldo, int num_sms, cudaStream_t stream) {
    const bool vec = (reinterpret_cast<uintptr_t>(x) & 7) == 0 && (M == 1 || ldx % 8 == 0);
    return launch_flat(q8_widen_kernel, M * (ldo / 8), num_sms, stream, x, ldx, M, K, out, ldo, vec);
}

cudaError_t launch_q8_align(const int8_t *w, long long ldw, int N, int K, int8_t *out,
                            long long ldo, int num_sms, cudaStream_t stream) {
    return launch_flat(q8_align_kernel, N * (ldo / 4), num_sms, stream, w, ldw, N, K, out, ldo);
}

}  // namespace sgemm
