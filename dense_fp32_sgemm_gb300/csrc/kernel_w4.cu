// Products of a few rows with 4-bit weights, and their quantisation.
//
//   y[m][n] = sum over groups G of  s[G][n] * sum over k in G of x[m][k] (q[k][n] - z[G][n])
//
// Bound: HBM, K N / 2 bytes of q read once.  At the card's rate that is 13.6
// weights per ns, so a lane has about 2.4 instructions for each, fewer where
// they are logic (half rate).  So the products go to the warp-level matrix
// instruction and the lanes only expand the weights: a word's eight values
// become four pairs of 16-bit floats, each by one logic instruction (the forms
// are described at expand).  The fifth-generation tensor cores would need the
// expanded weights in shared memory and gain nothing at 16 columns.
//
// Layout.  The instruction (m16n8k16) takes the weights as its 16 x 16
// operand, rows along n, and x as its 16 x 8 one, so up to eight rows of x
// cost one instruction.  The order of k inside an instruction is free, so the
// pairs come as a word gives them: (0,4), (1,5) in one instruction and (2,6),
// (3,7) in the next, and x read from shared memory is put in that order by four
// byte permutations.  Lane (g, t) = (lane / 4, lane % 4) of a warp takes eight
// columns' words of word row t of four; a unit is 128 k x 64 columns, 4 KB.
//
// Exactness.  q, z and q - z have at most five bits; 16-bit x enters as it is.
// With 16-bit x the zero points' part, z (or 128 + z) times the sum of x, comes
// off at the end of a group, its sum by one more instruction on a matrix of
// ones: a quarter fewer instructions.  The cancellation costs bf16 five bits of
// the FP32 sums' 24, far below the 8 bits of its y, and fp16 one or two.  FP32
// x keeps the exact form; it is the sum of three bf16 parts, each a row of its
// own of the x operand (made while x is staged).  Sums are FP32; each group's
// sum is scaled in FP32.
//
// Memory.  The time of such a product is a few round trips to HBM.  A warp
// keeps a ring of units of its own under way in shared memory: two TMA boxes of
// 32 columns each (128-byte swizzle; lanes take their columns in an order that
// makes the reads free of bank conflicts) and bulk copies of the scales and
// zero points, or, where rows do not start on 16 bytes, the aligned 16-byte
// pieces that cover them.  TMA because it costs one lane two instructions: as
// 16-byte copies by all lanes the first units alone held the warps up for 4000
// clocks of a 13 us call, and one warp asking for all others' units took 800
// clocks for each.
//
// Measured: 1 x 4096 x 12288 bf16 9.5 us (2.7 TB/s; 10.3 as a call), 16 x 12288 x
// 4096 16 us (18.3 as a call), 3 x 8191 x 8191 FP32 31 us (32.4); as calls also 1 x
// 16384 x 24576 49-53 us (4.0-4.2 TB/s) and 8 x 4096 x 12288 14.3 us.  More rows take a
// launch for every 16, each of which reads q again: 300 x 4096 x 4096 195 us, 4096 rows
// 2635 us (52 TFLOP/s).
// What bounds the larger ones is the latency of a warp's chain (shared read, expansion,
// matrix instructions, group scaling): shared memory leaves an SM two or three CTAs of
// four warps, which keep the issue slots 30-38 % and HBM 14-26 % busy.
//
// Split.  A CTA's four warps stand side by side on 64 columns each
// or behind one another along K (taking every n-th unit), or both: few rows of
// x favour K (more CTAs), many rows columns (x is staged once per CTA).  Warps
// along K add up through shared memory in warp order.  Where the columns give
// too few CTAs, a cluster shares K and adds its CTAs' sums in rank order
// through distributed shared memory: no atomics, no workspace.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "ops_common.cuh"
#include "tc_common.cuh"

namespace cg = cooperative_groups;

namespace sgemm {
namespace {

constexpr int kMaxDevices = 64;
constexpr int kThreads = kW4Warps * 32;
constexpr int kSteps = kW4UnitK / 32;
constexpr int kRows = kW4UnitK / 8;              // word rows of a unit
constexpr int kBoxBytes = kRows * 128;           // 32 columns of a unit
constexpr int kPlainPitch = 288;                 // bytes of a row of 64 + 3 words, banks apart

// A unit in shared memory: q (two boxes, or 16 rows of pieces), then a row of
// scales and one of zero points for each of its NG groups, as pieces.
template <int TYPE, int NG>
struct UnitLayout {
    static constexpr int kElem = TYPE == kTypeF32 ? 4 : 2;
    static constexpr int kScalePieces = kW4Cols * kElem / 16 + 1, kZeroPieces = kW4Cols / 16 + 1;
    static constexpr int kScale = kRows * kPlainPitch;
    static constexpr int kZero = kScale + NG * kScalePieces * 16;
    static constexpr int kBytes = (kZero + NG * kZeroPieces * 16 + 1023) / 1024 * 1024;
};
static_assert(2 * kBoxBytes <= kRows * kPlainPitch, "boxes fit in the plain rows' place");

// An aligned 16-byte piece of a row of a matrix into shared memory, as far as
// it lies inside the row: up to `end`, and not before the matrix's first
// element `base` (then element by element).
__device__ __forceinline__ void copy_piece(unsigned char *dst, const unsigned char *piece,
                                           const unsigned char *base, const unsigned char *end,
                                           int elem) {
    const long long left = end - piece;
    if (left <= 0) return;
    if (piece >= base && (left >= 16 || left % 4 == 0)) {
        cp_async16(reinterpret_cast<float *>(dst), reinterpret_cast<const float *>(piece),
                   left >= 16 ? 16 : (uint32_t)left);
    } else {
#pragma unroll 1
        for (int e = 0; e < 16 && e < left; e += elem) {
            if (piece + e < base) continue;
            if (elem == 1)
                dst[e] = piece[e];
            else if (elem == 2)
                *reinterpret_cast<uint16_t *>(dst + e) = *reinterpret_cast<const uint16_t *>(piece + e);
            else
                *reinterpret_cast<uint32_t *>(dst + e) = *reinterpret_cast<const uint32_t *>(piece + e);
        }
    }
}
__device__ __forceinline__ const unsigned char *piece_of(const unsigned char *p) {
    return reinterpret_cast<const unsigned char *>(reinterpret_cast<uintptr_t>(p) & ~uintptr_t(15));
}
// Where element n0 of the row starts in its first piece.
__device__ __forceinline__ int piece_shift(const void *base, long long elements, int elem) {
    return (int)((reinterpret_cast<uintptr_t>(base) + (unsigned long long)(elements * elem)) & 15);
}

template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// (w & mask) | magic in one instruction (left to itself the compiler makes two
// of it, as an instruction has room for one constant).
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t magic) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(magic));
    return r;
}

// How the lanes expand a word into pairs of 16-bit floats, and what is left to
// do for the zero points.
//   kPlainInt (fp16 x): the bits of two values, masked, are fp16 numbers as
//     they stand: subnormals, q 2^-24 for the low nibble of a byte and q 2^-20
//     for the high one, both exact.  The two kinds keep sums of their own;
//     z times the sum of x comes off at the end of a group.
//   kOffset (bf16 x): bf16 has no such room below, so q enters as 128 + q, and
//     128 + z times the sum of x comes off at the end.
//   kExact (FP32 x): as kOffset, but 128 + z comes off every value.
// Putting a few bits under a constant exponent by one logic instruction is a published
// method: Kim, Henry, Fahim and Awadalla, "Who Says Elephants Can't Run: Bringing Large
// Scale MoE Models into Cloud Scale Production", 2022.
enum : int { kPlainInt, kOffset, kExact };

// The pairs (0,4), (1,5), (2,6), (3,7) of a word.  magic: 128 twice in bf16;
// zero: 128 + z twice (kExact).
template <int FORM>
__device__ __forceinline__ void expand(uint32_t w, uint32_t magic, uint32_t zero, uint32_t (&p)[4]) {
    if constexpr (FORM == kPlainInt) {
        const uint32_t s = w >> 8;
        p[0] = w & 0x000F000Fu;
        p[1] = w & 0x00F000F0u;
        p[2] = s & 0x000F000Fu;
        p[3] = s & 0x00F000F0u;
    } else {
        const __nv_bfloat162 z = *reinterpret_cast<const __nv_bfloat162 *>(&zero);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = and_or(w >> (4 * i), 0x000F000Fu, magic);
            const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), z);
            p[i] = FORM == kOffset ? v : *reinterpret_cast<const uint32_t *>(&d);
        }
    }
}

// CTAs of one SM that the registers leave room for.
constexpr int ctas_per_sm(int type, int nt, int gs) {
    return nt == 1 && gs > 1 ? 4 : nt <= 2 && gs > 1 ? 3 : 2;
}

// TYPE: of x, scales and y.  NT: instructions' worth (8) of x rows.  GS: steps
// of 32 k that share a scale inside a unit.  VEC: rows of q, scales and zeros
// start on 16 bytes and N is a multiple of 16.
template <int TYPE, int NT, int GS, bool VEC>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(TYPE, NT, GS))
    w4_kernel(const __grid_constant__ CUtensorMap map, const W4Params p) {
    constexpr bool BF16 = TYPE != kTypeF16;
    constexpr int FORM = TYPE == kTypeF16 ? kPlainInt : TYPE == kTypeBF16 ? kOffset : kExact;
    constexpr int SUMS = FORM == kPlainInt ? 2 : 1;  // per accumulator
    constexpr int T16 = TYPE == kTypeF16 ? kTypeF16 : kTypeBF16;
    constexpr int P = TYPE == kTypeF32 ? 3 : 1;
    constexpr int NG = kSteps / GS;  // scales of a unit
    using L = UnitLayout<TYPE, NG>;
    extern __shared__ unsigned char w4_smem_raw[];
    __shared__ uint64_t full[kW4Warps][kW4Stages];  // TMA boxes of a warp's stages
    const uint32_t raw = smem_addr(w4_smem_raw);
    unsigned char *smem = w4_smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    unsigned char *xs = smem + kW4Warps * kW4Stages * L::kBytes;
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();

    const int tid = threadIdx.x, lane = tid % 32;
    const int warp = __shfl_sync(0xffffffffu, tid / 32, 0);
    const int warps_k = kW4Warps / p.warps_n;
    const int cols = kW4Cols * p.warps_n;             // of this CTA
    const int c0 = (int)(blockIdx.x / ranks) * cols;  // its first
    const int k_words = (p.K + 7) / 8;
    const int u0 = rank * p.cta_units, u1 = min(p.units, u0 + p.cta_units);
    const int rows = P * p.M;

    if (VEC && lane == 0) {
        for (int i = 0; i < kW4Stages; ++i) mbar_init(&full[warp][i], 1);
        fence_barrier_init();
    }
    __syncwarp();

    const int g = lane / 4, t = lane % 4;
    const int wn = warp % p.warps_n, wk = warp / p.warps_n;
    const int n0 = c0 + wn * kW4Cols;  // this warp's first column
    const int pitch = p.chunk_units * kW4UnitK * 2 + 64;  // 64 bytes apart modulo 128
    unsigned char *ring = smem + warp * (kW4Stages * L::kBytes);
    // The lane's columns: VEC, two runs of four, else every eighth.
    const int run = 4 * ((g >> 1) + 4 * (g & 1));

    auto group_of = [&](int k) { return p.group_shift >= 0 ? k >> p.group_shift : k / p.group; };

    // Asks for the warp's unit `u` (nothing when there is none).
    auto fetch = [&](int u, int stage) {
        if (u < u1 && n0 < p.N) {
            unsigned char *to = ring + stage * L::kBytes;
            if constexpr (VEC) {
                // Lane i brings group i's scales and zero points, lane 0 q.
                const int groups = min(NG, (p.K - u * kW4UnitK + GS * 32 - 1) / (GS * 32));
                const int cols_here = min(kW4Cols, p.N - n0);
                const int zero_bytes = p.zeros ? cols_here : 0;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[warp][stage],
                                          2 * kBoxBytes + groups * (cols_here * L::kElem + zero_bytes));
                    tma_load_2d(to, &map, &full[warp][stage], n0, u * kRows);
                    tma_load_2d(to + kBoxBytes, &map, &full[warp][stage], n0 + 32, u * kRows);
                }
                if (lane < groups) {
                    const int group = group_of(u * kW4UnitK + lane * GS * 32);
                    bulk_load(to + L::kScale + lane * (L::kScalePieces * 16),
                              static_cast<const unsigned char *>(p.scales) +
                                  (group * p.lds + n0) * L::kElem,
                              cols_here * L::kElem, &full[warp][stage]);
                    if (zero_bytes)
                        bulk_load(to + L::kZero + lane * (L::kZeroPieces * 16),
                                  p.zeros + group * p.ldz + n0, zero_bytes, &full[warp][stage]);
                }
            } else {
                // Two lanes to a row; 17 pieces cover 64 words wherever they
                // start.
                const int r = lane / 2, row = u * kRows + r;
                const uint32_t *q = p.q + row * p.ldq;
                const unsigned char *piece =
                    piece_of(reinterpret_cast<const unsigned char *>(q + n0)) + (lane % 2) * 16;
                unsigned char *dst = to + r * kPlainPitch + (lane % 2) * 16;
                if (u * kRows >= p.safe_rows && (u + 1) * kRows <= k_words - p.safe_rows) {
                    // All pieces lie inside the matrix.
#pragma unroll
                    for (int c = 0; c < 9; ++c)
                        if (c < 8 || lane % 2 == 0)
                            cp_async16(reinterpret_cast<float *>(dst + c * 32),
                                       reinterpret_cast<const float *>(piece + c * 32), 16);
                } else if (row < k_words) {
                    const unsigned char *base = reinterpret_cast<const unsigned char *>(p.q);
                    const unsigned char *end = reinterpret_cast<const unsigned char *>(q + p.N);
#pragma unroll 1
                    for (int c = 0; c < 9; ++c)
                        if (c < 8 || lane % 2 == 0)
                            copy_piece(dst + c * 32, piece + c * 32, base, end, 4);
                }
                constexpr int kScaleJobs = NG * L::kScalePieces, kZeroJobs = NG * L::kZeroPieces;
#pragma unroll 1
                for (int j = lane; j < kScaleJobs + (p.zeros ? kZeroJobs : 0); j += 32) {
                    const bool zero = j >= kScaleJobs;
                    const int jj = zero ? j - kScaleJobs : j;
                    const int per = zero ? L::kZeroPieces : L::kScalePieces;
                    const int i = jj / per, c = jj - i * per, k = u * kW4UnitK + i * GS * 32;
                    if (k < p.K) {
                        const unsigned char *base =
                            static_cast<const unsigned char *>(zero ? p.zeros : p.scales);
                        const int elem = zero ? 1 : L::kElem;
                        const unsigned char *row = base + group_of(k) * (zero ? p.ldz : p.lds) * elem;
                        copy_piece(to + (zero ? L::kZero : L::kScale) + jj * 16,
                                   piece_of(row + (long long)n0 * elem) + c * 16, base,
                                   row + (long long)p.N * elem, elem);
                    }
                }
            }
        }
        if constexpr (!VEC) cp_async_commit();
    };
    // Scale and zero point of the lane's columns of group i of unit u; what
    // was not loaded (columns beyond N, groups beyond K) is not used or
    // meets sums of zeros.
    auto scales_of = [&](const unsigned char *w, int u, int i, float (&sc)[8], uint32_t (&z)[2]) {
        const int k = u * kW4UnitK + i * GS * 32;
        const bool there = k < p.K;
        const unsigned char *s = w + L::kScale + i * L::kScalePieces * 16;
        const unsigned char *zs = w + L::kZero + i * L::kZeroPieces * 16;
        z[0] = z[1] = 0x08080808u;
        if constexpr (VEC) {
            s += run * L::kElem;
            zs += run;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (TYPE == kTypeF32) {
                    const float4 f = *reinterpret_cast<const float4 *>(s + 128 * h);
                    sc[4 * h] = f.x; sc[4 * h + 1] = f.y; sc[4 * h + 2] = f.z; sc[4 * h + 3] = f.w;
                } else {
                    const uint2 f = *reinterpret_cast<const uint2 *>(s + 64 * h);
                    const float2 a = unpack16<T16>(f.x), b = unpack16<T16>(f.y);
                    sc[4 * h] = a.x; sc[4 * h + 1] = a.y; sc[4 * h + 2] = b.x; sc[4 * h + 3] = b.y;
                }
                if (p.zeros) z[h] = *reinterpret_cast<const uint32_t *>(zs + 32 * h);
            }
        } else {
            const int group = group_of(k);
            s += piece_shift(p.scales, group * p.lds + n0, L::kElem) + g * L::kElem;
            if (p.zeros) {
                zs += piece_shift(p.zeros, group * p.ldz + n0, 1) + g;
                z[0] = z[1] = 0;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                sc[j] = load_as_float(s, TYPE, 8 * j);
                if (p.zeros) z[j / 4] |= (uint32_t)zs[8 * j] << (8 * (j % 4));
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (!there) sc[j] = 0.0f;
    };
    // x of units [a, b) into shared memory, one row of 16-bit values per row
    // of the x operand.  16-bit rows that start on 16 bytes are copied as they
    // are, without a register in between.
    const bool x_async = TYPE != kTypeF32 && p.x_vec;
    auto stage_x = [&](int a, int b) {
        const int octets = (b - a) * kRows, k0 = a * kW4UnitK;
        for (int o = tid; o < octets; o += kThreads) {
            const int left = p.K - k0 - o * 8;
            const long long at = k0 + o * 8;
            unsigned char *to = xs + o * 16;
            if constexpr (TYPE != kTypeF32) {
                const uint16_t *x = static_cast<const uint16_t *>(p.x) + at;
                if (x_async) {
                    const int n = min(max(left, 0), 8);
                    for (int m = 0; m < p.M; ++m, x += p.ldx, to += pitch)
                        cp_async16(reinterpret_cast<float *>(to),
                                   reinterpret_cast<const float *>(n ? x : p.x), n * 2);
                } else {
#pragma unroll 2
                    for (int m = 0; m < p.M; ++m) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = (2 * j < left ? __ldg(x + m * p.ldx + 2 * j) : 0u) |
                                   (2 * j + 1 < left ? (uint32_t)__ldg(x + m * p.ldx + 2 * j + 1) : 0u) << 16;
                        *reinterpret_cast<uint4 *>(to + m * pitch) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            } else {
                const float *x = static_cast<const float *>(p.x) + at;
#pragma unroll 2
                for (int m = 0; m < p.M; ++m) {
                    float v[8];
                    if (p.x_vec && left >= 8) {
                        const float4 c = __ldg(reinterpret_cast<const float4 *>(x + m * p.ldx));
                        const float4 d = __ldg(reinterpret_cast<const float4 *>(x + m * p.ldx) + 1);
                        v[0] = c.x; v[1] = c.y; v[2] = c.z; v[3] = c.w;
                        v[4] = d.x; v[5] = d.y; v[6] = d.z; v[7] = d.w;
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = j < left ? __ldg(x + m * p.ldx + j) : 0.0f;
                    }
                    float part[8][3];
#pragma unroll
                    for (int j = 0; j < 8; ++j) split3(v[j], part[j]);
#pragma unroll
                    for (int q = 0; q < 3; ++q)
                        *reinterpret_cast<uint4 *>(to + (q * p.M + m) * pitch) =
                            make_uint4(pack16<T16>(part[0][q], part[1][q]),
                                       pack16<T16>(part[2][q], part[3][q]),
                                       pack16<T16>(part[4][q], part[5][q]),
                                       pack16<T16>(part[6][q], part[7][q]));
                }
            }
        }
    };

    // Where the lane reads: q of a step with even and odd number (the TMA's
    // swizzle), and its row of x.
    const int read_even = t * 128 + ((run << 2) ^ (t << 4));
    const int read_odd = t * 128 + ((run << 2) ^ ((t + 4) << 4));
    int x_row[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) x_row[j] = min(8 * j + g, rows - 1) * pitch;

    float total[NT][4][4];
    // Kept in a register: see and_or.
    uint32_t magic;
    asm volatile("mov.b32 %0, %1;" : "=r"(magic) : "n"(0x43004300u));
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) total[j][b][e] = 0.0f;

    bool ok = true;
    int stage = 0;
    uint32_t parity = 0;
    int u = u0 + wk;
    if (x_async) stage_x(u0, min(u1, u0 + p.chunk_units));
    cp_async_commit();
#pragma unroll 1
    for (int i = 0; i < kW4Stages; ++i) fetch(u + i * warps_k, i);
    for (int a = u0; a < u1; a += p.chunk_units) {
        const int b = min(u1, a + p.chunk_units);
        if (a > u0) {
            __syncthreads();
            stage_x(a, b);
            cp_async_commit();
            cp_async_wait<0>();
        } else {
            if (!x_async) stage_x(a, b);
            cp_async_wait<VEC ? 0 : kW4Stages>();  // x; the units' copies came after it
        }
        __syncthreads();
        for (; ok && u < b; u += warps_k) {
            if constexpr (VEC) {
                if (n0 < p.N) ok = tc_wait(&full[warp][stage], parity, p.timeout_ns);
            } else {
                cp_async_wait<kW4Stages - 1>();
            }
            __syncwarp();
            if (!ok) break;
            const unsigned char *w = ring + stage * L::kBytes;
            const unsigned char *xu = xs + (size_t)(u - a) * kW4UnitK * 2 + t * 16;
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
                float sum[SUMS][NT][4][4], ones[NT][4], sc[8];
                uint32_t z[2];
                scales_of(w, u, gi, sc, z);
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        ones[j][e] = 0.0f;
#pragma unroll
                        for (int b2 = 0; b2 < 4; ++b2)
#pragma unroll
                            for (int k = 0; k < SUMS; ++k) sum[k][j][b2][e] = 0.0f;
                    }
#pragma unroll
                for (int st = 0; st < GS; ++st) {
                    const int i = gi * GS + st, r = 4 * i + t;
                    uint32_t wi[8];
                    if constexpr (VEC) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(
                                w + h * kBoxBytes + i * 512 + (i % 2 ? read_odd : read_even));
                            wi[4 * h] = v.x; wi[4 * h + 1] = v.y;
                            wi[4 * h + 2] = v.z; wi[4 * h + 3] = v.w;
                        }
                    } else {
                        // Where the row's first word lies in its first piece.
                        const int shift = piece_shift(p.q, (u * kRows + r) * p.ldq + n0, 4) / 4;
                        const uint32_t *from =
                            reinterpret_cast<const uint32_t *>(w + r * kPlainPitch) + shift + g;
#pragma unroll
                        for (int j = 0; j < 8; ++j) wi[j] = from[8 * j];
                    }
                    // x04, x15, x26, x37.  Columns beyond the rows of x
                    // repeat the last one; nobody reads what they add up to.
                    uint32_t xv[NT][4];
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(xu + x_row[j] + i * 64);
                        xv[j][0] = __byte_perm(v.x, v.z, 0x5410);
                        xv[j][1] = __byte_perm(v.x, v.z, 0x7632);
                        xv[j][2] = __byte_perm(v.y, v.w, 0x5410);
                        xv[j][3] = __byte_perm(v.y, v.w, 0x7632);
                        if constexpr (FORM != kExact) {
                            constexpr uint32_t kOne = BF16 ? 0x3F803F80u : 0x3C003C00u;
                            const uint32_t one[4] = {kOne, kOne, kOne, kOne};
                            mma<BF16>(ones[j], one, xv[j][0], xv[j][1]);
                            mma<BF16>(ones[j], one, xv[j][2], xv[j][3]);
                        }
                    }
#pragma unroll
                    for (int blk = 0; blk < 4; ++blk) {
                        uint32_t e0[4], e1[4], zero[2] = {};
                        if constexpr (FORM == kExact) {
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                zero[c] = 0x43004300u |
                                          ((z[blk / 2] >> (8 * (2 * (blk % 2) + c))) & 15u) * 0x00010001u;
                        }
                        expand<FORM>(wi[2 * blk], magic, zero[0], e0);
                        expand<FORM>(wi[2 * blk + 1], magic, zero[1], e1);
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            if constexpr (FORM == kPlainInt) {
                                // Low nibbles' pairs together, high nibbles' together.
                                const uint32_t lo[4] = {e0[0], e1[0], e0[2], e1[2]};
                                const uint32_t hi[4] = {e0[1], e1[1], e0[3], e1[3]};
                                mma<BF16>(sum[0][j][blk], lo, xv[j][0], xv[j][2]);
                                mma<BF16>(sum[SUMS - 1][j][blk], hi, xv[j][1], xv[j][3]);
                            } else {
                                const uint32_t a0[4] = {e0[0], e1[0], e0[1], e1[1]};
                                const uint32_t a1[4] = {e0[2], e1[2], e0[3], e1[3]};
                                mma<BF16>(sum[0][j][blk], a0, xv[j][0], xv[j][1]);
                                mma<BF16>(sum[0][j][blk], a1, xv[j][2], xv[j][3]);
                            }
                        }
                    }
                }
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    // z, or 128 + z: the byte dropped into the mantissa of 2^23.
                    const float off =
                        __uint_as_float(0x4B000000u | ((z[c / 4] >> (8 * (c % 4))) & 15u)) -
                        (FORM == kOffset ? 8388480.0f : 8388608.0f);
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int at = 2 * (c % 2) + e;
                            float v = sum[0][j][c / 2][at];
                            if constexpr (FORM == kPlainInt)
                                v = fmaf(16777216.0f, v, 1048576.0f * sum[SUMS - 1][j][c / 2][at]);
                            if constexpr (FORM != kExact) v = fmaf(-off, ones[j][e], v);
                            total[j][c / 2][at] = fmaf(sc[c], v, total[j][c / 2][at]);
                        }
                }
            }
            __syncwarp();
            fetch(u + kW4Stages * warps_k, stage);
            if (++stage == kW4Stages) {
                stage = 0;
                parity ^= 1;
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!ok && lane == 0) atomicOr(p.err, kErrWaitTimeout);
    if (__syncthreads_or(!ok)) {
        // Copies may still be under way: let them land before the staging
        // memory is used again.
        const long long start = clock64();
        while (clock64() - start < 4000000) {
        }
        __syncthreads();
    }

    // The warps' sums, then the cluster's, in order.
    float *red = reinterpret_cast<float *>(smem);  // [warp along K][row of x][column]
    {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int c = 8 * j + 2 * t + e;
                if (c < rows) {
                    float *to = red + (wk * rows + c) * cols + wn * kW4Cols;
#pragma unroll
                    for (int w = 0; w < 8; ++w)
                        to[VEC ? (w / 4) * 32 + run + w % 4 : 8 * w + g] = total[j][w / 2][2 * (w % 2) + e];
                }
            }
    }
    __syncthreads();
    float *mine = red + warps_k * rows * cols;  // [row of x][column], this CTA's sums
    const int outs = p.M * cols, shift = 31 - __clz(cols);
    for (int i = tid; i < outs; i += kThreads) {
        float v = 0.0f;
#pragma unroll 1
        for (int q = 0; q < P; ++q)
            for (int k = 0; k < warps_k; ++k) v += red[k * rows * cols + q * outs + i];
        if (ranks == 1) {
            const int n = c0 + (i & (cols - 1));
            if (n < p.N) store_from_float(p.y, TYPE, (long long)(i >> shift) * p.ldy + n, v);
        } else {
            mine[i] = v;
        }
    }
    if (ranks == 1) return;
    cluster.sync();
    for (int i = rank * kThreads + tid; i < outs; i += ranks * kThreads) {
        float v = 0.0f;
        for (int r = 0; r < ranks; ++r) v += cluster.map_shared_rank(mine, r)[i];
        const int n = c0 + (i & (cols - 1));
        if (n < p.N) store_from_float(p.y, TYPE, (long long)(i >> shift) * p.ldy + n, v);
    }
    cluster.sync();  // no CTA leaves while another reads its sums
}

template <int TYPE, int NT, int GS, bool VEC>
cudaError_t launch_one(const CUtensorMap &map, const W4Params &p, int cluster, cudaStream_t stream) {
    constexpr int P = TYPE == kTypeF32 ? 3 : 1;
    const int rows = P * p.M, cols = kW4Cols * p.warps_n;
    const size_t ring = kW4Warps * kW4Stages * UnitLayout<TYPE, kSteps / GS>::kBytes;
    const size_t x = (size_t)rows * (p.chunk_units * kW4UnitK * 2 + 64);
    const size_t reduce = (size_t)(kW4Warps / p.warps_n * rows + p.M) * cols * sizeof(float);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.N + cols - 1) / cols) * cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = std::max(ring + x, reduce) + 1024;
    cfg.stream = stream;
    static std::atomic<size_t> limit[kMaxDevices];  // set up so far, per device
    if (p.device >= kMaxDevices) return cudaErrorInvalidDevice;
    if (limit[p.device].load() < cfg.dynamicSmemBytes) {
        const size_t most = ring + kW4StageBytes + 8192 + 1024;
        const size_t want = std::max(cfg.dynamicSmemBytes, std::max(most, reduce + 1024));
        cudaError_t e = cudaFuncSetAttribute(w4_kernel<TYPE, NT, GS, VEC>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)want);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(w4_kernel<TYPE, NT, GS, VEC>,
                                     cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        if (e != cudaSuccess) return e;
        limit[p.device].store(want);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, w4_kernel<TYPE, NT, GS, VEC>, map, p);
}

template <int TYPE, int NT>
cudaError_t launch_nt(const CUtensorMap &map, const W4Params &p, bool vec, int cluster,
                      cudaStream_t stream) {
    if (p.group % 128 == 0)
        return vec ? launch_one<TYPE, NT, 4, true>(map, p, cluster, stream)
                   : launch_one<TYPE, NT, 4, false>(map, p, cluster, stream);
    if (p.group % 64 == 0)
        return vec ? launch_one<TYPE, NT, 2, true>(map, p, cluster, stream)
                   : launch_one<TYPE, NT, 2, false>(map, p, cluster, stream);
    return vec ? launch_one<TYPE, NT, 1, true>(map, p, cluster, stream)
               : launch_one<TYPE, NT, 1, false>(map, p, cluster, stream);
}

// ---------------------------------------------------------------------------
// Quantisation: one thread per column of a group, so a warp reads and writes
// along rows.  W is read twice, the second time from L2 where a group's rows fit
// there.  4096 x 12288 in groups of 128: 106 us from BF16 (its bytes once: 19), 143 us
// from FP32 (34); bound by a thread's chain of loads, one group of a column after the
// other.  It runs once per matrix.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) w4_quantize_kernel(const W4QuantParams p) {
    const int col_blocks = (p.N + 255) / 256;
    const int n = (int)(blockIdx.x % col_blocks) * 256 + threadIdx.x;
    if (n >= p.N) return;
    const int gi = blockIdx.x / col_blocks;
    const long long k0 = (long long)gi * p.group;
    const int count = (int)min((long long)p.group, p.K - k0);
    float lo = 0.0f, hi = 0.0f;
    // Four bits have no infinity or NaN (which a minimum passes over): the scale says it.
    bool finite = true;
    for (int k = 0; k < count; ++k) {
        const float w = load_as_float(p.W, p.type, (k0 + k) * p.ldw + n);
        lo = fminf(lo, w);
        hi = fmaxf(hi, w);
        finite = finite && fabsf(w) < INFINITY;
    }
    const float span = !finite  ? __int_as_float(0x7FC00000)
                       : p.zeros ? (hi - lo) / 15.0f
                                 : fmaxf(hi, -lo) / 7.0f;
    store_from_float(p.scales, p.type, (long long)gi * p.lds + n, span);
    const float scale = load_as_float(p.scales, p.type, (long long)gi * p.lds + n);
    const float zero = !p.zeros ? 8.0f
                       : scale > 0.0f ? fminf(fmaxf(rintf(-lo / scale), 0.0f), 15.0f) : 0.0f;
    if (p.zeros) p.zeros[(long long)gi * p.ldz + n] = (uint8_t)zero;
    for (int r = 0; r < count; r += 8) {
        uint32_t word = 0;
        for (int j = 0; j < 8; ++j) {
            float q = zero;
            if (r + j < count && scale > 0.0f) {
                const float w = load_as_float(p.W, p.type, (k0 + r + j) * p.ldw + n);
                q = fminf(fmaxf(rintf(w / scale) + zero, 0.0f), 15.0f);
            }
            word |= (uint32_t)q << (4 * j);
        }
        p.q[((k0 + r) / 8) * p.ldq + n] = word;
    }
}

}  // namespace

int w4_max_rows(int type) { return type == kTypeF32 ? 8 : 16; }

int w4_unit_bytes(int type, int M) { return (type == kTypeF32 ? 3 : 1) * M * kW4UnitK * 2; }

int w4_ctas_per_sm(int type, int M, int group, int units) {
    const int parts = type == kTypeF32 ? 3 : 1, nt = (parts * M + 7) / 8;
    const int gs = group % 128 == 0 ? 4 : group % 64 == 0 ? 2 : 1;
    auto ring = [&](auto type_of) {
        constexpr int t = decltype(type_of)::value;
        return gs == 4   ? UnitLayout<t, kSteps / 4>::kBytes
               : gs == 2 ? UnitLayout<t, kSteps / 2>::kBytes
                         : UnitLayout<t, kSteps>::kBytes;
    };
    const int stage = type == kTypeF32 ? ring(std::integral_constant<int, kTypeF32>())
                                       : ring(std::integral_constant<int, kTypeF16>());
    const int bytes = kW4Warps * kW4Stages * stage + parts * M * (units * kW4UnitK * 2 + 64) + 1024;
    // An SM's 228 KB, of which each CTA takes one for itself.
    return std::max(1, std::min(ctas_per_sm(type, nt, gs), 228 * 1024 / (bytes + 1024)));
}

cudaError_t launch_w4(const CUtensorMap &map, const W4Params &p, int type, bool vec, int cluster,
                      cudaStream_t stream) {
    if (type == kTypeF32) {
        if (3 * p.M <= 8) return launch_nt<kTypeF32, 1>(map, p, vec, cluster, stream);
        if (3 * p.M <= 16) return launch_nt<kTypeF32, 2>(map, p, vec, cluster, stream);
        return launch_nt<kTypeF32, 3>(map, p, vec, cluster, stream);
    }
    if (type == kTypeF16)
        return p.M <= 8 ? launch_nt<kTypeF16, 1>(map, p, vec, cluster, stream)
                        : launch_nt<kTypeF16, 2>(map, p, vec, cluster, stream);
    return p.M <= 8 ? launch_nt<kTypeBF16, 1>(map, p, vec, cluster, stream)
                    : launch_nt<kTypeBF16, 2>(map, p, vec, cluster, stream);
}

cudaError_t launch_w4_quantize(const W4QuantParams &p, cudaStream_t stream) {
    const long long blocks =
        (long long)((p.N + 255) / 256) * ((p.K + (long long)p.group - 1) / p.group);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    w4_quantize_kernel<<<(unsigned)blocks, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace sgemm
