// Products of a few rows with 4-bit weights, and their quantisation.
//
//   y[m][n] = sum over groups G of  s[G][n] * sum over k in G of x[m][k] (q[k][n] - z[G][n])
//
// Bound: HBM, K N / 2 bytes of q read once.  At the card's rate that is 13.6
// weights per ns, about 2.4 instructions a lane for each, so the products go
// to the warp-level matrix instruction and the lanes only expand the weights:
// a word's eight values become four pairs of 16-bit floats with one shift,
// four (and, or) instructions that drop the value into the mantissa of 1024
// (or 128 for bf16) and four exact subtractions of zero point and offset,
// about 1.2 instructions per weight.  The fifth-generation tensor cores would
// need the expanded weights in shared memory and gain nothing at 16 columns.
//
// Layout.  The instruction (m16n8k16) takes the weights as its 16 x 16
// operand, rows along n, and x as its 16 x 8 one, so up to eight rows of x
// cost one instruction.  The order of k inside an instruction is free, so the
// pairs come as a word gives them: (0,4), (1,5) in one instruction and (2,6),
// (3,7) in the next; x is staged in shared memory in that order.  Lane (g, t)
// = (lane / 4, lane % 4) of a warp reads four columns' words of word row t of
// four: a warp reads 4 rows x 128 contiguous bytes for 32 columns x 32 k.
//
// Exactness.  q - z has at most five bits; 16-bit x enters as it is.  FP32 x
// is the sum of three bf16 parts, each a row of its own of the x operand.
// Sums are FP32; each group's sum is scaled in FP32.
//
// Split.  A CTA owns 32 columns and a range of K; its eight warps take every
// eighth unit of 128 k and add up through shared memory in warp order.  Where
// N alone gives too few CTAs, a cluster shares K and adds its CTAs' sums in
// rank order through distributed shared memory: no atomics, no workspace.
#include <cooperative_groups.h>

#include <algorithm>

#include "ops_common.cuh"

namespace cg = cooperative_groups;

namespace sgemm {
namespace {

constexpr int kThreads = kW4Warps * 32;
constexpr int kSteps = kW4UnitK / 32;

__device__ __forceinline__ uint4 ld_stream(const uint32_t *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
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

// The four pairs (0,4), (1,5), (2,6), (3,7) of a word, minus the zero point.
// z0 holds offset + z twice: 1024 + z in fp16, 128 + z in bf16.  z1 (fp16
// only) holds -(64 + z) twice, for the pairs that sit four bits higher.
template <bool BF16>
__device__ __forceinline__ void expand(uint32_t w, uint32_t z0, uint32_t z1, uint32_t (&p)[4]) {
    if constexpr (BF16) {
        const __nv_bfloat162 z = *reinterpret_cast<const __nv_bfloat162 *>(&z0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
            const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), z);
            p[i] = *reinterpret_cast<const uint32_t *>(&d);
        }
    } else {
        const __half2 z = *reinterpret_cast<const __half2 *>(&z0);
        const __half2 zh = *reinterpret_cast<const __half2 *>(&z1);
        const uint32_t sixteenth = 0x2C002C00u;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t s = w >> (8 * i);
            const uint32_t lo = (s & 0x000F000Fu) | 0x64006400u;
            const uint32_t hi = (s & 0x00F000F0u) | 0x64006400u;
            const __half2 a = __hsub2(*reinterpret_cast<const __half2 *>(&lo), z);
            const __half2 b = __hfma2(*reinterpret_cast<const __half2 *>(&hi),
                                      *reinterpret_cast<const __half2 *>(&sixteenth), zh);
            p[2 * i] = *reinterpret_cast<const uint32_t *>(&a);
            p[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&b);
        }
    }
}

// TYPE: of x, scales and y.  NT: instructions' worth (8) of x rows.  GS: steps
// of 32 k that share a scale inside a unit.  VEC: four columns are read at once.
template <int TYPE, int NT, int GS, bool VEC>
__global__ void __launch_bounds__(kThreads, NT == 1 || (NT == 2 && TYPE != kTypeF32 && GS > 1) ? 2 : 1)
    w4_kernel(const W4Params p) {
    constexpr bool BF16 = TYPE != kTypeF16;
    constexpr int P = TYPE == kTypeF32 ? 3 : 1;
    constexpr int NG = kSteps / GS;  // scales of a unit
    extern __shared__ __align__(16) unsigned char smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
    const int n0 = (int)(blockIdx.x / ranks) * kW4Cols;
    const int rows = P * p.M;
    const int k_words = (p.K + 7) / 8;
    const int u0 = rank * p.cta_units, u1 = min(p.units, u0 + p.cta_units);
    const int chunk_k = p.chunk_units * kW4UnitK;
    const int pitch = chunk_k * 2 + 64;  // rows 64 bytes apart modulo 128: no bank conflicts

    // The lane's four columns, as offsets from n0.
    const int col0 = VEC ? 4 * g : g, col_step = VEC ? 1 : 8;
    bool col_ok[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) col_ok[j] = n0 + col0 + j * col_step < p.N;

    auto load_words = [&](int unit, uint32_t (&w)[kSteps][4]) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int r = unit * (kW4UnitK / 8) + 4 * i + t;
            const bool ok = unit < u1 && r < k_words;
            const uint32_t *q = p.q + (long long)r * p.ldq + n0 + col0;
            if constexpr (VEC) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (ok && col_ok[0]) v = ld_stream(q);
                w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) w[i][j] = ok && col_ok[j] ? __ldg(q + 8 * j) : 0u;
            }
        }
    };
    auto load_scales = [&](int unit, float (&s)[NG][4], uint32_t (&z)[NG]) {
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            const int k = unit * kW4UnitK + i * GS * 32;
            const bool ok = unit < u1 && k < p.K;
            const long long at = (long long)(k / p.group) * p.lds + n0 + col0;
            const long long zat = (long long)(k / p.group) * p.ldz + n0 + col0;
            z[i] = 0x08080808u;
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
            if constexpr (VEC) {
                if (ok && col_ok[0]) {
                    if constexpr (TYPE == kTypeF32) {
                        const float4 f =
                            __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p.scales) + at));
                        s[i][0] = f.x; s[i][1] = f.y; s[i][2] = f.z; s[i][3] = f.w;
                    } else {
                        const uint2 f = __ldg(reinterpret_cast<const uint2 *>(
                            static_cast<const uint16_t *>(p.scales) + at));
                        const float2 a = unpack16<TYPE>(f.x), b = unpack16<TYPE>(f.y);
                        s[i][0] = a.x; s[i][1] = a.y; s[i][2] = b.x; s[i][3] = b.y;
                    }
                    if (p.zeros) z[i] = __ldg(reinterpret_cast<const uint32_t *>(p.zeros + zat));
                }
            } else {
                if (p.zeros) z[i] = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (ok && col_ok[j]) {
                        s[i][j] = load_as_float(p.scales, TYPE, at + 8 * j);
                        if (p.zeros) z[i] |= (uint32_t)__ldg(p.zeros + zat + 8 * j) << (8 * j);
                    }
                }
            }
        }
    };

    float total[NT][2][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) total[j][b][e] = 0.0f;

    uint32_t w[kSteps][4];
    float s[NG][4];
    uint32_t z[NG];
    for (int c0 = u0; c0 < u1; c0 += p.chunk_units) {
        const int c1 = min(u1, c0 + p.chunk_units);
        // The first unit's weights are on their way while x is staged.
        load_words(min(c0 + warp, c1), w);
        load_scales(min(c0 + warp, c1), s, z);
        if (c0 > u0) __syncthreads();
        const int octets = (c1 - c0) * (kW4UnitK / 8);
        for (int i = tid; i < p.M * octets; i += kThreads) {
            const int m = i / octets, o = i % octets, k = c0 * kW4UnitK + o * 8;
            float x[8];
            const long long at = (long long)m * p.ldx + k;
            if (p.x_vec && k + 8 <= p.K) {
                if constexpr (TYPE == kTypeF32) {
                    const float4 *f = reinterpret_cast<const float4 *>(static_cast<const float *>(p.x) + at);
                    const float4 a = __ldg(f), b = __ldg(f + 1);
                    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
                    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
                } else {
                    const uint4 f = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.x) + at));
                    const float2 a = unpack16<TYPE>(f.x), b = unpack16<TYPE>(f.y);
                    const float2 c = unpack16<TYPE>(f.z), d = unpack16<TYPE>(f.w);
                    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
                    x[4] = c.x; x[5] = c.y; x[6] = d.x; x[7] = d.y;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    x[j] = k + j < p.K ? load_as_float(p.x, TYPE, at + j) : 0.0f;
            }
            unsigned char *to = smem + (size_t)m * pitch + o * 16;
            if constexpr (P == 1) {
                constexpr int T16 = TYPE == kTypeF16 ? kTypeF16 : kTypeBF16;
                *reinterpret_cast<uint4 *>(to) =
                    make_uint4(pack16<T16>(x[0], x[4]), pack16<T16>(x[1], x[5]),
                               pack16<T16>(x[2], x[6]), pack16<T16>(x[3], x[7]));
            } else {
                float part[8][3];
#pragma unroll
                for (int j = 0; j < 8; ++j) split3(x[j], part[j]);
#pragma unroll
                for (int q = 0; q < 3; ++q)
                    *reinterpret_cast<uint4 *>(to + (size_t)q * p.M * pitch) =
                        make_uint4(pack16<kTypeBF16>(part[0][q], part[4][q]),
                                   pack16<kTypeBF16>(part[1][q], part[5][q]),
                                   pack16<kTypeBF16>(part[2][q], part[6][q]),
                                   pack16<kTypeBF16>(part[3][q], part[7][q]));
            }
        }
        __syncthreads();

        for (int u = c0 + warp; u < c1; u += kW4Warps) {
            // The next unit's loads go out before this one is computed.
            uint32_t w2[kSteps][4];
            float s2[NG][4];
            uint32_t z2[NG];
            const int next = u + kW4Warps < c1 ? u + kW4Warps : u1;
            load_words(next, w2);
            load_scales(next, s2, z2);
            const unsigned char *xu = smem + (size_t)(u - c0) * kW4UnitK * 2 + t * 16;
#pragma unroll
            for (int gi = 0; gi < NG; ++gi) {
                float sum[NT][2][4];
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum[j][b][e] = 0.0f;
                uint32_t z0[4], z1[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t zj = (z[gi] >> (8 * j)) & 15u;
                    z0[j] = (BF16 ? 0x43004300u : 0x64006400u) | zj * 0x00010001u;
                    z1[j] = 0xD400D400u + zj * 0x00100010u;
                }
#pragma unroll
                for (int st = 0; st < GS; ++st) {
                    const int i = gi * GS + st;
                    uint32_t e[4][4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) expand<BF16>(w[i][j], z0[j], z1[j], e[j]);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        uint4 b = make_uint4(0, 0, 0, 0);
                        if (8 * j + g < rows)
                            b = *reinterpret_cast<const uint4 *>(xu + (size_t)(8 * j + g) * pitch +
                                                                 i * 64);
#pragma unroll
                        for (int blk = 0; blk < 2; ++blk) {
                            const uint32_t a0[4] = {e[2 * blk][0], e[2 * blk + 1][0],
                                                    e[2 * blk][1], e[2 * blk + 1][1]};
                            const uint32_t a1[4] = {e[2 * blk][2], e[2 * blk + 1][2],
                                                    e[2 * blk][3], e[2 * blk + 1][3]};
                            mma<BF16>(sum[j][blk], a0, b.x, b.y);
                            mma<BF16>(sum[j][blk], a1, b.z, b.w);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            total[j][b][e] = fmaf(s[gi][2 * b + e / 2], sum[j][b][e], total[j][b][e]);
            }
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) w[i][j] = w2[i][j];
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                z[i] = z2[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = s2[i][j];
            }
        }
    }

    // The warps' sums, then the cluster's, in order.
    __syncthreads();
    float *red = reinterpret_cast<float *>(smem);  // [warp][row of x][column]
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int c = 8 * j + 2 * t + e % 2;
                const int col = col0 + (2 * b + e / 2) * col_step;
                if (c < rows) red[(warp * rows + c) * kW4Cols + col] = total[j][b][e];
            }
    __syncthreads();
    float *mine = red + kW4Warps * rows * kW4Cols;  // [row of x][column], this CTA's sums
    const int outs = p.M * kW4Cols;
    for (int i = tid; i < outs; i += kThreads) {
        float v = 0.0f;
        for (int q = 0; q < P; ++q)
            for (int k = 0; k < kW4Warps; ++k) v += red[k * rows * kW4Cols + q * outs + i];
        if (ranks == 1) {
            const int n = n0 + i % kW4Cols;
            if (n < p.N) store_from_float(p.y, TYPE, (long long)(i / kW4Cols) * p.ldy + n, v);
        } else {
            mine[i] = v;
        }
    }
    if (ranks == 1) return;
    cluster.sync();
    for (int i = rank * kThreads + tid; i < outs; i += ranks * kThreads) {
        float v = 0.0f;
        for (int r = 0; r < ranks; ++r) v += cluster.map_shared_rank(mine, r)[i];
        const int n = n0 + i % kW4Cols;
        if (n < p.N) store_from_float(p.y, TYPE, (long long)(i / kW4Cols) * p.ldy + n, v);
    }
    cluster.sync();  // no CTA leaves while another reads its sums
}

template <int TYPE, int NT, int GS, bool VEC>
cudaError_t launch_one(const W4Params &p, int cluster, cudaStream_t stream) {
    constexpr int P = TYPE == kTypeF32 ? 3 : 1;
    const int rows = P * p.M;
    const size_t stage = (size_t)rows * (p.chunk_units * kW4UnitK * 2 + 64);
    const size_t reduce = (size_t)(kW4Warps * rows + p.M) * kW4Cols * sizeof(float);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.N + kW4Cols - 1) / kW4Cols) * cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = std::max(stage, reduce);
    cfg.stream = stream;
    if (cfg.dynamicSmemBytes > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(w4_kernel<TYPE, NT, GS, VEC>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kW4StageBytes + 16 * 1024);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, w4_kernel<TYPE, NT, GS, VEC>, p);
}

template <int TYPE, int NT>
cudaError_t launch_nt(const W4Params &p, bool vec, int cluster, cudaStream_t stream) {
    if (p.group % 128 == 0)
        return vec ? launch_one<TYPE, NT, 4, true>(p, cluster, stream)
                   : launch_one<TYPE, NT, 4, false>(p, cluster, stream);
    if (p.group % 64 == 0)
        return vec ? launch_one<TYPE, NT, 2, true>(p, cluster, stream)
                   : launch_one<TYPE, NT, 2, false>(p, cluster, stream);
    return vec ? launch_one<TYPE, NT, 1, true>(p, cluster, stream)
               : launch_one<TYPE, NT, 1, false>(p, cluster, stream);
}

// ---------------------------------------------------------------------------
// Quantisation: one thread per column of a group, so a warp reads and writes
// along rows.  Bound by HBM (W is read twice, the second time from L2 where a
// group's rows fit there); it runs once per matrix.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) w4_quantize_kernel(const W4QuantParams p) {
    const int col_blocks = (p.N + 255) / 256;
    const int n = (int)(blockIdx.x % col_blocks) * 256 + threadIdx.x;
    if (n >= p.N) return;
    const int gi = blockIdx.x / col_blocks;
    const long long k0 = (long long)gi * p.group;
    const int count = (int)min((long long)p.group, p.K - k0);
    float lo = 0.0f, hi = 0.0f;
    for (int k = 0; k < count; ++k) {
        const float w = load_as_float(p.W, p.type, (k0 + k) * p.ldw + n);
        lo = fminf(lo, w);
        hi = fmaxf(hi, w);
    }
    const float span = p.zeros ? (hi - lo) / 15.0f : fmaxf(hi, -lo) / 7.0f;
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

cudaError_t launch_w4(const W4Params &p, int type, bool vec, int cluster, cudaStream_t stream) {
    if (type == kTypeF32) {
        if (3 * p.M <= 8) return launch_nt<kTypeF32, 1>(p, vec, cluster, stream);
        if (3 * p.M <= 16) return launch_nt<kTypeF32, 2>(p, vec, cluster, stream);
        return launch_nt<kTypeF32, 3>(p, vec, cluster, stream);
    }
    if (type == kTypeF16)
        return p.M <= 8 ? launch_nt<kTypeF16, 1>(p, vec, cluster, stream)
                        : launch_nt<kTypeF16, 2>(p, vec, cluster, stream);
    return p.M <= 8 ? launch_nt<kTypeBF16, 1>(p, vec, cluster, stream)
                    : launch_nt<kTypeBF16, 2>(p, vec, cluster, stream);
}

cudaError_t launch_w4_quantize(const W4QuantParams &p, cudaStream_t stream) {
    const long long blocks =
        (long long)((p.N + 255) / 256) * ((p.K + (long long)p.group - 1) / p.group);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    w4_quantize_kernel<<<(unsigned)blocks, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace sgemm
