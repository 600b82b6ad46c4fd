// One AdamW step over many tensors in one launch, with 32-bit or 8-bit states.
//
//   m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g^2
//   p <- p (1 - lr wd) - lr / bc1 * m / (sqrt(v) / sqrt(bc2) + eps)
//
// Bound: HBM.  Per element p is read and written, g read, m and v read and
// written (28 bytes with everything in FP32; 14 with a bf16 gradient and 8-bit
// states).  So each element is touched once; a warp keeps three or four blocks' loads
// under way by asynchronous copies (with loads into registers the warps that fit
// had too little under way: 447 us at 134 M elements with 8-bit states); and
// all tensors share a launch: a CTA takes one chunk of
// up to kAdamChunk elements and finds its tensor by bisection over the tensors'
// first chunks, which travel with the pointers in the kernel's parameters
// (no table to upload, nothing kept on the device between steps).
//
// Measured, 134 M elements of FP32 with bf16 gradients: 8-bit states 338-342 us (5.6 TB/s,
// 82 % of a copy's rate), with 16-bit copies 379 us (84 %); 32-bit states 617 us (83 %),
// with copies 662 us (84 %).  bf16 parameters: 270 us (74 %) and 612 us (71 %).  300
// tensors of 3 M elements together with 32-bit states 18-20.6 us (60 %): chunks of 2048
// give a warp one block, so its ring is never filled but still limits an SM to two CTAs,
// and some 1600 CTAs go through five waves, each with its own bisection first.
//
// 8-bit states: a warp owns a block of 256 elements, eight per lane, so that
// the block's largest |m| and sqrt(v) are one warp reduction each.  The
// reduction compares the values' bit patterns as integers, which orders
// non-negative floats and puts NaN above everything, so a NaN reaches the
// scale.  Every operation that decides a code is a single correctly rounded
// FP32 one (no contraction, units as scale * (1/448) and (1/scale) * 448), so
// the codes are reproducible from the formula.
#include <atomic>

#include "ops_common.cuh"

namespace sgemm {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxDevices = 64;
// Blocks a warp has under way.
constexpr int stages_of(int bits) { return bits == 8 ? 4 : 3; }

extern __shared__ __align__(16) unsigned char adam_smem[];
constexpr float kTiny = 1.2621774483536189e-29f;  // 2^-96: the least scale
constexpr float kLeast = 0.001953125f;            // 2^-9: the least e4m3 value above zero

struct AdamTable {
    int count;
    AdamTensor t[kAdamTensors];
};

// A lane's eight elements of a block of 256 as loaded: eight consecutive ones
// in wide loads where the whole block exists and the array allows it, else
// every 32nd, element by element.
template <int BYTES>  // of an element: 4, 2 or 1
struct Raw {
    static constexpr int kWords = 2 * BYTES;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const void *p, unsigned block, int lane, int left) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j * 32 + lane >= left) continue;
            const unsigned at = block + j * 32 + lane;
            if constexpr (BYTES == 4) w[j] = __ldcs(static_cast<const uint32_t *>(p) + at);
            else if constexpr (BYTES == 2)
                w[j / 2] |= (uint32_t)__ldcs(static_cast<const uint16_t *>(p) + at) << (16 * (j % 2));
            else
                w[j / 4] |= (uint32_t)__ldcs(static_cast<const uint8_t *>(p) + at) << (8 * (j % 4));
        }
    }

    // The wide loads in two halves: an asynchronous copy to this lane's place in
    // shared memory, and the read from there.
    static __device__ __forceinline__ void fetch(unsigned char *to, const void *p, unsigned block,
                                                 int lane) {
        const unsigned char *q = static_cast<const unsigned char *>(p) + (block + 8u * lane) * BYTES;
        const uint32_t s = (uint32_t)__cvta_generic_to_shared(to);
        if constexpr (BYTES == 1) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(s + lane * 8), "l"(q) : "memory");
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s + i * 512 + lane * 16),
                             "l"(q + i * 16)
                             : "memory");
        }
    }
    __device__ __forceinline__ void take(const unsigned char *from, int lane) {
        if constexpr (BYTES == 1) {
            const uint2 a = *reinterpret_cast<const uint2 *>(from + lane * 8);
            w[0] = a.x; w[1] = a.y;
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 a = *reinterpret_cast<const uint4 *>(from + i * 512 + lane * 16);
                w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
            }
        }
    }

    __device__ __forceinline__ void store(void *p, unsigned block, int lane, int left, bool vec) const {
        if (vec) {
            unsigned char *q = static_cast<unsigned char *>(p) + (block + 8u * lane) * BYTES;
            if constexpr (BYTES == 1) {
                __stcs(reinterpret_cast<uint2 *>(q), make_uint2(w[0], w[1]));
            } else {
#pragma unroll
                for (int i = 0; i < kWords / 4; ++i)
                    __stcs(reinterpret_cast<uint4 *>(q) + i,
                           make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j * 32 + lane >= left) continue;
                const unsigned at = block + j * 32 + lane;
                if constexpr (BYTES == 4) __stcs(static_cast<uint32_t *>(p) + at, w[j]);
                else if constexpr (BYTES == 2)
                    __stcs(static_cast<uint16_t *>(p) + at, (uint16_t)(w[j / 2] >> (16 * (j % 2))));
                else
                    __stcs(static_cast<uint8_t *>(p) + at, (uint8_t)(w[j / 4] >> (8 * (j % 4))));
            }
        }
    }

    // 4 and 2 bytes: the values, by type.
    __device__ __forceinline__ void values(int type, float (&x)[8]) const {
        if constexpr (BYTES == 4) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(w[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = type == kTypeF16 ? unpack16<kTypeF16>(w[j % kWords])
                                                  : unpack16<kTypeBF16>(w[j % kWords]);
                x[2 * j] = f.x;
                x[2 * j + 1] = f.y;
            }
        }
    }
    __device__ __forceinline__ void set(int type, const float (&x)[8]) {
        if constexpr (BYTES == 4) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(x[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j % kWords] = type == kTypeF16 ? pack16<kTypeF16>(x[2 * j], x[2 * j + 1])
                                                 : pack16<kTypeBF16>(x[2 * j], x[2 * j + 1]);
        }
    }
};

__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
    uint32_t h;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(h) : "r"(two));
    return unpack16<kTypeF16>(h);
}

__device__ __forceinline__ uint32_t float2_to_e4m3x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\tcvt.rn.satfinite.e4m3x2.f32 c, %1, %2;\n\tcvt.u32.u16 %0, c;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}

// Eight codes times `unit`, and back.
__device__ __forceinline__ void decode(const Raw<1> &c, float unit, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = e4m3x2_to_float2((c.w[j / 2] >> (16 * (j % 2))) & 0xFFFFu);
        x[2 * j] = __fmul_rn(f.x, unit);
        x[2 * j + 1] = __fmul_rn(f.y, unit);
    }
}
__device__ __forceinline__ void encode(Raw<1> &c, const float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
        c.w[j] = float2_to_e4m3x2(x[4 * j], x[4 * j + 1]) |
                 float2_to_e4m3x2(x[4 * j + 2], x[4 * j + 3]) << 16;
}

__device__ __forceinline__ float approx_sqrt(float x) {
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The largest of a warp's non-negative values (or NaN).
__device__ __forceinline__ float warp_max_abs(float x) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x) & 0x7FFFFFFFu));
}

// PB, GB: bytes of a parameter and of a gradient.
template <int BITS, int PB, int GB>
__global__ void __launch_bounds__(kThreads, BITS == 8 ? 3 : 2)
    adamw_kernel(const __grid_constant__ AdamTable table, const AdamHyper h) {
    constexpr int SB = BITS == 32 ? 4 : 1;  // bytes of a state
    constexpr int kStages = stages_of(BITS);
    // The last tensor whose first chunk is not behind this one.
    int lo = 0, hi = table.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (table.t[mid].chunk0 <= blockIdx.x)
            lo = mid;
        else
            hi = mid;
    }
    const AdamTensor &t = table.t[lo];
    // The chunk's part of every array; from here on offsets are 32 bits.
    const long long first = (long long)(blockIdx.x - t.chunk0) * h.chunk;
    const int count = (int)min((long long)h.chunk, t.numel - first);
    unsigned char *const tp = static_cast<unsigned char *>(t.p) + first * PB;
    const unsigned char *const tg = static_cast<const unsigned char *>(t.g) + first * GB;
    unsigned char *const tm = static_cast<unsigned char *>(t.m) + first * SB;
    unsigned char *const tv = static_cast<unsigned char *>(t.v) + first * SB;
    float *const tms = BITS == 8 ? t.ms + first / kAdamBlock : nullptr;
    float *const tvs = BITS == 8 ? t.vs + first / kAdamBlock : nullptr;
    const int c_bytes = h.c_type == kTypeF32 ? 4 : 2;
    unsigned char *const tc = t.copy ? static_cast<unsigned char *>(t.copy) + first * c_bytes : nullptr;

    // A block's loads in a stage of the warp's ring: p, g, m, v, each lane's
    // bytes at its own place, so that no barrier is needed; the two scales
    // once per lane.
    constexpr int kG = 256 * PB, kM = kG + 256 * GB, kV = kM + 256 * SB, kS = kV + 256 * SB;
    constexpr int kStage = kS + (BITS == 8 ? 256 : 0);
    const int lane = threadIdx.x & 31, first_block = (threadIdx.x >> 5) * kAdamBlock;
    constexpr int kStride = kThreads / 32 * kAdamBlock;
    unsigned char *const ring = adam_smem + (threadIdx.x >> 5) * (kStages * kStage);
    auto fetch = [&](int block, int stage) {
        if (t.vec && block + kAdamBlock <= count) {
            unsigned char *to = ring + stage * kStage;
            Raw<GB>::fetch(to + kG, tg, block, lane);
            Raw<SB>::fetch(to + kM, tm, block, lane);
            Raw<SB>::fetch(to + kV, tv, block, lane);
            if constexpr (BITS == 8) {
                const uint32_t s = (uint32_t)__cvta_generic_to_shared(to + kS + lane * 8);
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(s),
                             "l"(tms + block / kAdamBlock) : "memory");
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(s + 4),
                             "l"(tvs + block / kAdamBlock) : "memory");
            }
            Raw<PB>::fetch(to, tp, block, lane);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) fetch(first_block + i * kStride, i);
    int stage = 0;
#pragma unroll 1
    for (int block = first_block; block < count; block += kStride) {
        const int left = count - block;
        const bool vec = t.vec && left >= kAdamBlock;
        Raw<PB> p;
        Raw<GB> g;
        Raw<SB> m, v;
        float ms = 0.0f, vs = 0.0f;
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        if (vec) {
            const unsigned char *from = ring + stage * kStage;
            g.take(from + kG, lane);
            m.take(from + kM, lane);
            v.take(from + kV, lane);
            if constexpr (BITS == 8) {
                const float2 f = *reinterpret_cast<const float2 *>(from + kS + lane * 8);
                ms = f.x;
                vs = f.y;
            }
            p.take(from, lane);
        } else {
            g.load(tg, block, lane, left);
            m.load(tm, block, lane, left);
            v.load(tv, block, lane, left);
            if constexpr (BITS == 8) {
                ms = __ldg(tms + block / kAdamBlock);
                vs = __ldg(tvs + block / kAdamBlock);
            }
            p.load(tp, block, lane, left);
        }
        float gg[8], mm[8], vv[8], r[8];
        g.values(h.g_type, gg);
        if constexpr (BITS == 32) {
            m.values(kTypeF32, mm);
            v.values(kTypeF32, vv);
        } else {
            decode(m, __fmul_rn(ms, 1.0f / 448.0f), mm);
            decode(v, __fmul_rn(vs, 1.0f / 448.0f), vv);
#pragma unroll
            for (int j = 0; j < 8; ++j) vv[j] = __fmul_rn(vv[j], vv[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float gj = __fmul_rn(gg[j], h.grad_scale);
            mm[j] = __fadd_rn(__fmul_rn(mm[j], h.beta1), __fmul_rn(gj, h.omb1));
            vv[j] = __fadd_rn(__fmul_rn(vv[j], h.beta2), __fmul_rn(__fmul_rn(gj, gj), h.omb2));
            // With 8-bit states the square root decides codes and is the
            // correctly rounded one.  Else it goes into the parameter's change
            // alone, as the division does: 2^-22 of the change each, below what the
            // sum with the parameter rounds off for changes up to a quarter of it.
            r[j] = BITS == 8 ? __fsqrt_rn(vv[j]) : approx_sqrt(vv[j]);
        }
        float pp[8];
        p.values(h.p_type, pp);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            pp[j] = fmaf(-h.step_size, __fdividef(mm[j], fmaf(r[j], h.inv_sqrt_bc2, h.eps)),
                         pp[j] * h.decay);
        p.set(h.p_type, pp);
        p.store(tp, block, lane, left, vec);
        if (tc) {
            if (h.c_type == kTypeF32) {
                Raw<4> c;
                c.set(kTypeF32, pp);
                c.store(tc, block, lane, left, vec);
            } else {
                Raw<2> c;
                c.set(h.c_type, pp);
                c.store(tc, block, lane, left, vec);
            }
        }
        if constexpr (BITS == 32) {
            m.set(kTypeF32, mm);
            v.set(kTypeF32, vv);
        } else {
            // Elements that are not there are zeros: they raise no maximum.
            uint32_t um = 0, ur = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                um = max(um, __float_as_uint(mm[j]) & 0x7FFFFFFFu);
                ur = max(ur, __float_as_uint(r[j]));
            }
            float top_m = warp_max_abs(__uint_as_float(um)), top_r = warp_max_abs(__uint_as_float(ur));
            if (top_m < kTiny) top_m = kTiny;
            if (top_r < kTiny) top_r = kTiny;
            const float km = __fmul_rn(__frcp_rn(top_m), 448.0f);
            const float kr = __fmul_rn(__frcp_rn(top_r), 448.0f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                mm[j] = __fmul_rn(mm[j], km);
                const float q = __fmul_rn(r[j], kr);
                r[j] = (r[j] > 0.0f && q < kLeast) ? kLeast : q;
            }
            encode(m, mm);
            encode(v, r);
            if (lane == 0) {
                tms[block / kAdamBlock] = top_m;
                tvs[block / kAdamBlock] = top_r;
            }
        }
        m.store(tm, block, lane, left, vec);
        v.store(tv, block, lane, left, vec);
        fetch(block + kStages * kStride, stage);
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
}

template <int BITS, int PB, int GB>
cudaError_t launch_one(const AdamTable &table, unsigned chunks, const AdamHyper &h, int device,
                       cudaStream_t stream) {
    constexpr int kState = BITS == 32 ? 4 : 1;
    constexpr int kBytes =
        kThreads / 32 * stages_of(BITS) * (256 * (PB + GB + 2 * kState) + (BITS == 8 ? 256 : 0));
    static std::atomic<bool> configured[kMaxDevices];
    if (device >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!configured[device].load()) {
        const cudaError_t e = cudaFuncSetAttribute(
            adamw_kernel<BITS, PB, GB>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
        if (e != cudaSuccess) return e;
        configured[device].store(true);
    }
    adamw_kernel<BITS, PB, GB><<<chunks, kThreads, kBytes, stream>>>(table, h);
    return cudaGetLastError();
}

template <int BITS>
cudaError_t launch_bits(const AdamTable &table, unsigned chunks, const AdamHyper &h, int device,
                        cudaStream_t stream) {
    const bool p32 = h.p_type == kTypeF32, g32 = h.g_type == kTypeF32;
    if (p32)
        return g32 ? launch_one<BITS, 4, 4>(table, chunks, h, device, stream)
                   : launch_one<BITS, 4, 2>(table, chunks, h, device, stream);
    return g32 ? launch_one<BITS, 2, 4>(table, chunks, h, device, stream)
               : launch_one<BITS, 2, 2>(table, chunks, h, device, stream);
}

}  // namespace

cudaError_t launch_adamw(const AdamTensor *tensors, int count, unsigned chunks, int state_bits,
                         const AdamHyper &h, int device, cudaStream_t stream) {
    if (chunks == 0) return cudaSuccess;
    AdamTable table;
    table.count = count;
    for (int i = 0; i < count; ++i) table.t[i] = tensors[i];
    return state_bits == 8 ? launch_bits<8>(table, chunks, h, device, stream)
                           : launch_bits<32>(table, chunks, h, device, stream);
}

}  // namespace sgemm
