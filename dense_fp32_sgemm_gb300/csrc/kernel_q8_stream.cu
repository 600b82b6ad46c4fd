// Products of 8-bit integers for a few rows of x, and 8-bit weights from a matrix.
//
// One pass over the weights: a CTA has a range of channels, cut into items of four
// channels by 512 k that its warps share out evenly; a lane multiplies 16 bytes of each
// of the four by the same 16 of every row of x (four at a time, summed into 32 bits).
// Sums are integers, so neither the sharing out nor the order of the additions
// changes them.  x lies in shared memory, zeros from K on.  The loads of three
// items are under way at a time.  Bound: HBM (1 x 4096 x 12288 11.4 us, 4.4 TB/s of the copy's
// 6.7, of which a launch and its first loads are 3; 1 x 8192 x 28672 44 us, 5.4 TB/s); from five
// rows on the multiplications too (8 x 4096 x 4096 11.3 us, 1.5 TB/s; larger matrices go to the tensor
// cores then).
#include <algorithm>
#include <atomic>

#include "device_common.cuh"
#include "kernels_q8.h"
#include "row_codes.cuh"

namespace sgemm {
namespace {

constexpr int kWarps = 16;
constexpr int kChannels = 4;       // of an item
constexpr int kItemK = 512;
constexpr int kAhead = 3;          // items on their way
constexpr int kCtaChannels = 256;  // most of a CTA
constexpr int kMaxDevices = 64;

__device__ __forceinline__ int4 load_weights(const int8_t *p) {
    int4 v;
    asm volatile("ld.global.L1::no_allocate.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// ROWS: rows of x (those from M on are zero).
template <int ROWS>
__global__ void __launch_bounds__(kWarps * 32, 1)
    q8_stream_kernel(const Q8StreamParams p, int type, int stage_k) {
    extern __shared__ __align__(16) int8_t s_x[];  // ROWS x stage_k
    __shared__ int s_sum[kCtaChannels * ROWS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // Channels of this CTA.
    const int n0 = (int)((long long)blockIdx.x * p.N / gridDim.x);
    const int count = (int)((blockIdx.x + 1LL) * p.N / gridDim.x) - n0;
    const int groups = (count + kChannels - 1) / kChannels;
    for (int i = tid; i < count * ROWS; i += kWarps * 32) s_sum[i] = 0;
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");

    for (int k0 = 0; k0 < p.K; k0 += stage_k) {
        const int len = min(stage_k, p.K - k0), chunks = (len + kItemK - 1) / kItemK;
        const int items = groups * chunks;
        const int first = (int)((long long)warp * items / kWarps), end = (int)((warp + 1LL) * items / kWarps);
        int acc[kChannels][ROWS];
        auto clear = [&]() {
#pragma unroll
            for (int c = 0; c < kChannels; ++c)
#pragma unroll
                for (int m = 0; m < ROWS; ++m) acc[c][m] = 0;
        };
        auto flush = [&](int g) {
#pragma unroll
            for (int c = 0; c < kChannels; ++c)
#pragma unroll
                for (int m = 0; m < ROWS; ++m) {
                    const int v = __reduce_add_sync(0xffffffffu, acc[c][m]);
                    if (lane == 0 && g * kChannels + c < count)
                        atomicAdd(&s_sum[(g * kChannels + c) * ROWS + m], v);
                }
        };
        auto fetch = [&](int it, int4 (&w)[kChannels]) {
            const int g = it / chunks, k = (it - g * chunks) * kItemK + lane * 16;
#pragma unroll
            for (int c = 0; c < kChannels; ++c) {
                const int n = g * kChannels + c;
                w[c] = make_int4(0, 0, 0, 0);
                if (it < end && n < count && k < len) {
                    const int8_t *from = p.w + (long long)(n0 + n) * p.ldw + k0 + k;
                    if (k + 16 <= len || n0 + n + 1 < p.N) {
                        w[c] = load_weights(from);
                    } else {
                        // (the last row may end with the matrix)
                        int v[4] = {0, 0, 0, 0};
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (k + j < len) v[j / 4] |= (int)(uint8_t)from[j] << (8 * (j % 4));
                        w[c] = make_int4(v[0], v[1], v[2], v[3]);
                    }
                }
            }
        };
        // The first weights are on their way while x is brought in.
        int4 ahead[kAhead][kChannels];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) fetch(first + a, ahead[a]);

        if (k0) __syncthreads();
        for (int i = tid; i < p.M * chunks * (kItemK / 16); i += kWarps * 32) {
            const int m = i / (chunks * (kItemK / 16)), k = (i - m * (chunks * (kItemK / 16))) * 16;
            const int8_t *from = p.x + m * p.ldx + k0 + k;
            int w[4] = {0, 0, 0, 0};
            if (p.x_vec && k + 16 <= len) {
                const int4 v = __ldg(reinterpret_cast<const int4 *>(from));
                w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (k + j < len) w[j / 4] |= (int)(uint8_t)__ldg(from + j) << (8 * (j % 4));
            }
            *reinterpret_cast<int4 *>(s_x + m * stage_k + k) = make_int4(w[0], w[1], w[2], w[3]);
        }
        for (int i = p.M * stage_k + tid * 16; i < ROWS * stage_k; i += kWarps * 32 * 16)
            *reinterpret_cast<int4 *>(s_x + i) = make_int4(0, 0, 0, 0);
        __syncthreads();

        clear();
#pragma unroll 1
        for (int it0 = first; it0 < end; it0 += kAhead) {
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const int it = it0 + a;
                if (it >= end) break;
                const int g = it / chunks, k = (it - g * chunks) * kItemK + lane * 16;
#pragma unroll
                for (int m = 0; m < ROWS; ++m) {
                    const int4 x = *reinterpret_cast<const int4 *>(s_x + m * stage_k + k);
#pragma unroll
                    for (int c = 0; c < kChannels; ++c) {
                        acc[c][m] = __dp4a(ahead[a][c].x, x.x, acc[c][m]);
                        acc[c][m] = __dp4a(ahead[a][c].y, x.y, acc[c][m]);
                        acc[c][m] = __dp4a(ahead[a][c].z, x.z, acc[c][m]);
                        acc[c][m] = __dp4a(ahead[a][c].w, x.w, acc[c][m]);
                    }
                }
                fetch(it + kAhead, ahead[a]);
                if (it + 1 == end || (it + 1) / chunks != g) {
                    flush(g);
                    clear();
                }
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < count * p.M; i += kWarps * 32) {
        const int m = i / count, n = i - m * count;
        store_from_float(p.y, type, m * p.ldy + n0 + n,
                         (float)s_sum[n * ROWS + m] * __ldg(p.x_scales + m) * __ldg(p.w_scales + n0 + n));
    }
}

template <int ROWS>
cudaError_t launch_stream_rows(const Q8StreamParams &p, int type, int num_sms, cudaStream_t stream) {
    const auto kernel = q8_stream_kernel<ROWS>;
    constexpr int kMost = kQ8StreamBytes / ROWS / kItemK * kItemK;
    const int stage_k = std::min(kMost, (p.K + kItemK - 1) / kItemK * kItemK);
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    static std::atomic<bool> configured[kMaxDevices];
    if (device >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!configured[device].load()) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kQ8StreamBytes);
        if (e != cudaSuccess) return e;
        configured[device].store(true);
    }
    const long long least = (p.N + kCtaChannels - 1LL) / kCtaChannels;
    cudaLaunchConfig_t cfg = {};
    // Whole rounds of all SMs, channels shared out evenly (at least four a CTA).
    long long ctas = (least + num_sms - 1) / num_sms * num_sms;
    ctas = std::max(least, std::min<long long>(ctas, (p.N + kChannels - 1) / kChannels));
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = (size_t)ROWS * stage_k;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, type, stage_k);
}

// Columns of W as rows of codes: 32 columns a CTA; their largest magnitudes, then
// 128 k at a time through shared memory.
__global__ void __launch_bounds__(1024) q8_quantize_kernel(const Q8QuantParams p) {
    __shared__ unsigned s_most[32][33];
    __shared__ uint32_t s_word[32][33];
    const int tx = threadIdx.x, ty = threadIdx.y;
    const int n = blockIdx.x * 32 + tx;
    const bool live = n < p.N;
    unsigned most = 0;
    if (live)
        for (int k = ty; k < p.K; k += 32)
            most = max(most, __float_as_uint(load_as_float(p.W, p.type, k * p.ldw + n)) & 0x7FFFFFFFu);
    s_most[ty][tx] = most;
    __syncthreads();
    most = __reduce_max_sync(0xffffffffu, s_most[tx][ty]);
    __syncthreads();
    if (tx == 0) s_most[0][ty] = most;
    __syncthreads();
    most = s_most[0][tx];
    const bool bad = most >= 0x7F800000u;
    const float top = fmaxf(__uint_as_float(most), kRowTiny);
    const float inv = bad ? 0.0f : 127.0f / top;
    if (ty == 0 && live) p.scales[n] = bad ? __int_as_float(0x7FC00000) : top / 127.0f;
    const int out = blockIdx.x * 32 + ty;  // the row this thread stores to
    const bool words = (reinterpret_cast<uintptr_t>(p.q) & 3) == 0 && p.ldq % 4 == 0;
    for (int k0 = 0; k0 < p.K; k0 += 128) {
        uint32_t word = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = k0 + ty * 4 + j;
            int q = 0;
            if (live && !bad && k < p.K) {
                const float a = load_as_float(p.W, p.type, k * p.ldw + n);
                bool near;
                q = row_code(a, inv, fabsf(a * inv) * 0x1p-21f, near);
                if (near) q = row_code_exact(a, top, inv);
            }
            word |= (uint32_t)(q & 255) << (8 * j);
        }
        s_word[tx][ty] = word;
        __syncthreads();
        word = s_word[ty][tx];
        __syncthreads();
        if (out >= p.N) continue;
        const int k = k0 + tx * 4;
        int8_t *to = p.q + out * p.ldq + k;
        if (words && k + 4 <= p.K) {
            *reinterpret_cast<uint32_t *>(to) = word;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k + j < p.K) to[j] = (int8_t)(word >> (8 * j));
        }
    }
}

}  // namespace

cudaError_t launch_q8_stream(const Q8StreamParams &p, int type, int num_sms, cudaStream_t stream) {
    if (p.M == 1) return launch_stream_rows<1>(p, type, num_sms, stream);
    if (p.M == 2) return launch_stream_rows<2>(p, type, num_sms, stream);
    if (p.M <= 4) return launch_stream_rows<4>(p, type, num_sms, stream);
    return launch_stream_rows<8>(p, type, num_sms, stream);
}

cudaError_t launch_q8_quantize(const Q8QuantParams &p, cudaStream_t stream) {
    q8_quantize_kernel<<<(p.N + 31) / 32, dim3(32, 32), 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace sgemm
