// The root-mean-square norm, and the norm that leaves in 8 bits: row_kernel.cuh; and the
// norm of rows that do not start on 16 bytes, word by word.
#include <type_traits>

#include "row_kernel.cuh"

namespace sgemm {
namespace {

// Rows off 16 bytes.  A warp has a stretch of the row, cut into the 4-byte words of y:
// lane l has every 32nd of them, so that its reads of shared memory (where the
// aligned pieces that cover the stretch of x lie) start at any word without a conflict,
// two halves of words make one of y's, and stores are whole words.  The
// weight lies in shared memory in FP32, even and odd elements apart, as a word of y may begin
// with either.  8192 x 8191 FP16: 72 us (3.7 TB/s; its bytes take 40), 105 in pieces of 16 bytes
// that are shifted on the way in and out.  Bound: instructions (25 per element; 67 % of the issue
// slots), half of them at the ends of rows, in the ring's copies and in the sums.
constexpr int kWordThreads = 512;
constexpr int kWordFloats = 32;             // most elements of a thread
constexpr int kWordSmem = 112 * 1024;       // of a CTA, two an SM
constexpr int kWordSmemOne = 224 * 1024;    // of one alone

// Elements of a 4-byte word, and words of a thread.
constexpr int word_elements(int type) { return type == kTypeF32 ? 1 : 2; }
constexpr int most_words(int type) { return kWordFloats / word_elements(type); }
// 16-byte pieces that cover 32 `words` words from any byte on.
__host__ __device__ constexpr int word_pieces(int words) { return 8 * words + 1; }
// Stores the elements of a word of y or h.  WHOLE: all of them are the row's, and `to` is the
// address of a word; else the row has `n` from the word's first on, but perhaps not that one.
template <int TYPE, bool WHOLE>
__device__ __forceinline__ void put_word(char *to, const float (&v)[word_elements(TYPE)], int n, bool first) {
    if constexpr (TYPE == kTypeF32) {
        if (WHOLE || n > 0) *reinterpret_cast<float *>(to) = v[0];
    } else {
        const uint32_t w = pack16<TYPE>(v[0], v[1]);
        if constexpr (WHOLE) {
            *reinterpret_cast<uint32_t *>(to) = w;
        } else {
            if (first && n > 0) *reinterpret_cast<uint16_t *>(to) = (uint16_t)w;
            if (n > 1) *reinterpret_cast<uint16_t *>(to + 2) = (uint16_t)(w >> 16);
        }
    }
}

// words: of a thread.
template <int TYPE>
__global__ void __launch_bounds__(kWordThreads, 2) norm_words_kernel(const RowParams p, int words) {
    constexpr int PER = word_elements(TYPE), E = 4 / PER, NW = most_words(TYPE);
    __shared__ float s_sum[2][kWordThreads / 32];
    extern __shared__ uint4 s_dynamic[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = threadIdx.y;
    const int warps = blockDim.x >> 5;
    const bool two = p.b != nullptr;
    const int arrays = two ? 2 : 1, pieces = word_pieces(words);
    uint4 *const s_ring = s_dynamic + (size_t)(group * warps + warp) * p.stages * arrays * pieces;
    const int half = blockDim.x * words + 2;  // room for the weight's even elements, of every word
    float *const s_even = reinterpret_cast<float *>(s_dynamic + (size_t)blockDim.y * warps * p.stages * arrays * pieces);
    float *const s_odd = s_even + half + 1;  // (16-bit types) from -1 on
    const unsigned rows = (unsigned)p.rows, stride = gridDim.x * blockDim.y;
    const int k0 = warp * words * 32;  // the warp's first word

    // y's words hold the elements 2 k - phase and 2 k - phase + 1.  (The last bits of addresses
    // are had in 32 bits.)
    auto low = [&](const void *m, long long ld, unsigned row) {
        return (unsigned)reinterpret_cast<uintptr_t>(m) + row * (unsigned)ld * E;
    };
    auto phase_of = [&](unsigned row) { return PER == 1 ? 0 : (int)(low(p.y, p.ldy, row) / E & 1); };
    // How far into a piece the warp's stretch of a row begins (perhaps an element before the row).
    auto into = [&](const void *m, long long ld, unsigned row, int phase) {
        return (int)(low(m, ld, row) + (k0 * PER - phase) * E & 15);
    };
    auto start = [&](unsigned row, int stage) {
        if (row < rows) {
            const int phase = phase_of(row), bytes = p.cols * E;
            for (int a = 0; a < arrays; ++a) {
                const long long ld = a ? p.ldb : p.lda, before = ld * row * E;  // bytes, in the matrix
                const char *m = static_cast<const char *>(a ? p.b : p.a), *begin = m + before;
                const int at = (k0 * PER - phase) * E - into(m, ld, row, phase);  // from the row's beginning
                uint4 *to = s_ring + (stage * arrays + a) * pieces;
                const int whole = min(max(bytes - at, 0) / 16, pieces);
                const bool cut = at < 0 && before + at < 0;
                for (int i = cut && lane == 0 ? 32 : lane; i < whole; i += 32)
                    cp_async16(reinterpret_cast<float *>(to + i), reinterpret_cast<const float *>(begin + at + 16 * i), 16);
                // The last piece, and zeros behind it (copies of no bytes, from the row's first piece).
                for (int i = max(whole, (int)cut) + lane; i < pieces; i += 32) {
                    const int n = min(max(bytes - at - 16 * i, 0), 16);
                    const int from = n > 0 ? at + 16 * i : -(int)(reinterpret_cast<uintptr_t>(begin) & 15);
                    cp_async16(reinterpret_cast<float *>(to + i), reinterpret_cast<const float *>(begin + from), n);
                }
                // A piece that begins before the matrix: what lies there is not read.
                if (cut && lane == 0) {
                    using Bits = std::conditional_t<PER == 1, uint32_t, uint16_t>;
                    for (int e = 0; e < 16; e += E) {
                        const bool there = at + e >= 0 && at + e < bytes;
                        reinterpret_cast<Bits *>(to)[e / E] = there ? *reinterpret_cast<const Bits *>(begin + at + e) : Bits(0);
                    }
                }
            }
        }
        cp_async_commit();
    };

    asm volatile("griddepcontrol.wait;" ::: "memory");
    unsigned row = blockIdx.x * blockDim.y + group;
    for (int s = 0; s < p.stages; ++s) start(row + s * stride, s);
    for (int e = group * blockDim.x + tid; e < p.cols; e += blockDim.x * blockDim.y) {
        const float w = load_as_float(p.w, p.w_f32 ? kTypeF32 : TYPE, e);
        if (PER == 1 || e % 2 == 0) s_even[e / PER] = w;
        else s_odd[e / 2] = w;
    }
    __syncthreads();

    float keep[NW][PER];
    int ring = 0;
    bool flip = false;
    for (; row < rows; row += stride, flip = !flip) {
        const int phase = phase_of(row);
        // Elements from the lane's first word on.
        const int left = p.cols + phase - (k0 + lane) * PER;
        const bool before = PER == 2 && phase && k0 + lane == 0;  // the first of them is not the row's
        // Where the lane's first word lies in a matrix.
        auto place = [&](void *m, long long ld) {
            return static_cast<char *>(m) + ((long long)row * ld + (k0 + lane) * PER - phase) * E;
        };
        const bool all = (k0 > 0 || !phase) && (k0 + 32 * words) * PER <= p.cols + phase;
        // All but the last stages - 1 rows' copies have landed, the other lanes' too.
        if (p.stages == 1) cp_async_wait<0>();
        else if (p.stages == 2) cp_async_wait<1>();
        else cp_async_wait<2>();
        __syncwarp();
        // The lane's first words in the ring, and how far into one y's begin.
        const int at_a = into(p.a, p.lda, row, phase), at_b = into(p.b, p.ldb, row, phase);
        const uint32_t *from_a = reinterpret_cast<const uint32_t *>(s_ring + ring * arrays * pieces) + (at_a >> 2) + lane;
        const uint32_t *from_b = from_a - (at_a >> 2) + (at_b >> 2) + 4 * pieces;
        if (PER == 2 && phase && k0 == 0) {
            if (lane == 0) {
                reinterpret_cast<uint16_t *>(s_ring + ring * arrays * pieces)[at_a / 2] = 0;
                if (two) reinterpret_cast<uint16_t *>(s_ring + (ring * arrays + 1) * pieces)[at_b / 2] = 0;
            }
            __syncwarp();
        }
        auto take = [&](const uint32_t *from, int at, int i, float (&v)[PER]) {
            if constexpr (PER == 1) {
                v[0] = __uint_as_float(from[32 * i]);
            } else {
                const float2 e = unpack16<TYPE>(__funnelshift_r(from[32 * i], from[32 * i + 1], (at & 2) * 8));
                v[0] = e.x;
                v[1] = e.y;
            }
        };
        char *const to_h = place(p.h, p.ldh);
        float sum = 0.0f;
        auto read = [&](auto whole) {
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                if (i >= words) continue;
                take(from_a, at_a, i, keep[i]);
                if (two) {
                    float r[PER];
                    take(from_b, at_b, i, r);
#pragma unroll
                    for (int j = 0; j < PER; ++j) keep[i][j] += r[j];
                }
#pragma unroll
                for (int j = 0; j < PER; ++j) sum = fmaf(keep[i][j], keep[i][j], sum);
                if (p.h) put_word<TYPE, decltype(whole)::value>(to_h + 128 * i, keep[i], left - 32 * PER * i, i > 0 || !before);
            }
        };
        if (all && (reinterpret_cast<uintptr_t>(to_h) & 3) == 0) read(std::true_type());
        else read(std::false_type());

#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (warps > 1) {
            // (a group's warps wait for one another alone)
            if (lane == 0) s_sum[flip][group * warps + warp] = sum;
            asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"((int)blockDim.x) : "memory");
            sum = (lane & 15) < warps ? s_sum[flip][group * warps + (lane & 15)] : 0.0f;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        const float rstd = rsqrtf(fmaf(sum, p.inv_cols, p.eps));
        char *const to_y = place(p.y, p.ldy);
        const float *w0 = (phase ? s_odd - 1 : s_even) + k0 + lane, *w1 = (phase ? s_even : s_odd) + k0 + lane;
        auto write = [&](auto whole) {
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                if (i >= words) continue;
                float y[PER];
                y[0] = keep[i][0] * rstd * w0[32 * i];
                if constexpr (PER == 2) y[1] = keep[i][1] * rstd * w1[32 * i];
                put_word<TYPE, decltype(whole)::value>(to_y + 128 * i, y, left - 32 * PER * i, i > 0 || !before);
            }
        };
        if (all) write(std::true_type());
        else write(std::false_type());
        // (here its addresses need no registers beside the row's elements)
        start(row + p.stages * stride, ring);
        if (++ring == p.stages) ring = 0;
    }
}

// Whether there are many rows of p and they fit (with two CTAs an SM or one), and the launch.  Few
// are faster piece by piece, with nothing to lay out first (100 x 4097 BF16 4.4 us, 7.0 here; 300 x
// 1025 FP32 4.9 and 6.9), many here (1817 x 2816 FP32 15.1 us and 12.6 here, 8000 x 1025 25.9 and
// 17.7, 4000 x 4097 BF16 50.5 and 35.6; only short ones lose a little, 16000 x 233 13.9 and 15.1).
template <int TYPE>
bool launch_words(const RowParams &p, int num_sms, cudaStream_t stream, cudaError_t &e) {
    constexpr int PER = word_elements(TYPE), NW = most_words(TYPE);
    // With few rows four words a thread, else as many as it holds.
    const int count = (p.cols + 2 * (PER - 1)) / PER, arrays = p.b ? 2 : 1;
    const int target = p.rows <= 2 * num_sms ? 4 : NW;
    const int threads = std::min(((count + target - 1) / target + 31) / 32 * 32, kWordThreads);
    const int words = (count + threads - 1) / threads;
    if (words > NW || few_rows<TYPE, kRowNorm>(p, num_sms)) return false;
    int groups = kWordThreads / threads;
    if (p.rows <= 2 * num_sms) groups = 1;
    const size_t weight = 4 * ((size_t)(threads * words + 2) * PER + 4);
    const size_t stage = (size_t)groups * (threads / 32) * arrays * word_pieces(words) * 16;
    const int per_sm = weight + stage <= kWordSmem ? 2 : 1;
    const size_t room = per_sm == 2 ? kWordSmem : kWordSmemOne;
    if (weight + stage > room) return false;
    RowParams q = p;
    q.stages = (int)std::min<size_t>(3, (room - weight) / stage);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<long long>((p.rows + groups - 1) / groups, (long long)num_sms * per_sm));
    cfg.blockDim = dim3(threads, groups);
    cfg.stream = stream;
    cfg.dynamicSmemBytes = weight + stage * q.stages;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    static std::atomic<bool> configured[kMaxDevices];
    e = p.device < kMaxDevices ? cudaSuccess : cudaErrorInvalidDevice;
    if (e == cudaSuccess && !configured[p.device].load()) {
        e = cudaFuncSetAttribute(norm_words_kernel<TYPE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kWordSmemOne);
        if (e == cudaSuccess) configured[p.device].store(true);
    }
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, norm_words_kernel<TYPE>, q, words);
    return true;
}

}  // namespace

cudaError_t launch_norm(const RowParams &p, int type, bool q8, bool vec, int num_sms,
                        cudaStream_t stream) {
    if (q8) return launch_rows_of<kRowNormQ8, -1>(p, type, vec, num_sms, stream);
    cudaError_t e;
    if (!vec && (type == kTypeF32   ? launch_words<kTypeF32>(p, num_sms, stream, e)
                 : type == kTypeF16 ? launch_words<kTypeF16>(p, num_sms, stream, e)
                                    : launch_words<kTypeBF16>(p, num_sms, stream, e)))
        return e;
    return launch_rows_of<kRowNorm, -1>(p, type, vec, num_sms, stream);
}

}  // namespace sgemm
