// Pieces of a row: V consecutive elements (16 bytes) of a matrix, in FP32.
//
// Rows that do not start on 16 bytes are read through the two aligned pieces that
// cover a piece, shifted into place, and written through shared memory, a warp's 512
// bytes at a time: aligned pieces of the destination, and its ends element by
// element.  (One element per lane and instruction took 145 us for the norm of 8192 x 8191
// FP16, where the whole traffic takes 40.)
#pragma once

#include "device_common.cuh"
#include "ops_common.cuh"

namespace sgemm {

// Elements of a 16-byte piece.
constexpr int piece_elements(int type) { return type == kTypeF32 ? 4 : 8; }

// A row to read.  inside: aligned pieces which reach over its ends (by less than 16 bytes)
// stay inside the matrix; first: those over its beginning do not.
struct RowSource {
    const char *row;
    int bytes;  // of the row
    bool first, inside;
};
__device__ __forceinline__ RowSource row_source(const void *p, long long row, int cols, long long ld,
                                                int element, long long rows) {
    const long long before = row * ld * element, behind = (rows - 1 - row) * ld * element;
    return {static_cast<const char *>(p) + before, cols * element, before < 16, before >= 16 && behind >= 16};
}

// w >> (8 * shift) over eight words, the first four of it; shift in 0 .. 15, even.
__device__ __forceinline__ uint4 shift_pieces(uint4 a, uint4 b, int shift) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t u[7], t[5], o[4];
#pragma unroll
    for (int k = 0; k < 7; ++k) u[k] = shift & 4 ? w[k + 1] : w[k];
#pragma unroll
    for (int k = 0; k < 5; ++k) t[k] = shift & 8 ? u[k + 2] : u[k];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = __funnelshift_r(t[k], t[k + 1], (shift & 2) * 8);
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int TYPE>
__device__ __forceinline__ void unpack_piece(uint4 f, float (&v)[piece_elements(TYPE)]) {
    const uint32_t w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (TYPE == kTypeF32) {
            v[j] = __uint_as_float(w[j]);
        } else {
            const float2 e = unpack16<TYPE>(w[j]);
            v[2 * j] = e.x;
            v[2 * j + 1] = e.y;
        }
    }
}
template <int TYPE>
__device__ __forceinline__ uint4 pack_piece(const float (&v)[piece_elements(TYPE)]) {
    if constexpr (TYPE == kTypeF32)
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                          __float_as_uint(v[3]));
    else
        return make_uint4(pack16<TYPE>(v[0], v[1]), pack16<TYPE>(v[2], v[3]), pack16<TYPE>(v[4], v[5]),
                          pack16<TYPE>(v[6], v[7]));
}

// n (at least 1) elements of a row from byte `at` (a multiple of 16) on, as they lie in
// memory, zeros for the others up to a piece.  ALIGNED: the row is on 16 bytes.
template <int TYPE, bool ALIGNED>
__device__ __forceinline__ uint4 load_piece(const RowSource &m, int at, int n) {
    constexpr int V = piece_elements(TYPE), E = 16 / V;
    const char *p = m.row + at;
    const int shift = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(m.row) & 15);
    if (n >= V) {
        if (ALIGNED || shift == 0) return *reinterpret_cast<const uint4 *>(p);
        if (m.inside || (at >= shift && at - shift + 32 <= m.bytes)) {
            const uint4 *first = reinterpret_cast<const uint4 *>(p - shift);
            return shift_pieces(first[0], first[1], shift);
        }
    }
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (j < n) {
            if constexpr (E == 4)
                w[j] = *reinterpret_cast<const uint32_t *>(p + 4 * j);
            else
                w[j / 2] |= (uint32_t)*reinterpret_cast<const uint16_t *>(p + 2 * j) << (16 * (j % 2));
        }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// Bytes of shared memory for a piece on its way: the aligned pieces that cover it.
constexpr int piece_slots(bool aligned) { return aligned ? 1 : 2; }

// Starts copying what covers a row's piece (from byte `at` on, a multiple of 16 below the
// row's length) into `slot` and, for rows off 16 bytes, slot[pitch]; zeros behind the row's
// end.  Only the matrix's first piece cannot be had this way, when the row before
// it is not there: take_piece() loads it.
template <bool ALIGNED>
__device__ __forceinline__ void start_piece(uint4 *slot, int pitch, const RowSource &m, int at) {
    const int shift = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(m.row) & 15);
    const int left = m.bytes - at + shift;
    const char *first = m.row + at - shift;
    if (!ALIGNED && m.first && at < shift) return;
    cp_async16(reinterpret_cast<float *>(slot), reinterpret_cast<const float *>(first), min(16, left));
    if (!ALIGNED && shift)
        cp_async16(reinterpret_cast<float *>(slot + pitch),
                   reinterpret_cast<const float *>(left > 16 ? first + 16 : first),
                   max(0, min(16, left - 16)));
}
template <int TYPE, bool ALIGNED>
__device__ __forceinline__ uint4 take_piece(const uint4 *slot, int pitch, const RowSource &m, int at) {
    if constexpr (ALIGNED) {
        return *slot;
    } else {
        const int shift = (int)(reinterpret_cast<uintptr_t>(m.row) & 15);
        if (shift == 0) return *slot;
        if (m.first && at < shift) return load_piece<TYPE, false>(m, at, (m.bytes - at) / (16 / piece_elements(TYPE)));
        return shift_pieces(slot[0], slot[pitch], shift);
    }
}

template <int TYPE, bool ALIGNED>
__device__ __forceinline__ void load_values(const RowSource &m, int at, int n,
                                            float (&v)[piece_elements(TYPE)]) {
    unpack_piece<TYPE>(load_piece<TYPE, ALIGNED>(m, at, n), v);
}

// n (at least 1) elements of the norm's weight from c on; its type is TYPE or FP32.
template <int TYPE, bool ALIGNED>
__device__ __forceinline__ void load_weight(const RowSource &m, bool f32, int c, int n,
                                            float (&v)[piece_elements(TYPE)]) {
    if constexpr (TYPE == kTypeF32) {
        load_values<TYPE, ALIGNED>(m, 4 * c, n, v);
    } else if (!f32) {
        load_values<TYPE, ALIGNED>(m, 2 * c, n, v);
    } else {
        float a[4], b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        load_values<kTypeF32, ALIGNED>(m, 4 * c, n, a);
        if (n > 4) load_values<kTypeF32, ALIGNED>(m, 4 * c + 16, n - 4, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = a[j];
            v[4 + j] = b[j];
        }
    }
}

// Shared memory of a warp for store_piece().
constexpr int kStageWords = 33 * 4;  // 32 pieces, and one that a read may reach into

// A whole warp's pieces, lane by lane from `p` on (the address of lane 0's): n
// elements of each lane's exist (none where n < 1).  Every lane calls it.
template <int TYPE, bool ALIGNED>
__device__ __forceinline__ void store_piece(char *p, int n, uint4 w, uint32_t *stage) {
    constexpr int V = piece_elements(TYPE), E = 16 / V;
    const int lane = threadIdx.x & 31;
    const int shift = ALIGNED ? 0 : (int)(reinterpret_cast<uintptr_t>(p) & 15);
    if (ALIGNED || shift == 0) {
        char *to = p + 16 * lane;
        if (n >= V) {
            *reinterpret_cast<uint4 *>(to) = w;
        } else {
            const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < n) {
                    if constexpr (E == 4)
                        reinterpret_cast<uint32_t *>(to)[j] = e[j];
                    else
                        reinterpret_cast<uint16_t *>(to)[j] = (uint16_t)(e[j / 2] >> (16 * (j % 2)));
                }
        }
        return;
    }
    __syncwarp();
    reinterpret_cast<uint4 *>(stage)[lane] = w;
    __syncwarp();
    const int bytes = __reduce_add_sync(0xffffffffu, max(0, min(n, V))) * E;
    const int head = 16 - shift;  // bytes before the destination's first aligned piece
    const int at = head + 16 * lane;
    if (at + 16 <= bytes) {
        const uint4 *from = reinterpret_cast<const uint4 *>(stage) + lane;
        *reinterpret_cast<uint4 *>(p + at) = shift_pieces(from[0], from[1], head);
    }
    // The ends: before `head`, and behind the last whole piece.
    const int tail = bytes > head ? head + (bytes - head) / 16 * 16 : bytes;
    const int i = (lane & 15) * E, off = lane < 16 ? i : tail + i;
    if (lane < 16 ? i < min(head, bytes) : off < bytes) {
        if constexpr (E == 4)
            *reinterpret_cast<uint32_t *>(p + off) = stage[off / 4];
        else
            *reinterpret_cast<uint16_t *>(p + off) = reinterpret_cast<const uint16_t *>(stage)[off / 2];
    }
}

}  // namespace sgemm
