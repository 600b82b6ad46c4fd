// Device helpers of the feed-forward operators: element types, conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "kernels_ffn.h"

namespace sgemm {

// Element `i` of an array of `type` elements, in FP32.
__device__ __forceinline__ float load_as_float(const void *p, int type, long long i) {
    if (type == kTypeF32) return static_cast<const float *>(p)[i];
    if (type == kTypeF16) return __half2float(static_cast<const __half *>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

// The same, rounded to nearest even.
__device__ __forceinline__ void store_from_float(void *p, int type, long long i, float v) {
    if (type == kTypeF32)
        static_cast<float *>(p)[i] = v;
    else if (type == kTypeF16)
        static_cast<__half *>(p)[i] = __float2half_rn(v);
    else
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

// Two 16-bit values of `type` packed in a word, the first in the low half.
template <int TYPE>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
    if constexpr (TYPE == kTypeF16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

template <int TYPE>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
    if constexpr (TYPE == kTypeF16) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    } else {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
}

// x rounded to bf16; a finite x that would round to infinity is cut instead.
__device__ __forceinline__ float bf16_part(float x) {
    const float hi = __bfloat162float(__float2bfloat16_rn(x));
    return fabsf(hi) == INFINITY ? __uint_as_float(__float_as_uint(x) & 0xFFFF0000u) : hi;
}
// What is left of x after its part, exact in FP32: nothing of an infinity or NaN.
// (Selects, no branches: with branches a lane's elements go one after the other.)
__device__ __forceinline__ float bf16_rest(float x, float part) {
    return fabsf(part) < INFINITY ? x - part : 0.0f;
}
// x as the sum of three bf16 values (its 24 significant bits in parts of 8),
// each the rounded rest of those before it; an infinity or NaN is its first part
// alone.  (In a product with another value's parts an infinity meets zero parts, so
// the sum it enters is NaN.)
__device__ __forceinline__ void split3(float x, float (&part)[3]) {
    part[0] = bf16_part(x);
    const float r = bf16_rest(x, part[0]);
    part[1] = __bfloat162float(__float2bfloat16_rn(r));
    part[2] = r - part[1];
}

}  // namespace sgemm
