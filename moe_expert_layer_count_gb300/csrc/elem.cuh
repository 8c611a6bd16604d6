// Element types of the 16/32-bit training operators (bf16, fp16, fp32): loads, one
// rounding per stored value, 16-byte vectors and the dispatch from enum moe_dtype.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"

namespace moe {

using bf16 = __nv_bfloat16;
using fp16 = __half;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(fp16 v) { return __half2float(v); }

// Round-to-nearest-even to T (fp16 overflows to infinity).
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ fp16 from_f32<fp16>(float v) { return __float2half_rn(v); }

// Two values rounded to T in one conversion, the first in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack2_f32(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2_f32<bf16>(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2_f32<fp16>(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// V consecutive values of T, moved with one load or store where V * sizeof(T) is 16.
template <typename T, int V>
struct alignas(V * sizeof(T)) Vec {
    T v[V];
};

inline int dtype_bytes(int dtype) {
    return dtype == MOE_DT_F32 ? 4 : dtype == MOE_DT_BF16 || dtype == MOE_DT_F16 ? 2 : 0;
}

// Calls f with a null pointer of the element type that `dtype` names.
template <typename F>
int with_dtype(int dtype, F&& f) {
    switch (dtype) {
        case MOE_DT_F32: return f(static_cast<float*>(nullptr));
        case MOE_DT_BF16: return f(static_cast<bf16*>(nullptr));
        case MOE_DT_F16: return f(static_cast<fp16*>(nullptr));
        default: return MOE_ERR_INVALID_ARG;
    }
}

inline bool misaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace moe
