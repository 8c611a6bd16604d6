// Kept activations in 8 bits: e4m3 codes and, for every 16 values of a row, one byte s for the
// scale 2^(s - 127), the smallest power of two (2^-126 or more) that brings the 16 values within
// e4m3's +-448. A power of two makes every step but the rounding to e4m3 exact (no division, and
// packing what was unpacked changes nothing), and costs no precision: e4m3 is a floating format.
// 16 values because that is what one warp of the gated product holds of a row's gate or up.
// A group that holds an infinity or a NaN has the byte 255 and comes back as NaN.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <float.h>

#include "elem.cuh"

namespace moe {

constexpr int kCkptGroup = 16;  // values that share a scale

// The scale's byte from the bits of the largest absolute value. 448 = 1.75 * 2^8: a larger mantissa
// carries into the exponent.
__device__ __forceinline__ uint32_t ckpt_byte(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return 255u;
    return (uint32_t)max((int)((amax_bits + 0x1fffffu) >> 23) - 8, 1);
}
// 2^-(s - 127) for bytes 1..247 (as ckpt_byte gives them); NaN for 255.
__device__ __forceinline__ float ckpt_inverse(uint32_t byte) {
    return __uint_as_float(byte == 255u ? 0x7fffffffu : (254u - byte) << 23);
}
// 2^(s - 127), whatever the byte; NaN for 255.
__device__ __forceinline__ float ckpt_scale(uint32_t byte) {
    return __uint_as_float(byte == 255u ? 0x7fffffffu : byte == 0u ? 0x00400000u : byte << 23);
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The codes of four values of one group.
__device__ __forceinline__ uint32_t ckpt_encode4(float a, float b, float c, float d, float inverse) {
    return (uint32_t)f32x2_to_e4m3x2(a * inverse, b * inverse) | (uint32_t)f32x2_to_e4m3x2(c * inverse, d * inverse) << 16;
}

template <typename T>
__device__ __forceinline__ float largest();
template <>
__device__ __forceinline__ float largest<float>() { return FLT_MAX; }
template <>
__device__ __forceinline__ float largest<bf16>() { return __uint_as_float(0x7f7f0000u); }
template <>
__device__ __forceinline__ float largest<fp16>() { return 65504.f; }

// The value of a code under its scale, within T's range (NaN stays NaN). Exact in T but where it is subnormal.
template <typename T>
__device__ __forceinline__ float ckpt_value(float code, float scale) {
    float v;  // the smaller magnitude with the first one's sign
    asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(v) : "f"(code * scale), "f"(largest<T>()));
    return v;
}
template <typename T>
__device__ __forceinline__ void ckpt_decode4(uint32_t codes, float scale, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes >> 16 * i), __NV_E4M3));
        v[2 * i] = ckpt_value<T>(__low2float(h), scale);
        v[2 * i + 1] = ckpt_value<T>(__high2float(h), scale);
    }
}

// Two 16-bit values of one word.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    const Vec<T, 2> v = *reinterpret_cast<const Vec<T, 2>*>(&w);
    return make_float2(to_f32(v.v[0]), to_f32(v.v[1]));
}

// One group of 16-bit values (two 16-byte pieces) to its codes and scale byte.
template <typename T>
__device__ __forceinline__ uint4 ckpt_encode16(const uint4& lo, const uint4& hi, uint32_t& byte) {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    float2 v[8];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = unpack2<T>(w[i]);
        amax = __vmaxu2(amax, w[i] & 0x7fff7fffu);  // magnitudes of one type order as their bits
    }
    byte = ckpt_byte(abs_bits(unpack2<T>(max(amax >> 16, amax & 0xffff)).x));
    const float inv = ckpt_inverse(byte);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = ckpt_encode4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y, inv);
    return make_uint4(c[0], c[1], c[2], c[3]);
}

// The same of a group that two neighbouring lanes hold a half of each: this lane's eight codes.
template <typename T>
__device__ __forceinline__ uint2 ckpt_encode8(const uint4& piece, uint32_t& byte) {
    const uint32_t w[4] = {piece.x, piece.y, piece.z, piece.w};
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) amax = __vmaxu2(amax, w[i] & 0x7fff7fffu);
    amax = max(amax >> 16, amax & 0xffff);
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    byte = ckpt_byte(abs_bits(unpack2<T>(amax).x));
    const float inv = ckpt_inverse(byte);
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 a = unpack2<T>(w[2 * i]), b = unpack2<T>(w[2 * i + 1]);
        c[i] = ckpt_encode4(a.x, a.y, b.x, b.y, inv);
    }
    return make_uint2(c[0], c[1]);
}

// And back.
template <typename T>
__device__ __forceinline__ void ckpt_decode16(const uint4& codes, uint32_t byte, uint4& lo, uint4& hi) {
    const uint32_t c[4] = {codes.x, codes.y, codes.z, codes.w};
    const float scale = ckpt_scale(byte);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v[4];
        ckpt_decode4<T>(c[i], scale, v);
#pragma unroll
        for (int j = 0; j < 2; ++j) w[2 * i + j] = pack2_f32<T>(v[2 * j], v[2 * j + 1]);
    }
    lo = make_uint4(w[0], w[1], w[2], w[3]);
    hi = make_uint4(w[4], w[5], w[6], w[7]);
}

}  // namespace moe
