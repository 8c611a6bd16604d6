// Activations kept in 8 bits for the backward pass (the form of ckpt.cuh), and read back.
#include <climits>

#include "ckpt.cuh"
#include "elem.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Rows of whole groups on 16-byte boundaries: a thread has one group.
template <typename T>
__global__ void __launch_bounds__(kThreads) pack_groups_kernel(const T* __restrict__ x, int64_t groups, uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales) {
    pdl_wait();
    pdl_trigger();
    const int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (g >= groups) return;
    const uint4* p = reinterpret_cast<const uint4*>(x + g * kCkptGroup);
    uint32_t byte;
    uint4 c;
    if constexpr (sizeof(T) == 2) {
        c = ckpt_encode16<T>(p[0], p[1], byte);
    } else {
        uint4 q[4];
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            q[i] = p[i];
            amax = max(max(amax, max(q[i].x & 0x7fffffffu, q[i].y & 0x7fffffffu)), max(q[i].z & 0x7fffffffu, q[i].w & 0x7fffffffu));
        }
        byte = ckpt_byte(amax);
        const float inv = ckpt_inverse(byte);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = ckpt_encode4(__uint_as_float(q[i].x), __uint_as_float(q[i].y), __uint_as_float(q[i].z), __uint_as_float(q[i].w), inv);
        c = make_uint4(w[0], w[1], w[2], w[3]);
    }
    reinterpret_cast<uint4*>(codes)[g] = c;
    scales[g] = (uint8_t)byte;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) unpack_groups_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                                 int64_t groups, T* __restrict__ x) {
    pdl_wait();
    pdl_trigger();
    const int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (g >= groups) return;
    const uint4 c = reinterpret_cast<const uint4*>(codes)[g];
    const uint32_t byte = scales[g];
    uint4* o = reinterpret_cast<uint4*>(x + g * kCkptGroup);
    if constexpr (sizeof(T) == 2) {
        uint4 lo, hi;
        ckpt_decode16<T>(c, byte, lo, hi);
        o[0] = lo;
        o[1] = hi;
    } else {
        const float scale = ckpt_scale(byte);
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[4];
            ckpt_decode4<T>(w[i], scale, v);
            o[i] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        }
    }
}

// Any width and alignment: 16 lanes have a group, a value each. `per_row`: groups of a row.
template <typename T>
__global__ void __launch_bounds__(kThreads) pack_values_kernel(const T* __restrict__ x, int64_t groups, int K, int per_row,
                                                               uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    pdl_wait();
    pdl_trigger();
    const int64_t g = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / kCkptGroup;
    const int64_t row = g / per_row;
    const int col = (int)(g - row * per_row) * kCkptGroup + (threadIdx.x & (kCkptGroup - 1));
    const bool in = g < groups && col < K;
    const float v = in ? to_f32(x[row * K + col]) : 0.f;
    uint32_t amax = abs_bits(v);
#pragma unroll
    for (int o = kCkptGroup / 2; o; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const uint32_t byte = ckpt_byte(amax);
    if (!in) return;
    codes[row * K + col] = (uint8_t)f32x2_to_e4m3x2(v * ckpt_inverse(byte), 0.f);
    if ((threadIdx.x & (kCkptGroup - 1)) == 0) scales[g] = (uint8_t)byte;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) unpack_values_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                                 int64_t groups, int K, int per_row, T* __restrict__ x) {
    pdl_wait();
    pdl_trigger();
    const int64_t g = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / kCkptGroup;
    const int64_t row = g / per_row;
    const int col = (int)(g - row * per_row) * kCkptGroup + (threadIdx.x & (kCkptGroup - 1));
    if (g >= groups || col >= K) return;
    float v[4];
    ckpt_decode4<T>(codes[row * K + col], ckpt_scale(scales[g]), v);
    x[row * K + col] = from_f32<T>(v[0]);
}

// Sizes of both directions; the groups' number.
bool sizes_ok(int64_t M, int K, int dtype, int64_t& groups) {
    if (M < 0 || K < 1 || K > 1 << 30 || !dtype_bytes(dtype) || M > ((int64_t)1 << 46) / K) return false;
    groups = M * ((K + kCkptGroup - 1) / kCkptGroup);
    return groups <= (int64_t)INT32_MAX * (kThreads / kCkptGroup);  // one grid
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

MOE_API int moe_checkpoint_pack(const void* x, int64_t M, int K, int dtype, uint8_t* codes, uint8_t* scales, moe_stream_t stream) {
    int64_t groups = 0;
    if (!sizes_ok(M, K, dtype, groups)) return MOE_ERR_INVALID_ARG;
    const size_t z = dtype_bytes(dtype), n = (size_t)M * K;
    if (M > 0 && (!x || !codes || !scales)) return MOE_ERR_INVALID_ARG;
    if (misaligned(x, z) || overlap(x, n * z, codes, n) || overlap(x, n * z, scales, groups) || overlap(codes, n, scales, groups))
        return MOE_ERR_INVALID_ARG;
    if (M == 0) return MOE_OK;
    if (int st = check_device(nullptr)) return st;
    return with_dtype(dtype, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        cudaStream_t s = (cudaStream_t)stream;
        const T* in = static_cast<const T*>(x);
        if (K % kCkptGroup == 0 && !misaligned(x, 16) && !misaligned(codes, 16)) {
            launch_k(pack_groups_kernel<T>, (unsigned)((groups + kThreads - 1) / kThreads), kThreads, 0, s, in, groups, codes, scales);
        } else {
            const int per = kThreads / kCkptGroup, per_row = (K + kCkptGroup - 1) / kCkptGroup;
            launch_k(pack_values_kernel<T>, (unsigned)((groups + per - 1) / per), kThreads, 0, s, in, groups, K, per_row, codes, scales);
        }
        note_launches(1);
        return launch_status();
    });
}

MOE_API int moe_checkpoint_unpack(const uint8_t* codes, const uint8_t* scales, int64_t M, int K, int dtype, void* x,
                                  moe_stream_t stream) {
    int64_t groups = 0;
    if (!sizes_ok(M, K, dtype, groups)) return MOE_ERR_INVALID_ARG;
    const size_t z = dtype_bytes(dtype), n = (size_t)M * K;
    if (M > 0 && (!x || !codes || !scales)) return MOE_ERR_INVALID_ARG;
    if (misaligned(x, z) || overlap(x, n * z, codes, n) || overlap(x, n * z, scales, groups)) return MOE_ERR_INVALID_ARG;
    if (M == 0) return MOE_OK;
    if (int st = check_device(nullptr)) return st;
    return with_dtype(dtype, [&](auto* t) {
        using T = std::remove_pointer_t<decltype(t)>;
        cudaStream_t s = (cudaStream_t)stream;
        T* out = static_cast<T*>(x);
        if (K % kCkptGroup == 0 && !misaligned(x, 16) && !misaligned(codes, 16)) {
            launch_k(unpack_groups_kernel<T>, (unsigned)((groups + kThreads - 1) / kThreads), kThreads, 0, s, codes, scales, groups, out);
        } else {
            const int per = kThreads / kCkptGroup, per_row = (K + kCkptGroup - 1) / kCkptGroup;
            launch_k(unpack_values_kernel<T>, (unsigned)((groups + per - 1) / per), kThreads, 0, s, codes, scales, groups, K, per_row, out);
        }
        note_launches(1);
        return launch_status();
    });
}

}  // extern "C"
