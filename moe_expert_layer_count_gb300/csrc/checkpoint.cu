// Activations kept in 8 bits for the backward pass (the form of ckpt.cuh), and read back.
#include <climits>
#include <type_traits>

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

// `bytes` bytes between global and shared memory by all threads of the block, 16 at a time but for the
// ends. Both addresses have the same offset from a 16-byte boundary; a value's size divides them.
template <int kSize>
__device__ __forceinline__ void move_flat(uint8_t* to, const uint8_t* from, int bytes) {
    using U = std::conditional_t<kSize == 4, uint32_t, std::conditional_t<kSize == 2, uint16_t, uint8_t>>;
    const int head = min((int)(-reinterpret_cast<uintptr_t>(from) & 15), bytes), whole = (bytes - head) & ~15, tail = head + whole;
    for (int i = threadIdx.x * 16; i < whole; i += kThreads * 16)
        *reinterpret_cast<uint4*>(to + head + i) = *reinterpret_cast<const uint4*>(from + head + i);
    const int i = threadIdx.x * kSize;
    if (i < head) *reinterpret_cast<U*>(to + i) = *reinterpret_cast<const U*>(from + i);
    if (tail + i < bytes) *reinterpret_cast<U*>(to + tail + i) = *reinterpret_cast<const U*>(from + tail + i);
}

// Any width and alignment. A block has kThreads groups one after the other, whose values are contiguous in
// memory whatever the rows' length: they go through shared memory, so that global memory is moved 16 bytes
// at a time, and a thread has one group there. Lane l takes its values from the (l / 2)-th on, which spreads
// the lanes over the banks for values of 1, 2 and 4 bytes alike. `per_row`: groups of a row.
template <typename T, bool kPack>
__global__ void __launch_bounds__(kThreads) rows_kernel(T* __restrict__ x, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                                                        int64_t groups, int K, int per_row) {
    __shared__ __align__(16) uint8_t x_mem[kThreads * kCkptGroup * sizeof(T) + 16];
    __shared__ __align__(16) uint8_t c_mem[kThreads * kCkptGroup + 16];
    pdl_wait();
    pdl_trigger();
    const int64_t g0 = (int64_t)blockIdx.x * kThreads, row0 = g0 / per_row;
    const int first = (int)(g0 - row0 * per_row), n = (int)min((int64_t)kThreads, groups - g0);
    // the i-th group's first value from the first group's, and its length
    auto start = [&](int i, int& length) {
        const int row = (first + i) / per_row, col = (first + i - row * per_row) * kCkptGroup;
        length = min(kCkptGroup, K - col);
        return row * K + col - first * kCkptGroup;
    };
    int length;
    const int values = start(n - 1, length) + length;
    const int64_t at = row0 * K + (int64_t)first * kCkptGroup;
    uint8_t* xg = reinterpret_cast<uint8_t*>(x + at);
    uint8_t* cg = codes + at;
    uint8_t* xr = x_mem + (reinterpret_cast<uintptr_t>(xg) & 15);
    uint8_t* cs = c_mem + (reinterpret_cast<uintptr_t>(cg) & 15);
    T* xs = reinterpret_cast<T*>(xr);
    if (kPack)
        move_flat<sizeof(T)>(xr, xg, values * (int)sizeof(T));
    else
        move_flat<1>(cs, cg, values);
    __syncthreads();
    const int i = threadIdx.x;
    if (i < n) {
        const int s = start(i, length), turn = (threadIdx.x & 31) >> 1;
        if (kPack) {
            float v[kCkptGroup];
            uint32_t amax = 0;
#pragma unroll
            for (int j = 0; j < kCkptGroup; ++j) {
                const int e = (j + turn) & (kCkptGroup - 1);
                v[j] = e < length ? to_f32(xs[s + e]) : 0.f;
                amax = max(amax, abs_bits(v[j]));
            }
            const uint32_t byte = ckpt_byte(amax);
            const float inv = ckpt_inverse(byte);
#pragma unroll
            for (int j = 0; j < kCkptGroup; j += 2) {
                const uint32_t two = f32x2_to_e4m3x2(v[j] * inv, v[j + 1] * inv);
                const int e = (j + turn) & (kCkptGroup - 1), f = (j + 1 + turn) & (kCkptGroup - 1);
                if (e < length) cs[s + e] = (uint8_t)two;
                if (f < length) cs[s + f] = (uint8_t)(two >> 8);
            }
            scales[g0 + i] = (uint8_t)byte;
        } else {
            const float scale = ckpt_scale(scales[g0 + i]);
#pragma unroll
            for (int j = 0; j < kCkptGroup; j += 4) {
                uint32_t four = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int e = (j + q + turn) & (kCkptGroup - 1);
                    if (e < length) four |= (uint32_t)cs[s + e] << 8 * q;
                }
                float v[4];
                ckpt_decode4<T>(four, scale, v);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int e = (j + q + turn) & (kCkptGroup - 1);
                    if (e < length) xs[s + e] = from_f32<T>(v[q]);
                }
            }
        }
    }
    __syncthreads();
    if (kPack)
        move_flat<1>(cg, cs, values);
    else
        move_flat<sizeof(T)>(xg, xr, values * (int)sizeof(T));
}

// Sizes of both directions; the groups' number.
bool sizes_ok(int64_t M, int K, int dtype, int64_t& groups) {
    if (M < 0 || K < 1 || K > 1 << 30 || !dtype_bytes(dtype) || M > ((int64_t)1 << 46) / K) return false;
    groups = M * ((K + kCkptGroup - 1) / kCkptGroup);
    return groups <= (int64_t)INT32_MAX * kThreads;  // one grid
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
            launch_k(rows_kernel<T, true>, (unsigned)((groups + kThreads - 1) / kThreads), kThreads, 0, s, const_cast<T*>(in), codes, scales,
                     groups, K, (K + kCkptGroup - 1) / kCkptGroup);
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
            launch_k(rows_kernel<T, false>, (unsigned)((groups + kThreads - 1) / kThreads), kThreads, 0, s, out, const_cast<uint8_t*>(codes),
                     const_cast<uint8_t*>(scales), groups, K, (K + kCkptGroup - 1) / kCkptGroup);
        }
        note_launches(1);
        return launch_status();
    });
}

}  // extern "C"
