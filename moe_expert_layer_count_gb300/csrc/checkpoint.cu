// Activations kept in 8 bits for the backward pass (the form of ckpt.cuh), and read back: x * 2^-e rounded to
// e4m3, e one exponent for 16 values. Each value is read and written once, so DRAM bounds it where rows are
// whole groups: 65536 x 2048 bf16 58 us packed and 60 read back, 6.8-7.1 TB/s (its floor at the copy rate: 61), fp32
// 99 and 97 (100). Rows of other widths cost instructions and shared memory's queue instead (an issue in 73 % of
// the slots from and to 16 bits, in 59 % to fp32, DRAM at a quarter to a half): 30011 x 1111 bf16 22 us both ways (floor 15),
// fp32 32 and 28-29 (25).
#include <climits>
#include <type_traits>

#include "ckpt.cuh"
#include "elem.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
// rows_kernel: a block's groups, and those of a thread. Two share the work of finding the block's place and of
// the ends (65536 x 1000 bf16: 44 -> 40 us); packing fp32, whose values fill registers, has one (two: 56 -> 71 us).
constexpr int kRowGroups = 256;
template <typename T, bool kPack>
__host__ __device__ constexpr int per_thread() { return kPack && sizeof(T) == 4 ? 1 : 2; }

// Rows of whole groups on 16-byte boundaries: a thread has one group and needs no shared memory (65536 x 2048 bf16
// packed and read back 60 and 60 us, by rows_kernel 68 and 72; fp32 99 and 97, 103 and 99).
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
    if constexpr (sizeof(T) == 2) {
        const int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x;
        if (g >= groups) return;
        uint4 lo, hi;
        ckpt_decode16<T>(reinterpret_cast<const uint4*>(codes)[g], scales[g], lo, hi);
        uint4* o = reinterpret_cast<uint4*>(x) + 2 * g;
        o[0] = lo;
        o[1] = hi;
    } else {
        // four values at a time, so that a warp writes 512 bytes in a row (65536 x 2048: 64 bytes a thread 130 us)
        const int64_t q0 = (int64_t)blockIdx.x * (4 * kThreads) + threadIdx.x;
        uint32_t c[4], byte[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t q = q0 + i * kThreads;
            const bool live = q < 4 * groups;
            c[i] = live ? reinterpret_cast<const uint32_t*>(codes)[q] : 0;
            byte[i] = live ? scales[q >> 2] : 0;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[4];
            ckpt_decode4<T>(c[i], ckpt_scale(byte[i]), v);
            const int64_t q = q0 + i * kThreads;
            if (q < 4 * groups) reinterpret_cast<float4*>(x)[q] = make_float4(v[0], v[1], v[2], v[3]);
        }
    }
}

// `bytes` bytes from global to shared memory or back by all threads of the block, 16 at a time but for the
// ends. Shared memory holds them at the address's offset from a 16-byte boundary; kSize, a value's size,
// divides them. At most 16 * kTurns bytes a group.
template <int kSize, bool kIn, int kTurns, int kRowThreads>
__device__ __forceinline__ void move_flat(uint4 (&mem)[kTurns * kRowGroups + kTurns + 1], uint8_t* global, int bytes) {
    using U = std::conditional_t<kSize == 4, uint32_t, std::conditional_t<kSize == 2, uint16_t, uint8_t>>;
    const int skew = (int)(reinterpret_cast<uintptr_t>(global) & 15), end = skew + bytes;
    uint4* g = reinterpret_cast<uint4*>(global - skew);
    // whole vectors [lo, hi)
    const int lo = skew ? 1 : 0, hi = end >> 4;
#pragma unroll
    for (int k = 0; k < kTurns * kRowGroups / kRowThreads + 1; ++k) {
        const int i = threadIdx.x + k * kRowThreads;
        if (i >= lo && i < hi) kIn ? mem[i] = g[i] : g[i] = mem[i];
    }
    // the ends: the first threads have the values before lo and from hi on
    U* m = reinterpret_cast<U*>(mem);
    U* v = reinterpret_cast<U*>(g);
    constexpr int kPer = 16 / kSize;
    if (threadIdx.x < 2 * kPer) {
        const int vec = threadIdx.x < kPer ? 0 : hi, i = vec * kPer + (threadIdx.x & (kPer - 1));
        // a first vector that is no whole one, and the last one's part (once, where both are the same)
        if ((threadIdx.x < kPer ? lo == 1 : hi >= lo) && i * kSize >= skew && i * kSize < end) kIn ? m[i] = v[i] : v[i] = m[i];
    }
}

// Any width and alignment. A block has kRowGroups groups one after the other, whose values are contiguous in
// memory whatever the rows' length: they go through shared memory, so that global memory is moved 16 bytes
// at a time, and a thread has one group there or two (per_thread), which start anywhere. It takes a group's quads, and the
// values of a quad, in an order that goes by its lane, so that the lanes' values lie in different banks.
// `per_row`: groups of a row.
template <typename T, bool kPack>
__global__ void __launch_bounds__(kRowGroups / per_thread<T, kPack>())
    rows_kernel(T* __restrict__ x, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t groups, int K, Divisor per_row) {
    constexpr int kPer = per_thread<T, kPack>(), kRowThreads = kRowGroups / kPer;
    // one vector for the offset from a boundary; a short last group is looked at as a whole one
    __shared__ uint4 x_mem[sizeof(T) * kRowGroups + sizeof(T) + 1], c_mem[kRowGroups + 2];
    static_assert(kCkptGroup == sizeof(uint4), "a thread's codes are one vector");
    pdl_wait();
    pdl_trigger();
    const int64_t g0 = (int64_t)blockIdx.x * kRowGroups, row0 = groups <= INT32_MAX ? per_row.of((int)g0) : g0 / per_row.d;
    const int first = (int)(g0 - row0 * per_row.d), n = (int)min((int64_t)kRowGroups, groups - g0);
    // the i-th group's first value from the first group's, and its length
    auto start = [&](int i, int& length) {
        const int row = per_row.of(first + i), col = (first + i - row * per_row.d) * kCkptGroup;
        length = min(kCkptGroup, K - col);
        return row * K + col - first * kCkptGroup;
    };
    int length;
    const int values = start(n - 1, length) + length;
    const int64_t at = row0 * K + (int64_t)first * kCkptGroup;
    uint8_t* xg = reinterpret_cast<uint8_t*>(x + at);
    uint8_t* cg = codes + at;
    const int lane = threadIdx.x & 31;
    uint32_t bytes[kPer] = {};
    if (kPack) {
        move_flat<sizeof(T), true, sizeof(T), kRowThreads>(x_mem, xg, values * (int)sizeof(T));
    } else {
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            if (threadIdx.x + k * kRowThreads < n) bytes[k] = scales[g0 + threadIdx.x + k * kRowThreads];
        move_flat<1, true, 1, kRowThreads>(c_mem, cg, values);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = threadIdx.x + k * kRowThreads;
        uint32_t byte = bytes[k];
        const int s = start(i, length);
        if (i >= n) length = 0;
        // indices, and not pointers, so that every access is one of shared memory
        T* xm = reinterpret_cast<T*>(x_mem);
        uint8_t* cm = reinterpret_cast<uint8_t*>(c_mem);
        const int xs = (int)(reinterpret_cast<uintptr_t>(xg) & 15) / (int)sizeof(T) + s;
        const int cs = (int)(reinterpret_cast<uintptr_t>(cg) & 15) + s;
        // fp32: groups are 16 words apart, so lanes 0, 2, 4, 6 take different quads, lanes 8 apart other values of
        // a quad; 16 bits, 8 words apart: lanes 0, 4, 8, 12 and lanes 16 apart take different quads. The codes'
        // groups are 4 words apart: lanes 8 apart take different quads
        const int quad = sizeof(T) == 4 ? (lane >> 1) + (lane >> 3) : (lane >> 2) + (lane >> 4);
        const int turn = sizeof(T) == 4 ? lane >> 3 : 0;
        const int in_quad[4] = {turn, (turn + 1) & 3, (turn + 2) & 3, (turn + 3) & 3};
        // whole: no lane of the warp has a short group, so that nothing is compared with its length
        auto group = [&](auto whole) {
            auto in = [&](int e) { return decltype(whole)::value || e < length; };
            if (kPack) {
                uint32_t amax = 0;
                float v[kCkptGroup];
                if constexpr (sizeof(T) == 2) {
                    // words, and the next one where the group starts in the middle of one, in order; the
                    // values' bits are compared two at a time
                    const uint32_t* words = reinterpret_cast<const uint32_t*>(x_mem);
                    const uint32_t shift = 16 * (uint32_t)(xs & 1);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int base = ((quad + q) & 3) * 4;
                        const uint32_t* w = words + ((xs + base) >> 1);
                        const uint32_t w0 = w[0], w1 = w[1], w2 = w[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint32_t two = __funnelshift_r(j ? w1 : w0, j ? w2 : w1, shift);
                            if (!in(base + 2 * j)) two = 0;
                            if (!in(base + 2 * j + 1)) two &= 0xffff;
                            amax = __vmaxu2(amax, two & 0x7fff7fffu);
                            const float2 f = unpack2<T>(two);
                            v[4 * q + 2 * j] = f.x;
                            v[4 * q + 2 * j + 1] = f.y;
                        }
                    }
                    amax = max(amax >> 16, amax & 0xffff);
                    amax = abs_bits(unpack2<T>(amax).x);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int base = ((quad + q) & 3) * 4;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float u = to_f32(xm[xs + base + in_quad[j]]);
                            v[4 * q + j] = in(base + in_quad[j]) ? u : 0.f;
                            amax = max(amax, abs_bits(v[4 * q + j]));
                        }
                    }
                }
                byte = ckpt_byte(amax);
                const float inv = ckpt_inverse(byte);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int base = ((quad + q) & 3) * 4;
                    uint32_t c = ckpt_encode4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3], inv);
                    if (sizeof(T) == 4) c = __funnelshift_l(c, c, 8 * turn);  // back in order
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (in(base + j)) cm[cs + base + j] = (uint8_t)(c >> 8 * j);
                }
            } else {
                const float scale = ckpt_scale(byte);
                const uint32_t* words = reinterpret_cast<const uint32_t*>(c_mem);
                const uint32_t shift = 8 * (uint32_t)(cs & 3);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int at_quad = (quad + q) & 3, base = at_quad * 4;
                    uint32_t c = __funnelshift_r(words[(cs >> 2) + at_quad], words[(cs >> 2) + at_quad + 1], shift);
                    if (sizeof(T) == 4) c = __funnelshift_r(c, c, 8 * turn);
                    float v[4];
                    ckpt_decode4<T>(c, scale, v);
                    bool stored = false;
                    if constexpr (sizeof(T) == 2) if (decltype(whole)::value) {
                        // two words, or half a word, a word and half a word
                        stored = true;
                        const uint32_t lo = pack2_f32<T>(v[0], v[1]), hi = pack2_f32<T>(v[2], v[3]);
                        const int to = xs + base;
                        uint16_t* halves = reinterpret_cast<uint16_t*>(x_mem);
                        uint32_t* pairs = reinterpret_cast<uint32_t*>(x_mem) + (to >> 1);
                        if (to & 1) {
                            halves[to] = (uint16_t)lo;
                            pairs[1] = __funnelshift_r(lo, hi, 16);
                            halves[to + 3] = (uint16_t)(hi >> 16);
                        } else {
                            pairs[0] = lo;
                            pairs[1] = hi;
                        }
                    }
                    if (!stored) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (in(base + in_quad[j])) xm[xs + base + in_quad[j]] = from_f32<T>(v[j]);
                    }
                }
            }
        };
        if (__all_sync(0xffffffffu, length == kCkptGroup))
            group(std::true_type());
        else
            group(std::false_type());
        if (kPack && i < n) scales[g0 + i] = (uint8_t)byte;
    }
    __syncthreads();
    if (kPack)
        move_flat<1, false, 1, kRowThreads>(c_mem, cg, values);
    else
        move_flat<sizeof(T), false, sizeof(T), kRowThreads>(x_mem, xg, values * (int)sizeof(T));
}

// Sizes of both directions; the groups' number.
bool sizes_ok(int64_t M, int K, int dtype, int64_t& groups) {
    if (M < 0 || K < 1 || K > 1 << 30 || !dtype_bytes(dtype) || M > ((int64_t)1 << 40) / K) return false;  // grids
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
            const int per_row = (K + kCkptGroup - 1) / kCkptGroup;
            launch_k(rows_kernel<T, true>, (unsigned)((groups + kRowGroups - 1) / kRowGroups),
                     kRowGroups / per_thread<T, true>(), 0, s, const_cast<T*>(in), codes, scales, groups, K, Divisor{per_row, magic_of(per_row)});
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
            const int per_row = (K + kCkptGroup - 1) / kCkptGroup;
            launch_k(rows_kernel<T, false>, (unsigned)((groups + kRowGroups - 1) / kRowGroups),
                     kRowGroups / per_thread<T, false>(), 0, s, out, const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales), groups, K, Divisor{per_row, magic_of(per_row)});
        }
        note_launches(1);
        return launch_status();
    });
}

}  // extern "C"
