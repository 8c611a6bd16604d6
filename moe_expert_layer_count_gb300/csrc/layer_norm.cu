// Layer norm over the last dimension and its gradients.
//   forward   mean = sum x / K, rstd = 1 / sqrt(sum (x - mean)^2 / K + eps),
//             y = (x - mean) * rstd * weight + bias
//   backward  with xh = (x - mean) * rstd, g = dy * weight:
//             dx = rstd * (g - sum g / K - xh * sum(g xh) / K)
//             d_weight = sum over rows of dy xh, d_bias = sum over rows of dy
// Memory is their floor: x (and dy) are read once, kept in registers in their own type
// while the row's sums are taken, and written from there. Rows that start on 16-byte
// boundaries move 16 bytes at a time (V values), others one value at a time.
// A thread has 16 columns, their parameters in registers; a row takes K / 16 threads, and a
// block every G-th row, the next ones on their way to shared memory while a row is summed.
// The backward pass keeps the sums of d_weight and d_bias for its columns in registers; the
// blocks' partial sums are added in a fixed order by a second kernel.
// What bounds them now is latency at few warps (16384 x 2048 bf16: 23-29 % of the warps that fit, an instruction
// in 55-57 % of the issue slots, no pipe above a third, DRAM at 46-59 %): the registers that hold a row, and
// in the backward pass the two column sums, are what limits the warps.
// Rows longer than 1024 threads' columns (or the ring) take the looping kernels, which read
// them again from L2.
#include <atomic>
#include <type_traits>

#include "elem.cuh"

namespace moe {
namespace {

constexpr int kRowThreads = 256;
constexpr int kColParts = 152;  // row ranges of the looping kernels' partial sums

// Columns of a thread: their weights (and biases, or the two column sums) stay in registers.
template <int V>
constexpr int cols_of = V == 1 ? 8 : 16;

// How the row kernels divide rows of K values: the threads of a row, the rows of a block (as many
// as fill `block` threads) and the blocks that an SM holds at once with `resident` threads.
struct Rows {
    int threads, per_block, per_sm;
    Rows(int K, int columns, int block, int resident) {
        threads = ((K + columns - 1) / columns + 31) / 32 * 32;
        per_block = threads < block ? block / threads : 1;
        const int n = resident / (threads * per_block);
        per_sm = n > 1 ? n : 1;
    }
};
// The most threads of the small variant of the forward kernel.
template <int V>
constexpr int most_threads = V == 1 ? 256 : 128;
template <int V>
Rows forward_rows(int K) { return Rows(K, cols_of<V>, V == 1 ? 1 : 128, V == 1 ? 1280 : 640); }
template <int V>
Rows backward_rows(int K) { return Rows(K, cols_of<V>, V == 1 ? 1 : 256, V == 1 ? 1120 : 512); }

constexpr int kMostColumns = 1 << 24;
constexpr int kSms = 152;
// Partial sums of the backward kernel, its blocks: each is 2 K floats that the fold reads again.
template <int V>
int parts_of(int K) { return kSms * backward_rows<V>(K).per_sm; }

// Sum over the block, the same value in every thread. `s`: one float per warp.
__device__ __forceinline__ float block_sum(float v, float* s) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = warp_sum((threadIdx.x & 31) < kRowThreads / 32 ? s[threadIdx.x & 31] : 0.f);
    __syncthreads();
    return v;
}

// Two fp32 values; the arithmetic on them is packed (one instruction for both).
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
template <typename T>
__device__ __forceinline__ uint32_t bits_of(T v) {
    if constexpr (sizeof(T) == 4)
        return __float_as_uint(v);
    else
        return *reinterpret_cast<const uint16_t*>(&v);
}

// One thread's share of a row: IT vectors of V values, held as the 32-bit words they are loaded in
// (V = 1: as fp32). A warp has 32 * IT vectors in a row; a lane every 32nd of them, from vector
// `base` on, so that their addresses differ by constants. The share is used as pairs of values,
// whichever vectors these lie in.
template <typename T, int V, int IT>
struct Share {
    static constexpr int kPairs = V * IT / 2;
    static constexpr int kWords = V > 1 ? V * (int)sizeof(T) / 4 : 1;  // of a vector
    uint32_t w[IT * kWords];
    static __device__ __forceinline__ int base() { return (threadIdx.x & ~31u) * IT + (threadIdx.x & 31); }
    // whether this warp's vectors all lie within K values and can be moved as such
    static __device__ __forceinline__ bool whole(int K, bool vec) {
        return ((int)(threadIdx.x >> 5) + 1) * 32 * IT * V <= K && (V == 1 || vec);
    }
    // values at or past K are zero; `vec`: the row starts on a 16-byte boundary (else one load per
    // value, the same values to the same threads: results do not depend on the alignment); `whole`: as
    // above, the way without checks
    __device__ __forceinline__ void load(const T* __restrict__ row, int K, int base, bool vec, bool whole) {
        row += base * V;
        if (V > 1 && whole) {
#pragma unroll
            for (int i = 0; i < IT; ++i)
#pragma unroll
                for (int j = 0; j < kWords; j += 4) {
                    const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(row + i * 32 * V) + j);
                    uint32_t* o = w + i * kWords + j;
                    o[0] = u.x, o[1] = u.y, o[2] = u.z, o[3] = u.w;
                }
            return;
        }
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            uint32_t* o = w + i * kWords;
            const T* at = row + i * 32 * V;
            if (!whole && (base + i * 32) * V >= K) {
#pragma unroll
                for (int j = 0; j < kWords; ++j) o[j] = 0;
            } else if constexpr (V == 1) {
                o[0] = __float_as_uint(to_f32(at[0]));
            } else if (vec) {
#pragma unroll
                for (int j = 0; j < kWords; j += 4) {
                    const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(at) + j);
                    o[j] = u.x, o[j + 1] = u.y, o[j + 2] = u.z, o[j + 3] = u.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < kWords; ++j)
                    o[j] = sizeof(T) == 4 ? bits_of(at[j]) : bits_of(at[2 * j]) | bits_of(at[2 * j + 1]) << 16;
            }
        }
    }
    __device__ __forceinline__ void store(T* __restrict__ row, int K, int base, bool vec, bool whole) const {
        row += base * V;
        if constexpr (V > 1) {
            if (whole) {
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    const uint32_t* o = w + i * kWords;
                    *reinterpret_cast<uint4*>(row + i * 32 * V) = make_uint4(o[0], o[1], o[2], o[3]);
                }
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const uint32_t* o = w + i * kWords;
            T* at = row + i * 32 * V;
            if (!whole && (base + i * 32) * V >= K) continue;
            if constexpr (V == 1) {
                at[0] = from_f32<T>(__uint_as_float(o[0]));
            } else if (vec) {
                *reinterpret_cast<uint4*>(at) = make_uint4(o[0], o[1], o[2], o[3]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if constexpr (sizeof(T) == 4)
                        at[j] = __uint_as_float(o[j]);
                    else
                        reinterpret_cast<uint16_t*>(at)[j] = (uint16_t)(o[j / 2] >> (j % 2 * 16));
                }
            }
        }
    }
    __device__ __forceinline__ float2 get(int p) const {
        if constexpr (V == 1 || sizeof(T) == 4)
            return make_float2(__uint_as_float(w[2 * p]), __uint_as_float(w[2 * p + 1]));
        else if constexpr (std::is_same<T, bf16>::value)
            return make_float2(__uint_as_float(w[p] << 16), __uint_as_float(w[p] & 0xffff0000u));
        else
            return __half22float2(*reinterpret_cast<const __half2*>(&w[p]));
    }
    __device__ __forceinline__ void set(int p, float2 f) {
        if constexpr (V == 1 || sizeof(T) == 4) {
            w[2 * p] = __float_as_uint(f.x);
            w[2 * p + 1] = __float_as_uint(f.y);
        } else if constexpr (std::is_same<T, bf16>::value) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
            w[p] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __half2 h = __floats2half2_rn(f.x, f.y);
            w[p] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    // the columns of a pair's two values
    static __device__ __forceinline__ int first(int p, int base) {
        return V > 1 ? (base + 2 * p / V * 32) * V + 2 * p % V : base + 2 * p * 32;
    }
    static __device__ __forceinline__ int second(int p, int base) { return first(p, base) + (V > 1 ? 1 : 32); }
};

// The warps' sums of N rows (or rows of pairs), 32 places each: read four values at a time, so on
// 16-byte boundaries.
template <typename F, int N>
struct alignas(16) WarpSums {
    F v[N * 32];
};

// Sums over the threads of a row (blockDim.x of them, a row per threadIdx.y), the same in all.
// `sums`: a place per row, other ones at the next call, so that one barrier is enough.
template <int N>
__device__ __forceinline__ float row_sum(float v, WarpSums<float, N>& sums) {
    static_assert(alignof(WarpSums<float, N>) >= alignof(float4), "read as float4");
    v = warp_sum(v);
    if (blockDim.x == 32) return v;
    float* s = sums.v + threadIdx.y * 32;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    if (blockDim.x == 128) {
        const float4 f = *reinterpret_cast<const float4*>(s);
        return (f.x + f.y) + (f.z + f.w);
    }
    return warp_sum((threadIdx.x & 31) < (blockDim.x >> 5) ? s[threadIdx.x & 31] : 0.f);
}
__device__ __forceinline__ float2 warp_sum2(float2 v) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v = __fadd2_rn(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
    return v;
}
// The sums of kR rows at once: one barrier, and their exchanges overlap.
template <int kR, int N>
__device__ __forceinline__ void row_sums(float2 (&v)[kR], WarpSums<float2, N>& sums) {
    static_assert(alignof(WarpSums<float2, N>) >= alignof(float4), "read as float4");
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int k = 0; k < kR; ++k)
            v[k] = __fadd2_rn(v[k], make_float2(__shfl_xor_sync(0xffffffffu, v[k].x, o), __shfl_xor_sync(0xffffffffu, v[k].y, o)));
    if (blockDim.x == 32) return;
    float2* s = sums.v + threadIdx.y * 32 * kR;
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
#pragma unroll
        for (int k = 0; k < kR; ++k) s[k * 32 + (threadIdx.x >> 5)] = v[k];
    }
    __syncthreads();
    if (blockDim.x == 128) {
#pragma unroll
        for (int k = 0; k < kR; ++k) {
            const float4 f = *reinterpret_cast<const float4*>(s + k * 32), g = *reinterpret_cast<const float4*>(s + k * 32 + 2);
            v[k] = make_float2((f.x + f.z) + (g.x + g.z), (f.y + f.w) + (g.y + g.w));
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < kR; ++k) v[k] = warp_sum2(lane < (int)(blockDim.x >> 5) ? s[k * 32 + lane] : both(0.f));
}

__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ring_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

// A block's next rows, some of them in turn, on their way from global to shared memory by
// cp.async. V > 1: every thread copies and reads only its own share, no barrier is needed.
template <typename T, int V, int IT>
struct Ring {
    static constexpr int kBytes = V * (int)sizeof(T);  // of a vector
    uint8_t* mine;  // this thread's first vector; the others `stride` bytes apart
    int stride;
    __device__ __forceinline__ Ring(uint8_t* smem, int stages, const T*, int64_t, int K) {
        const int n = blockDim.x * blockDim.y;
        mine = smem + (threadIdx.y * blockDim.x + threadIdx.x) * kBytes;
        stride = n * kBytes;
        for (int i = 0; i < stages * IT; ++i)
            if ((Share<T, V, IT>::base() + i % IT * 32) * V >= K)  // what no column fills is zero
                for (int j = 0; j < kBytes / 4; ++j) reinterpret_cast<uint32_t*>(mine + i * stride)[j] = 0;
    }
    // bytes of a stage
    static __host__ __device__ size_t bytes(int K, int threads, int per_block) {
        return (size_t)threads * per_block * IT * kBytes;
    }
    __device__ __forceinline__ void fetch(int stage, const T* __restrict__ row, int K, int base, bool vec, bool whole) {
        row += base * V;
        if (whole) {
#pragma unroll
            for (int i = 0; i < IT; ++i) copy16(mine + (stage * IT + i) * stride, row + i * 32 * V);
            return;
        }
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            if ((base + i * 32) * V >= K) continue;
            uint8_t* to = mine + (stage * IT + i) * stride;
            const T* at = row + i * 32 * V;
            if (vec)
                copy16(to, at);
            else
                for (int j = 0; j < V; ++j) reinterpret_cast<T*>(to)[j] = at[j];
        }
    }
    __device__ __forceinline__ void read(int stage, const T*, int, int, bool, Share<T, V, IT>& s) const {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const uint4 u = *reinterpret_cast<const uint4*>(mine + (stage * IT + i) * stride);
            s.w[4 * i] = u.x, s.w[4 * i + 1] = u.y, s.w[4 * i + 2] = u.z, s.w[4 * i + 3] = u.w;
        }
    }
    static __device__ __forceinline__ void landed() {}
};
// V = 1: the threads of a row copy the 16-byte pieces that it lies in together (a row may start
// anywhere), and read single values from there after a barrier. A piece that is not wholly inside
// the tensor is copied value by value.
template <typename T, int IT>
struct Ring<T, 1, IT> {
    uint8_t* mine;  // this row's first stage
    int stride;     // bytes of a stage of the block
    const T *first, *last;
    __device__ __forceinline__ Ring(uint8_t* smem, int stages, const T* x, int64_t n, int K) : first(x), last(x + n) {
        const int row = row_bytes(K);
        mine = smem + threadIdx.y * row;
        stride = row * blockDim.y;
    }
    static __host__ __device__ int row_bytes(int K) { return (K * (int)sizeof(T) + 15) / 16 * 16 + 16; }
    static __host__ __device__ size_t bytes(int K, int threads, int per_block) { return (size_t)row_bytes(K) * per_block; }
    __device__ __forceinline__ void fetch(int stage, const T* __restrict__ row, int K, int, bool, bool) {
        const T* from = reinterpret_cast<const T*>(reinterpret_cast<uintptr_t>(row) & ~uintptr_t(15));
        constexpr int N = 16 / sizeof(T);
        T* to = reinterpret_cast<T*>(mine + stage * stride);
        for (int c = threadIdx.x * N; from + c < row + K; c += blockDim.x * N) {
            if (from + c >= first && from + c + N <= last)
                copy16(to + c, from + c);
            else
                for (int j = 0; j < N; ++j)
                    if (from + c + j >= row && from + c + j < row + K) to[c + j] = from[c + j];
        }
    }
    __device__ __forceinline__ void read(int stage, const T* row, int K, int base, bool whole, Share<T, 1, IT>& s) const {
        const T* at = reinterpret_cast<const T*>(mine + stage * stride + (reinterpret_cast<uintptr_t>(row) & 15)) + base;
#pragma unroll
        for (int i = 0; i < IT; ++i) s.w[i] = whole || base + i * 32 < K ? __float_as_uint(to_f32(at[i * 32])) : 0u;
    }
    static __device__ __forceinline__ void landed() {
        if (blockDim.x == 32)
            __syncwarp();
        else
            __syncthreads();
    }
};

template <int V>
constexpr int its = cols_of<V> / V;  // vectors of a thread
// S, below: the stages of a block's ring. 0 (backward only): none -- single fp32 values, coalesced
// as they are, are loaded straight into registers, one row ahead (30011 x 1111: 92 us, with a
// ring 109).

// Block b takes the rows b * blockDim.y + threadIdx.y, then gridDim.x * blockDim.y further on.
struct Turns {
    int64_t row, step;
    int all, mine;  // rows of the block's first row of threads (each row of threads goes as far), of this one
    __device__ __forceinline__ explicit Turns(int64_t M) {
        const int64_t first = (int64_t)blockIdx.x * blockDim.y;
        step = (int64_t)gridDim.x * blockDim.y;
        row = first + threadIdx.y;
        all = (int)((M - first + step - 1) / step);
        mine = row < M ? (int)((M - row + step - 1) / step) : 0;
    }
};

// sum / K in one rounding, from the reciprocal of K; infinities and NaN as they are.
__device__ __forceinline__ float mean_of(float sum, float K, float inv_k) {
    const float q = div_rn_by(sum, K, inv_k);
    return fabsf(sum) <= 3.402823466e38f ? q : sum;
}

// kThreads, here and below: the most threads of a block.
template <typename T, typename P, int V, int S, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 128 ? 5 : kThreads == 256 ? 4 : 1)
    layer_norm_rows_kernel(const T* x, int64_t M, int K, float inv_k, const P* __restrict__ weight, const P* __restrict__ bias,
                           float eps, T* y, float* __restrict__ mean_out, float* __restrict__ rstd_out, bool vec) {
    using Sh = Share<T, V, its<V>>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ WarpSums<float, 4> s[4];  // at most four rows a block
    pdl_wait();
    pdl_trigger();
    const int tx = threadIdx.x;
    Share<P, V, its<V>> w, bs;
    const int base = Sh::base();
    const bool whole = Sh::whole(K, vec);
    w.load(weight, K, base, vec, whole);
    bs.load(bias ? bias : weight, bias ? K : 0, base, vec, false);  // no bias: zeros
    const Turns turn(M);
    Sh xs;
    Ring<T, V, its<V>> ring(smem, S, x, M * K, K);
    const int64_t hop = turn.step * K;
    int64_t here = turn.row * K, ahead = here;  // this row's values, and the next row's to fetch
    auto fetch = [&](int i) {
        if (i < turn.mine) ring.fetch(i % S, x + ahead, K, base, vec, whole);
        ring_commit();
        ahead += hop;
    };
    for (int i = 0; i < S - 1; ++i) fetch(i);
    int at = 0;
    int64_t q = turn.row;
    for (int i = 0; i < turn.all; ++i, q += turn.step, here += hop) {
        fetch(i + S - 1);
        ring_wait<S - 1>();
        ring.landed();
        ring.read(i % S, x + here, K, base, whole, xs);
        float2 a = both(0.f);
#pragma unroll
        for (int p = 0; p < Sh::kPairs; ++p) a = __fadd2_rn(a, xs.get(p));
        const float mean = mean_of(row_sum(a.x + a.y, s[at]), (float)K, inv_k);
        a = both(0.f);
        if (whole) {
#pragma unroll
            for (int p = 0; p < Sh::kPairs; ++p) {
                const float2 d = __fadd2_rn(xs.get(p), both(-mean));
                a = __ffma2_rn(d, d, a);
            }
        } else {
#pragma unroll
            for (int p = 0; p < Sh::kPairs; ++p) {
                float2 d = __fadd2_rn(xs.get(p), both(-mean));
                if (Sh::first(p, base) >= K) d.x = 0.f;
                if (Sh::second(p, base) >= K) d.y = 0.f;
                a = __ffma2_rn(d, d, a);
            }
        }
        const float rstd = rsqrtf(fmaf(row_sum(a.x + a.y, s[at + 1]), inv_k, eps));
        at ^= 2;
        if (i < turn.mine) {
#pragma unroll
            for (int p = 0; p < Sh::kPairs; ++p) {
                const float2 h = __fmul2_rn(__fadd2_rn(xs.get(p), both(-mean)), both(rstd));
                xs.set(p, __ffma2_rn(h, w.get(p), bs.get(p)));
            }
            xs.store(y + here, K, base, vec, whole);
            if (tx == 0) {
                if (mean_out) mean_out[q] = mean;
                if (rstd_out) rstd_out[q] = rstd;
            }
        }
    }
    ring_wait<0>();
}

// Rows that the backward pass takes at once: two where a thread has the registers for it, so that
// the wait at the barrier is shared.
template <typename T, int V, int S, int kThreads>
constexpr int rows_at_once = sizeof(T) == 2 && V > 1 && S >= 4 && kThreads <= 512 ? 2 : 1;

// x - mean is one subtraction, so that its error does not grow with the mean; x * rstd - mean * rstd in one
// rounding would save an instruction a pair (8192 x 2048 bf16: 23.8 against 23.9 us) and at a mean of 1000
// spreads gives the weight's gradient an error of 2e-5.
template <typename T, typename P, int V, int S, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads > 256 ? 1 : 2)
    layer_norm_backward_kernel(const T* dy, const T* __restrict__ x, int64_t M, int K, float inv_k,
                               const P* __restrict__ weight, const float* __restrict__ mean_in,
                               const float* __restrict__ rstd_in, T* dx, float* __restrict__ parts, bool vec) {
    using Sh = Share<T, V, its<V>>;
    __shared__ WarpSums<float2, 2 * 8> s[2];  // two rows at once, at most eight rows a block
    extern __shared__ __align__(16) uint8_t smem[];  // the ring; at the end 2 K floats where a block has several rows
    pdl_wait();
    pdl_trigger();
    const int tx = threadIdx.x, threads = blockDim.x;
    Share<P, V, its<V>> w;
    const int base = Sh::base();
    const bool whole = Sh::whole(K, vec);
    w.load(weight, K, base, vec, whole);
    float2 dw[Sh::kPairs], db[Sh::kPairs];
#pragma unroll
    for (int p = 0; p < Sh::kPairs; ++p) dw[p] = db[p] = both(0.f);
    const Turns turn(M);
    constexpr int kR = rows_at_once<T, V, S, kThreads>;
    constexpr int kAhead = S > 0 ? S - kR : 1;  // rows fetched ahead
    Sh xs[kR], ds[kR];
    using R = Ring<T, V, its<V>>;
    R rx(smem, S, x, M * K, K), rd(smem + S * R::bytes(K, threads, blockDim.y), S, dy, M * K, K);
    const int64_t hop = turn.step * K;
    int64_t here = turn.row * K, ahead = here;  // this row's values, and the next row's to fetch
    Sh xn, dn;  // S = 0
    auto fetch = [&](int i) {
        const bool in = i < turn.mine;
        if constexpr (S > 0) {
            if (in) {
                rx.fetch(i % S, x + ahead, K, base, vec, whole);
                rd.fetch(i % S, dy + ahead, K, base, vec, whole);
            }
            ring_commit();
        } else {
            if (in) {
                xn.load(x + ahead, K, base, false, whole);
                dn.load(dy + ahead, K, base, false, whole);
            }
        }
        ahead += hop;
    };
    float mean_n[kR], rstd_n[kR];
    int64_t q = turn.row;
    auto statistics = [&](int i) {
#pragma unroll
        for (int k = 0; k < kR; ++k) {
            mean_n[k] = i + k < turn.mine ? __ldg(mean_in + q) : 0.f;
            rstd_n[k] = i + k < turn.mine ? __ldg(rstd_in + q) : 0.f;
            q += turn.step;
        }
    };
    for (int i = 0; i < kAhead; ++i) fetch(i);
    statistics(0);
    for (int i = 0; i < turn.all; i += kR) {
        if constexpr (S > 0) {
#pragma unroll
            for (int k = 0; k < kR; ++k) fetch(i + kAhead + k);
            ring_wait<kAhead>();
            R::landed();
#pragma unroll
            for (int k = 0; k < kR; ++k) {
                rx.read((i + k) % S, x + here + k * hop, K, base, whole, xs[k]);
                rd.read((i + k) % S, dy + here + k * hop, K, base, whole, ds[k]);
            }
        } else {
            xs[0] = xn;
            ds[0] = dn;
            if (i + 1 < turn.all) fetch(i + 1);
        }
        float rstd[kR], mean[kR];
        float2 a[kR], b[kR];
#pragma unroll
        for (int k = 0; k < kR; ++k) {
            rstd[k] = rstd_n[k];
            mean[k] = mean_n[k];
            a[k] = b[k] = both(0.f);
        }
        statistics(i + kR);
#pragma unroll
        for (int k = 0; k < kR; ++k)
            if (i + k < turn.mine) {
#pragma unroll
                for (int p = 0; p < Sh::kPairs; ++p) {
                    const float2 d = ds[k].get(p), h = __fmul2_rn(__fadd2_rn(xs[k].get(p), both(-mean[k])), both(rstd[k])),
                                 g = __fmul2_rn(d, w.get(p));
                    a[k] = __fadd2_rn(a[k], g);
                    b[k] = __ffma2_rn(g, h, b[k]);
                    dw[p] = __ffma2_rn(d, h, dw[p]);
                    db[p] = __fadd2_rn(db[p], d);
                }
            }
#pragma unroll
        for (int k = 0; k < kR; ++k) a[k] = make_float2(a[k].x + a[k].y, b[k].x + b[k].y);
        row_sums<kR>(a, s[i / kR & 1]);
#pragma unroll
        for (int k = 0; k < kR; ++k)
            if (i + k < turn.mine) {
                // rstd * (g - a - (x - mean) (rstd b))
                const float2 c = both(-a[k].x * inv_k * rstd[k]), e = both(-a[k].y * inv_k * rstd[k]);
#pragma unroll
                for (int p = 0; p < Sh::kPairs; ++p) {
                    const float2 h = __fadd2_rn(xs[k].get(p), both(-mean[k])), g = __fmul2_rn(ds[k].get(p), w.get(p));
                    xs[k].set(p, __ffma2_rn(__ffma2_rn(h, e, g), both(rstd[k]), c));
                }
                xs[k].store(dx + here + k * hop, K, base, vec, whole);
            }
        here += kR * hop;
    }
    if constexpr (S > 0) ring_wait<0>();
    float* cols = reinterpret_cast<float*>(smem);
    float* out = blockDim.y > 1 ? cols : parts + (int64_t)blockIdx.x * 2 * K;
    for (int y = 0; y < blockDim.y; ++y) {  // the block's rows one after the other
        if (blockDim.y > 1) __syncthreads();
        if (threadIdx.y == y) {
#pragma unroll
            for (int p = 0; p < Sh::kPairs; ++p) {
                const int c = Sh::first(p, base), c2 = Sh::second(p, base);
                if (c < K) {
                    out[c] = dw[p].x + (y ? out[c] : 0.f);
                    out[K + c] = db[p].x + (y ? out[K + c] : 0.f);
                }
                if (c2 < K) {
                    out[c2] = dw[p].y + (y ? out[c2] : 0.f);
                    out[K + c2] = db[p].y + (y ? out[K + c2] : 0.f);
                }
            }
        }
    }
    if (blockDim.y == 1) return;
    __syncthreads();
    out = parts + (int64_t)blockIdx.x * 2 * K;
    for (int c = threadIdx.y * threads + tx; c < 2 * K; c += threads * blockDim.y) out[c] = cols[c];
}

template <typename T, typename P>
__global__ void __launch_bounds__(kRowThreads)
    layer_norm_kernel(const T* x, int K, const P* __restrict__ weight, const P* __restrict__ bias, float eps, T* y,
                      float* __restrict__ mean_out, float* __restrict__ rstd_out) {
    __shared__ float s[kRowThreads / 32];
    pdl_wait();
    pdl_trigger();
    const T* row = x + (int64_t)blockIdx.x * K;
    T* out = y + (int64_t)blockIdx.x * K;
    float a = 0.f;
    for (int i = threadIdx.x; i < K; i += kRowThreads) a += to_f32(row[i]);
    const float mean = block_sum(a, s) / K;
    a = 0.f;
    for (int i = threadIdx.x; i < K; i += kRowThreads) {
        const float d = to_f32(row[i]) - mean;
        a = fmaf(d, d, a);
    }
    const float rstd = 1.f / sqrtf(block_sum(a, s) / K + eps);
    for (int i = threadIdx.x; i < K; i += kRowThreads)
        out[i] = from_f32<T>(fmaf((to_f32(row[i]) - mean) * rstd, to_f32(weight[i]), bias ? to_f32(bias[i]) : 0.f));
    if (threadIdx.x == 0) {
        if (mean_out) mean_out[blockIdx.x] = mean;
        if (rstd_out) rstd_out[blockIdx.x] = rstd;
    }
}

template <typename T, typename P>
__global__ void __launch_bounds__(kRowThreads)
    layer_norm_dx_kernel(const T* dy, const T* __restrict__ x, int K, const P* __restrict__ weight,
                         const float* __restrict__ mean_in, const float* __restrict__ rstd_in, T* dx) {
    __shared__ float s[kRowThreads / 32];
    pdl_wait();
    pdl_trigger();
    const int64_t base = (int64_t)blockIdx.x * K;
    const float mean = mean_in[blockIdx.x], rstd = rstd_in[blockIdx.x];
    float a = 0.f, b = 0.f;
    for (int i = threadIdx.x; i < K; i += kRowThreads) {
        const float g = to_f32(dy[base + i]) * to_f32(weight[i]);
        a += g;
        b = fmaf(g, (to_f32(x[base + i]) - mean) * rstd, b);
    }
    a = block_sum(a, s) / K;
    b = block_sum(b, s) / K;
    for (int i = threadIdx.x; i < K; i += kRowThreads) {
        const float g = to_f32(dy[base + i]) * to_f32(weight[i]);
        dx[base + i] = from_f32<T>(rstd * (g - a - (to_f32(x[base + i]) - mean) * rstd * b));
    }
}

// Block (x, p): columns [32 x, 32 x + 32) summed over the p-th range of rows.
template <typename T>
__global__ void __launch_bounds__(256)
    layer_norm_cols_kernel(const T* __restrict__ dy, const T* __restrict__ x, int64_t M, int K,
                           const float* __restrict__ mean, const float* __restrict__ rstd, float* __restrict__ parts) {
    __shared__ float s[2][8][33];
    pdl_wait();
    pdl_trigger();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + tx;
    const int64_t per = (M + gridDim.y - 1) / gridDim.y;
    const int64_t r0 = per * blockIdx.y, r1 = r0 + per < M ? r0 + per : M;
    float dw = 0.f, db = 0.f;
    if (c < K)
        for (int64_t r = r0 + ty; r < r1; r += 8) {
            const float d = to_f32(dy[r * K + c]);
            dw = fmaf(d, (to_f32(x[r * K + c]) - mean[r]) * rstd[r], dw);
            db += d;
        }
    s[0][ty][tx] = dw;
    s[1][ty][tx] = db;
    __syncthreads();
    if (ty < 2 && c < K) {
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) a += s[ty][i][tx];
        parts[((int64_t)blockIdx.y * 2 + ty) * K + c] = a;
    }
}

// Adds the n partial sums of 32 columns of d_weight or d_bias (blockIdx.y): 32 threads per
// column, each every 32nd part, then their sums in order.
template <typename P>
__global__ void __launch_bounds__(1024)
    layer_norm_fold_kernel(const float* __restrict__ parts, int n, int K, P* __restrict__ dw, P* __restrict__ db) {
    __shared__ float s[32][33];
    pdl_wait();
    pdl_trigger();
    const int tx = threadIdx.x, ty = threadIdx.y;
    const int c = blockIdx.x * 32 + tx;
    float a = 0.f;
    if (c < K) {
#pragma unroll 8
        for (int p = ty; p < n; p += 32) a += parts[((int64_t)p * 2 + blockIdx.y) * K + c];
    }
    s[ty][tx] = a;
    __syncthreads();
    a = warp_sum(s[tx][ty]);  // column blockIdx.x * 32 + ty
    P* out = blockIdx.y ? db : dw;
    if (tx == 0 && out && blockIdx.x * 32 + ty < K) out[blockIdx.x * 32 + ty] = from_f32<P>(a);
}

bool norm_args_ok(int64_t M, int K, int dtype, int param_dtype) {
    return M >= 0 && M <= INT32_MAX && K >= 1 && K <= kMostColumns && dtype_bytes(dtype) && (param_dtype == dtype || param_dtype == MOE_DT_F32);
}

// Calls f with the stages of a ring that has `bytes` a stage in each of `per_sm` blocks, as a
// constant, and returns what it returns; kNoRing where not even two fit.
constexpr int kNoRing = -1;
constexpr size_t kRingRoom = 200 * 1024;
template <bool kRing, typename F>
int with_stages(size_t bytes, int per_sm, F&& f) {
    if constexpr (!kRing) return f(std::integral_constant<int, 0>{});
    const size_t room = kRingRoom / per_sm;
    if (4 * bytes <= room) return f(std::integral_constant<int, 4>{});
    if (3 * bytes <= room) return f(std::integral_constant<int, 3>{});
    if (2 * bytes <= room) return f(std::integral_constant<int, 2>{});
    return kNoRing;
}
// The kernel's shared memory beyond 48 KB needs permission, which is a state of the kernel on the device: given
// once, for the largest ring, and never lowered, so that calls of other widths beside this one do not
// matter.
constexpr int kMaxDevices = 64;
template <auto kKernel, typename... Args>
int launch_ring(unsigned grid, dim3 block, size_t smem, cudaStream_t stream, Args&&... args) {
    static std::atomic<bool> allowed[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MOE_ERR_CUDA;
    if (!allowed[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingRoom) != cudaSuccess) {
            launch_status();
            return MOE_ERR_CUDA;
        }
        allowed[dev].store(true, std::memory_order_release);
    }
    launch_k(kKernel, grid, block, smem, stream, std::forward<Args>(args)...);
    note_launches(1);
    return launch_status();
}

// Calls f(T*, P*) with the element types of x and of the parameters.
template <typename F>
int with_types(int dtype, int param_dtype, F&& f) {
    return with_dtype(dtype, [&](auto* t) {
        if (param_dtype == MOE_DT_F32) return f(t, static_cast<float*>(nullptr));
        return f(t, t);
    });
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

MOE_API int moe_layer_norm(const void* x, int64_t M, int K, int dtype, const void* weight, const void* bias,
                           int param_dtype, float eps, void* y, float* mean, float* rstd, moe_stream_t stream) {
    if (!norm_args_ok(M, K, dtype, param_dtype) || !(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
    if (M == 0) return MOE_OK;
    const int z = dtype_bytes(dtype), zp = dtype_bytes(param_dtype);
    if (!x || !weight || !y || misaligned(x, z) || misaligned(y, z) || misaligned(weight, zp) || misaligned(bias, zp) ||
        misaligned(mean, 4) || misaligned(rstd, 4))
        return MOE_ERR_INVALID_ARG;
    const size_t n = (size_t)M * K * z;
    const size_t nm = mean ? (size_t)M * 4 : 0, nr = rstd ? (size_t)M * 4 : 0, nw = (size_t)K * zp, nb = bias ? nw : 0;
    if ((y != x && overlap(y, n, x, n)) || overlap(y, n, weight, nw) || overlap(y, n, bias, nb)) return MOE_ERR_INVALID_ARG;
    // the statistics, too, are written while other blocks still read
    if (overlap(mean, nm, x, n) || overlap(mean, nm, y, n) || overlap(mean, nm, weight, nw) || overlap(mean, nm, bias, nb) ||
        overlap(rstd, nr, x, n) || overlap(rstd, nr, y, n) || overlap(rstd, nr, weight, nw) || overlap(rstd, nr, bias, nb) ||
        overlap(mean, nm, rstd, nr))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if (int st = check_device(&sms)) return st;
    return with_types(dtype, param_dtype, [&](auto* t, auto* p) {
        using T = std::remove_pointer_t<decltype(t)>;
        using P = std::remove_pointer_t<decltype(p)>;
        constexpr int V = 16 / sizeof(T);
        const bool vec = !misaligned(x, 16) && !misaligned(y, 16) && !misaligned(weight, 16) && !misaligned(bias, 16);
        auto rows = [&](auto vc) -> int {
            constexpr int W = decltype(vc)::value;
            const Rows g = forward_rows<W>(K);
            if (g.threads > 1024) return kNoRing;
            const int64_t blocks = (M + g.per_block - 1) / g.per_block, most = (int64_t)sms * g.per_sm;
            const dim3 block(g.threads, g.per_block);
            const size_t bytes = Ring<T, W, its<W>>::bytes(K, g.threads, g.per_block);
            return with_stages<true>(bytes, g.per_sm, [&](auto sc) {
                constexpr int S = decltype(sc)::value;
                auto go = [&](auto tc) {
                    return launch_ring<layer_norm_rows_kernel<T, P, W, S, decltype(tc)::value>>(
                        (unsigned)(blocks < most ? blocks : most), block, bytes * S, (cudaStream_t)stream,
                        static_cast<const T*>(x), M, K, 1.f / K, static_cast<const P*>(weight), static_cast<const P*>(bias),
                        eps, static_cast<T*>(y), mean, rstd, vec);
                };
                if (g.threads <= most_threads<W>) return go(std::integral_constant<int, most_threads<W>>{});
                if (g.threads <= 512) return go(std::integral_constant<int, 512>{});
                return go(std::integral_constant<int, 1024>{});
            });
        };
        const int st = K % V == 0 ? rows(std::integral_constant<int, V>{}) : rows(std::integral_constant<int, 1>{});
        if (st != kNoRing) return st;
        launch_k(layer_norm_kernel<T, P>, (unsigned)M, kRowThreads, 0, (cudaStream_t)stream, static_cast<const T*>(x), K,
                 static_cast<const P*>(weight), static_cast<const P*>(bias), eps, static_cast<T*>(y), mean, rstd);
        note_launches(1);
        return launch_status();
    });
}

MOE_API size_t moe_layer_norm_workspace_size(int64_t M, int K) {
    if (M < 0 || K < 1 || K > kMostColumns) return 0;
    // whichever way the rows are divided (by their type and alignment), the looping kernels too; never more
    // partial sums than rows, and one for no rows, so that there is a workspace to name
    int n = parts_of<1>(K) > parts_of<8>(K) ? parts_of<1>(K) : parts_of<8>(K);
    if (n < kColParts) n = kColParts;
    if (n > M) n = M > 1 ? (int)M : 1;
    return (size_t)n * 2 * K * sizeof(float);
}

MOE_API int moe_layer_norm_backward(const void* dy, const void* x, int64_t M, int K, int dtype, const void* weight,
                                    int param_dtype, const float* mean, const float* rstd, void* dx, void* d_weight,
                                    void* d_bias, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    if (!norm_args_ok(M, K, dtype, param_dtype) || !d_weight || !workspace || misaligned(workspace, 16))
        return MOE_ERR_INVALID_ARG;
    const int z = dtype_bytes(dtype), zp = dtype_bytes(param_dtype);
    if (misaligned(d_weight, zp) || misaligned(d_bias, zp)) return MOE_ERR_INVALID_ARG;
    if (M > 0 && (!dy || !x || !weight || !mean || !rstd || !dx || misaligned(dy, z) || misaligned(x, z) ||
                  misaligned(dx, z) || misaligned(weight, zp) || misaligned(mean, 4) || misaligned(rstd, 4)))
        return MOE_ERR_INVALID_ARG;
    const size_t n = (size_t)M * K * z;
    if ((dx != dy && overlap(dx, n, dy, n)) || overlap(dx, n, x, n) || overlap(workspace, workspace_bytes, dy, n) ||
        overlap(workspace, workspace_bytes, x, n) || overlap(workspace, workspace_bytes, dx, n))
        return MOE_ERR_INVALID_ARG;
    const size_t need = moe_layer_norm_workspace_size(M, K);
    if (workspace_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
    // dx and the partial sums are written while other blocks still read the weight and the statistics, the
    // column sums (which may lie over any of the inputs) while the partial sums are read
    const size_t nm = (size_t)M * 4, nw = (size_t)K * zp, nb = d_bias ? nw : 0, nin = M > 0 ? nw : 0;
    if (overlap(dx, n, weight, nin) || overlap(dx, n, mean, nm) || overlap(dx, n, rstd, nm) || overlap(dx, n, d_weight, nw) ||
        overlap(dx, n, d_bias, nb) || overlap(workspace, need, weight, nin) || overlap(workspace, need, mean, nm) ||
        overlap(workspace, need, rstd, nm) || overlap(workspace, need, d_weight, nw) || overlap(workspace, need, d_bias, nb) ||
        overlap(d_weight, nw, d_bias, nb))
        return MOE_ERR_INVALID_ARG;
    if (int st = check_device(nullptr)) return st;
    return with_types(dtype, param_dtype, [&](auto* t, auto* p) {
        using T = std::remove_pointer_t<decltype(t)>;
        using P = std::remove_pointer_t<decltype(p)>;
        cudaStream_t s = (cudaStream_t)stream;
        float* parts = static_cast<float*>(workspace);
        int n_parts = 0;
        constexpr int V = 16 / sizeof(T);
        const bool vec = !misaligned(x, 16) && !misaligned(dy, 16) && !misaligned(dx, 16) && !misaligned(weight, 16);
        auto rows = [&](auto vc) -> int {
            constexpr int W = decltype(vc)::value;
            const Rows g = backward_rows<W>(K);
            if (g.threads > 1024) return kNoRing;
            const dim3 block(g.threads, g.per_block);
            const int64_t blocks = (M + g.per_block - 1) / g.per_block;
            n_parts = (int)(blocks < parts_of<W>(K) ? blocks : parts_of<W>(K));
            const size_t bytes = 2 * Ring<T, W, its<W>>::bytes(K, g.threads, g.per_block);
            return with_stages<(W * sizeof(T) != 4)>(bytes, g.per_sm, [&](auto sc) {
                constexpr int S = decltype(sc)::value;
                const size_t sums = g.per_block > 1 ? 2 * K * sizeof(float) : 0;
                auto go = [&](auto tc) {
                    return launch_ring<layer_norm_backward_kernel<T, P, W, S, decltype(tc)::value>>(
                        (unsigned)n_parts, block, bytes * S < sums ? sums : bytes * S, s, static_cast<const T*>(dy),
                        static_cast<const T*>(x), M, K, 1.f / K, static_cast<const P*>(weight), mean, rstd,
                        static_cast<T*>(dx), parts, vec);
                };
                if (g.threads <= 256) return go(std::integral_constant<int, 256>{});
                if (g.threads <= 512) return go(std::integral_constant<int, 512>{});
                return go(std::integral_constant<int, 1024>{});
            });
        };
        // a launch that was refused is not followed by one that reads its results
        if (M > 0) {
            int st = K % V == 0 ? rows(std::integral_constant<int, V>{}) : rows(std::integral_constant<int, 1>{});
            if (st == kNoRing) {
                n_parts = (int)(M < kColParts ? M : kColParts);
                // the column sums read dy before dx, which may be the same buffer, is written
                launch_k(layer_norm_cols_kernel<T>, dim3((unsigned)((K + 31) / 32), (unsigned)n_parts), 256, 0, s,
                         static_cast<const T*>(dy), static_cast<const T*>(x), M, K, mean, rstd, parts);
                note_launches(1);
                if ((st = launch_status()) != MOE_OK) return st;
                launch_k(layer_norm_dx_kernel<T, P>, (unsigned)M, kRowThreads, 0, s, static_cast<const T*>(dy),
                         static_cast<const T*>(x), K, static_cast<const P*>(weight), mean, rstd, static_cast<T*>(dx));
                note_launches(1);
                st = launch_status();
            }
            if (st != MOE_OK) return st;
        }
        launch_k(layer_norm_fold_kernel<P>, dim3((unsigned)((K + 31) / 32), d_bias ? 2 : 1), dim3(32, 32), 0, s, parts, n_parts, K,
                 static_cast<P*>(d_weight), static_cast<P*>(d_bias));
        note_launches(1);
        return launch_status();
    });
}

}  // extern "C"
