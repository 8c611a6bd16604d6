// Layer norm over the last dimension and its gradients.
//   forward   mean = sum x / K, rstd = 1 / sqrt(sum (x - mean)^2 / K + eps),
//             y = (x - mean) * rstd * weight + bias
//   backward  with xh = (x - mean) * rstd, g = dy * weight:
//             dx = rstd * (g - sum g / K - xh * sum(g xh) / K)
//             d_weight = sum over rows of dy xh, d_bias = sum over rows of dy
// Both are bound by memory: x (and dy) are read once, kept in registers in their own type
// while the row's sums are taken, and written from there. Rows that start on 16-byte
// boundaries move 16 bytes at a time (V values), others one value at a time.
//  * forward: a warp per row up to 8 vectors a lane (no barriers), else a block per row.
//  * backward: each block takes every G-th row and keeps the sums of d_weight and d_bias for its
//    columns in registers, the next row's loads under way during the current row's sums; G
//    partial sums are added in a fixed order by a second kernel.
// Rows too long for registers (over 8 vectors in 1024 threads; backward over 16 values in each)
// take the looping kernels, which read them again from L2.
#include <type_traits>

#include "elem.cuh"

namespace moe {
namespace {

constexpr int kRowThreads = 256;
constexpr int kColParts = 152;  // row ranges of the looping kernels' partial sums

// Partial sums of the backward kernel (its blocks): as many per SM as keep enough loads under
// way, up to eight; each partial sum is 2 K floats that the fold reads again, 10 MB in all.
int most_parts(int K) {
    const int n = 1250000 / K / 152;
    return 152 * (n < 1 ? 1 : n > 8 ? 8 : n);
}

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

// One thread's share of a row: IT vectors of V values, `threads` vectors apart, held as the
// 32-bit words they are loaded in (V = 1: as fp32). The share is used as pairs of values,
// whichever vectors these lie in.
template <typename T, int V, int IT>
struct Share {
    static constexpr int kPairs = V * IT / 2;
    static constexpr int kWords = V > 1 ? V * (int)sizeof(T) / 4 : 1;  // of a vector
    uint32_t w[IT * kWords];
    // values at or past K are zero; `vec`: the row starts on a 16-byte boundary (else one load
    // per value, the same values to the same threads: results do not depend on the alignment)
    __device__ __forceinline__ void load(const T* __restrict__ row, int K, int tx, int threads, bool vec) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = (i * threads + tx) * V;
            uint32_t* o = w + i * kWords;
            if (c >= K) {
#pragma unroll
                for (int j = 0; j < kWords; ++j) o[j] = 0;
            } else if constexpr (V == 1) {
                o[0] = __float_as_uint(to_f32(row[c]));
            } else if (vec) {
#pragma unroll
                for (int j = 0; j < kWords; j += 4) {
                    const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(row + c) + j);
                    o[j] = u.x, o[j + 1] = u.y, o[j + 2] = u.z, o[j + 3] = u.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < kWords; ++j)
                    o[j] = sizeof(T) == 4 ? bits_of(row[c + j]) : bits_of(row[c + 2 * j]) | bits_of(row[c + 2 * j + 1]) << 16;
            }
        }
    }
    __device__ __forceinline__ void store(T* __restrict__ row, int K, int tx, int threads, bool vec) const {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = (i * threads + tx) * V;
            const uint32_t* o = w + i * kWords;
            if (c >= K) continue;
            if constexpr (V == 1) {
                row[c] = from_f32<T>(__uint_as_float(o[0]));
            } else if (vec) {
                *reinterpret_cast<uint4*>(row + c) = make_uint4(o[0], o[1], o[2], o[3]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if constexpr (sizeof(T) == 4)
                        row[c + j] = __uint_as_float(o[j]);
                    else
                        reinterpret_cast<uint16_t*>(row)[c + j] = (uint16_t)(o[j / 2] >> (j % 2 * 16));
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
    // the column of the pair's first value (the second: the next, or `threads` on where V is 1)
    static __device__ __forceinline__ int column(int p, int tx, int threads) {
        return V > 1 ? (2 * p / V * threads + tx) * V + 2 * p % V : 2 * p * threads + tx;
    }
};

// Sums over the threads of a row (blockDim.x of them, a row per threadIdx.y), the same in all.
// `s`: 32 places per row, another one at the next call, so that one barrier is enough.
__device__ __forceinline__ float2 row_sum(float2 v, float2* s) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v = __fadd2_rn(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
    if (blockDim.x == 32) return v;
    s += threadIdx.y * 32;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = s[0];
    for (int i = 1; i < (int)(blockDim.x >> 5); ++i) v = __fadd2_rn(v, s[i]);
    return v;
}

// kThreads, here and below: the most threads of a block. The number of blocks that an SM is
// to hold bounds the registers, so that enough rows are under way.
template <typename T, typename P, int V, int IT, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 128 ? 6 : 1)
    layer_norm_rows_kernel(const T* x, int64_t M, int K, const P* __restrict__ weight, const P* __restrict__ bias, float eps,
                           T* y, float* __restrict__ mean_out, float* __restrict__ rstd_out, bool vec) {
    using S = Share<T, V, IT>;
    __shared__ float2 s[2][4 * 32];
    pdl_wait();
    pdl_trigger();
    const int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool in = r < M;  // threads of absent rows keep the barriers company
    const int tx = threadIdx.x, threads = blockDim.x;
    S xs;
    xs.load(x + (in ? r : 0) * K, in ? K : 0, tx, threads, vec);
    float2 a = both(0.f);
#pragma unroll
    for (int p = 0; p < S::kPairs; ++p) a = __fadd2_rn(a, xs.get(p));
    a = row_sum(both(a.x + a.y), s[0]);
    const float mean = a.x / K;
    a = both(0.f);
#pragma unroll
    for (int p = 0; p < S::kPairs; ++p) {
        float2 d = __fadd2_rn(xs.get(p), both(-mean));
        if (S::column(p, tx, threads) >= K) d = both(0.f);
        if (V == 1 && S::column(p, tx, threads) + threads >= K) d.y = 0.f;
        a = __ffma2_rn(d, d, a);
    }
    a = row_sum(both(a.x + a.y), s[1]);
    const float rstd = 1.f / sqrtf(a.x / K + eps);
    if (!in) return;
    // a vector (V = 1: a pair) of parameters at a time
    constexpr int kStep = V > 1 ? V / 2 : 1;
#pragma unroll
    for (int p0 = 0; p0 < S::kPairs; p0 += kStep) {
        const int c = S::column(p0, tx, threads);
        if (c >= K) break;
        Share<P, V, (V > 1 ? 1 : 2)> w, b;
        w.load(weight + c, K - c, 0, threads, vec);
        if (bias) b.load(bias + c, K - c, 0, threads, vec);
#pragma unroll
        for (int q = 0; q < kStep; ++q) {
            const float2 h = __fmul2_rn(__fadd2_rn(xs.get(p0 + q), both(-mean)), both(rstd));
            xs.set(p0 + q, __ffma2_rn(h, w.get(q), bias ? b.get(q) : both(0.f)));
        }
    }
    xs.store(y + r * K, K, tx, threads, vec);
    if (tx == 0) {
        if (mean_out) mean_out[r] = mean;
        if (rstd_out) rstd_out[r] = rstd;
    }
}

// Block b takes the rows b * blockDim.y + threadIdx.y, then gridDim.x * blockDim.y further on.
// (x - mean) * rstd is taken as x * rstd - mean * rstd in one rounding.
template <typename T, typename P, int V, int IT, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads > 256 ? 1 : V * IT > 8 ? 2 : 3)
    layer_norm_backward_kernel(const T* dy, const T* __restrict__ x, int64_t M, int K, const P* __restrict__ weight,
                               const float* __restrict__ mean_in, const float* __restrict__ rstd_in, T* dx,
                               float* __restrict__ parts, bool vec) {
    using S = Share<T, V, IT>;
    __shared__ float2 s[2][8 * 32];
    extern __shared__ float cols[];  // 2 * K, where the block has several rows at a time
    pdl_wait();
    pdl_trigger();
    const int tx = threadIdx.x, threads = blockDim.x;
    Share<P, V, IT> w;
    w.load(weight, K, tx, threads, vec);
    float2 dw[S::kPairs], db[S::kPairs];
#pragma unroll
    for (int p = 0; p < S::kPairs; ++p) dw[p] = db[p] = both(0.f);
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    S xs, ds, xn, dn;
    float mean_n = 0.f, rstd_n = 0.f;
    auto fetch = [&](int64_t r) {
        const bool in = r < M;
        xn.load(x + (in ? r : 0) * K, in ? K : 0, tx, threads, vec);
        dn.load(dy + (in ? r : 0) * K, in ? K : 0, tx, threads, vec);
        mean_n = in ? __ldg(mean_in + r) : 0.f;
        rstd_n = in ? __ldg(rstd_in + r) : 0.f;
    };
    int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    fetch(r);
    int turn = 0;
    // all rows of the block take the same number of turns (absent ones are zeros)
    for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < M; r0 += step, r += step, turn ^= 1) {
        xs = xn;
        ds = dn;
        const float rstd = rstd_n, shift = -mean_n * rstd_n;
        if (r0 + step < M) fetch(r + step);
        float2 a = both(0.f), b = both(0.f);
#pragma unroll
        for (int p = 0; p < S::kPairs; ++p) {
            const float2 d = ds.get(p), h = __ffma2_rn(xs.get(p), both(rstd), both(shift)), g = __fmul2_rn(d, w.get(p));
            a = __fadd2_rn(a, g);
            b = __ffma2_rn(g, h, b);
            dw[p] = __ffma2_rn(d, h, dw[p]);
            db[p] = __fadd2_rn(db[p], d);
        }
        a = row_sum(make_float2(a.x + a.y, b.x + b.y), s[turn]);
        if (r < M) {
            // rstd * (g - a - h b)
            const float2 c = both(-a.x / K * rstd), e = both(-a.y / K);
#pragma unroll
            for (int p = 0; p < S::kPairs; ++p) {
                const float2 h = __ffma2_rn(xs.get(p), both(rstd), both(shift)), g = __fmul2_rn(ds.get(p), w.get(p));
                xs.set(p, __ffma2_rn(__ffma2_rn(h, e, g), both(rstd), c));
            }
            xs.store(dx + r * K, K, tx, threads, vec);
        }
    }
    float* out = parts + (int64_t)blockIdx.x * 2 * K;
    if (blockDim.y > 1) out = cols;
    for (int y = 0; y < blockDim.y; ++y) {  // the block's rows one after the other
        if (y) __syncthreads();
        if (threadIdx.y == y) {
#pragma unroll
            for (int p = 0; p < S::kPairs; ++p) {
                const int c = S::column(p, tx, threads), c2 = V > 1 ? c + 1 : c + threads;
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
#pragma unroll 4
        for (int p = ty; p < n; p += 32) a += parts[((int64_t)p * 2 + blockIdx.y) * K + c];
    }
    s[ty][tx] = a;
    __syncthreads();
    a = warp_sum(s[tx][ty]);  // column blockIdx.x * 32 + ty
    P* out = blockIdx.y ? db : dw;
    if (tx == 0 && out && blockIdx.x * 32 + ty < K) out[blockIdx.x * 32 + ty] = from_f32<P>(a);
}

bool norm_args_ok(int64_t M, int K, int dtype, int param_dtype) {
    return M >= 0 && M <= INT32_MAX && K >= 1 && dtype_bytes(dtype) && (param_dtype == dtype || param_dtype == MOE_DT_F32);
}

// Calls f with `it` (a power of two up to kMost) as a constant.
template <int kMost, typename F>
void with_it(int it, F&& f) {
    if (it == kMost)
        f(std::integral_constant<int, kMost>{});
    else if constexpr (kMost > 1)
        with_it<kMost / 2>(it, f);
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
    if (!x || !weight || !y || misaligned(x, z) || misaligned(y, z) || misaligned(weight, zp) || misaligned(bias, zp))
        return MOE_ERR_INVALID_ARG;
    const size_t n = (size_t)M * K * z;
    if ((y != x && overlap(y, n, x, n)) || overlap(y, n, weight, (size_t)K * zp) ||
        overlap(y, n, bias, bias ? (size_t)K * zp : 0))
        return MOE_ERR_INVALID_ARG;
    if (int st = check_device(nullptr)) return st;
    return with_types(dtype, param_dtype, [&](auto* t, auto* p) {
        using T = std::remove_pointer_t<decltype(t)>;
        using P = std::remove_pointer_t<decltype(p)>;
        constexpr int V = 16 / sizeof(T);
        const bool vec = !misaligned(x, 16) && !misaligned(y, 16) && !misaligned(weight, 16) && !misaligned(bias, 16);
        auto rows = [&](auto vc) -> bool {
            constexpr int W = decltype(vc)::value;
            const int nv = (K + W - 1) / W;
            if (nv > 8 * 1024) return false;
            const int it = nv > 128 ? 8 : nv > 64 ? 4 : nv > 32 || W == 1 ? 2 : 1;
            const int threads = nv <= 256 ? 32 : ((nv + 7) / 8 + 31) / 32 * 32;
            const dim3 block(threads, threads == 32 ? 4 : 1);
            with_it<8>(it, [&](auto ic) {
                constexpr int IT = decltype(ic)::value;
                auto kernel = layer_norm_rows_kernel<T, P, W, (IT * W > 1 ? IT : 2), 128>;
                if constexpr (IT == 8)  // more than a warp per row: always 8 vectors a thread
                    if (threads > 128) kernel = layer_norm_rows_kernel<T, P, W, IT, 1024>;
                launch_k(kernel, (unsigned)((M + block.y - 1) / block.y), block, 0,
                         (cudaStream_t)stream, static_cast<const T*>(x), M, K, static_cast<const P*>(weight),
                         static_cast<const P*>(bias), eps, static_cast<T*>(y), mean, rstd, vec);
            });
            return true;
        };
        if (!(K % V == 0 ? rows(std::integral_constant<int, V>{}) : rows(std::integral_constant<int, 1>{})))
            launch_k(layer_norm_kernel<T, P>, (unsigned)M, kRowThreads, 0, (cudaStream_t)stream, static_cast<const T*>(x), K,
                     static_cast<const P*>(weight), static_cast<const P*>(bias), eps, static_cast<T*>(y), mean, rstd);
        note_launches(1);
        return launch_status();
    });
}

MOE_API size_t moe_layer_norm_workspace_size(int64_t M, int K) {
    if (M < 0 || K < 1) return 0;
    return (size_t)most_parts(K) * 2 * K * sizeof(float);
}

MOE_API int moe_layer_norm_backward(const void* dy, const void* x, int64_t M, int K, int dtype, const void* weight,
                                    int param_dtype, const float* mean, const float* rstd, void* dx, void* d_weight,
                                    void* d_bias, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    if (!norm_args_ok(M, K, dtype, param_dtype) || !d_weight || !workspace || misaligned(workspace, 16))
        return MOE_ERR_INVALID_ARG;
    const int z = dtype_bytes(dtype), zp = dtype_bytes(param_dtype);
    if (misaligned(d_weight, zp) || misaligned(d_bias, zp)) return MOE_ERR_INVALID_ARG;
    if (M > 0 && (!dy || !x || !weight || !mean || !rstd || !dx || misaligned(dy, z) || misaligned(x, z) ||
                  misaligned(dx, z) || misaligned(weight, zp)))
        return MOE_ERR_INVALID_ARG;
    const size_t n = (size_t)M * K * z;
    if ((dx != dy && overlap(dx, n, dy, n)) || overlap(dx, n, x, n) || overlap(workspace, workspace_bytes, dy, n) ||
        overlap(workspace, workspace_bytes, x, n) || overlap(workspace, workspace_bytes, dx, n))
        return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < moe_layer_norm_workspace_size(M, K)) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (int st = check_device(nullptr)) return st;
    return with_types(dtype, param_dtype, [&](auto* t, auto* p) {
        using T = std::remove_pointer_t<decltype(t)>;
        using P = std::remove_pointer_t<decltype(p)>;
        cudaStream_t s = (cudaStream_t)stream;
        float* parts = static_cast<float*>(workspace);
        int n_parts = 0;
        constexpr int V = 16 / sizeof(T);
        const bool vec = !misaligned(x, 16) && !misaligned(dy, 16) && !misaligned(dx, 16) && !misaligned(weight, 16);
        auto rows = [&](auto vc) -> bool {
            constexpr int W = decltype(vc)::value;
            const int nv = (K + W - 1) / W;
            // up to 16 columns a thread: their weights and two sums each stay in registers
            constexpr int kMostIt = 16 / W;
            if (nv > kMostIt * 1024) return false;
            int it = W == 1 ? 2 : 1;
            while (it < kMostIt && nv > 256 * it) it *= 2;
            const int threads = ((nv + it - 1) / it + 31) / 32 * 32;
            const dim3 block(threads, threads <= 128 ? 256 / threads : 1);
            const int64_t blocks = (M + block.y - 1) / block.y;
            n_parts = (int)(blocks < most_parts(K) ? blocks : most_parts(K));
            with_it<kMostIt>(it, [&](auto ic) {
                constexpr int IT = decltype(ic)::value;
                if constexpr (IT * W <= 16 && IT * W > 1) {
                    auto kernel = layer_norm_backward_kernel<T, P, W, IT, 256>;
                    if constexpr (IT == kMostIt)
                        if (threads > 256)
                            kernel = threads > 512 ? layer_norm_backward_kernel<T, P, W, IT, 1024>
                                                   : layer_norm_backward_kernel<T, P, W, IT, 512>;
                    launch_k(kernel, (unsigned)n_parts, block,
                             block.y > 1 ? 2 * K * sizeof(float) : 0, s, static_cast<const T*>(dy), static_cast<const T*>(x), M,
                             K, static_cast<const P*>(weight), mean, rstd, static_cast<T*>(dx), parts, vec);
                }
            });
            note_launches(1);
            return true;
        };
        if (M > 0 && !(K % V == 0 ? rows(std::integral_constant<int, V>{}) : rows(std::integral_constant<int, 1>{}))) {
            n_parts = (int)(M < kColParts ? M : kColParts);
            // the column sums read dy before dx, which may be the same buffer, is written
            launch_k(layer_norm_cols_kernel<T>, dim3((unsigned)((K + 31) / 32), (unsigned)n_parts), 256, 0, s,
                     static_cast<const T*>(dy), static_cast<const T*>(x), M, K, mean, rstd, parts);
            launch_k(layer_norm_dx_kernel<T, P>, (unsigned)M, kRowThreads, 0, s, static_cast<const T*>(dy),
                     static_cast<const T*>(x), K, static_cast<const P*>(weight), mean, rstd, static_cast<T*>(dx));
            note_launches(2);
        }
        launch_k(layer_norm_fold_kernel<P>, dim3((unsigned)((K + 31) / 32), d_bias ? 2 : 1), dim3(32, 32), 0, s, parts, n_parts, K,
                 static_cast<P*>(d_weight), static_cast<P*>(d_bias));
        note_launches(1);
        return launch_status();
    });
}

}  // extern "C"
