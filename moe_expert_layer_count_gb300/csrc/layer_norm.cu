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
// Rows too long for registers (over 8 vectors in 1024 threads; backward over 8192 values)
// take the looping kernels, which read them again from L2.
#include "elem.cuh"

namespace moe {
namespace {

constexpr int kRowThreads = 256;
constexpr int kColParts = 152;  // row ranges of the looping kernels' partial sums

// Partial sums of the backward kernel (its blocks): four an SM while a row is short, so that
// enough loads are under way; each partial sum is 2 K floats that the fold reads again.
int most_parts(int K) { return K <= 2048 ? 608 : K <= 4096 ? 304 : 152; }

// V values from p; `vec`: p lies on a vector's boundary (else one load per value, the same values
// to the same threads: results do not depend on the alignment).
template <typename P, int V>
__device__ __forceinline__ Vec<P, V> load_vec(const P* __restrict__ p, bool vec) {
    Vec<P, V> r;
    if (!vec) {
#pragma unroll
        for (int j = 0; j < V; ++j) r.v[j] = p[j];
    } else if constexpr (V * sizeof(P) <= 16) {
        r = *reinterpret_cast<const Vec<P, V>*>(p);
    } else {  // 8 fp32 values: two loads
        constexpr int N = 16 / sizeof(P);
#pragma unroll
        for (int i = 0; i < V; i += N) {
            const Vec<P, N> h = *reinterpret_cast<const Vec<P, N>*>(p + i);
#pragma unroll
            for (int j = 0; j < N; ++j) r.v[i + j] = h.v[j];
        }
    }
    return r;
}
template <typename P, int V>
__device__ __forceinline__ void store_vec(P* p, const Vec<P, V>& v, bool vec) {
    if (vec) {
        *reinterpret_cast<Vec<P, V>*>(p) = v;
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) p[j] = v.v[j];
    }
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

// kThreads: the most threads of a block, 256 or 1024 (which leaves 64 registers a thread).

// The raw values of one thread's share of a row: IT vectors, `threads` vectors apart.
template <typename T, int V, int IT>
struct Share {
    Vec<T, V> v[IT];
    // vectors at or past K are zero; `vec`: the row starts on a vector's boundary
    __device__ __forceinline__ void load(const T* __restrict__ row, int K, int tx, int threads, bool vec) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = (i * threads + tx) * V;
            if (c < K) {
                v[i] = load_vec<T, V>(row + c, vec);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) v[i].v[j] = from_f32<T>(0.f);
            }
        }
    }
};

// Sum over the threads of a row (blockDim.x of them, a row per threadIdx.y), the same in all.
// `s`: 32 floats per row; called in turn with two buffers, so that one barrier is enough.
__device__ __forceinline__ float row_sum(float v, float* s) {
    v = warp_sum(v);
    if (blockDim.x == 32) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) s[threadIdx.y * 32 + (threadIdx.x >> 5)] = v;
    __syncthreads();
    return warp_sum(lane < (blockDim.x >> 5) ? s[threadIdx.y * 32 + lane] : 0.f);
}

template <typename T, typename P, int V, int IT, int kThreads>
__global__ void __launch_bounds__(kThreads)
    layer_norm_rows_kernel(const T* x, int64_t M, int K, const P* __restrict__ weight, const P* __restrict__ bias, float eps,
                           T* y, float* __restrict__ mean_out, float* __restrict__ rstd_out, bool vec) {
    __shared__ float s[2][8 * 32];
    pdl_wait();
    pdl_trigger();
    const int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool in = r < M;  // threads of absent rows keep the barriers company
    const int tx = threadIdx.x, threads = blockDim.x;
    Share<T, V, IT> xs;
    xs.load(x + (in ? r : 0) * K, in ? K : 0, tx, threads, vec);
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) a += to_f32(xs.v[i].v[j]);
    const float mean = row_sum(a, s[0]) / K;
    a = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i)
        if ((i * threads + tx) * V < K) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = to_f32(xs.v[i].v[j]) - mean;
                a = fmaf(d, d, a);
            }
        }
    const float rstd = 1.f / sqrtf(row_sum(a, s[1]) / K + eps);
    if (!in) return;
    T* out = y + r * K;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = (i * threads + tx) * V;
        if (c < K) {
            const Vec<P, V> w = load_vec<P, V>(weight + c, vec);
            Vec<P, V> b = {};
            if (bias) b = load_vec<P, V>(bias + c, vec);
            Vec<T, V> o;
#pragma unroll
            for (int j = 0; j < V; ++j)
                o.v[j] = from_f32<T>(fmaf((to_f32(xs.v[i].v[j]) - mean) * rstd, to_f32(w.v[j]), bias ? to_f32(b.v[j]) : 0.f));
            store_vec(out + c, o, vec);
        }
    }
    if (tx == 0) {
        if (mean_out) mean_out[r] = mean;
        if (rstd_out) rstd_out[r] = rstd;
    }
}

// Block b takes the rows b * blockDim.y + threadIdx.y, then gridDim.x * blockDim.y further on.
template <typename T, typename P, int V, int IT, int kThreads>
__global__ void __launch_bounds__(kThreads)
    layer_norm_backward_kernel(const T* dy, const T* __restrict__ x, int64_t M, int K, const P* __restrict__ weight,
                               const float* __restrict__ mean_in, const float* __restrict__ rstd_in, T* dx,
                               float* __restrict__ parts, bool vec) {
    __shared__ float s[4][8 * 32];
    extern __shared__ float cols[];  // 2 * K, where the block has several rows at a time
    pdl_wait();
    pdl_trigger();
    const int tx = threadIdx.x, threads = blockDim.x;
    float w[IT][V], dw[IT][V], db[IT][V];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int c = (i * threads + tx) * V;
        Vec<P, V> p = {};
        if (c < K) p = load_vec<P, V>(weight + c, vec);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            w[i][j] = c < K ? to_f32(p.v[j]) : 0.f;
            dw[i][j] = db[i][j] = 0.f;
        }
    }
    const int64_t step = (int64_t)gridDim.x * blockDim.y;
    Share<T, V, IT> xs, ds, xn, dn;
    float mean = 0.f, rstd = 0.f, mean_n = 0.f, rstd_n = 0.f;
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
    for (int64_t r0 = (int64_t)blockIdx.x * blockDim.y; r0 < M; r0 += step, r += step, turn ^= 2) {
        xs = xn;
        ds = dn;
        mean = mean_n;
        rstd = rstd_n;
        if (r0 + step < M) fetch(r + step);
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float d = to_f32(ds.v[i].v[j]), h = (to_f32(xs.v[i].v[j]) - mean) * rstd, g = d * w[i][j];
                a += g;
                b = fmaf(g, h, b);
                dw[i][j] = fmaf(d, h, dw[i][j]);
                db[i][j] += d;
            }
        a = warp_sum(a);
        b = warp_sum(b);
        if (threads > 32) {
            const int lane = tx & 31, n = threads >> 5, base = threadIdx.y * 32;
            if (lane == 0) {
                s[turn][base + (tx >> 5)] = a;
                s[turn + 1][base + (tx >> 5)] = b;
            }
            __syncthreads();
            a = warp_sum(lane < n ? s[turn][base + lane] : 0.f);
            b = warp_sum(lane < n ? s[turn + 1][base + lane] : 0.f);
        }
        a /= K;
        b /= K;
        if (r < M) {
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int c = (i * threads + tx) * V;
                if (c < K) {
                    Vec<T, V> o;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float h = (to_f32(xs.v[i].v[j]) - mean) * rstd;
                        o.v[j] = from_f32<T>(rstd * (to_f32(ds.v[i].v[j]) * w[i][j] - a - h * b));
                    }
                    store_vec(dx + r * K + c, o, vec);
                }
            }
        }
    }
    float* out = parts + (int64_t)blockIdx.x * 2 * K;
    if (blockDim.y == 1) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int c = (i * threads + tx) * V;
            if (c < K) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    out[c + j] = dw[i][j];
                    out[K + c + j] = db[i][j];
                }
            }
        }
        return;
    }
    for (int y = 0; y < blockDim.y; ++y) {  // the block's rows one after the other
        __syncthreads();
        if (threadIdx.y == y) {
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int c = (i * threads + tx) * V;
                if (c < K) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        cols[c + j] = dw[i][j] + (y ? cols[c + j] : 0.f);
                        cols[K + c + j] = db[i][j] + (y ? cols[K + c + j] : 0.f);
                    }
                }
            }
        }
    }
    __syncthreads();
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

// Calls f with `it` (1, 2, 4 or 8) as a constant.
template <typename F>
void with_it(int it, F&& f) {
    if (it == 1) f(std::integral_constant<int, 1>{});
    if (it == 2) f(std::integral_constant<int, 2>{});
    if (it == 4) f(std::integral_constant<int, 4>{});
    if (it == 8) f(std::integral_constant<int, 8>{});
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
            const int it = nv > 128 ? 8 : nv > 64 ? 4 : nv > 32 ? 2 : 1;
            const int threads = nv <= 256 ? 32 : ((nv + 7) / 8 + 31) / 32 * 32;
            const dim3 block(threads, threads == 32 ? 4 : 1);
            with_it(it, [&](auto ic) {
                constexpr int IT = decltype(ic)::value;
                launch_k(threads <= 256 ? layer_norm_rows_kernel<T, P, W, IT, 256> : layer_norm_rows_kernel<T, P, W, IT, 1024>,
                         (unsigned)((M + block.y - 1) / block.y), block, 0,
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
            // 8 columns a thread at most: their weights and two sums each stay in registers
            constexpr int kMostIt = 8 / W;
            if (nv > kMostIt * 1024) return false;
            int it = 1;
            while (it < kMostIt && nv > 128 * it) it *= 2;
            const int threads = ((nv + it - 1) / it + 31) / 32 * 32;
            const dim3 block(threads, threads <= 128 ? 256 / threads : 1);
            const int64_t blocks = (M + block.y - 1) / block.y;
            n_parts = (int)(blocks < most_parts(K) ? blocks : most_parts(K));
            with_it(it, [&](auto ic) {
                constexpr int IT = decltype(ic)::value;
                if constexpr (IT * W <= 8)
                    launch_k(threads <= 256 ? layer_norm_backward_kernel<T, P, W, IT, 256>
                                            : layer_norm_backward_kernel<T, P, W, IT, 1024>,
                             (unsigned)n_parts, block,
                             block.y > 1 ? 2 * K * sizeof(float) : 0, s, static_cast<const T*>(dy), static_cast<const T*>(x), M,
                             K, static_cast<const P*>(weight), mean, rstd, static_cast<T*>(dx), parts, vec);
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
