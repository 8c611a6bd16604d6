// Layer norm over the last dimension and its gradients.
//   forward   mean = sum x / K, rstd = 1 / sqrt(sum (x - mean)^2 / K + eps),
//             y = (x - mean) * rstd * weight + bias
//   backward  with xh = (x - mean) * rstd, g = dy * weight:
//             dx = rstd * (g - sum g / K - xh * sum(g xh) / K)
//             d_weight = sum over rows of dy xh, d_bias = sum over rows of dy
// One block per row for y and dx; d_weight and d_bias as partial sums of row ranges,
// added in a fixed order by a second kernel.
#include "elem.cuh"

namespace moe {
namespace {

constexpr int kRowThreads = 256;
constexpr int kColParts = 152;  // row ranges of the partial sums (one per SM)

// Sum over the block, the same value in every thread. `s`: one float per warp.
__device__ __forceinline__ float block_sum(float v, float* s) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = warp_sum((threadIdx.x & 31) < kRowThreads / 32 ? s[threadIdx.x & 31] : 0.f);
    __syncthreads();
    return v;
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

template <typename P>
__global__ void __launch_bounds__(256)
    layer_norm_fold_kernel(const float* __restrict__ parts, int n, int K, P* __restrict__ dw, P* __restrict__ db) {
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= K) return;
    float a = 0.f, b = 0.f;
    for (int p = 0; p < n; ++p) {
        a += parts[(int64_t)p * 2 * K + c];
        b += parts[((int64_t)p * 2 + 1) * K + c];
    }
    dw[c] = from_f32<P>(a);
    if (db) db[c] = from_f32<P>(b);
}

bool norm_args_ok(int64_t M, int K, int dtype, int param_dtype) {
    return M >= 0 && M <= INT32_MAX && K >= 1 && dtype_bytes(dtype) && (param_dtype == dtype || param_dtype == MOE_DT_F32);
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
        launch_k(layer_norm_kernel<T, P>, (unsigned)M, kRowThreads, 0, (cudaStream_t)stream, static_cast<const T*>(x), K,
                 static_cast<const P*>(weight), static_cast<const P*>(bias), eps, static_cast<T*>(y), mean, rstd);
        note_launches(1);
        return launch_status();
    });
}

MOE_API size_t moe_layer_norm_workspace_size(int64_t M, int K) {
    if (M < 0 || K < 1) return 0;
    return (size_t)kColParts * 2 * K * sizeof(float);
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
        const int n_parts = (int)(M < kColParts ? M : kColParts);
        if (M > 0) {
            // the column sums read dy before dx, which may be the same buffer, is written
            launch_k(layer_norm_cols_kernel<T>, dim3((unsigned)((K + 31) / 32), (unsigned)n_parts), 256, 0, s,
                     static_cast<const T*>(dy), static_cast<const T*>(x), M, K, mean, rstd, parts);
            launch_k(layer_norm_dx_kernel<T, P>, (unsigned)M, kRowThreads, 0, s, static_cast<const T*>(dy),
                     static_cast<const T*>(x), K, static_cast<const P*>(weight), mean, rstd, static_cast<T*>(dx));
            note_launches(2);
        }
        launch_k(layer_norm_fold_kernel<P>, (unsigned)((K + 255) / 256), 256, 0, s, parts, n_parts, K,
                 static_cast<P*>(d_weight), static_cast<P*>(d_bias));
        note_launches(1);
        return launch_status();
    });
}

}  // extern "C"
