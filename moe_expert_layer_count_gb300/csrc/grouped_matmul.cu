// Matrix products of ragged row groups with one 16-bit weight matrix per group (the
// experts of an MoE layer in training, or served from 16-bit weights):
//   forward   y[r]  = W_l x[r]                     for the rows r of group l
//   dgrad     dx[r] = W_l^T dy[r]
//   wgrad     dW_l  = sum over the rows r of group l of dy[r] x[r]^T   (0 if it has none)
// One 64x64 output tile per block, operands through shared memory, fp32 FMAs.
#include <climits>

#include "elem.cuh"
#include "route.cuh"

namespace moe {
namespace {

constexpr int kTile = 64, kDepth = 16;
enum { kFwd = 0, kDgrad = 1, kWgrad = 2 };

// Rows [lo, hi) of group l, never outside [0, R).
__device__ __forceinline__ void group_rows(const int32_t* off, const int32_t* cnt, int l, int R, int& lo, int& hi) {
    lo = min(max(off[l], 0), R);
    const int end = cnt ? (int)min((int64_t)lo + max(cnt[l], 0), (int64_t)R) : off[l + 1];
    hi = max(min(end, R), lo);
}

template <int MODE, typename T, typename O>
__global__ void __launch_bounds__(256)
    grouped_simple_kernel(const T* __restrict__ a, const T* __restrict__ b, const int32_t* __restrict__ off,
                          const int32_t* __restrict__ cnt, int El, int R, int N, int K, O* __restrict__ out) {
    __shared__ float sa[kDepth][kTile + 1], sb[kDepth][kTile + 1];
    pdl_wait();
    pdl_trigger();
    // this block's group and its tile within the group
    int l, lo, hi, m0;
    if (MODE == kWgrad) {
        l = blockIdx.z;
        group_rows(off, cnt, l, R, lo, hi);
        m0 = blockIdx.x * kTile;
    } else {
        int t = blockIdx.x;
        for (l = 0; l < El; ++l) {
            group_rows(off, cnt, l, R, lo, hi);
            const int n = (hi - lo + kTile - 1) / kTile;
            if (t < n) break;
            t -= n;
        }
        if (l == El) return;
        m0 = lo + t * kTile;
    }
    const int n0 = blockIdx.y * kTile;
    const int m_end = MODE == kWgrad ? N : hi, n_end = MODE == kFwd ? N : K;
    const int d0 = MODE == kWgrad ? lo : 0, d_end = MODE == kWgrad ? hi : MODE == kFwd ? K : N;
    const T* w = b + (MODE == kWgrad ? 0 : (int64_t)l * N * K);
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int d = d0; d < d_end; d += kDepth) {
        for (int i = threadIdx.x; i < kTile * kDepth; i += 256) {
            // the fastest index runs along each operand's contiguous direction
            int m = MODE == kWgrad ? i % kTile : i / kDepth, k = MODE == kWgrad ? i / kTile : i % kDepth;
            float v = 0.f;
            if (m0 + m < m_end && d + k < d_end)
                v = MODE == kFwd     ? to_f32(a[(int64_t)(m0 + m) * K + d + k])
                    : MODE == kDgrad ? to_f32(a[(int64_t)(m0 + m) * N + d + k])
                                     : to_f32(a[(int64_t)(d + k) * N + m0 + m]);
            sa[k][m] = v;
            m = MODE == kFwd ? i / kDepth : i % kTile, k = MODE == kFwd ? i % kDepth : i / kTile;
            v = 0.f;
            if (n0 + m < n_end && d + k < d_end)
                v = MODE == kFwd ? to_f32(w[(int64_t)(n0 + m) * K + d + k]) : to_f32(w[(int64_t)(d + k) * K + n0 + m]);
            sb[k][m] = v;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kDepth; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty + 16 * i], sb[k][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
    O* o = out + (MODE == kWgrad ? (int64_t)l * N * K : 0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m < m_end && n < n_end) o[(int64_t)m * n_end + n] = from_f32<O>(acc[i][j]);
        }
}

template <int MODE, typename T, typename O>
int launch_simple(const void* a, const void* b, const int32_t* off, const int32_t* cnt, int El, int64_t R, int N, int K,
                  void* out, cudaStream_t stream) {
    const int64_t tiles = MODE == kWgrad ? (N + kTile - 1) / kTile : (R + kTile - 1) / kTile + El;
    const int n_out = MODE == kFwd ? N : K;
    if (n_out > 65535 * kTile) return MOE_ERR_INVALID_ARG;
    const dim3 grid((unsigned)tiles, (unsigned)((n_out + kTile - 1) / kTile), MODE == kWgrad ? (unsigned)El : 1u);
    launch_k(grouped_simple_kernel<MODE, T, O>, grid, 256, 0, stream, static_cast<const T*>(a), static_cast<const T*>(b), off,
             cnt, El, (int)R, N, K, static_cast<O*>(out));
    note_launches(1);
    return launch_status();
}

// a, b: the operands (x and w; dy and w; dy and x). The checks of all three entry points.
template <int MODE>
int grouped_impl(const void* a, const void* b, const int32_t* off, const int32_t* cnt, int El, int64_t R, int N, int K,
                 int dtype, int out_dtype, void* out, moe_stream_t stream) {
    if (El < 1 || El > kMaxLocalExperts || R < 0 || R > INT32_MAX || N < 8 || K < 8 || N % 8 || K % 8 || !off ||
        (dtype != MOE_DT_BF16 && dtype != MOE_DT_F16) || (out_dtype != dtype && out_dtype != MOE_DT_F32))
        return MOE_ERR_INVALID_ARG;
    if (((R > 0 || MODE == kWgrad) && !out) || (R > 0 && (!a || !b)) || misaligned(a, 16) || misaligned(b, 16) || misaligned(out, 16)) return MOE_ERR_INVALID_ARG;
    if (R == 0 && MODE != kWgrad) return MOE_OK;
    const size_t wn = (size_t)El * N * K;
    const size_t a_bytes = (size_t)R * (MODE == kFwd ? K : N) * 2;
    const size_t b_bytes = MODE == kWgrad ? (size_t)R * K * 2 : wn * 2;
    const size_t o_bytes = (MODE == kWgrad ? wn : (size_t)R * (MODE == kFwd ? N : K)) * dtype_bytes(out_dtype);
    if (overlap(out, o_bytes, a, a_bytes) || overlap(out, o_bytes, b, b_bytes)) return MOE_ERR_INVALID_ARG;
    if (int st = check_device(nullptr)) return st;
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == MOE_DT_BF16)
        return out_dtype == MOE_DT_F32 ? launch_simple<MODE, bf16, float>(a, b, off, cnt, El, R, N, K, out, s)
                                       : launch_simple<MODE, bf16, bf16>(a, b, off, cnt, El, R, N, K, out, s);
    return out_dtype == MOE_DT_F32 ? launch_simple<MODE, fp16, float>(a, b, off, cnt, El, R, N, K, out, s)
                                   : launch_simple<MODE, fp16, fp16>(a, b, off, cnt, El, R, N, K, out, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

MOE_API int moe_grouped_matmul(const void* x, int64_t R, const void* w, int local_num_experts, int n_out, int k_in,
                               const int32_t* expert_offsets, const int32_t* expert_num_tokens, int dtype, int out_dtype,
                               void* out, moe_stream_t stream) {
    return grouped_impl<kFwd>(x, w, expert_offsets, expert_num_tokens, local_num_experts, R, n_out, k_in, dtype, out_dtype,
                              out, stream);
}

MOE_API int moe_grouped_matmul_dgrad(const void* dy, int64_t R, const void* w, int local_num_experts, int n_out, int k_in,
                                     const int32_t* expert_offsets, const int32_t* expert_num_tokens, int dtype,
                                     int out_dtype, void* dx, moe_stream_t stream) {
    return grouped_impl<kDgrad>(dy, w, expert_offsets, expert_num_tokens, local_num_experts, R, n_out, k_in, dtype,
                                out_dtype, dx, stream);
}

MOE_API int moe_grouped_matmul_wgrad(const void* dy, const void* x, int64_t R, int local_num_experts, int n_out, int k_in,
                                     const int32_t* expert_offsets, const int32_t* expert_num_tokens, int dtype,
                                     int out_dtype, void* dw, moe_stream_t stream) {
    return grouped_impl<kWgrad>(dy, x, expert_offsets, expert_num_tokens, local_num_experts, R, n_out, k_in, dtype,
                                out_dtype, dw, stream);
}

}  // extern "C"
