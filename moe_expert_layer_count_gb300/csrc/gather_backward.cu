// Gradients of the gather with the top-k weight-and-reduce: with r = src2dst[t, k],
//   d_y[r] = w[t, k] * dout[t],   d_w[t, k] = sum over c of y[r, c] * dout[t, c].
// DRAM bounds it: dout, y and d_y once each, 84 us for 8192 tokens, top-8, of 2048 columns (571 MB at
// 6.77 TB/s, the copy rate).
// Small calls are the host's: 1.6-3.3 us on the device for 17 to 1023 tokens, 7-9 us a call.
#include <climits>

#include "elem.cuh"
#include "route.cuh"

namespace moe {
namespace {

constexpr int kMaxWarps = 8;

// A block has a token, a warp one of its slots at a time, so that dout's row comes from DRAM once and from L1
// for the other slots, and no sum crosses a warp: a lane holds pieces of 8 columns.
// Products and sums in fp32; w * dout is rounded once.
__global__ void __launch_bounds__(32 * kMaxWarps)
    gather_backward_kernel(const bf16* __restrict__ dout, const bf16* __restrict__ y, const int32_t* __restrict__ src2dst,
                           const float* __restrict__ weights, int topk, int K, int rows, bf16* __restrict__ d_y,
                           float* __restrict__ d_weights) {
    pdl_wait();
    pdl_trigger();
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 31;
    for (int k = threadIdx.x >> 5; k < topk; k += blockDim.x >> 5) {
        const int r = src2dst[t * topk + k];
        float sum = 0.f;
        if (r >= 0 && r < rows) {
            const float w = weights ? weights[t * topk + k] : 1.f;
            for (int c = lane * 8; c < K; c += 256) {
                const Vec<bf16, 8> g = *reinterpret_cast<const Vec<bf16, 8>*>(dout + t * K + c);
                Vec<bf16, 8> o;
#pragma unroll
                for (int i = 0; i < 8; ++i) o.v[i] = from_f32<bf16>(w * to_f32(g.v[i]));
                if (d_weights) {
                    const Vec<bf16, 8> v = *reinterpret_cast<const Vec<bf16, 8>*>(y + (int64_t)r * K + c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum = fmaf(to_f32(v.v[i]), to_f32(g.v[i]), sum);
                }
                *reinterpret_cast<Vec<bf16, 8>*>(d_y + (int64_t)r * K + c) = o;
            }
        }
        sum = warp_sum(sum);
        if (d_weights && lane == 0) d_weights[t * topk + k] = sum;
    }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" MOE_API int moe_gather_weight_reduce_backward(const void* dout, const void* y, int64_t rows, const int32_t* src2dst,
                                                         const float* topk_weights, int64_t M, int topk, int K,
                                                         int apply_router_weight_on_input, void* d_y, float* d_topk_weights,
                                                         moe_stream_t stream) {
    const bool unit = apply_router_weight_on_input != 0;
    if (M < 0 || topk < 1 || topk > 32 || M > INT32_MAX / topk || K < 128 || K % 128 || K > 1 << 30 || rows < 0 || rows > INT32_MAX)
        return MOE_ERR_INVALID_ARG;
    if (M > 0 && (!dout || !src2dst || (rows > 0 && !d_y) || (!unit && !topk_weights) || (d_topk_weights && rows > 0 && !y)))
        return MOE_ERR_INVALID_ARG;
    if (unit && d_topk_weights) return MOE_ERR_INVALID_ARG;
    if (misaligned(dout, 16) || misaligned(y, 16) || misaligned(d_y, 16) || misaligned(src2dst, 4) || misaligned(topk_weights, 4) ||
        misaligned(d_topk_weights, 4))
        return MOE_ERR_INVALID_ARG;
    const size_t n = (size_t)M * topk, row = (size_t)K * 2, y_bytes = d_topk_weights ? rows * row : 0;
    const size_t w_bytes = unit ? 0 : n * 4, dw_bytes = d_topk_weights ? n * 4 : 0;
    if (overlap(d_y, rows * row, dout, M * row) || overlap(d_y, rows * row, y, y_bytes) || overlap(d_y, rows * row, src2dst, n * 4) ||
        overlap(d_y, rows * row, topk_weights, w_bytes) || overlap(d_topk_weights, dw_bytes, d_y, rows * row) ||
        overlap(d_topk_weights, dw_bytes, dout, M * row) || overlap(d_topk_weights, dw_bytes, y, y_bytes) ||
        overlap(d_topk_weights, dw_bytes, src2dst, n * 4) || overlap(d_topk_weights, dw_bytes, topk_weights, w_bytes))
        return MOE_ERR_INVALID_ARG;
    if (M == 0) return MOE_OK;
    if (int st = check_device(nullptr)) return st;
    launch_k(gather_backward_kernel, (unsigned)M, 32 * (topk < kMaxWarps ? topk : kMaxWarps), 0, (cudaStream_t)stream,
             static_cast<const bf16*>(dout), static_cast<const bf16*>(y), src2dst, unit ? nullptr : topk_weights, topk, K, (int)rows,
             static_cast<bf16*>(d_y), d_topk_weights);
    note_launches(1);
    return launch_status();
}
