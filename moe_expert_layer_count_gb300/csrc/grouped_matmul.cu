// Matrix products of ragged row groups with one 16-bit weight matrix per group (the
// experts of an MoE layer in training, or served from 16-bit weights), on the
// 5th-generation tensor cores (tcgen05, sm_103a):
//   forward   y[r]  = W_l x[r]                     for the rows r of group l
//   dgrad     dx[r] = W_l^T dy[r]
//   wgrad     dW_l  = sum over the rows r of group l of dy[r] x[r]^T   (0 if it has none)
// The kernel is in grouped_tc.cuh.
//
// What it measured (one GB300, times of one call in bursts of a few tens of ms, SM clock 2070 MHz; in
// brackets after a second of load, when the power cap holds it at 1290-1575 MHz; 8192 x 8192 x 8192 in the
// library's dense product: 540-555 us):
//   one group of 8192 rows, 8192 x 8192      590-610 us forward, 596 us [700] wgrad   1.8, 1.84 PFLOP/s
//   128 groups of 512 rows, 1536 x 2048      248-257 us [292] forward, 287 us [322] wgrad   1.65, 1.44
//   65536 rows over 128 groups, Zipf 1.2     275-279 us forward, 343-354 us wgrad   1.5, 1.2
//   512 rows over 128 groups (decode)        116-127 us forward: 750-806 MB of weights at 6.4 TB/s
//                                            132 us wgrad: as much written at 6.1 TB/s
// Where the time goes (variants that leave one part out, 512 rows a group):
//   forward: without loads 187 us, without MMAs 211 us (DRAM gives 6 TB/s for the 1.27 GB that has
//   to move), the full kernel 250 us, as the two hide each other only in part;
//   wgrad: without loads 190 us, without stores 216 us, without MMAs 244 us: 3.2 GB into the SMs
//   and 0.8 GB out of them, 16.4 TB/s, which is about what they take (64 bytes a clock each).
// What it is sensitive to: the MMA loop has to issue from uniform registers (a loop that one lane
// runs alone takes 130 clocks an MMA: 750 us dense), the look-up of a tile is on the MMA warp's
// way between tiles, and a signal to the other CTA must not be a cluster-wide release by a thread that
// stores, which it waits for (2000 clocks).

#include "grouped_tc.cuh"

namespace moe {
namespace {

// wgrad of few tiles over many rows (a router's gate, a few large experts): each group's rows are
// split into parts whose tiles fill the pairs, their sums joined by fold_parts_kernel in a fixed
// order. The parts have 512 rows or more on average; one more costs 4 bytes written and read per
// weight (8192 rows, 128 x 2048: 38.5 us in one part, 14.7 us in nine).
constexpr int kPartRows = 512, kMostParts = 16;

int wgrad_parts(int64_t R, int El, int N, int K) {
    const int64_t tiles = El * (((int64_t)N + kPairM - 1) / kPairM) * (((int64_t)K + kMaxN - 1) / kMaxN);
    int64_t parts = kSms / 2 / tiles;
    if (parts > R / El / kPartRows) parts = R / El / kPartRows;
    return (int)(parts < 2 ? 1 : parts > kMostParts ? kMostParts : parts);
}

template <typename O>
__global__ void __launch_bounds__(256) fold_parts_kernel(const float4* __restrict__ parts, int n, int64_t n4, O* __restrict__ out) {
    pdl_wait();
    pdl_trigger();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n4) return;
    float4 a = parts[i];
    for (int p = 1; p < n; ++p) {
        const float4 v = parts[p * n4 + i];
        a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    }
    Vec<O, 4> o;
    o.v[0] = from_f32<O>(a.x), o.v[1] = from_f32<O>(a.y), o.v[2] = from_f32<O>(a.z), o.v[3] = from_f32<O>(a.w);
    reinterpret_cast<Vec<O, 4>*>(out)[i] = o;
}

// a, b: the operands (x and w; dy and w; dy and x). The checks of all three entry points.
template <int MODE>
int grouped_impl(const void* a, const void* b, const int32_t* off, const int32_t* cnt, int El, int64_t R, int N, int K,
                 int dtype, int out_dtype, void* out, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    if (El < 1 || El > kMaxLocalExperts || R < 0 || R > INT32_MAX || N < 8 || K < 8 || N % 8 || K % 8 || !off ||
        (dtype != MOE_DT_BF16 && dtype != MOE_DT_F16) || (out_dtype != dtype && out_dtype != MOE_DT_F32))
        return MOE_ERR_INVALID_ARG;
    if (((R > 0 || MODE == kWgrad) && !out) || (R > 0 && (!a || !b)) || misaligned(a, 16) || misaligned(b, 16) ||
        misaligned(out, 16) || misaligned(off, 4) || misaligned(cnt, 4))
        return MOE_ERR_INVALID_ARG;
    // tiles are counted in 32 bits (choose_rows takes fewer rows only where that makes few more)
    const int64_t m_tiles = ((int64_t)(MODE == kDgrad ? K : N) + kPairM - 1) / kPairM;
    if ((MODE == kWgrad ? El * m_tiles * (((int64_t)K + kMaxN - 1) / kMaxN) : (R / kMaxN + El) * m_tiles) > INT32_MAX / 2)
        return MOE_ERR_INVALID_ARG;
    if (R == 0 && MODE != kWgrad) return MOE_OK;
    const size_t wn = (size_t)El * N * K;
    const size_t a_bytes = (size_t)R * (MODE == kFwd ? K : N) * 2;
    const size_t b_bytes = MODE == kWgrad ? (size_t)R * K * 2 : wn * 2;
    const size_t o_bytes = (MODE == kWgrad ? wn : (size_t)R * (MODE == kFwd ? N : K)) * dtype_bytes(out_dtype);
    const size_t off_bytes = ((size_t)El + 1) * 4, cnt_bytes = cnt ? (size_t)El * 4 : 0;  // read by every CTA as it starts
    if (overlap(out, o_bytes, a, a_bytes) || overlap(out, o_bytes, b, b_bytes) || overlap(out, o_bytes, off, off_bytes) ||
        overlap(out, o_bytes, cnt, cnt_bytes))
        return MOE_ERR_INVALID_ARG;
    if (MODE == kWgrad) {
        const size_t need = moe_grouped_matmul_wgrad_workspace_size(R, El, N, K);
        if (need > 0 && (!workspace || workspace_bytes < need)) return MOE_ERR_WORKSPACE_TOO_SMALL;
        if (need > 0 && (misaligned(workspace, 16) || overlap(workspace, need, a, a_bytes) || overlap(workspace, need, b, b_bytes) ||
                         overlap(workspace, need, out, o_bytes) || overlap(workspace, need, off, off_bytes) ||
                         overlap(workspace, need, cnt, cnt_bytes)))
            return MOE_ERR_INVALID_ARG;
    }
    int sms = 0;
    if (int st = check_device(&sms)) return st;
    cudaStream_t s = (cudaStream_t)stream;
    if constexpr (MODE == kWgrad) {
        const int parts = wgrad_parts(R, El, N, K);
        if (parts > 1) {
            if (int st = launch_grouped<kWgrad, float>(a, b, off, cnt, El, R, N, K, dtype, workspace, parts, sms, s)) return st;
            const int64_t n4 = (int64_t)wn / 4;  // n_out and k_in are multiples of 8
            const unsigned grid = (unsigned)((n4 + 255) / 256);
            const float4* from = static_cast<const float4*>(workspace);
            if (out_dtype == MOE_DT_F32)
                launch_k(fold_parts_kernel<float>, grid, 256, 0, s, from, parts, n4, static_cast<float*>(out));
            else if (dtype == MOE_DT_BF16)
                launch_k(fold_parts_kernel<bf16>, grid, 256, 0, s, from, parts, n4, static_cast<bf16*>(out));
            else
                launch_k(fold_parts_kernel<fp16>, grid, 256, 0, s, from, parts, n4, static_cast<fp16*>(out));
            note_launches(1);
            return launch_status();
        }
    }
    if (out_dtype == MOE_DT_F32) return launch_grouped<MODE, float>(a, b, off, cnt, El, R, N, K, dtype, out, 1, sms, s);
    if (dtype == MOE_DT_BF16) return launch_grouped<MODE, bf16>(a, b, off, cnt, El, R, N, K, dtype, out, 1, sms, s);
    return launch_grouped<MODE, fp16>(a, b, off, cnt, El, R, N, K, dtype, out, 1, sms, s);
}

}  // namespace

int read_grouped_error(int clear) { return read_error_word(clear); }

}  // namespace moe

using namespace moe;

extern "C" {

MOE_API int moe_grouped_matmul(const void* x, int64_t R, const void* w, int local_num_experts, int n_out, int k_in,
                               const int32_t* expert_offsets, const int32_t* expert_num_tokens, int dtype, int out_dtype,
                               void* out, moe_stream_t stream) {
    return grouped_impl<kFwd>(x, w, expert_offsets, expert_num_tokens, local_num_experts, R, n_out, k_in, dtype, out_dtype,
                              out, nullptr, 0, stream);
}

MOE_API int moe_grouped_matmul_dgrad(const void* dy, int64_t R, const void* w, int local_num_experts, int n_out, int k_in,
                                     const int32_t* expert_offsets, const int32_t* expert_num_tokens, int dtype,
                                     int out_dtype, void* dx, moe_stream_t stream) {
    return grouped_impl<kDgrad>(dy, w, expert_offsets, expert_num_tokens, local_num_experts, R, n_out, k_in, dtype,
                                out_dtype, dx, nullptr, 0, stream);
}

MOE_API int moe_grouped_matmul_wgrad(const void* dy, const void* x, int64_t R, int local_num_experts, int n_out, int k_in,
                                     const int32_t* expert_offsets, const int32_t* expert_num_tokens, int dtype, int out_dtype,
                                     void* dw, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    return grouped_impl<kWgrad>(dy, x, expert_offsets, expert_num_tokens, local_num_experts, R, n_out, k_in, dtype,
                                out_dtype, dw, workspace, workspace_bytes, stream);
}

MOE_API size_t moe_grouped_matmul_wgrad_workspace_size(int64_t R, int local_num_experts, int n_out, int k_in) {
    if (R < 0 || local_num_experts < 1 || n_out < 1 || k_in < 1) return 0;
    const int parts = wgrad_parts(R, local_num_experts, n_out, k_in);
    return parts > 1 ? (size_t)parts * local_num_experts * n_out * k_in * sizeof(float) : 0;
}

}  // extern "C"
