// The gated feed-forward part of an MoE layer's experts with 16-bit weights: both input projections
// of a ragged row group and the activation in one product, and its backward pass up to the gradients
// of the two projections. With W_g, W_u the first and last N rows of w13[l]:
//   forward   g = W_g x[r], u = W_u x[r], h[r] = a(g) * u            for the rows r of group l
//   backward  dh = w2[l]^T dy[r], dg = dh * u * a'(g), du = dh * a(g), h[r] = a(g) * u again
// The kernel is in grouped_tc.cuh. What is kept of g and u for the backward pass leaves the same
// epilogue, in 16 bits or in the 8-bit form of ckpt.cuh.
//
// What it measured (one GB300, times of one call with L2 flushed, in short runs at the full clock; sizes N = 768,
// K = 2048, 128 groups):
//   512 rows a group       forward 250-261 us, 265-277 with g and u kept in 16 bits or in 8 (the ungated product of
//                          the same weights: 252-259); backward 214-222 us from either
//   65536 rows, Zipf 1.2   forward 271-283 us, 285-300 with g and u kept; backward 210-214 us from either. Passes that
//                          follow one another for seconds, where the power cap holds the clock at 1290-1575 MHz:
//                          322-342 us with g and u kept in 16 bits, backward 212-227
//   512 rows, decode       forward 122-126 us: 790 MB at 6.3-6.5 TB/s
// What bounds it. Forward: as the ungated product (tensor pipe active 81 %, 74 % with g and u stored): MMAs
// and the weights' way from DRAM hide each other only in part; without an epilogue 247 us at 512 rows a
// group. Backward: 1.17 GB from and to DRAM at 5.3-5.5 TB/s (its floor at the copy rate is 174 us); without
// MMAs it takes as long, without its stores or without reading g and u 181 us each, without both 156.
// What did not help: asking for the next tile's weights in L2 (258 -> 306-330 us by either kind of prefetch: what the
// SMs take in is short, not time), asking for g and u by TMA (220 -> 240 us), streaming stores (equal) and loads
// (214 -> 222 us).
#include "grouped_tc.cuh"

namespace moe {
namespace {

// Whether a product of sizes is at most 2^46, more than any memory holds.
bool fits(int64_t a, int64_t b, int64_t c) { return (long double)a * (long double)b * (long double)c <= 0x1p46L; }

struct Span {
    const void* p;
    size_t n;
};
bool apart(const Span& a, std::initializer_list<Span> others) {
    for (const Span& b : others)
        if (overlap(a.p, a.n, b.p, b.n)) return false;
    return true;
}

// What both directions check of their sizes; tile: outputs of a tile.
bool sizes_ok(int El, int64_t R, int N, int K, int act, int keep, int dtype, const int32_t* off, int tile) {
    if (El < 1 || El > kMaxLocalExperts || R < 0 || R > INT32_MAX || N < 8 || N > INT32_MAX / 2 || K < 8 || N % 8 || K % 8 ||
        !off || (dtype != MOE_DT_BF16 && dtype != MOE_DT_F16) || (act != MOE_ACT_SILU && act != MOE_ACT_GELU_TANH) ||
        keep < MOE_KEEP_NONE || keep > MOE_KEEP_E4M3 || (keep == MOE_KEEP_E4M3 && N % kCkptGroup))
        return false;
    // tiles are counted in 32 bits (choose_rows takes fewer rows only where that makes few more)
    return (R / kMaxN + El) * (((int64_t)N + tile - 1) / tile) <= INT32_MAX / 2 && fits(El, 2 * (int64_t)N, K) &&
           fits(R, 2 * (int64_t)N, 1) && fits(R, K, 1);
}

}  // namespace

int read_gated_error(int clear) { return read_error_word(clear); }

}  // namespace moe

using namespace moe;

extern "C" {

MOE_API int moe_grouped_gated(const void* x, int64_t R, const void* w13, int local_num_experts, int N, int K,
                              const int32_t* expert_offsets, const int32_t* expert_num_tokens, int activation, int dtype,
                              void* h, int keep, void* pre, uint8_t* pre_scale, moe_stream_t stream) {
    const int El = local_num_experts;
    if (!sizes_ok(El, R, N, K, activation, keep, dtype, expert_offsets, tile_outputs<kGated>())) return MOE_ERR_INVALID_ARG;
    if ((R > 0 && (!x || !w13 || !h)) || misaligned(x, 16) || misaligned(w13, 16) || misaligned(h, 16) || misaligned(pre, 16) ||
        misaligned(expert_offsets, 4) || misaligned(expert_num_tokens, 4))
        return MOE_ERR_INVALID_ARG;
    if ((keep == MOE_KEEP_NONE ? pre != nullptr : R > 0 && !pre) || (keep == MOE_KEEP_E4M3 ? R > 0 && !pre_scale : pre_scale != nullptr))
        return MOE_ERR_INVALID_ARG;
    if (R == 0) return MOE_OK;
    const size_t n = (size_t)R * N;
    const Span in_x{x, (size_t)R * K * 2}, in_w{w13, (size_t)El * 2 * N * K * 2}, in_off{expert_offsets, ((size_t)El + 1) * 4},
        in_cnt{expert_num_tokens, expert_num_tokens ? (size_t)El * 4 : 0};
    const Span out_h{h, n * 2}, out_pre{pre, keep == MOE_KEEP_NONE ? 0 : keep == MOE_KEEP_16BIT ? n * 4 : n * 2},
        out_scale{pre_scale, keep == MOE_KEEP_E4M3 ? n * 2 / kCkptGroup : 0};
    if (!apart(out_h, {in_x, in_w, in_off, in_cnt, out_pre, out_scale}) || !apart(out_pre, {in_x, in_w, in_off, in_cnt, out_scale}) ||
        !apart(out_scale, {in_x, in_w, in_off, in_cnt}))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if (int st = check_device(&sms)) return st;
    const Gated gated{activation, keep, nullptr, pre, pre_scale};
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == MOE_DT_BF16)
        return launch_grouped<kGated, bf16>(x, w13, expert_offsets, expert_num_tokens, El, R, N, K, dtype, h, 1, sms, s, gated);
    return launch_grouped<kGated, fp16>(x, w13, expert_offsets, expert_num_tokens, El, R, N, K, dtype, h, 1, sms, s, gated);
}

MOE_API int moe_grouped_gated_backward(const void* dy, int64_t R, const void* w2, int local_num_experts, int N, int K,
                                       const int32_t* expert_offsets, const int32_t* expert_num_tokens, int activation,
                                       int dtype, int keep, const void* pre, const uint8_t* pre_scale, void* d_pre, void* h,
                                       moe_stream_t stream) {
    const int El = local_num_experts;
    if (!sizes_ok(El, R, N, K, activation, keep, dtype, expert_offsets, tile_outputs<kGatedBwd>()) || keep == MOE_KEEP_NONE)
        return MOE_ERR_INVALID_ARG;
    if ((R > 0 && (!dy || !w2 || !pre || !d_pre)) || misaligned(dy, 16) || misaligned(w2, 16) || misaligned(pre, 16) ||
        misaligned(d_pre, 16) || misaligned(h, 16) || misaligned(expert_offsets, 4) || misaligned(expert_num_tokens, 4))
        return MOE_ERR_INVALID_ARG;
    if (keep == MOE_KEEP_E4M3 ? R > 0 && !pre_scale : pre_scale != nullptr) return MOE_ERR_INVALID_ARG;
    if (R == 0) return MOE_OK;
    const size_t n = (size_t)R * N;
    const bool eight = keep == MOE_KEEP_E4M3;
    const Span in_dy{dy, (size_t)R * K * 2}, in_w{w2, (size_t)El * N * K * 2}, in_off{expert_offsets, ((size_t)El + 1) * 4},
        in_cnt{expert_num_tokens, expert_num_tokens ? (size_t)El * 4 : 0}, in_pre{pre, eight ? n * 2 : n * 4},
        in_scale{pre_scale, eight ? n * 2 / kCkptGroup : 0};
    const Span out_d{d_pre, n * 4}, out_h{h, h ? n * 2 : 0};
    // a gradient may take the place of the 16-bit value that it was made from: the same warp has read it
    const bool in_place = !eight && d_pre == pre;
    if ((!in_place && !apart(out_d, {in_pre})) || !apart(out_d, {in_dy, in_w, in_off, in_cnt, in_scale, out_h}) ||
        !apart(out_h, {in_dy, in_w, in_off, in_cnt, in_pre, in_scale}))
        return MOE_ERR_INVALID_ARG;
    int sms = 0;
    if (int st = check_device(&sms)) return st;
    const Gated gated{activation, keep, pre, d_pre, const_cast<uint8_t*>(pre_scale)};
    cudaStream_t s = (cudaStream_t)stream;
    // w2 [El, K, N]: dgrad's n_out is K, its k_in N
    if (dtype == MOE_DT_BF16)
        return launch_grouped<kGatedBwd, bf16>(dy, w2, expert_offsets, expert_num_tokens, El, R, K, N, dtype, h, 1, sms, s, gated);
    return launch_grouped<kGatedBwd, fp16>(dy, w2, expert_offsets, expert_num_tokens, El, R, K, N, dtype, h, 1, sms, s, gated);
}

}  // extern "C"
