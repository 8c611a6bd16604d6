// The top-k router: for every token the topk experts with the largest logits (or biased
// scores), their weights, and the gradient of the weights with respect to the logits.
//
//   softmax  s_j = exp(l_j) / sum_m exp(l_m)        sigmoid  s_j = 1 / (1 + exp(-l_j))
//   w_i = scale * s_i,  or  scale * s_i / S  with S the sum over the chosen experts
// Gradient, g_i = dL/dw_i, sums over the chosen experts:
//   softmax               dl_j = s_j * scale * ([j chosen] g_j - sum_i s_i g_i)
//   softmax, renormalised dl_i = scale * q_i * (g_i - sum_m q_m g_m),  q_i = s_i / S; 0 elsewhere
//   sigmoid               dl_i = scale * g_i * s_i * (1 - s_i)
//   sigmoid, renormalised dl_i = scale * q_i * (g_i - sum_m q_m g_m) * (1 - s_i)
// The general forward kernel takes one warp per token: lane i holds the V consecutive logits
// [i*V, (i+1)*V) in registers, so a tie goes to the lowest lane and then to its first value.
// Without a bias and up to 16 choices the forward pass runs as router_list_kernel or, for large
// batches of 16-bit logits, as router_pair_kernel.
#include <climits>
#include <type_traits>

#include "elem.cuh"
#include "route.cuh"

namespace moe {
namespace {

constexpr int kRouterWarps = 8;
constexpr int kMaxRouterExperts = 1024;
constexpr float kFltMax = 3.402823466e38f;

// A logit as the router sees it: NaN is -inf (not available), +inf the largest finite value.
__device__ __forceinline__ float clean_logit(float l) { return l != l ? -INFINITY : fminf(l, kFltMax); }

// Order-preserving key of a value; 0 (below every other) for -inf and NaN: not available.
// -0 and +0 share a key.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);
    const uint32_t k = (u & 0x80000000u) ? ~u : u | 0x80000000u;
    return v > -INFINITY ? k : 0u;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// 1 / (1 + exp(-l)), without overflow on either side.
__device__ __forceinline__ float sigmoid(float l) {
    const float e = expf(-fabsf(l));
    return l >= 0.f ? 1.f / (1.f + e) : e / (1.f + e);
}

// The ratios s_i / S of sigmoid scores, one chosen logit per lane (-inf: none): each score
// times exp(-m), m = min(0, largest chosen logit), so that scores too small for fp32 keep
// their ratios. All of the warp's lanes call it.
__device__ __forceinline__ float sigmoid_share(float l) {
    const float m = fminf(0.f, warp_max(l));
    const float s = l > -INFINITY ? expf(fminf(l, 0.f) - m) / (1.f + expf(-fabsf(l))) : 0.f;
    const float S = warp_sum(s);
    return S > 0.f ? s / S : 0.f;
}

// exp(x) of a softmax over logits of type T. For fp32 it is good to 2 ulp. For 16-bit logits the faster
// form, whose relative error grows as |x| * 2^-24: what is written in 16 bits rounds by 2^-12 or more, and the fp32
// weights only have it in their sum, where a term that is far from the maximum counts for little.
template <typename T>
__device__ __forceinline__ float exp_of(float x) {
    if constexpr (sizeof(T) == 4)
        return expf(x);
    else
        return __expf(x);
}

// The V logits of this lane (absent ones -inf).
template <typename T, int V, bool kVec>
__device__ __forceinline__ void load_logits(const T* __restrict__ row, int lane, int E, float (&v)[V]) {
    if constexpr (kVec) {  // E is a multiple of V and rows start on V * sizeof(T) bytes
        Vec<T, V> r;
        const bool in = lane * V < E;
        if (in) r = *reinterpret_cast<const Vec<T, V>*>(row + lane * V);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = in ? clean_logit(to_f32(r.v[j])) : -INFINITY;
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = lane * V + j;
            v[j] = e < E ? clean_logit(to_f32(row[e])) : -INFINITY;
        }
    }
}

template <typename T, typename TId, int V, bool kVec>
__global__ void __launch_bounds__(kRouterWarps * 32)
    router_kernel(const T* __restrict__ logits, int64_t M, int E, int topk, int scoring, const float* __restrict__ bias,
                  int renorm, float scale, float* __restrict__ out_w, TId* __restrict__ out_id) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kRouterWarps + (threadIdx.x >> 5);
    if (t >= M) return;
    float v[V];
    load_logits<T, V, kVec>(logits + t * E, lane, E, v);
    const bool soft = scoring == MOE_SCORE_SOFTMAX;
    float top = 0.f, sum = 1.f;
    if (soft && (bias || !renorm)) {
        top = -INFINITY;
#pragma unroll
        for (int j = 0; j < V; ++j) top = fmaxf(top, v[j]);
        top = warp_max(top);
        sum = 0.f;
        if (top > -INFINITY) {
#pragma unroll
            for (int j = 0; j < V; ++j) sum += expf(v[j] - top);
        }
        sum = warp_sum(sum);
    }
    uint32_t key[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float s = v[j];
        if (bias) {
            const int e = lane * V + j;
            s = v[j] > -INFINITY && e < E ? (soft ? expf(v[j] - top) / sum : sigmoid(v[j])) + __ldg(bias + e) : -INFINITY;
        }
        key[j] = order_key(s);
    }
    int my_id = -1;
    float my_logit = -INFINITY;
    for (int i = 0; i < topk; ++i) {
        uint32_t best = 0;
        int at = 0;
        float l = -INFINITY;
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (key[j] > best) {
                best = key[j];
                at = j;
                l = v[j];
            }
        const uint32_t most = __reduce_max_sync(0xffffffffu, best);
        if (most == 0) break;  // no available expert is left
        const int win = __ffs(__ballot_sync(0xffffffffu, best == most)) - 1;
        const int id = __shfl_sync(0xffffffffu, lane * V + at, win);
        l = __shfl_sync(0xffffffffu, l, win);
        if (lane == i) {
            my_id = id;
            my_logit = l;
        }
        if (lane == win) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j == at) key[j] = 0;
        }
    }
    // lane i: slot i
    float w = 0.f;
    if (soft) {
        if (renorm) {
            // relative to the largest chosen logit, so that small scores do not vanish first
            const float m = warp_max(my_logit);
            const float e = my_id >= 0 ? expf(my_logit - m) : 0.f;
            const float S = warp_sum(e);
            w = my_id >= 0 ? e / S : 0.f;
        } else if (my_id >= 0) {
            w = expf(my_logit - top) / sum;
        }
    } else if (renorm) {
        w = sigmoid_share(my_logit);
    } else if (my_id >= 0) {
        w = sigmoid(my_logit);
    }
    if (lane < topk) {
        out_w[t * topk + lane] = w * scale;
        out_id[t * topk + lane] = (TId)my_id;
    }
}

// ------------------------------------------------------------------ unbiased choice
// Four lanes per token, eight tokens per warp. A lane takes 8 of every 32 logits, turns each into
// a key that holds the logit's order and, below it, the index (so that keys are distinct and a
// tie goes to the lower index), keeps the L largest keys in a sorted list by sorting networks, and
// merges its list with its neighbours' (two exchanges). A 16-bit logit has 13 or 16 zero bits
// below its fp32 form: its key is 32 bits and a comparator is two instructions; fp32 takes 64.
// What bounds it is the ALU pipe (minima and maxima), not memory: about 110 instructions per
// token of 128 16-bit logits against 256 bytes read.
constexpr int kListThreads = 128;
constexpr int kLanes = 4;             // per token
constexpr uint32_t kIndexMask = 0x3ff;

template <typename T>
struct KeyOf {
    using type = uint32_t;
    static __device__ __forceinline__ uint32_t make(uint32_t order, int e) { return (order & ~kIndexMask) | (kIndexMask - e); }
    static __device__ __forceinline__ int index(uint32_t k) { return kIndexMask - (k & kIndexMask); }
    // the logit; NaN for key 0 (no logit)
    static __device__ __forceinline__ float logit(uint32_t k) {
        return __uint_as_float(k & 0x80000000u ? (k & ~kIndexMask) ^ 0x80000000u : ~(k | kIndexMask));
    }
};
template <>
struct KeyOf<float> {
    using type = uint64_t;
    static __device__ __forceinline__ uint64_t make(uint32_t order, int e) { return (uint64_t)order << 32 | (kIndexMask - e); }
    static __device__ __forceinline__ int index(uint64_t k) { return kIndexMask - ((uint32_t)k & kIndexMask); }
    static __device__ __forceinline__ float logit(uint64_t k) {
        const uint32_t o = (uint32_t)(k >> 32);
        return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
    }
};

// a >= b afterwards.
template <typename K>
__device__ __forceinline__ void order2(K& a, K& b) {
    const K hi = a > b ? a : b, lo = a > b ? b : a;
    a = hi;
    b = lo;
}

// Batcher's odd-even merge sort, descending (L a power of two).
template <typename K, int L>
__device__ __forceinline__ void sort_list(K (&a)[L]) {
#pragma unroll
    for (int p = 1; p < L; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < L; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < L && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order2(a[i + j], a[i + j + k]);
}

// The L largest of two descending lists, descending: the larger of a[i] and b[L - 1 - i] are
// they, as a bitonic sequence.
template <typename K, int L>
__device__ __forceinline__ void merge_lists(K (&a)[L], const K (&b)[L]) {
#pragma unroll
    for (int i = 0; i < L; ++i) a[i] = a[i] > b[L - 1 - i] ? a[i] : b[L - 1 - i];
#pragma unroll
    for (int s = L / 2; s >= 1; s /= 2)
#pragma unroll
        for (int i = 0; i < L; ++i)
            if (!(i & s)) order2(a[i], a[i + s]);
}

// 8 logits of one lane of a 32-logit chunk and their experts. kVec: 8 in a row (E a multiple
// of 8, rows on 16-byte boundaries), else every fourth.
template <bool kVec>
__device__ __forceinline__ int expert_at(int chunk, int lane, int j) {
    return kVec ? chunk * 32 + lane * 8 + j : chunk * 32 + j * kLanes + lane;
}
template <typename T, bool kVec>
__device__ __forceinline__ void load8(const T* __restrict__ row, int chunk, int lane, int E, float (&v)[8]) {
    if constexpr (kVec) {
        constexpr int N = 16 / sizeof(T);
        if (chunk * 32 + lane * 8 < E) {
#pragma unroll
            for (int h = 0; h < 8; h += N) {
                const Vec<T, N> r = *reinterpret_cast<const Vec<T, N>*>(row + chunk * 32 + lane * 8 + h);
#pragma unroll
                for (int j = 0; j < N; ++j) v[h + j] = to_f32(r.v[j]);
            }
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = -INFINITY;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = expert_at<false>(chunk, lane, j);
            v[j] = e < E ? to_f32(row[e]) : -INFINITY;
        }
    }
}

template <typename T, typename TId, int L, bool kVec>
__global__ void __launch_bounds__(kListThreads)
    router_list_kernel(const T* __restrict__ logits, int64_t M, int E, int topk, int scoring, int renorm, float scale,
                       float* __restrict__ out_w, TId* __restrict__ out_id) {
    using Key = KeyOf<T>;
    using K = typename Key::type;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & (kLanes - 1);
    int64_t t = (int64_t)blockIdx.x * (kListThreads / kLanes) + threadIdx.x / kLanes;
    const bool real = t < M;  // the lanes past the last token go along on the last one's row
    if (!real) t = M - 1;
    const T* row = logits + t * E;
    const int chunks = (E + 31) / 32;  // absent logits are -inf: they cannot displace a real one, nor be chosen
    K best[L];
#pragma unroll
    for (int i = 0; i < L; ++i) best[i] = 0;
#pragma unroll 4
    for (int c = 0; c < chunks; c += L / 8) {
        K now[L];
#pragma unroll
        for (int h = 0; h < L; h += 8) {
            float v[8];
            load8<T, kVec>(row, c + h / 8, lane, E, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // -0 becomes +0, NaN -inf; an fp32 +inf is the largest finite value itself, while that lies above
                // every 16-bit logit, as +inf's key does
                float l = fmaxf(v[j] + 0.f, -INFINITY);
                if constexpr (sizeof(T) == 4) l = fminf(l, kFltMax);
                const uint32_t u = __float_as_uint(l);
                const uint32_t order = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
                now[h + j] = Key::make(order, expert_at<kVec>(c + h / 8, lane, j) & kIndexMask);
            }
        }
        sort_list(now);
        merge_lists(best, now);
    }
#pragma unroll
    for (int o = 1; o < kLanes; o *= 2) {
        K other[L];
#pragma unroll
        for (int i = 0; i < L; ++i) other[i] = __shfl_xor_sync(0xffffffffu, best[i], o);
        merge_lists(best, other);
    }
    // all four lanes have the list; lane q takes places q, q + 4, ...
    const bool soft = scoring == MOE_SCORE_SOFTMAX;
    const float top = fminf(Key::logit(best[0]), kFltMax);
    float w[L / kLanes], sum = 0.f;
    int id[L / kLanes];
#pragma unroll
    for (int i = 0; i < L / kLanes; ++i) {
        K k = best[i * kLanes];
#pragma unroll
        for (int q = 1; q < kLanes; ++q)
            if (lane == q) k = best[i * kLanes + q];
        const float value = Key::logit(k), l = fminf(value, kFltMax);
        const bool chosen = value > -INFINITY && i * kLanes + lane < topk;  // not for key 0, whose logit is NaN
        id[i] = chosen ? Key::index(k) : -1;
        if (soft)
            w[i] = chosen ? expf(l - top) : 0.f;
        else if (renorm)  // as sigmoid_share has it
            w[i] = chosen ? expf(fminf(l, 0.f) - fminf(0.f, top)) / (1.f + expf(-fabsf(l))) : 0.f;
        else
            w[i] = chosen ? sigmoid(l) : 0.f;
        sum += w[i];
    }
    if (soft && !renorm) {
        sum = 0.f;
        for (int c = 0; c < chunks; ++c) {
            float v[8];
            load8<T, kVec>(row, c, lane, E, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += exp_of<T>(clean_logit(v[j]) - top);
        }
    }
    if (soft || renorm) {
#pragma unroll
        for (int o = 1; o < kLanes; o *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        scale = sum > 0.f ? scale / sum : 0.f;  // 0 or NaN: nothing was chosen, all w are 0
    }
    if (!real) return;
#pragma unroll
    for (int i = 0; i < L / kLanes; ++i) {
        const int at = i * kLanes + lane;
        if (at < topk) {
            out_w[t * topk + at] = w[i] * scale;
            out_id[t * topk + at] = (TId)id[i];
        }
    }
}

// The same for large batches of up to 128 16-bit logits and 8 choices: two lanes per token, so that
// less of the work is merging, and keys made from packed pairs. Order and tie rules are those of
// router_list_kernel. Bound by the ALU pipe like it: 2^20 tokens of 128 bf16 logits take 98.5 us
// (3.4 TB/s, half of the copy rate) against its 141.
constexpr int kPairThreads = 128;
constexpr int kPairExperts = 128;
// Smaller batches do not fill the SMs with two lanes a token.
constexpr int64_t kPairTokens = 16384;

__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b, const bf16*) {
    const __nv_bfloat162 r = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b, const fp16*) {
    const __half2 r = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b, const bf16*) {
    const __nv_bfloat162 r = __hadd2_rn(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b, const fp16*) {
    const __half2 r = __hadd2_rn(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

template <typename T, typename TId>
__global__ void __launch_bounds__(kPairThreads)
    router_pair_kernel(const T* __restrict__ logits, int64_t M, int E, int topk, int scoring, int renorm, float scale,
                       float* __restrict__ out_w, TId* __restrict__ out_id) {
    constexpr uint32_t kLow = std::is_same<T, bf16>::value ? 0xff80ff80u : 0xfc00fc00u;  // a pair of -inf
    constexpr T* kType = nullptr;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 1;
    int64_t t = (int64_t)blockIdx.x * (kPairThreads / 2) + threadIdx.x / 2;
    const bool real = t < M;
    if (!real) t = M - 1;
    const T* row = logits + t * E + lane * 8;  // this lane's 8 of every 16 logits
    uint4 raw[kPairExperts / 16];
#pragma unroll
    for (int c = 0; c < kPairExperts / 16; ++c) {
        raw[c] = make_uint4(kLow, kLow, kLow, kLow);
        if (c * 16 + lane * 8 < E) raw[c] = *reinterpret_cast<const uint4*>(row + c * 16);
    }
    uint32_t best[8];
#pragma unroll
    for (int c = 0; c < kPairExperts / 16; ++c) {
        if (c > 0 && c * 16 >= E) break;
        uint32_t now[8];
        const uint32_t w4[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // NaN becomes -inf, -0 becomes +0, then each half the order of its value
            const uint32_t w = hadd2(hmax2(w4[j], kLow, kType), 0u, kType);
            const uint32_t order = w ^ ((w >> 15 & 0x00010001u) * 0x7fffu + 0x80008000u);
            const uint32_t index = kIndexMask - (c * 16 + 2 * j);
            now[2 * j] = order * 65536u + index;
            now[2 * j + 1] = (order & 0xffff0000u) | (index - 1);
        }
        sort_list(now);
        if (c == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) best[i] = now[i];
        } else {
            merge_lists(best, now);
        }
    }
    uint32_t other[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) best[i] -= lane * 8;  // the index counted from the row's start
#pragma unroll
    for (int i = 0; i < 8; ++i) other[i] = __shfl_xor_sync(0xffffffffu, best[i], 1);
    merge_lists(best, other);
    // lane q has places 4q to 4q + 3
    const bool soft = scoring == MOE_SCORE_SOFTMAX;
    auto logit_of = [&](uint32_t k) {
        const uint32_t o = k >> 16;
        const uint16_t u = (uint16_t)(o & 0x8000u ? o ^ 0x8000u : ~o);
        return to_f32(*reinterpret_cast<const T*>(&u));
    };
    const float top = fminf(logit_of(best[0]), kFltMax);
    float w[4], sum = 0.f;
    int id[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t k = lane ? best[4 + i] : best[i];
        const float value = logit_of(k), l = fminf(value, kFltMax);
        const bool chosen = value > -INFINITY && lane * 4 + i < topk;  // not for key 0, whose logit is NaN
        id[i] = chosen ? (int)(kIndexMask - (k & kIndexMask)) : -1;
        if (soft)
            w[i] = chosen ? expf(l - top) : 0.f;
        else if (renorm)  // as sigmoid_share has it
            w[i] = chosen ? expf(fminf(l, 0.f) - fminf(0.f, top)) / (1.f + expf(-fabsf(l))) : 0.f;
        else
            w[i] = chosen ? sigmoid(l) : 0.f;
        sum += w[i];
    }
    if (soft && !renorm) {
        sum = 0.f;
#pragma unroll
        for (int c = 0; c < kPairExperts / 16; ++c) {
            if (c * 16 >= E) break;
            const uint32_t w4[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint16_t u = (uint16_t)(w4[j / 2] >> (j % 2 * 16));
                sum += exp_of<T>(clean_logit(to_f32(*reinterpret_cast<const T*>(&u))) - top);
            }
        }
    }
    if (soft || renorm) {
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        scale = sum > 0.f ? scale / sum : 0.f;  // 0 or NaN: nothing was chosen, all w are 0
    }
    if (!real) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = lane * 4 + i;
        if (at < topk) {
            out_w[t * topk + at] = w[i] * scale;
            out_id[t * topk + at] = (TId)id[i];
        }
    }
}

// ------------------------------------------------------------------ gradient
// Eight lanes per token. A lane takes the slots lane, lane + 8, ... and 8 of every 64 logits. The
// row is read twice where its softmax is needed (the second time from L1): once for the maximum
// and the sum, once for the values that are written.
constexpr int kGradThreads = 128;
constexpr int kGradLanes = 8;
constexpr int kSlots = 32 / kGradLanes;

__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = 1; o < kGradLanes; o *= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = 1; o < kGradLanes; o *= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// V = 8: in a row (E a multiple of 8, rows on 16-byte boundaries); else every eighth.
template <bool kVec>
__device__ __forceinline__ int grad_expert(int chunk, int lane, int j) {
    return kVec ? chunk * 64 + lane * 8 + j : chunk * 64 + j * kGradLanes + lane;
}

template <typename T, typename TId, bool kVec>
__global__ void __launch_bounds__(kGradThreads)
    router_backward_kernel(const T* logits, int64_t M, int E, const TId* __restrict__ ids, int topk, int scoring,
                           int renorm, float scale, const float* __restrict__ dw, T* d_logits) {
    constexpr int N = 16 / sizeof(T);
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & (kGradLanes - 1);
    int64_t t = (int64_t)blockIdx.x * (kGradThreads / kGradLanes) + threadIdx.x / kGradLanes;
    const bool real = t < M;  // the lanes past the last token go along on the last one's row, and write nothing
    if (!real) t = M - 1;
    const bool soft = scoring == MOE_SCORE_SOFTMAX;
    const T* row = logits + t * E;
    // this lane's slots
    int id[kSlots];
    float g[kSlots], l[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        const int at = i * kGradLanes + lane;
        id[i] = -1;
        g[i] = 0.f;
        l[i] = -INFINITY;
        if (at < topk) {
            const TId raw = ids[t * topk + at];
            if (raw >= 0 && raw < TId(E)) {
                id[i] = (int)raw;
                g[i] = scale * dw[t * topk + at];
                l[i] = clean_logit(to_f32(row[id[i]]));
            }
        }
    }
    auto load = [&](int c, float (&v)[8]) {
        if constexpr (kVec) {
            if (c * 64 + lane * 8 < E) {
#pragma unroll
                for (int h = 0; h < 8; h += N) {
                    const Vec<T, N> r = *reinterpret_cast<const Vec<T, N>*>(row + c * 64 + lane * 8 + h);
#pragma unroll
                    for (int j = 0; j < N; ++j) v[h + j] = clean_logit(to_f32(r.v[j]));
                }
                return;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = grad_expert<kVec>(c, lane, j);
            v[j] = !kVec && e < E ? clean_logit(to_f32(row[e])) : -INFINITY;
        }
    };
    const int chunks = (E + 63) / 64;
    float d[kSlots];
    float top = 0.f, rest = 0.f;  // what an expert that was not chosen gets: rest * exp(logit - top)
    if (soft && !renorm) {
        float m = -INFINITY, sum = 0.f;
#pragma unroll 2
        for (int c = 0; c < chunks; ++c) {
            float v[8], most = m;
            load(c, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) most = fmaxf(most, v[j]);
            if (most > -INFINITY) {
                sum *= exp_of<T>(m - most);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum += exp_of<T>(v[j] - most);
                m = most;
            }
        }
        top = group_max(m);
        sum = group_sum(m > -INFINITY ? sum * exp_of<T>(m - top) : 0.f);
        const float r = sum > 0.f ? 1.f / sum : 0.f;
        float s[kSlots], dot = 0.f;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            s[i] = l[i] > -INFINITY ? expf(l[i] - top) * r : 0.f;
            dot = fmaf(s[i], g[i], dot);
        }
        dot = group_sum(dot);
#pragma unroll
        for (int i = 0; i < kSlots; ++i) d[i] = s[i] * (g[i] - dot);
        rest = -dot * r;
    } else {
        // the share of a chosen score in the chosen scores' sum, each taken times exp(-low) so that
        // scores too small for fp32 keep their ratios (renormalised), or the score itself
        float m = -INFINITY, S = 0.f, dot = 0.f, q[kSlots];
#pragma unroll
        for (int i = 0; i < kSlots; ++i) m = fmaxf(m, l[i]);
        m = group_max(m);
        if (!soft) m = renorm ? fminf(0.f, m) : 0.f;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            const bool in = l[i] > -INFINITY;
            q[i] = !in ? 0.f : soft ? expf(l[i] - m) : expf(fminf(l[i], 0.f) - m) / (1.f + expf(-fabsf(l[i])));
            S += q[i];
        }
        if (renorm) {
            S = group_sum(S);
            const float r = S > 0.f ? 1.f / S : 0.f;
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                q[i] *= r;
                dot = fmaf(q[i], g[i], dot);
            }
            dot = group_sum(dot);
        }
#pragma unroll
        for (int i = 0; i < kSlots; ++i) d[i] = q[i] * (g[i] - dot) * (soft ? 1.f : sigmoid(-l[i]));
    }
    __syncwarp();  // the chosen logits are read: d_logits may be logits
    T* out = d_logits + t * E;
#pragma unroll 2
    for (int c = 0; c < chunks; ++c) {
        float v[8];
        if (rest != 0.f) {
            load(c, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = rest * exp_of<T>(v[j] - top);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.f;
        }
        if (!real) continue;
        if constexpr (kVec) {
            if (c * 64 + lane * 8 < E) {
#pragma unroll
                for (int h = 0; h < 8; h += N) {
                    Vec<T, N> r;
#pragma unroll
                    for (int j = 0; j < N; ++j) r.v[j] = from_f32<T>(v[h + j]);
                    *reinterpret_cast<Vec<T, N>*>(out + c * 64 + lane * 8 + h) = r;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int e = grad_expert<false>(c, lane, j);
                if (e < E) out[e] = from_f32<T>(v[j]);
            }
        }
    }
    __syncwarp();  // the chosen experts' values replace the ones just written
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
        if (real && id[i] >= 0) out[id[i]] = from_f32<T>(d[i]);
}

bool router_args_ok(int64_t M, int E, int dtype, int topk, int scoring) {
    return M >= 0 && E >= 1 && E <= kMaxRouterExperts && topk >= 1 && topk <= 32 && topk <= E && M <= INT32_MAX / topk &&
           dtype_bytes(dtype) && (scoring == MOE_SCORE_SOFTMAX || scoring == MOE_SCORE_SIGMOID);
}

// Calls f(V) with V = the smallest power of two that covers E with 32 lanes.
template <typename F>
int with_v(int E, F&& f) {
    if (E <= 32) return f(std::integral_constant<int, 1>{});
    if (E <= 64) return f(std::integral_constant<int, 2>{});
    if (E <= 128) return f(std::integral_constant<int, 4>{});
    if (E <= 256) return f(std::integral_constant<int, 8>{});
    if (E <= 512) return f(std::integral_constant<int, 16>{});
    return f(std::integral_constant<int, 32>{});
}

// Vector accesses move at most 16 bytes: a lane's V values are one vector only while they fit.
template <typename T, int V>
constexpr bool fits_vec() { return V > 1 && V * sizeof(T) <= 16; }

template <typename TId>
int router_impl(const void* logits, int64_t M, int E, int dtype, int topk, int scoring, const float* bias, int renorm,
                float scale, float* w, TId* ids, moe_stream_t stream) {
    if (!router_args_ok(M, E, dtype, topk, scoring)) return MOE_ERR_INVALID_ARG;
    if (M == 0) return MOE_OK;
    if (!logits || !w || !ids || misaligned(logits, dtype_bytes(dtype)) || misaligned(bias, 4) || misaligned(w, 4) ||
        misaligned(ids, sizeof(TId)))
        return MOE_ERR_INVALID_ARG;
    const size_t nl = (size_t)M * E * dtype_bytes(dtype), nw = (size_t)M * topk * 4, ni = (size_t)M * topk * sizeof(TId);
    const size_t nb = bias ? (size_t)E * 4 : 0;
    if (overlap(w, nw, logits, nl) || overlap(ids, ni, logits, nl) || overlap(w, nw, ids, ni) || overlap(w, nw, bias, nb) ||
        overlap(ids, ni, bias, nb))
        return MOE_ERR_INVALID_ARG;
    if (int st = check_device(nullptr)) return st;
    const unsigned grid = (unsigned)((M + kRouterWarps - 1) / kRouterWarps);
    return with_dtype(dtype, [&](auto* p) {
        using T = std::remove_pointer_t<decltype(p)>;
        if (!bias && topk <= 16) {
            auto go = [&](auto kernel, int per = kListThreads / kLanes) {
                static_assert(kListThreads == kPairThreads, "one block size");
                launch_k(kernel, (unsigned)((M + per - 1) / per), kListThreads, 0, (cudaStream_t)stream,
                         static_cast<const T*>(logits), M, E, topk, scoring, renorm ? 1 : 0, scale, w, ids);
                note_launches(1);
                return launch_status();
            };
            const bool vec = E % 8 == 0 && !misaligned(logits, 16);
            if constexpr (sizeof(T) == 2)
                if (vec && topk <= 8 && E <= kPairExperts && M >= kPairTokens)
                    return go(router_pair_kernel<T, TId>, kPairThreads / 2);
            if (topk <= 8) return vec ? go(router_list_kernel<T, TId, 8, true>) : go(router_list_kernel<T, TId, 8, false>);
            return vec ? go(router_list_kernel<T, TId, 16, true>) : go(router_list_kernel<T, TId, 16, false>);
        }
        return with_v(E, [&](auto vc) {
            constexpr int V = decltype(vc)::value;
            auto go = [&](auto kernel) {
                launch_k(kernel, grid, kRouterWarps * 32, 0, (cudaStream_t)stream, static_cast<const T*>(logits), M, E,
                         topk, scoring, bias, renorm ? 1 : 0, scale, w, ids);
                note_launches(1);
                return launch_status();
            };
            if constexpr (fits_vec<T, V>())
                if (E % V == 0 && !misaligned(logits, V * sizeof(T))) return go(router_kernel<T, TId, V, true>);
            return go(router_kernel<T, TId, V, false>);
        });
    });
}

template <typename TId>
int router_backward_impl(const void* logits, int64_t M, int E, int dtype, const TId* ids, int topk, int scoring,
                         int renorm, float scale, const float* dw, void* d_logits, moe_stream_t stream) {
    if (!router_args_ok(M, E, dtype, topk, scoring)) return MOE_ERR_INVALID_ARG;
    if (M == 0) return MOE_OK;
    if (!logits || !ids || !dw || !d_logits || misaligned(logits, dtype_bytes(dtype)) ||
        misaligned(d_logits, dtype_bytes(dtype)) || misaligned(ids, sizeof(TId)) || misaligned(dw, 4))
        return MOE_ERR_INVALID_ARG;
    const size_t nl = (size_t)M * E * dtype_bytes(dtype);
    if ((d_logits != logits && overlap(d_logits, nl, logits, nl)) ||
        overlap(d_logits, nl, ids, (size_t)M * topk * sizeof(TId)) || overlap(d_logits, nl, dw, (size_t)M * topk * 4))
        return MOE_ERR_INVALID_ARG;
    if (int st = check_device(nullptr)) return st;
    return with_dtype(dtype, [&](auto* p) {
        using T = std::remove_pointer_t<decltype(p)>;
        constexpr int per = kGradThreads / kGradLanes;
        const bool vec = E % 8 == 0 && !misaligned(logits, 16) && !misaligned(d_logits, 16);
        launch_k(vec ? router_backward_kernel<T, TId, true> : router_backward_kernel<T, TId, false>,
                 (unsigned)((M + per - 1) / per), kGradThreads, 0, (cudaStream_t)stream, static_cast<const T*>(logits), M, E, ids,
                 topk, scoring, renorm ? 1 : 0, scale, dw, static_cast<T*>(d_logits));
        note_launches(1);
        return launch_status();
    });
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

MOE_API int moe_router_topk(const void* logits, int64_t M, int E, int dtype, int topk, int scoring, const float* bias,
                            int renormalize, float scale, float* topk_weights, int32_t* topk_ids, moe_stream_t stream) {
    return router_impl(logits, M, E, dtype, topk, scoring, bias, renormalize, scale, topk_weights, topk_ids, stream);
}

MOE_API int moe_router_topk_i64(const void* logits, int64_t M, int E, int dtype, int topk, int scoring,
                                const float* bias, int renormalize, float scale, float* topk_weights, int64_t* topk_ids,
                                moe_stream_t stream) {
    return router_impl(logits, M, E, dtype, topk, scoring, bias, renormalize, scale, topk_weights, topk_ids, stream);
}

MOE_API int moe_router_topk_backward(const void* logits, int64_t M, int E, int dtype, const int32_t* topk_ids, int topk,
                                     int scoring, int renormalize, float scale, const float* d_topk_weights,
                                     void* d_logits, moe_stream_t stream) {
    return router_backward_impl(logits, M, E, dtype, topk_ids, topk, scoring, renormalize, scale, d_topk_weights, d_logits,
                                stream);
}

MOE_API int moe_router_topk_backward_i64(const void* logits, int64_t M, int E, int dtype, const int64_t* topk_ids,
                                         int topk, int scoring, int renormalize, float scale,
                                         const float* d_topk_weights, void* d_logits, moe_stream_t stream) {
    return router_backward_impl(logits, M, E, dtype, topk_ids, topk, scoring, renormalize, scale, d_topk_weights, d_logits,
                                stream);
}

}  // extern "C"
