// The 2-norm of all values of a list of tensors and clipping by it:
//   norm = sqrt(sum over tensors and values of g^2);  g' = g * (norm > max ? max / norm : 1)
// Bound by memory: two reads and a write of every value (the norm has to be known first).
// The tensors are cut into chunks; each block adds the squares of its chunks (fp32 per
// thread and chunk, fp64 above that) into one partial sum. The chunks go to the blocks by
// their number alone, so the sum's order does not change from call to call. The clip pass
// adds the partial sums in every block and scales the chunks, last chunk first: the end
// of the list is what the first pass has left in L2. 604 M bf16 values, over several GPUs: the
// norm alone 172-185 us (7.0-6.5 TB/s), with the clipping 545-569 us (6.65-6.4 TB/s over the
// three passes).
#include <algorithm>
#include <memory>
#include <new>

#include "elem.cuh"

namespace moe {
namespace {

constexpr int kNormThreads = 256;
constexpr int kMaxBlocks = 1216;  // 152 SMs x 8 blocks of 256 threads
// Tensors per launch: a table travels as a kernel argument, and a short list takes a short one
// (48 tensors: 9.0 us of host time for both launches with the long table).
constexpr int kTensors = 256, kFewTensors = 64;
// Values of a piece: a thread adds the squares of its share of one in fp32. A chunk, what a block
// takes at a time, is one piece, or four where the list is long enough to fill the SMs with those
// (1.2 GB of bf16, same GPU: the norm 178 -> 172 us).
constexpr int64_t kPiece = 16384, kLong = kPiece * 4 * kMaxBlocks;

template <int N>
struct Table {
    const void* in[N];
    void* out[N];
    int64_t n[N];
    int64_t chunk0[N + 1];  // first chunk of each tensor
    int64_t chunk;          // values of a chunk
    uint8_t dtype[N];
    int count;
    bool in_place;  // every output is its input
};

// Values before the first 16-byte boundary of a tensor.
template <typename T>
__host__ __device__ __forceinline__ int64_t head_of(const void* p, int64_t n) {
    const int64_t h = (int64_t)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (int64_t)sizeof(T);
    return h < n ? h : n;
}

// Chunk c of a tensor: [lo, hi), lo on a 16-byte boundary but for chunk 0, which has the head too.
template <typename T>
__device__ __forceinline__ void chunk_range(const void* p, int64_t n, int64_t c, int64_t chunk, int64_t& head, int64_t& lo,
                                            int64_t& hi) {
    head = head_of<T>(p, n);
    lo = c == 0 ? 0 : head + c * chunk;
    hi = min(head + (c + 1) * chunk, n);
}

template <int N>
__device__ __forceinline__ int tensor_of(const Table<N>& t, int64_t chunk) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.chunk0[mid] <= chunk) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Sum of the squares of this thread's values of n at g (a piece or less; on a 16-byte boundary
// for n >= V). fp32 holds it while it neither overflows nor sinks to where the squares lose bits
// (values below ~1e-17); otherwise the thread's values are read again in fp64.
template <typename T>
__device__ __forceinline__ double piece_squares(const T* __restrict__ g, int n) {
    constexpr int V = 16 / sizeof(T);
    float a = 0.f, most = 0.f;  // `most`: to tell zeros from vanished squares
    auto add = [&](float x) {
        a = fmaf(x, x, a);
        most = fmaxf(most, fabsf(x));
    };
    const int nv = n / V;
    if (n == kPiece) {  // eight loads under way in every thread
        const uint4* from = reinterpret_cast<const uint4*>(g) + threadIdx.x;
#pragma unroll
        for (int h = 0; h < kPiece / V / kNormThreads; h += 8) {
            uint4 r[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) r[k] = from[(h + k) * kNormThreads];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const T* v = reinterpret_cast<const T*>(&r[k]);
#pragma unroll
                for (int j = 0; j < V; ++j) add(to_f32(v[j]));
            }
        }
    } else {
        for (int i = threadIdx.x; i < nv; i += kNormThreads) {
            const Vec<T, V> r = reinterpret_cast<const Vec<T, V>*>(g)[i];
#pragma unroll
            for (int j = 0; j < V; ++j) add(to_f32(r.v[j]));
        }
        for (int i = nv * V + threadIdx.x; i < n; i += kNormThreads) add(to_f32(g[i]));
    }
    if (a >= 1e-30f && a <= 3e38f) return (double)a;
    if (most == 0.f && a == 0.f) return 0.0;
    double d = 0.0;
    for (int i = threadIdx.x; i < nv; i += kNormThreads)
        for (int j = 0; j < V; ++j) {
            const double x = to_f32(g[i * V + j]);
            d += x * x;
        }
    for (int i = nv * V + threadIdx.x; i < n; i += kNormThreads) d += (double)to_f32(g[i]) * to_f32(g[i]);
    return d;
}

template <typename T>
__device__ double chunk_squares(const void* p, int64_t n, int64_t c, int64_t chunk) {
    const T* g = static_cast<const T*>(p);
    int64_t head, lo, hi;
    chunk_range<T>(p, n, c, chunk, head, lo, hi);
    double d = 0.0;
    if (c == 0 && head > 0) {  // fewer than V values
        d = piece_squares(g, (int)head);
        lo = head;
    }
    for (; lo < hi; lo += kPiece) d += piece_squares(g + lo, (int)min(hi - lo, kPiece));
    return d;
}

__device__ __forceinline__ double block_sum(double v, double* s) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < kNormThreads / 32; ++i) v += s[i];
    __syncthreads();
    return v;
}

template <int N>
__global__ void __launch_bounds__(kNormThreads) squares_kernel(const __grid_constant__ Table<N> t, double* __restrict__ parts) {
    __shared__ double s[kNormThreads / 32];
    pdl_wait();
    pdl_trigger();
    double a = 0.0;
    for (int64_t c = blockIdx.x; c < t.chunk0[t.count]; c += gridDim.x) {
        const int k = tensor_of(t, c);
        const int64_t i = c - t.chunk0[k];
        switch (t.dtype[k]) {
            case MOE_DT_F32: a += chunk_squares<float>(t.in[k], t.n[k], i, t.chunk); break;
            case MOE_DT_BF16: a += chunk_squares<bf16>(t.in[k], t.n[k], i, t.chunk); break;
            default: a += chunk_squares<fp16>(t.in[k], t.n[k], i, t.chunk); break;
        }
    }
    a = block_sum(a, s);
    if (threadIdx.x == 0) parts[blockIdx.x] = a;
}

// The norm from the n partial sums: the same order, so the same value, in every block.
__device__ __forceinline__ float norm_of(const double* __restrict__ parts, int n, double* s) {
    double a = 0.0;
    for (int i = threadIdx.x; i < n; i += kNormThreads) a += parts[i];
    return (float)sqrt(block_sum(a, s));
}

__global__ void __launch_bounds__(kNormThreads) norm_kernel(const double* __restrict__ parts, int n, float* __restrict__ norm) {
    __shared__ double s[kNormThreads / 32];
    pdl_wait();
    pdl_trigger();
    const float v = norm_of(parts, n, s);
    if (threadIdx.x == 0) *norm = v;
}

template <typename T>
__device__ void scale_chunk(const void* p, void* q, int64_t n, int64_t c, int64_t chunk, float coef) {
    constexpr int V = 16 / sizeof(T);
    const T* g = static_cast<const T*>(p);
    T* o = static_cast<T*>(q);
    int64_t head, lo, hi;
    chunk_range<T>(p, n, c, chunk, head, lo, hi);
    const int64_t v0 = c == 0 ? head : lo;
    const bool same = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(q)) & 15) == 0;
    const int64_t nv = same ? (hi - v0) / V : 0;
    for (int64_t i = lo + threadIdx.x; i < v0; i += kNormThreads) o[i] = from_f32<T>(to_f32(g[i]) * coef);
    const uint4* from = reinterpret_cast<const uint4*>(g + v0);
    uint4* to = reinterpret_cast<uint4*>(o + v0);
    auto scaled = [&](uint4 r) {
        T* v = reinterpret_cast<T*>(&r);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = from_f32<T>(to_f32(v[j]) * coef);
        return r;
    };
    int64_t i = threadIdx.x;
    for (; i + 7 * kNormThreads < nv; i += 8 * kNormThreads) {
        uint4 r[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) r[k] = from[i + k * kNormThreads];
#pragma unroll
        for (int k = 0; k < 8; ++k) to[i + k * kNormThreads] = scaled(r[k]);
    }
    for (; i < nv; i += kNormThreads) to[i] = scaled(from[i]);
    for (i = v0 + nv * V + threadIdx.x; i < hi; i += kNormThreads) o[i] = from_f32<T>(to_f32(g[i]) * coef);
}

template <int N>
__global__ void __launch_bounds__(kNormThreads)
    clip_kernel(const __grid_constant__ Table<N> t, const double* __restrict__ parts, int n, float max_norm,
                float* __restrict__ norm) {
    __shared__ double s[kNormThreads / 32];
    pdl_wait();
    pdl_trigger();
    const float v = norm_of(parts, n, s);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
    const float coef = v > max_norm && v <= 3.402823466e38f ? max_norm / v : 1.f;
    if (coef == 1.f && t.in_place) return;  // nothing to clip
    for (int64_t c = t.chunk0[t.count] - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
        const int k = tensor_of(t, c);
        const int64_t i = c - t.chunk0[k];
        switch (t.dtype[k]) {
            case MOE_DT_F32: scale_chunk<float>(t.in[k], t.out[k], t.n[k], i, t.chunk, coef); break;
            case MOE_DT_BF16: scale_chunk<bf16>(t.in[k], t.out[k], t.n[k], i, t.chunk, coef); break;
            default: scale_chunk<fp16>(t.in[k], t.out[k], t.n[k], i, t.chunk, coef); break;
        }
    }
}

int launches_of(int n_tensors) { return (n_tensors + kTensors - 1) / kTensors; }

// The table of tensors [first, first + N); returns its number of chunks.
template <int N>
int64_t fill(Table<N>& t, const void* const* in, void* const* out, const int64_t* numel, const int32_t* dtypes, int first,
             int n_tensors) {
    t.count = n_tensors - first < N ? n_tensors - first : N;
    int64_t chunks = 0, total = 0;
    for (int i = 0; i < t.count; ++i) total += numel[first + i];
    t.chunk = total >= kLong ? 4 * kPiece : kPiece;
    t.in_place = true;
    for (int i = 0; i < t.count; ++i) {
        const int64_t n = numel[first + i];
        t.in[i] = in[first + i];
        t.out[i] = out ? out[first + i] : nullptr;
        t.n[i] = n;
        t.in_place = t.in_place && t.out[i] == t.in[i];
        t.dtype[i] = (uint8_t)dtypes[first + i];
        t.chunk0[i] = chunks;
        const int64_t head = dtypes[first + i] == MOE_DT_F32 ? head_of<float>(in[first + i], n) : head_of<bf16>(in[first + i], n);
        if (n > 0) chunks += n - head > 0 ? (n - head + t.chunk - 1) / t.chunk : 1;
    }
    t.chunk0[t.count] = chunks;
    return chunks;
}

int blocks_of(int64_t chunks) { return (int)(chunks < 1 ? 1 : chunks < kMaxBlocks ? chunks : kMaxBlocks); }

template <int N>
int run(const void* const* in, void* const* outs, const int64_t* numel, const int32_t* dtypes, int n_tensors, bool clip,
        float max_norm, float* norm, double* parts, cudaStream_t stream) {
    int n_parts = 0;
    Table<N> t;
    for (int first = 0; first < n_tensors; first += N) {
        const int grid = blocks_of(fill(t, in, outs, numel, dtypes, first, n_tensors));
        launch_k(squares_kernel<N>, grid, kNormThreads, 0, stream, t, parts + n_parts);
        note_launches(1);
        n_parts += grid;
    }
    if (int st = launch_status()) return st;  // nothing is scaled by sums that were not made
    if (!clip || n_tensors == 0) {
        launch_k(norm_kernel, 1, kNormThreads, 0, stream, parts, n_parts, norm);
        note_launches(1);
        return launch_status();
    }
    for (int first = (n_tensors - 1) / N * N; first >= 0; first -= N) {
        if (n_tensors > N || !outs) fill(t, in, outs ? outs : const_cast<void* const*>(in), numel, dtypes, first, n_tensors);
        launch_k(clip_kernel<N>, blocks_of(t.chunk0[t.count]), kNormThreads, 0, stream, t, parts, n_parts, max_norm, norm);
        note_launches(1);
    }
    return launch_status();
}

// Bytes that the clip pass reads or writes.
struct Span {
    uintptr_t lo, hi;
    bool written;
};

// Whether the clip pass would write what another block reads or writes too: the tensors, their outputs, the
// norm and the partial sums (a tensor that is its own output is one span). A sweep over the spans in
// the order of their addresses.
int check_spans(const void* const* in, void* const* outs, const int64_t* numel, const int32_t* dtypes, int n_tensors,
                const float* norm, const void* workspace, size_t need) {
    constexpr int kFew = 130;  // 64 tensors and their outputs
    Span few[kFew];
    std::unique_ptr<Span[]> many;
    const size_t most = 2 * (size_t)n_tensors + 2;
    if (most > kFew) many.reset(new (std::nothrow) Span[most]);
    Span* s = most > kFew ? many.get() : few;
    if (!s) return MOE_ERR_CUDA;  // no host memory for a list of this length
    size_t n = 0;
    auto add = [&](const void* p, size_t bytes, bool written) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        if (bytes) s[n++] = Span{lo, lo + bytes, written};
    };
    for (int i = 0; i < n_tensors; ++i) {
        const size_t b = (size_t)numel[i] * dtype_bytes(dtypes[i]);
        const bool same = !outs || outs[i] == in[i];
        add(in[i], b, same);
        if (!same) add(outs[i], b, true);
    }
    add(norm, sizeof(float), true);
    add(workspace, need, true);
    std::sort(s, s + n, [](const Span& a, const Span& b) { return a.lo < b.lo; });
    uintptr_t end = 0, written_end = 0;  // of the spans so far
    for (size_t i = 0; i < n; ++i) {
        if (s[i].lo < (s[i].written ? end : written_end)) return MOE_ERR_INVALID_ARG;
        end = std::max(end, s[i].hi);
        if (s[i].written) written_end = std::max(written_end, s[i].hi);
    }
    return MOE_OK;
}

int norm_impl(const void* const* in, const int64_t* numel, const int32_t* dtypes, int n_tensors, bool clip, float max_norm,
              void* const* outs, float* norm, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (n_tensors < 0 || !norm || misaligned(norm, 4) || !workspace || misaligned(workspace, 16) ||
        (n_tensors > 0 && (!in || !numel || !dtypes)) || (clip && !(max_norm >= 0.f)))
        return MOE_ERR_INVALID_ARG;
    for (int i = 0; i < n_tensors; ++i) {
        const int z = dtype_bytes(dtypes[i]);
        if (numel[i] < 0 || !z) return MOE_ERR_INVALID_ARG;
        if (numel[i] == 0) continue;
        const void* o = outs ? outs[i] : in[i];
        const size_t b = (size_t)numel[i] * z;
        if (!in[i] || !o || misaligned(in[i], z) || misaligned(o, z) || (o != in[i] && overlap(o, b, in[i], b)) ||
            overlap(workspace, workspace_bytes, o, b) || overlap(workspace, workspace_bytes, in[i], b))
            return MOE_ERR_INVALID_ARG;
    }
    const size_t need = moe_grad_norm_workspace_size(numel, n_tensors);
    if (workspace_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
    if (clip)
        if (int st = check_spans(in, outs, numel, dtypes, n_tensors, norm, workspace, need)) return st;
    if (int st = check_device(nullptr)) return st;
    double* parts = static_cast<double*>(workspace);
    if (n_tensors <= kFewTensors)
        return run<kFewTensors>(in, outs, numel, dtypes, n_tensors, clip, max_norm, norm, parts, stream);
    return run<kTensors>(in, outs, numel, dtypes, n_tensors, clip, max_norm, norm, parts, stream);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

MOE_API size_t moe_grad_norm_workspace_size(const int64_t* numel, int n_tensors) {
    if (n_tensors < 0 || (n_tensors > 0 && !numel)) return 0;
    for (int i = 0; i < n_tensors; ++i)
        if (numel[i] < 0) return 0;
    return (size_t)(n_tensors ? launches_of(n_tensors) : 1) * kMaxBlocks * sizeof(double);
}

MOE_API int moe_grad_norm(const void* const* tensors, const int64_t* numel, const int32_t* dtypes, int n_tensors,
                          float* norm, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
    return norm_impl(tensors, numel, dtypes, n_tensors, false, 0.f, nullptr, norm, workspace, workspace_bytes,
                     (cudaStream_t)stream);
}

MOE_API int moe_clip_grad_norm(void* const* tensors, const int64_t* numel, const int32_t* dtypes, int n_tensors,
                               float max_norm, void* const* outs, float* norm, void* workspace, size_t workspace_bytes,
                               moe_stream_t stream) {
    return norm_impl(const_cast<const void* const*>(tensors), numel, dtypes, n_tensors, true, max_norm, outs, norm, workspace,
                     workspace_bytes, (cudaStream_t)stream);
}

}  // extern "C"
