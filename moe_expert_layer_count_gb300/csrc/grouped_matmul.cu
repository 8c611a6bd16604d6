// Matrix products of ragged row groups with one 16-bit weight matrix per group (the
// experts of an MoE layer in training, or served from 16-bit weights), on the
// 5th-generation tensor cores (tcgen05, sm_103a):
//   forward   y[r]  = W_l x[r]                     for the rows r of group l
//   dgrad     dx[r] = W_l^T dy[r]
//   wgrad     dW_l  = sum over the rows r of group l of dy[r] x[r]^T   (0 if it has none)
//
// Two CTAs (one cluster, two neighbouring SMs) work on one 256-row tile with
// tcgen05.mma.cta_group::2; each holds 128 rows of A and half of B's columns in shared
// memory and 128 rows of the fp32 accumulator in TMEM.
//  * forward and dgrad compute the transposed product: the M side (256 rows) runs over the
//    weights' outputs, which have no ragged edge, and the N side over a group's rows. N may
//    be any multiple of 16 up to 256, so a group of c rows costs ceil(c / 16) * 16 columns
//    and not a multiple of 128, and a group of a few rows (decode) just streams its weights.
//  * wgrad: M over n_out, N over k_in, the sum over the group's rows in steps of 64. The
//    last step's rows past the group's end are another group's (or anything): a warp of each
//    CTA zeroes them in shared memory, in both operands (0 * NaN is NaN).
// The operand that TMA loads with its reduced index outermost (the weights of dgrad, both
// operands of wgrad) is read as an MN-major tile: 64 x 64 boxes, no transposition in memory.
// A persistent grid of CTA pairs; per CTA: warps 0-3 epilogue, warp 4 TMA, warp 5 MMA (issued
// by the pair's first CTA), warps 6 and 7 wgrad's ragged ends. Two TMEM accumulators, so that a tile's
// epilogue runs under the next tile's MMAs. Every pipeline wait gives up after 2 s, sets a device
// error word and ends the kernel.
//
// What it measured (one GB300, times of one call in bursts of a few tens of ms, SM clock 2070 MHz; in
// brackets after a second of load, when the power cap holds it at 1290-1575 MHz; 8192 x 8192 x 8192 in the
// library's dense product: 540-555 us):
//   one group of 8192 rows, 8192 x 8192      590-610 us forward, 596 us [700] wgrad   1.8, 1.84 PFLOP/s
//   128 groups of 512 rows, 1536 x 2048      248-257 us [292] forward, 287 us [322] wgrad   1.65, 1.44
//   65536 rows over 128 groups, Zipf 1.2     285-305 us [327] forward, 343-354 us wgrad   1.4, 1.2
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

#include <cudaTypedefs.h>

#include <atomic>
#include <climits>
#include <mutex>

#include "elem.cuh"
#include "route.cuh"
#include "sm100_ptx.cuh"

namespace moe {

__device__ int g_grouped_error;  // set to 1 when a pipeline wait ran out of time

namespace {

enum { kFwd = 0, kDgrad = 1, kWgrad = 2 };

constexpr int kPairM = 256;        // rows of a tile (both CTAs)
constexpr int kMaxN = 256;         // columns of a tile
constexpr int kDepth = 64;         // reduced index per stage: 64 16-bit values = one 128-byte swizzled row
constexpr int kOperandBytes = 128 * kDepth * 2;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kMaxStages = 6;
constexpr int kEpiWarps = 4, kTmaWarp = 4, kMmaWarp = 5, kTailWarp = 6;
constexpr int kBoxBytes = 4096;    // wgrad output box: 32 rows x 128 bytes
constexpr int kBoxes = 2;          // boxes of a warp in turn (four would cost two stages: 302 against 289 us)
// forward and dgrad stage two 32-row x 64-byte buffers per warp
template <int MODE>
__host__ __device__ constexpr int staging_bytes() { return kEpiWarps * kBoxBytes * (MODE == kWgrad ? kBoxes : 1); }
constexpr int kSmemLimit = 232448;
constexpr int kRowBoxes = 5;       // boxes of 8, 16, 32, 64, 128 rows
template <int MODE>
__host__ __device__ constexpr int threads_of() { return MODE == kWgrad ? 256 : 192; }  // the tail warps are wgrad's
constexpr int kBuckets = 128;      // steps of cost that the groups are sorted by
constexpr int kSms = 152;           // what a workspace size is computed for
constexpr int kMaxDevices = 64;
constexpr uint64_t kTimeoutNs = 2000000000ull;

struct Maps {
    CUtensorMap a;             // M side: weights (forward, dgrad) or dy (wgrad)
    CUtensorMap b[kRowBoxes];  // N side: rows in boxes of 8 << i (forward, dgrad); b[0]: x (wgrad)
    CUtensorMap o;             // wgrad's output
};

struct __align__(8) Tail {
    uint64_t full[kMaxStages];   // first CTA: both CTAs' loads of a stage have landed
    uint64_t empty[kMaxStages];
    uint64_t land[kMaxStages];   // wgrad: this CTA's loads of a group's ragged last stage have landed
    uint64_t ready[kMaxStages];  // wgrad, first CTA: both CTAs have zeroed what the stage must not hold
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort;
    int tiles;
    int bucket[kBuckets];
};

// Shared memory without the stages: alignment, staging, the groups, barriers.
template <int MODE>
size_t fixed_smem(int El) { return 1024 + staging_bytes<MODE>() + sizeof(Tail) + (size_t)El * 16; }


// ------------------------------------------------------------------ PTX of the CTA pair
__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of this CTA's shared variable `a` in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t map_to(uint32_t a, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
// Arrivals on a barrier of the pair's other CTA. With nothing in memory to publish (an accumulator that
// has been read, ordered by tcgen05.fence) the arrival is relaxed; without a scope it would be a release
// among this CTA's threads, which says nothing to the other CTA.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The arrival that makes this warp's shared-memory writes visible to the other CTA's waiter (which takes
// wait_phase<true>). It waits for the thread's own global stores; the tail warps have none.
__device__ __forceinline__ void arrive_cluster_release(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(1000000u)
        : "memory");
    return ok != 0;
}
// Tile loads whose completion may count on the barrier of the pair's other CTA.
__device__ __forceinline__ void load_2d_pair(uint32_t dst, const CUtensorMap* m, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void load_3d_pair(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void store_3d(const CUtensorMap* m, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(cols) : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t t, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(t), "r"(cols) : "memory");
}
// D[tmem of both CTAs] (+)= A * B^T over 16 values of the reduced index, 16-bit operands.
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives on `bar` of both CTAs once the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

// Shared-memory descriptor of 16 values of the reduced index (the i-th) of an operand tile with
// the 128-byte swizzle; `addr`: its address / 16. K-major (the reduced index innermost): rows
// of 128 bytes, groups of 8 rows 1024 bytes apart (stride offset). MN-major: boxes of 64
// values x kDepth rows of 128 bytes, the boxes 8192 bytes apart (leading offset), groups of 8
// rows of the reduced index 1024 bytes apart.
template <bool kMn>
__device__ __forceinline__ uint64_t operand(uint32_t addr, int i) {
    const uint32_t lo = addr + (uint32_t)i * (kMn ? 2048 >> 4 : 32 >> 4) | (kMn ? kOperandBytes / 2 >> 4 : 1u) << 16;
    constexpr uint32_t hi = 1024 >> 4 | 1u << 14 | 2u << 29;  // stride offset, version, 128-byte swizzle
    return (uint64_t)hi << 32 | lo;
}

template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// TMEM columns [t, t + N) of this warp's 32 lanes: thread i gets lane i.
__device__ __forceinline__ void load_columns(uint32_t t, uint32_t (&r)[32]) { ptx::tmem_ld_32x32b_x32(t, r); }
__device__ __forceinline__ void load_columns(uint32_t t, uint32_t (&r)[64]) {
    ptx::tmem_ld_32x32b_x32(t, *reinterpret_cast<uint32_t(*)[32]>(r));
    ptx::tmem_ld_32x32b_x32(t + 32, *reinterpret_cast<uint32_t(*)[32]>(r + 32));
}
__device__ __forceinline__ void wait_columns(uint32_t (&r)[32]) { ptx::tmem_wait_ld_regs32(r); }
__device__ __forceinline__ void wait_columns(uint32_t (&r)[64]) {
    ptx::tmem_wait_ld_regs32(*reinterpret_cast<uint32_t(*)[32]>(r));
    ptx::tmem_wait_ld_regs32(*reinterpret_cast<uint32_t(*)[32]>(r + 32));
}
// 16 lanes x 32 columns as 8 x 8 fragments: registers 4i .. 4i + 3 of thread T hold columns
// 8i + 2 (T % 4) and the next of lane T / 4, then of lane T / 4 + 8.
__device__ __forceinline__ void load_fragments16(uint32_t t, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t)
        : "memory");
}
// The warp's 32 lanes x 32 columns: lanes 0-15 in r[0..15], lanes 16-31 in r[16..31].
__device__ __forceinline__ void load_fragments(uint32_t t, uint32_t (&r)[32]) {
    load_fragments16(t, r);
    load_fragments16(t + (16u << 16), r + 16);
}
// Four 8 x 8 fragments of 16-bit values, transposed; lane i addresses row i % 8 of fragment i / 8.
__device__ __forceinline__ void store_transposed(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}
// Two fp32 rounded to O, the first in the low half.
template <typename O>
__device__ __forceinline__ uint32_t pack2(uint32_t lo, uint32_t hi) {
    Vec<O, 2> v;
    v.v[0] = from_f32<O>(__uint_as_float(lo));
    v.v[1] = from_f32<O>(__uint_as_float(hi));
    return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Instruction descriptor of kind::f16 for M = 256 without N (N / 8 goes to bit 17).
uint32_t idesc_base(int mode, int dtype) {
    const uint32_t f = dtype == MOE_DT_BF16 ? 1u : 0u;
    return 1u << 4 | f << 7 | f << 10 | (mode != kFwd ? 1u << 15 : 0u) | (mode == kWgrad ? 1u << 16 : 0u) |
           (uint32_t)(kPairM >> 4) << 24;
}

// Waits for a phase; false when the kernel was given up or the time ran out. kCluster: the barrier's
// arrivals come from both CTAs and publish, or hand over, what the waiter uses next.
template <bool kCluster = false>
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int* abort, bool check_abort = true) {
    auto done = [&] { return kCluster ? try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity); };
    if (done()) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
        if (done()) return true;
        if ((i & 31) == 0) {
            if (check_abort && *abort) return false;
            if (ptx::globaltimer_ns() - t0 > kTimeoutNs) {
                *abort = 1;
                atomicExch(&g_grouped_error, 1);
                return false;
            }
        }
    }
}

// ------------------------------------------------------------------ tiles
// A group of rows: its first row, its row count, its number (low 16 bits of `id`) and, forward
// and dgrad, its first tile and the rows of each of its tiles (high 16 bits of `id`; equal
// parts of at most 256, whole 16s). wgrad has the groups in falling order of rows.
struct __align__(16) Group {
    int start, lo, rows;
    uint32_t id;
};
// ceil(n / d) for n >= 0, without n + d overflowing.
__device__ __forceinline__ int ceil_div(int n, int d) { return n > 0 ? (n - 1) / d + 1 : 0; }
// wgrad: the bucket of a group of so many rows, four buckets an octave, the largest first.
__device__ __forceinline__ int bucket_of(int rows) {
    return kBuckets - 1 - ((int)(__float_as_uint((float)rows + 1.f) >> 21) - 508);
}

// i / d for 0 <= i < 2^31 by a multiplication; magic_of(d) = floor(2^32 / d) + 1 overshoots by
// less than one.
uint32_t magic_of(int64_t d) { return d == 1 ? 0 : (uint32_t)((1ull << 32) / (uint64_t)d + 1); }
struct Divisor {
    int d;
    uint32_t magic;
    __device__ __forceinline__ int of(int i) const {
        if (d == 1) return i;
        const int q = (int)__umulhi((uint32_t)i, magic);
        return q * (int64_t)d > i ? q - 1 : q;
    }
};
struct Shape {
    Divisor m_tiles;      // tiles along the M side
    Divisor group_tiles;  // wgrad: tiles of a group, all its parts'
    Divisor part_tiles;   // wgrad: tiles of one part
    int parts;            // wgrad: parts that a group's rows are split into
    int depth;            // forward, dgrad: the reduced length
};

// Where a tile lies. forward, dgrad: outputs [m0, m0 + 256) x rows [lo, lo + rows) of group
// l, n = rows rounded up to 16. wgrad: [m0, m0 + 256) x [n0, n0 + 256) of the part-th sum of
// dW_l, over rows [lo, lo + rows). steps: stages of the reduced index.
struct Tile {
    int l, part, lo, rows, m0, n0, n, steps;
};

// All lanes of a warp call it together (forward and dgrad look the group up with two votes).
template <int MODE>
__device__ __forceinline__ Tile tile_at(int tile, const Group* groups, int El, const Shape& sh) {
    Tile t;
    if (MODE == kWgrad) {
        const int at = sh.group_tiles.of(tile);
        int i = tile - at * sh.group_tiles.d;
        t.part = sh.part_tiles.of(i);
        i -= t.part * sh.part_tiles.d;
        const int p = sh.m_tiles.of(i);
        const Group g = groups[at];
        t.l = g.id & 0xffff;
        t.m0 = (i - p * sh.m_tiles.d) * kPairM;
        t.n0 = p * kMaxN;
        t.n = kMaxN;
        t.lo = g.lo;
        t.rows = g.rows;
        t.steps = ceil_div(t.rows, kDepth);
        if (sh.parts > 1) {  // whole steps to every part
            const int from = (int)((int64_t)t.steps * t.part / sh.parts), to = (int)((int64_t)t.steps * (t.part + 1) / sh.parts);
            t.lo += from * kDepth;
            t.rows = min(t.rows - from * kDepth, (to - from) * kDepth);
            t.steps = to - from;
        }
    } else {
        // the last group whose first tile is not past this one (an empty group starts where
        // the next one does): the block of `stride` groups, then the group
        const int lane = threadIdx.x & 31, stride = (El + 31) >> 5;
        int l = lane * stride;
        l = __popc(__ballot_sync(0xffffffffu, l < El && groups[l].start <= tile)) * stride - stride;
        l += __popc(__ballot_sync(0xffffffffu, lane < stride && l + lane < El && groups[l + lane].start <= tile)) - 1;
        const Group g = groups[l];
        const int i = tile - g.start, per = g.id >> 16;
        const int p = sh.m_tiles.of(i);
        t.l = g.id & 0xffff;
        t.m0 = (i - p * sh.m_tiles.d) * kPairM;
        t.lo = g.lo + p * per;
        t.rows = min(per, g.rows - p * per);
        t.n = (t.rows + 15) & ~15;
        t.n0 = t.part = 0;
        t.steps = ceil_div(sh.depth, kDepth);
    }
    return t;
}

// wgrad: whether stage k of a tile ends between two multiples of 16 rows, so that the MMAs
// would read rows past the group's end.
__device__ __forceinline__ bool ragged(const Tile& t, int k) { return k + 1 == t.steps && (t.rows & 15) != 0; }

__device__ __forceinline__ int warp_prefix(int v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int w = __shfl_up_sync(0xffffffffu, v, o);
        if ((int)(threadIdx.x & 31) >= o) v += w;
    }
    return v;
}

template <int MODE, typename O>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads_of<MODE>(), 1)
    grouped_kernel(const __grid_constant__ Maps maps, const int32_t* __restrict__ off, const int32_t* __restrict__ cnt,
                   int El, int R, int N, int K, Shape sh, uint32_t idesc0, int stages, O* __restrict__ out) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* staging = smem + stages * kStageBytes;
    Group* groups = reinterpret_cast<Group*>(staging + staging_bytes<MODE>());
    Tail* st = reinterpret_cast<Tail*>(groups + El);
    volatile int* abort = &st->abort;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();
    const int P = MODE == kDgrad ? K : N;  // length of the M side

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            ptx::mbar_init(ptx::smem_addr(&st->full[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&st->empty[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&st->land[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&st->ready[s]), 2);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(ptx::smem_addr(&st->tfull[b]), 1);
            ptx::mbar_init(ptx::smem_addr(&st->tempty[b]), 2 * kEpiWarps);
        }
        ptx::mbar_init(ptx::smem_addr(&st->mma_done), 1);
        st->abort = 0;
        ptx::fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc_pair(ptx::smem_addr(&st->tmem_base), 512);
        tmem_relinquish_pair();
        ptx::tc_fence_before();
    }
    pdl_wait();
    pdl_trigger();
    // the groups' rows, never outside [0, R)
    Group* unsorted = MODE == kWgrad ? reinterpret_cast<Group*>(smem) : groups;  // in the still unused stages
    if (MODE == kWgrad) {
        for (int i = threadIdx.x; i < kBuckets; i += threads_of<MODE>()) st->bucket[i] = 0;
        __syncthreads();
    }
    for (int l = threadIdx.x; l < El; l += threads_of<MODE>()) {
        const int lo = min(max(__ldg(off + l), 0), R);
        const int end = cnt ? (int)min((int64_t)lo + max(__ldg(cnt + l), 0), (int64_t)R) : min(__ldg(off + l + 1), R);
        const int rows = max(end - lo, 0);
        const int parts = max(ceil_div(rows, kMaxN), 1);
        const int per = (ceil_div(rows, parts) + 15) & ~15;
        const int b = MODE == kWgrad ? bucket_of(rows) : 0;
        unsorted[l] = Group{b, lo, rows, (uint32_t)per << 16 | l};
        if (MODE == kWgrad) atomicAdd(&st->bucket[b], 1);
    }
    __syncthreads();
    if (warp == 0) {
        if (MODE == kWgrad) {
            // a counting sort that every CTA does alike: the first place of every bucket (lane i
            // has buckets [4i, 4i + 4)), then the groups in their order
            int n[kBuckets / 32], sum = 0;
#pragma unroll
            for (int i = 0; i < kBuckets / 32; ++i) {
                n[i] = sum;
                sum += st->bucket[lane * (kBuckets / 32) + i];
            }
            const int before = warp_prefix(sum) - sum;
#pragma unroll
            for (int i = 0; i < kBuckets / 32; ++i) st->bucket[lane * (kBuckets / 32) + i] = before + n[i];
            __syncwarp();
            for (int l0 = 0; l0 < El; l0 += 32) {
                const bool in = l0 + lane < El;
                const Group g = in ? unsorted[l0 + lane] : Group{-1, 0, 0, 0};
                const unsigned same = __match_any_sync(0xffffffffu, g.start);
                const int place = in ? st->bucket[g.start] + __popc(same & lanemask_lt()) : 0;
                __syncwarp();
                if (in) {
                    groups[place] = g;
                    if (same >> lane == 1u) st->bucket[g.start] = place + 1;  // the last of its bucket
                }
                __syncwarp();
            }
        } else {
            // prefix sums of the groups' tiles
            int base = 0;
            for (int l0 = 0; l0 < El; l0 += 32) {
                const int l = l0 + lane;
                const int mine = l < El ? ceil_div(groups[l].rows, kMaxN) * sh.m_tiles.d : 0;
                const int sum = warp_prefix(mine);
                if (l < El) groups[l].start = base + sum - mine;
                base += __shfl_sync(0xffffffffu, sum, 31);
            }
            if (lane == 0) st->tiles = base;
        }
    }
    if (MODE == kWgrad) ptx::fence_proxy_async_smem();  // TMA writes the stages next
    __syncthreads();
    cluster_sync();  // barriers and TMEM of both CTAs are in place
    ptx::tc_fence_after();
    const uint32_t tmem = st->tmem_base;
    const int tiles = MODE == kWgrad ? El * sh.group_tiles.d : st->tiles;
    // Pair p takes the tiles p, p + pairs, ...; wgrad, whose tiles come from the dearest to the
    // cheapest, p, 2 * pairs - 1 - p, 2 * pairs + p, ..., so that the pairs' sums stay close
    // (skewed groups of 65536 rows: 378 -> 345 us). Forward and dgrad are bound by what the SMs
    // take in from L2, not by the spread of the pairs' work: sorted, they measured no faster.
    const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
    const int turn = MODE == kWgrad ? 2 * (pairs - pair) - 1 : pairs;

    if (warp == kTmaWarp) {
        const bool lead = elect_one();
        const uint32_t pair_full = map_to(ptx::smem_addr(&st->full[0]), 0);  // both CTAs' loads count on the first's
        int s = 0;
        uint32_t ph = 0, filled = 0, landed = 0;
        bool ok = true;
        for (int tile = pair, gap = turn; ok && tile < tiles; tile += gap, gap = 2 * pairs - gap) {
            const Tile t = tile_at<MODE>(tile, groups, El, sh);
            int box = 0;  // the smallest box that holds this CTA's half of the columns
            while (MODE != kWgrad && (8 << box) < t.n / 2) ++box;
            const int row = t.lo + (int)rank * (t.n / 2);
            const int m = t.m0 + (int)rank * 128, n = t.n0 + (int)rank * 128;
            for (int k = 0; k < t.steps; ++k) {
                ok = __all_sync(0xffffffffu, wait_phase(ptx::smem_addr(&st->empty[s]), ph ^ 1, abort));
                if (!ok) break;
                const uint32_t a = ptx::smem_addr(smem + s * kStageBytes), b = a + kOperandBytes;
                const uint32_t full = ptx::smem_addr(&st->full[s]), bar = pair_full + 8 * s;
                const int d = k * kDepth;
                if (MODE == kWgrad && ragged(t, k)) {  // this CTA's tail warps come first
                    if (lead) {
                        const uint32_t land = ptx::smem_addr(&st->land[s]);
                        ptx::mbar_arrive_expect_tx(land, kStageBytes);
                        ptx::tma_load_2d(a, &maps.a, m, t.lo + d, land);
                        ptx::tma_load_2d(a + kOperandBytes / 2, &maps.a, m + 64, t.lo + d, land);
                        ptx::tma_load_2d(b, &maps.b[0], n, t.lo + d, land);
                        ptx::tma_load_2d(b + kOperandBytes / 2, &maps.b[0], n + 64, t.lo + d, land);
                    }
                    landed ^= 1u << s;
                } else {
                    if (lead) {
                        if (rank == 0)
                            ptx::mbar_arrive_expect_tx(full, MODE == kWgrad ? 2 * kStageBytes : 2 * (kOperandBytes + (1024u << box)));
                        if (MODE == kWgrad) {
                            load_2d_pair(a, &maps.a, m, t.lo + d, bar);
                            load_2d_pair(a + kOperandBytes / 2, &maps.a, m + 64, t.lo + d, bar);
                            load_2d_pair(b, &maps.b[0], n, t.lo + d, bar);
                            load_2d_pair(b + kOperandBytes / 2, &maps.b[0], n + 64, t.lo + d, bar);
                        } else {
                            if (MODE == kFwd) {
                                load_3d_pair(a, &maps.a, d, m, t.l, bar);
                            } else {
                                load_3d_pair(a, &maps.a, m, d, t.l, bar);
                                load_3d_pair(a + kOperandBytes / 2, &maps.a, m + 64, d, t.l, bar);
                            }
                            load_2d_pair(b, &maps.b[box], d, row, bar);
                        }
                    }
                    filled ^= 1u << s;
                }
                if (++s == stages) s = 0, ph ^= 1;
            }
        }
        // never leave with copies in flight: every stage's last loads must have landed
        // (`filled`, `landed`: the parity of each barrier's uses, odd after the first)
        for (int i = 0; i < stages; ++i) {
            if (rank == 0) wait_phase(ptx::smem_addr(&st->full[i]), (filled >> i & 1) ^ 1, abort, false);
            if (MODE == kWgrad) wait_phase(ptx::smem_addr(&st->land[i]), (landed >> i & 1) ^ 1, abort, false);
        }
    } else if (warp == kMmaWarp) {
        if (rank == 0) {
            // the whole warp runs the loop, so that what the MMAs take stays in uniform registers;
            // one elected lane issues
            const bool lead = elect_one();
            const uint32_t base = ptx::smem_addr(smem) >> 4;
            int s = 0, b = 0;
            uint32_t tph = 0, filled = 0, landed = 0;
            bool ok = true;
            for (int tile = pair, gap = turn; ok && tile < tiles; tile += gap, gap = 2 * pairs - gap) {
                const Tile t = tile_at<MODE>(tile, groups, El, sh);
                if (t.steps == 0) continue;
                const uint32_t idesc = idesc0 | (uint32_t)(t.n >> 3) << 17;
                const uint32_t d = tmem + (uint32_t)(b * kMaxN);
                ok = __all_sync(0xffffffffu, wait_phase<true>(ptx::smem_addr(&st->tempty[b]), tph ^ 1, abort));
                if (!ok) break;
                for (int k = 0; k < t.steps; ++k) {
                    bool got;
                    if (MODE == kWgrad && ragged(t, k)) {
                        got = wait_phase<true>(ptx::smem_addr(&st->ready[s]), landed >> s & 1, abort);
                        landed ^= 1u << s;
                    } else {
                        got = wait_phase(ptx::smem_addr(&st->full[s]), filled >> s & 1, abort);
                        filled ^= 1u << s;
                    }
                    ok = __all_sync(0xffffffffu, got);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    const uint32_t a = base + (uint32_t)s * (kStageBytes >> 4), w = a + (kOperandBytes >> 4);
                    const int left = (MODE == kWgrad ? t.rows : sh.depth) - k * kDepth;
                    if (left > kDepth - 16) {
                        if (lead) {
#pragma unroll
                            for (int i = 0; i < kDepth / 16; ++i)
                                mma_pair(d, operand<MODE != kFwd>(a, i), operand<MODE == kWgrad>(w, i), idesc,
                                         i > 0 || k > 0 ? 1u : 0u);
                            commit_pair(ptx::smem_addr(&st->empty[s]));
                        }
                    } else if (lead) {
                        for (int i = 0; i * 16 < left; ++i)
                            mma_pair(d, operand<MODE != kFwd>(a, i), operand<MODE == kWgrad>(w, i), idesc, (i | k) ? 1u : 0u);
                        commit_pair(ptx::smem_addr(&st->empty[s]));
                    }
                    if (++s == stages) s = 0;
                }
                if (ok && lead) commit_pair(ptx::smem_addr(&st->tfull[b]));
                if (++b == 2) b = 0, tph ^= 1;
            }
            // never leave with MMAs in flight
            if (lead) {
                commit_pair(ptx::smem_addr(&st->mma_done));
                wait_phase(ptx::smem_addr(&st->mma_done), 0, abort, false);
            }
        }
    } else if (MODE == kWgrad && warp >= kTailWarp) {
        // a group's last stage, the first warp's where it lies in an even stage (each warp sees all phases of its
        // stages' barriers; one warp alone, with the wait for its writes to reach the cluster, took longer than
        // the rest of a decode-sized tile: 512 rows over 128 groups 143.8 -> 131.6 us): the rows past the group's end within the last 16 that the MMAs
        // read become zeros in all four boxes of this CTA
        int s = 0;
        uint32_t landed = 0;
        for (int tile = pair, gap = turn; tile < tiles; tile += gap, gap = 2 * pairs - gap) {
            const Tile t = tile_at<MODE>(tile, groups, El, sh);
            if (t.steps == 0) continue;
            s = (s + t.steps - 1) % stages;
            if (ragged(t, t.steps - 1) && (s & 1) == warp - kTailWarp) {
                const bool ok = wait_phase(ptx::smem_addr(&st->land[s]), landed >> s & 1, abort);
                if (!__all_sync(0xffffffffu, ok)) break;
                landed ^= 1u << s;
                uint8_t* p = smem + s * kStageBytes;
                const int left = t.rows - (t.steps - 1) * kDepth;
                const int n = (-left & 15) * 8;  // 16-byte pieces of a box
                p += left * 128 + lane * 16;
                for (int i = lane; i < n; i += 32, p += 512)
#pragma unroll
                    for (int box = 0; box < 4; ++box)
                        *reinterpret_cast<uint4*>(p + box * (kOperandBytes / 2)) = make_uint4(0, 0, 0, 0);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) arrive_cluster_release(map_to(ptx::smem_addr(&st->ready[s]), 0));
            }
            if (++s == stages) s = 0;
        }
    } else {
        // ---------------------------------------------------------------- epilogue
        int b = 0, boxes = 0;
        uint32_t tph = 0;
        const uint32_t slab = (uint32_t)(warp * 32) << 16;
        for (int tile = pair, gap = turn; tile < tiles; tile += gap, gap = 2 * pairs - gap) {
            const Tile t = tile_at<MODE>(tile, groups, El, sh);
            const int m = t.m0 + (int)rank * 128 + warp * 32;  // this warp's first row of the tile
            if (t.steps > 0) {
                bool ok = wait_phase(ptx::smem_addr(&st->tfull[b]), tph, abort);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ptx::tc_fence_after();
            }
            const uint32_t acc = tmem + slab + (uint32_t)(b * kMaxN);
            // the accumulator is free for the MMAs once this warp has read its last columns
            auto release = [&] {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster(map_to(ptx::smem_addr(&st->tempty[b]), 0));
            };
            if constexpr (MODE == kWgrad) {
                constexpr int kCols = 128 / sizeof(O);  // columns of a 128-byte-wide box
                const int cols = min(kMaxN, K - t.n0);
                // 32 rows x 128 bytes in TMA's 128-byte swizzle, kBoxes boxes in turn
                auto put = [&](const uint32_t (&v)[kCols], int c) {
                    uint8_t* box = staging + (warp * kBoxes + boxes) * kBoxBytes;
                    if (++boxes == kBoxes) boxes = 0;
                    if (lane == 0) bulk_wait_read<kBoxes - 1>();
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        Vec<O, 16 / sizeof(O)> w;
#pragma unroll
                        for (int j = 0; j < 16 / (int)sizeof(O); ++j)
                            w.v[j] = from_f32<O>(__uint_as_float(v[q * (16 / sizeof(O)) + j]));
                        *reinterpret_cast<Vec<O, 16 / sizeof(O)>*>(box + lane * 128 + ((q ^ (lane & 7)) << 4)) = w;
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (m < P) store_3d(&maps.o, ptx::smem_addr(box), t.n0 + c, m, t.part * El + t.l);
                        ptx::bulk_commit();
                    }
                };
                uint32_t u[kCols], v[kCols];
                if (t.steps == 0) {
#pragma unroll
                    for (int j = 0; j < kCols; ++j) u[j] = 0;
                    for (int c = 0; c < cols; c += kCols) put(u, c);
                } else {
                    // the next box's columns are on their way while this one's are stored
                    auto step_box = [&](uint32_t (&now)[kCols], uint32_t (&next)[kCols], int c) {
                        wait_columns(now);
                        if (c + kCols < cols)
                            load_columns(acc + c + kCols, next);
                        else
                            release();
                        put(now, c);
                    };
                    load_columns(acc, u);
                    for (int c = 0; c < cols; c += 2 * kCols) {
                        step_box(u, v, c);
                        if (c + kCols < cols) step_box(v, u, c + kCols);
                    }
                }
            } else if constexpr (sizeof(O) == 4) {
                // lane = output column: 128 bytes of one row per store
                const bool in = m + lane < P;
                O* o = out + (int64_t)t.lo * P + m + lane;
                uint32_t u[32], v[32];
                auto step_rows = [&](uint32_t (&now)[32], uint32_t (&next)[32], int c) {
                    __syncwarp();
                    wait_columns(now);
                    if (c + 32 < t.rows)
                        load_columns(acc + c + 32, next);
                    else
                        release();
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (in && c + j < t.rows) o[(int64_t)(c + j) * P] = __uint_as_float(now[j]);
                };
                load_columns(acc, u);
                for (int c = 0; c < t.rows; c += 64) {
                    step_rows(u, v, c);
                    if (c + 32 < t.rows) step_rows(v, u, c + 32);
                }
            } else {
                // 32 rows of the result x this warp's 32 outputs at a time: read as 8 x 8 fragments,
                // transposed into shared memory (64 bytes a row, 16-byte pieces swizzled so that
                // neither side has bank conflicts), stored as 64-byte pieces of rows
                uint8_t* stage = staging + warp * kBoxBytes;
                const int piece = lane & 3;
                const bool in = m + piece * 8 < P;
                O* o = out + ((int64_t)t.lo + (lane >> 2)) * P + m + piece * 8;
                const uint32_t put_at = (uint32_t)((lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4));
                const uint32_t get_at = (uint32_t)((lane >> 2) * 64 + ((piece ^ ((lane >> 3) & 3)) << 4));
                uint32_t u[32], v[32];
                auto step_rows = [&](uint32_t (&now)[32], uint32_t (&next)[32], int c) {
                    __syncwarp();
                    wait_columns(now);
                    if (c + 32 < t.rows)
                        load_fragments(acc + c + 32, next);
                    else
                        release();
                    uint8_t* buf = stage + (c & 32) * 64;
                    const uint32_t to = ptx::smem_addr(buf) + put_at;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        store_transposed(to + i * 512, pack2<O>(now[4 * i], now[4 * i + 1]),
                                         pack2<O>(now[4 * i + 2], now[4 * i + 3]), pack2<O>(now[16 + 4 * i], now[16 + 4 * i + 1]),
                                         pack2<O>(now[16 + 4 * i + 2], now[16 + 4 * i + 3]));
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 w = *reinterpret_cast<const uint4*>(buf + get_at + i * 512);
                        if (in && c + i * 8 + (lane >> 2) < t.rows) *reinterpret_cast<uint4*>(o + (int64_t)(c + i * 8) * P) = w;
                    }
                };
                load_fragments(acc, u);
                for (int c = 0; c < t.rows; c += 64) {
                    step_rows(u, v, c);
                    if (c + 32 < t.rows) step_rows(v, u, c + 32);
                }
                __syncwarp();
            }
            if (t.steps > 0)
                if (++b == 2) b = 0, tph ^= 1;
        }
        if (MODE == kWgrad && lane == 0) ptx::bulk_wait0();
    }
    __syncwarp();
    __syncthreads();
    cluster_sync();  // no CTA leaves while the other still signals its barriers or uses its TMEM
    if (warp == kMmaWarp) {
        // The MMAs' completions are signalled to both CTAs by the hardware, outside of any thread's order: the
        // first CTA has seen the last of them, the second may not leave before it has arrived there too (its
        // shared memory may by then be another kernel's).
        if (rank == 1) wait_phase(ptx::smem_addr(&st->mma_done), 0, abort, false);
        __syncwarp();
        ptx::tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ------------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// Tensor [z, y, x] (z = 1: two dimensions) of 2- or 4-byte elements, boxes of box_y rows x 128
// bytes with the 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* base, int esize, uint64_t x, uint64_t y, uint64_t z, uint32_t box_y, int dims) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t size[3] = {x, y, z}, stride[2] = {x * esize, x * y * esize};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / esize), box_y, 1}, one[3] = {1, 1, 1};
    return fn(m, esize == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, (cuuint32_t)dims,
              const_cast<void*>(base), size, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

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

template <int MODE, typename O>
int launch_grouped(const void* a, const void* b, const int32_t* off, const int32_t* cnt, int El, int64_t R, int N, int K,
                   int dtype, void* out, int parts, int num_sms, cudaStream_t stream) {
    Maps maps{};
    bool ok = true;
    if (MODE == kWgrad) {
        const uint64_t rows = R > 0 ? (uint64_t)R : 1;  // R = 0: nothing is loaded
        const void* any = out;
        ok = make_map(&maps.a, R > 0 ? a : any, 2, N, rows, 1, kDepth, 2) &&
             make_map(&maps.b[0], R > 0 ? b : any, 2, K, rows, 1, kDepth, 2) &&
             make_map(&maps.o, out, sizeof(O), K, N, (uint64_t)El * parts, 32, 3);
    } else {
        ok = make_map(&maps.a, b, 2, K, N, El, MODE == kFwd ? 128 : kDepth, 3);
        for (int i = 0; i < kRowBoxes; ++i) ok = ok && make_map(&maps.b[i], a, 2, MODE == kFwd ? K : N, R, 1, 8u << i, 2);
    }
    if (!ok) return MOE_ERR_CUDA;
    int dev = 0;
    static std::atomic<bool> attr_set[kMaxDevices];
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MOE_ERR_CUDA;
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(grouped_kernel<MODE, O>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit) !=
            cudaSuccess)
            return MOE_ERR_CUDA;
        attr_set[dev].store(true, std::memory_order_release);
    }
    int stages = (int)((kSmemLimit - fixed_smem<MODE>(El)) / kStageBytes);
    if (stages > kMaxStages) stages = kMaxStages;
    const size_t smem = fixed_smem<MODE>(El) + (size_t)stages * kStageBytes;
    const int64_t m_tiles = ((int64_t)(MODE == kDgrad ? K : N) + kPairM - 1) / kPairM;
    const int64_t part_tiles = m_tiles * (((int64_t)K + kMaxN - 1) / kMaxN), group_tiles = part_tiles * parts;
    const Shape sh{{(int)m_tiles, magic_of(m_tiles)}, {(int)group_tiles, magic_of(group_tiles)},
                   {(int)part_tiles, magic_of(part_tiles)}, parts, MODE == kDgrad ? N : K};
    // no more pairs than tiles (an upper bound: the groups' sizes are not known here)
    const int64_t most = MODE == kWgrad ? El * group_tiles : (R / kMaxN + (R < El ? R : El)) * m_tiles;
    const int pairs = (int)(most < num_sms / 2 ? most : num_sms / 2);
    launch_k(grouped_kernel<MODE, O>, 2 * pairs, threads_of<MODE>(), smem, stream, maps, off, cnt, El, (int)R, N, K,
             sh, idesc_base(MODE, dtype), stages, static_cast<O*>(out));
    note_launches(1);
    return launch_status();
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
    // tiles are counted in 32 bits
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

int read_grouped_error(int clear) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_grouped_error, sizeof(int)) != cudaSuccess) return -1;
    if (clear && v) {
        const int z = 0;
        cudaMemcpyToSymbol(g_grouped_error, &z, sizeof(int));
    }
    return v;
}

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
