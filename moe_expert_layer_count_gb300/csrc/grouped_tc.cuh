// The kernel behind the matrix products of ragged row groups with one 16-bit weight matrix per
// group, on the 5th-generation tensor cores (tcgen05, sm_103a): forward, its two gradients, and the
// gated forms with an activation in the epilogue. Included by the files that launch it.
//
// Two CTAs (one cluster, two neighbouring SMs) work on one 256-row tile with
// tcgen05.mma.cta_group::2; each holds 128 rows of A and half of B's columns in shared
// memory and 128 rows of the fp32 accumulator in TMEM.
//  * forward and dgrad compute the transposed product: the M side (256 rows) runs over the
//    weights' outputs, which have no ragged edge, and the N side over a group's rows. N may
//    be any multiple of 16 up to 256, so a group of c rows costs ceil(c / 16) * 16 columns
//    and not a multiple of 128, and a group of a few rows (decode) just streams its weights.
//  * the gated forward product's 256 rows are 128 outputs' gate rows and up rows, 16 and 16 by
//    turns, so that an epilogue thread has both of an output in its registers.
//  * wgrad: M over n_out, N over k_in, the sum over the group's rows in steps of 64. The
//    last step's rows past the group's end are another group's (or anything): a warp of each
//    CTA zeroes them in shared memory, in both operands (0 * NaN is NaN).
// The operand that TMA loads with its reduced index outermost (the weights of dgrad, both
// operands of wgrad) is read as an MN-major tile: 64 x 64 boxes, no transposition in memory.
// A persistent grid of CTA pairs; per CTA: warps 0-3 epilogue, warp 4 TMA, warp 5 MMA (issued
// by the pair's first CTA), warps 6 and 7 wgrad's ragged ends, or warps 6-17 the gated forms' epilogues
// too. Two TMEM accumulators, so that a tile's epilogue runs under the next tile's MMAs. Every pipeline
// wait gives up after 2 s, sets a device error word and ends the kernel.
#pragma once

#include <atomic>
#include <climits>
#include <type_traits>

#include "ckpt.cuh"
#include "elem.cuh"
#include "route.cuh"
#include "sm100_ptx.cuh"
#include "tensor_map.cuh"
#include "tile_rows.cuh"

namespace moe {

namespace {

__device__ int g_grouped_error;  // set to 1 when a pipeline wait ran out of time; one for each file with kernels

// kGated: two forward products of the same rows (gate and up) whose results meet in the epilogue;
// kGatedBwd: dgrad with the activation's gradients in the epilogue.
enum { kFwd = 0, kDgrad = 1, kWgrad = 2, kGated = 3, kGatedBwd = 4 };
__host__ __device__ constexpr bool like_fwd(int mode) { return mode == kFwd || mode == kGated; }
__host__ __device__ constexpr bool like_dgrad(int mode) { return mode == kDgrad || mode == kGatedBwd; }

constexpr int kPairM = 256;        // rows of a tile (both CTAs)
constexpr int kDepth = 64;         // reduced index per stage: 64 16-bit values = one 128-byte swizzled row
constexpr int kOperandBytes = 128 * kDepth * 2;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kMaxStages = 6;
constexpr int kEpiWarps = 4, kTmaWarp = 4, kMmaWarp = 5, kTailWarp = 6;
constexpr int kBoxBytes = 4096;    // wgrad output box: 32 rows x 128 bytes
constexpr int kScaleBytes = 256 * 8;  // kGated: a tile's scale bytes, 4 of gate and 4 of up a row
constexpr int kBoxes = 2;          // boxes of a warp in turn (four would cost two stages: 302 against 289 us)
// The gated forms' epilogues take kStep rows at a time and have kSets warps for each quarter of the
// accumulator's lanes, whose steps' chains of loads, special functions and exchanges overlap.
constexpr int kStep = 8, kSets = 4;
template <int MODE>
__host__ __device__ constexpr int epi_warps() { return MODE == kGated || MODE == kGatedBwd ? kSets * kEpiWarps : kEpiWarps; }
// a warp's kStep rows of the gated forms: 64 bytes of gate and up (kGatedBwd: of each) and h of 32 (kGatedBwd: 64)
template <int MODE>
__host__ __device__ constexpr int gated_bytes() { return kStep * (MODE == kGatedBwd ? 192 : 96); }
// forward and dgrad stage two 32-row x 64-byte buffers per warp
template <int MODE>
__host__ __device__ constexpr int staging_bytes() {
    if (MODE == kGated) return epi_warps<MODE>() * gated_bytes<MODE>() + 2 * kScaleBytes + kSets * 8;  // and a barrier for each set
    return epi_warps<MODE>() * (MODE == kGatedBwd ? gated_bytes<MODE>() : kBoxBytes * (MODE == kWgrad ? kBoxes : 1));
}
// results along the M side of a tile: kGated's rows are half gate and half up
template <int MODE>
__host__ __device__ constexpr int tile_outputs() { return MODE == kGated ? kPairM / 2 : kPairM; }
constexpr int kSmemLimit = 232448;
constexpr int kRowBoxes = 5;       // boxes of 8, 16, 32, 64, 128 rows
template <int MODE>
__host__ __device__ constexpr int threads_of() {  // the tail warps are wgrad's
    return MODE == kWgrad ? 256 : 32 * (epi_warps<MODE>() + 2);
}
constexpr int kBuckets = 128;      // steps of cost that the groups are sorted by
constexpr int kSms = 152;           // what a workspace size is computed for
constexpr int kMaxDevices = 64;
constexpr uint64_t kTimeoutNs = 2000000000ull;

struct Maps {
    CUtensorMap a;             // M side: weights (forward, dgrad) or dy (wgrad)
    CUtensorMap b[kRowBoxes];  // N side: rows in boxes of 8 << i (forward, dgrad); b[0]: x (wgrad)
    CUtensorMap o;             // wgrad's output
};

// What the gated epilogues read and write beside `out` (h).
struct Gated {
    int act, keep;       // enum moe_activation, enum moe_keep
    const void* pre_in;  // kGatedBwd: gate and up as they were kept, [R, 2 P] (16 bits or codes)
    void* pre_out;       // kGated: gate and up to keep, or null; kGatedBwd: their gradients (16 bits)
    uint8_t* scale;      // the codes' scale bytes [R, 2 P / 16]: written by kGated, read by kGatedBwd
};

// Forward and dgrad go through the parts, all tiles along the M side of one after the other. A part of a long
// group finds its weights in L2, where the group's other parts have left them, and is bound by the MMAs; a group of one
// part is bound by its weights' way from DRAM: one kind after the other, each leaves idle what bounds the other. So
// the two kinds are taken by turns in proportion, where there is enough of both (by_turns); else all groups are
// taken in their own order, as groups of several parts.
struct Order {
    int singles, several;       // groups
    int single_parts, parts;    // parts of the former; of all groups
    uint32_t step;              // about 2^32 * single_parts / parts
    // How many of the first `part` parts are groups of their own: it grows by 0 or 1 a part and leaves, at
    // either end, as many of each kind as there are.
    __device__ __forceinline__ int singles_before(int part) const {
        return min(max((int)__umulhi((uint32_t)part, step), part - (parts - single_parts)), single_parts);
    }
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
    int bucket[kBuckets];        // wgrad
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
__device__ __forceinline__ void load_4d_pair(uint32_t dst, const CUtensorMap* m, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
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
// The warp's 32 lanes x 8 columns: lanes 0-15 in r[0..3], lanes 16-31 in r[4..7].
__device__ __forceinline__ void load_fragments(uint32_t t, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(t)
                 : "memory");
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(t + (16u << 16))
                 : "memory");
}
__device__ __forceinline__ void wait_columns(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
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
// Two of them; lanes 0-15 give the addresses.
__device__ __forceinline__ void store_transposed(uint32_t addr, uint32_t a, uint32_t b) {
    asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
// The other way: four 8 x 8 fragments read from rows of 16 bytes, transposed.
__device__ __forceinline__ void load_transposed(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
                 : "r"(addr)
                 : "memory");
}
// Two fp32 rounded to O, the first in the low half.
template <typename O>
__device__ __forceinline__ uint32_t pack2(uint32_t lo, uint32_t hi) {
    return pack2_f32<O>(__uint_as_float(lo), __uint_as_float(hi));
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Instruction descriptor of kind::f16 for M = 256 without N (N / 8 goes to bit 17).
uint32_t idesc_base(int mode, int dtype) {
    const uint32_t f = dtype == MOE_DT_BF16 ? 1u : 0u;
    return 1u << 4 | f << 7 | f << 10 | (!like_fwd(mode) ? 1u << 15 : 0u) | (mode == kWgrad ? 1u << 16 : 0u) |
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

// ------------------------------------------------------------------ activations
constexpr float kGeluA = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Both activations are a(g) = g s with s = 1 / (1 + exp(-q)): q = g for SiLU and, since
// (1 + tanh z) / 2 = 1 / (1 + exp(-2 z)), q = 2 sqrt(2 / pi) (g + 0.044715 g^3) for GELU's tanh form. The cubic and
// exp(-q) may overflow: s is 0 or 1 then, as it should be. A NaN gate makes s NaN, so no step of this may take its
// place by a number (the smaller or larger of NaN and a bound is the bound). Exponential and reciprocal are the
// approximate ones, which flush what is subnormal: a few fp32 ulp where the result is rounded to 16 bits (the forms that
// keep subnormals cost another seven instructions a value), but s below 2^-126 is 0: |a| below 2^-119 may be 0.
// Two values at once: products and sums in packed instructions.
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
template <bool kGelu>
__device__ __forceinline__ float2 act_gate(float2 g) {
    float2 q;
    if (kGelu)
        q = __fmul2_rn(g, __ffma2_rn(both(-kLog2e * kGeluA * kGeluB), __fmul2_rn(g, g), both(-kLog2e * kGeluA)));
    else
        q = __fmul2_rn(both(-kLog2e), g);
    const float2 d = __fadd2_rn(both(1.f), make_float2(ex2_approx(q.x), ex2_approx(q.y)));
    return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}
template <bool kGelu>
__device__ __forceinline__ float2 act_of(float2 g) { return __fmul2_rn(g, act_gate<kGelu>(g)); }
// a(g) and its derivative s + g q' s (1 - s), q' = 1 or 2 sqrt(2 / pi) (1 + 3 * 0.044715 g^2). GELU's g q' is taken at
// most at |g| = 32, where s (1 - s) is 0 already, since infinity times that were NaN; 0 * g leaves it as it is but where g
// is infinite or NaN: there the derivative is NaN, as by its formula, for both activations.
template <bool kGelu>
__device__ __forceinline__ void act_and_slope(float2 g, float2& a, float2& slope) {
    const float2 s = act_gate<kGelu>(g);
    a = __fmul2_rn(g, s);
    float2 gq = g;
    if (kGelu) {
        const float2 c = make_float2(fminf(fmaxf(g.x, -32.f), 32.f), fminf(fmaxf(g.y, -32.f), 32.f));
        gq = __ffma2_rn(both(0.f), g, __fmul2_rn(c, __ffma2_rn(both(3.f * kGeluA * kGeluB), __fmul2_rn(c, c), both(kGeluA))));
    }
    slope = __ffma2_rn(__ffma2_rn(make_float2(-s.x, -s.y), s, s), gq, s);
}

// ------------------------------------------------------------------ tiles
// A group of rows: its first row, its row count, its number (low 16 bits of `id`) and, forward
// and dgrad, its first part and the rows of each of its parts (high 16 bits of `id`; equal
// parts of at most 256, whole 16s). wgrad has the groups in falling order of rows; forward and dgrad
// have the groups of several parts in their own order from the front, the others from the back, and
// count both kinds' parts from 0.
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

struct Shape {
    Divisor m_tiles;      // tiles along the M side
    Divisor group_tiles;  // wgrad: tiles of a group, all its parts'
    Divisor part_tiles;   // wgrad: tiles of one part
    int parts;            // wgrad: parts that a group's rows are split into
    int depth;            // forward, dgrad: the reduced length
    float share;          // forward, dgrad: tiles along the M side for each pair of CTAs
};

// Where a tile lies. forward, dgrad: outputs [m0, m0 + 256) x rows [lo, lo + rows) of group
// l, n = rows rounded up to 16. wgrad: [m0, m0 + 256) x [n0, n0 + 256) of the part-th sum of
// dW_l, over rows [lo, lo + rows). steps: stages of the reduced index.
struct Tile {
    int l, part, lo, rows, m0, n0, n, steps;
};

// All lanes of a warp call it together (forward and dgrad look the group up with two votes).
template <int MODE>
__device__ __forceinline__ Tile tile_at(int tile, const Group* groups, const Order& order, const Shape& sh) {
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
        const int part = sh.m_tiles.of(tile), i = tile - part * sh.m_tiles.d;
        bool single = order.several == 0;
        int before = single ? part : 0;
        if (order.several > 0 && order.single_parts > 0) {
            before = order.singles_before(part);
            single = order.singles_before(part + 1) > before;
        }
        const int at = single ? before : part - before, n = single ? order.singles : order.several;
        const Group* of = single ? groups + (order.singles + order.several - 1) : groups;
        const int way = single ? -1 : 1;
        // the last group whose first part is not past this one (an empty group starts where
        // the next one does): the block of `stride` groups, then the group
        const int lane = threadIdx.x & 31, stride = (n + 31) >> 5;
        int l = lane * stride;
        l = __popc(__ballot_sync(0xffffffffu, l < n && of[way * l].start <= at)) * stride - stride;
        l += __popc(__ballot_sync(0xffffffffu, lane < stride && l + lane < n && of[way * (l + lane)].start <= at)) - 1;
        const Group g = of[way * l];
        const int p = at - g.start, per = g.id >> 16;
        t.l = g.id & 0xffff;
        t.m0 = i * tile_outputs<MODE>();
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

// Forward and dgrad put the groups in place in two steps, in each of which every warp has 32 groups at a time (one warp
// alone for all takes 200 clocks for every 32). First, for each choice of a tile's rows, how many parts of each kind
// these groups have; then, once all are known, the choice, and the groups behind those of the other warps.
struct __align__(16) Block {
    // x: groups of several parts and, in the high 16 bits, the parts of the others; y: the former's parts
    uint2 of[kRowChoices];
    unsigned rows16, longest;  // as in RowSums
};
// More parts come only of groups that lie over one another (rows are fewer than 2^31); 32 bits might not count them.
constexpr unsigned kPartsLimit = 1u << 26;

__device__ __forceinline__ void sum_groups(int rows, Block* block) {
    const unsigned any = __ballot_sync(0xffffffffu, rows > 0);
    Block b;
#pragma unroll
    for (int c = 0; c < kRowChoices; ++c) {
        const bool mine = rows > kMaxN >> c;
        const unsigned several = __ballot_sync(0xffffffffu, mine);
        b.of[c] = make_uint2(__popc(several) | __popc(any & ~several) << 16, 0);
        if (several)
            b.of[c].y = min(__reduce_add_sync(0xffffffffu, mine ? ((unsigned)rows + (kMaxN >> c) - 1) >> (8 - c) : 0), kPartsLimit);
    }
    b.rows16 = __reduce_add_sync(0xffffffffu, ((unsigned)rows + 15) >> 4);
    b.longest = __reduce_max_sync(0xffffffffu, (unsigned)rows);
    if ((threadIdx.x & 31) == 0) *block = b;
}

template <int MODE>
__device__ __forceinline__ Order place_groups(const Group* unsorted, const Block* blocks, Group* groups, int El, const Shape& sh) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Block block{};
    if (lane < (El + 31) >> 5) block = blocks[lane];
    const unsigned longest = __reduce_max_sync(0xffffffffu, block.longest);
    int down = 0;
    if (longest > kLeastN) {  // where no group is longer than the fewest rows all choices are one
        RowSums sums;
#pragma unroll
        for (int c = 0; c < kRowChoices; ++c) sums.parts[c] = __reduce_add_sync(0xffffffffu, block.of[c].y + (block.of[c].x >> 16));
        sums.rows16 = __reduce_add_sync(0xffffffffu, block.rows16);
        sums.longest = longest;
        down = choose_rows<MODE == kGatedBwd>(sums, (float)ceil_div(sh.depth, kDepth), sh.share);
    }
    const int cap = kMaxN >> down;
    uint2 of = down == 0 ? block.of[0] : down == 1 ? block.of[1] : block.of[2];
    unsigned counts = __reduce_add_sync(0xffffffffu, of.x), several_parts = __reduce_add_sync(0xffffffffu, of.y);
    // by turns (see Order), or all groups in their own order, as groups of several parts
    const bool turns = several_parts == 0 || by_turns(several_parts, counts & 0xffff, counts >> 16);
    if (!turns) {
        of = make_uint2(min(32, max(El - 32 * lane, 0)), of.y + (of.x >> 16));
        several_parts += counts >> 16;
        counts = (unsigned)El;
    }
    for (int l0 = warp * 32; l0 < El; l0 += threads_of<MODE>()) {
        const int l = l0 + lane;
        const unsigned before = __reduce_add_sync(0xffffffffu, lane < l0 >> 5 ? of.x : 0);
        Group g = l < El ? unsorted[l] : Group{0, 0, 0, 0};
        const bool several = turns ? g.rows > cap : l < El;
        const unsigned those = __ballot_sync(0xffffffffu, several), ones = __ballot_sync(0xffffffffu, g.rows > 0 && !several);
        const int several_before = (int)(before & 0xffff) + __popc(those & lanemask_lt());
        int per = g.rows;
        g.start = (int)(before >> 16) + __popc(ones & lanemask_lt());
        if (those) {
            const int mine = several ? (int)(((unsigned)g.rows + cap - 1) >> (8 - down)) : 0, sum = warp_prefix(mine);
            const int parts_before = (int)__reduce_add_sync(0xffffffffu, lane < l0 >> 5 ? of.y : 0);
            if (several) per = ceil_div(g.rows, mine), g.start = parts_before + sum - mine;
        }
        g.id |= (uint32_t)((per + 15) & ~15) << 16;
        if (l < El) groups[several ? several_before : El - 1 - (l - several_before)] = g;
    }
    const int several = (int)(counts & 0xffff), single_parts = (int)(counts >> 16);
    const unsigned all = several_parts + single_parts;
    const bool fits = several_parts < kPartsLimit && (uint64_t)all * (unsigned)sh.m_tiles.d <= INT_MAX - 4096u;  // else no tiles
    Order order{El - several, several, single_parts, fits ? (int)all : 0, 0};
    if (several > 0 && single_parts > 0)
        order.step = __float2uint_rz(fminf(__fdividef((float)single_parts, (float)all) * 4294967296.f, 4294967040.f));
    return order;
}

template <int MODE, typename O>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads_of<MODE>(), 1)
    grouped_kernel(const __grid_constant__ Maps maps, const int32_t* __restrict__ off, const int32_t* __restrict__ cnt,
                   int El, int R, int N, int K, Shape sh, uint32_t idesc0, int stages, O* __restrict__ out,
                   const Gated gated) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* staging = smem + stages * kStageBytes;
    Group* groups = reinterpret_cast<Group*>(staging + staging_bytes<MODE>());
    Tail* st = reinterpret_cast<Tail*>(groups + El);
    volatile int* abort = &st->abort;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();
    const int P = like_dgrad(MODE) ? K : N;  // length of the M side

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            ptx::mbar_init(ptx::smem_addr(&st->full[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&st->empty[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&st->land[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&st->ready[s]), 2);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(ptx::smem_addr(&st->tfull[b]), 1);
            ptx::mbar_init(ptx::smem_addr(&st->tempty[b]), 2 * epi_warps<MODE>());
        }
        ptx::mbar_init(ptx::smem_addr(&st->mma_done), 1);
        if (MODE == kGated)
            for (int set = 0; set < kSets; ++set)
                ptx::mbar_init(ptx::smem_addr(staging + epi_warps<MODE>() * gated_bytes<MODE>() + 2 * kScaleBytes + 8 * set), 4);
        st->abort = 0;
        ptx::fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc_pair(ptx::smem_addr(&st->tmem_base), 512);
        tmem_relinquish_pair();
        ptx::tc_fence_before();
    }
    if (MODE == kWgrad)
        for (int i = threadIdx.x; i < kBuckets; i += threads_of<MODE>()) st->bucket[i] = 0;
    // barriers and TMEM of both CTAs are in place; before the wait for the kernel before this one, whose last CTAs this
    // is hidden under (900 clocks)
    cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tmem = st->tmem_base;
    pdl_wait();
    pdl_trigger();
    // the groups' rows, never outside [0, R)
    Group* unsorted = reinterpret_cast<Group*>(smem);  // in the still unused stages
    Block* blocks = reinterpret_cast<Block*>(unsorted + kMaxLocalExperts);
    for (int l0 = warp * 32; l0 < El; l0 += threads_of<MODE>()) {
        const int l = l0 + lane;
        int rows = 0;
        if (l < El) {
            const int lo = min(max(__ldg(off + l), 0), R);
            const int end = cnt ? (int)min((int64_t)lo + max(__ldg(cnt + l), 0), (int64_t)R) : min(__ldg(off + l + 1), R);
            rows = max(end - lo, 0);
            const int b = MODE == kWgrad ? bucket_of(rows) : 0;
            unsorted[l] = Group{b, lo, rows, (uint32_t)l};
            if (MODE == kWgrad) atomicAdd(&st->bucket[b], 1);
        }
        if (MODE != kWgrad) sum_groups(rows, blocks + (l0 >> 5));
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
        }
    }
    Order order;
    if (MODE != kWgrad) order = place_groups<MODE>(unsorted, blocks, groups, El, sh);
    ptx::fence_proxy_async_smem();  // TMA writes the stages next
    __syncthreads();
    const int tiles = MODE == kWgrad ? El * sh.group_tiles.d : order.parts * sh.m_tiles.d;
    // Pair p takes the tiles p, p + pairs, ...; wgrad, whose tiles come from the dearest to the
    // cheapest, p, 2 * pairs - 1 - p, 2 * pairs + p, ..., so that the pairs' sums stay close
    // (skewed groups of 65536 rows: 378 -> 345 us). Forward and dgrad, sorted, measured no faster: what
    // counts there is that tiles bound by DRAM and by MMAs run at the same time (see Order).
    const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
    const int turn = MODE == kWgrad ? 2 * (pairs - pair) - 1 : pairs;

    if (warp == kTmaWarp) {
        const bool lead = elect_one();
        const uint32_t pair_full = map_to(ptx::smem_addr(&st->full[0]), 0);  // both CTAs' loads count on the first's
        int s = 0;
        uint32_t ph = 0, filled = 0, landed = 0;
        bool ok = true;
        for (int tile = pair, gap = turn; ok && tile < tiles; tile += gap, gap = 2 * pairs - gap) {
            const Tile t = tile_at<MODE>(tile, groups, order, sh);
            const int half = t.n / 2;  // this CTA's rows on the N side
            int box = 0;               // the smallest box that holds them (exact ones, several a stage, measured slower)
            while (MODE != kWgrad && (8 << box) < half) ++box;
            const int row = t.lo + (int)rank * half;
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
                            if (MODE == kGated) {
                                // every warp's 32 lanes of the accumulator: 16 gate rows, then the up rows of
                                // the same outputs
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    load_4d_pair(a + i * (kOperandBytes / 4), &maps.a, d, t.m0 + (int)rank * 64 + i * 16, 0, t.l, bar);
                            } else if (MODE == kFwd) {
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
                const Tile t = tile_at<MODE>(tile, groups, order, sh);
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
                                mma_pair(d, operand<!like_fwd(MODE)>(a, i), operand<MODE == kWgrad>(w, i), idesc,
                                         i > 0 || k > 0 ? 1u : 0u);
                            commit_pair(ptx::smem_addr(&st->empty[s]));
                        }
                    } else if (lead) {
                        for (int i = 0; i * 16 < left; ++i)
                            mma_pair(d, operand<!like_fwd(MODE)>(a, i), operand<MODE == kWgrad>(w, i), idesc, (i | k) ? 1u : 0u);
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
            const Tile t = tile_at<MODE>(tile, groups, order, sh);
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
        uint32_t tph = 0, turns = 0;
        const int quarter = warp & 3;  // of the accumulator's lanes: what a warp can read goes by its number
        const int set = warp < 4 ? 0 : (warp - 2) >> 2;
        const uint32_t slab = (uint32_t)(quarter * 32) << 16;
        for (int tile = pair, gap = turn; tile < tiles; tile += gap, gap = 2 * pairs - gap) {
            const Tile t = tile_at<MODE>(tile, groups, order, sh);
            const int m = t.m0 + (int)rank * (tile_outputs<MODE>() / 2) + quarter * (tile_outputs<MODE>() / 8);  // this warp's first output
            // kGatedBwd: a step's gate and up, row lane / 4; 16 bits: the lane's 16-byte piece of each; 8 bits: one
            // group's codes and scale, of gate or up
            uint4 in[2];
            uint32_t sc;
            auto fetch = [&](int c) {
                const int r = lane >> 2;
                const int64_t P2 = 2 * (int64_t)P, row = ((int64_t)t.lo + c + r) * P2;
                if (gated.keep == MOE_KEEP_E4M3) {
                    const int j = m + (lane & 1) * 16;
                    const bool live = j < P && c + r < t.rows;
                    const int64_t at = row + ((lane >> 1) & 1) * (int64_t)P + j;
                    const uint8_t* codes = static_cast<const uint8_t*>(gated.pre_in) + at;
                    in[0] = live ? __ldcg(reinterpret_cast<const uint4*>(codes)) : make_uint4(0, 0, 0, 0);
                    sc = live ? __ldcg(gated.scale + at / kCkptGroup) : 127u;
                } else {
                    const int j = m + (lane & 3) * 8;
                    const bool live = j < P && c + r < t.rows;
                    const O* pre = static_cast<const O*>(gated.pre_in) + row + j;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        in[i] = live ? __ldcg(reinterpret_cast<const uint4*>(pre + i * (int64_t)P)) : make_uint4(0, 0, 0, 0);
                }
            };
            if constexpr (MODE == kGatedBwd) {
                // ask for what the quarters will read while the tile's product is under way, one of them for each
                // line of 128 bytes (not at all: 28940 rows of 1376 x 512 100 -> 118 us; each quarter for itself: 102;
                // a tile ahead: 116)
                const bool eight = gated.keep == MOE_KEEP_E4M3;
                const uint8_t* p = static_cast<const uint8_t*>(gated.pre_in);
                const int64_t P2 = 2 * (int64_t)P;
                const int z = eight ? 1 : 2, first = set * kStep, r = (lane >> 1) & 7;
                if (first < t.rows) fetch(first);
                if (m < P && (quarter & (eight ? 3 : 1)) == 0)  // two steps' rows at a time
                    for (int c = first + kSets * kStep * (1 + (lane >> 4)); c + r < t.rows; c += 2 * kSets * kStep) {
                        const int64_t at = (t.lo + (int64_t)c + r) * P2 + (lane & 1) * (int64_t)P + m;
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(p + at * z) : "memory");
                    }
            }
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
            } else if constexpr (MODE == kGated) {
                // Lanes 0-15 of the accumulator are the gates of this warp's 16 outputs, lanes 16-31 their ups, so
                // that a thread's registers j and 4 + j are the gate and up of one output. Rounded to 16 bits they
                // are transposed into shared memory, rows of 64 bytes (16 gates, 16 ups) and of 32 bytes (h), and
                // leave it as 16-byte pieces of rows.
                uint8_t* stage = staging + (set * 4 + quarter) * gated_bytes<MODE>();
                uint8_t* hbuf = stage + kStep * 64;
                const uint32_t put_pre = ptx::smem_addr(stage) + (uint32_t)((lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4));
                const uint32_t put_h = ptx::smem_addr(hbuf) + (uint32_t)((lane & 7) * 32 + ((((lane >> 3) & 1) ^ ((lane >> 2) & 1)) << 4));
                const int64_t P2 = 2 * (int64_t)P;
                uint8_t* bytes = staging + epi_warps<MODE>() * gated_bytes<MODE>() + (turns & 1) * kScaleBytes;
                const int r = lane >> 2, piece = lane & 3;             // of gate and up
                const int hr = (lane >> 1) & 7, side = lane & 1;       // of h
                if (set * kStep >= t.rows) release();
#pragma unroll 1
                for (int c = set * kStep; c < t.rows; c += kSets * kStep) {
                    uint32_t v[8], h[2];
                    load_fragments(acc + c, v);
                    __syncwarp();
                    wait_columns(v);
                    if (c + kSets * kStep >= t.rows) release();
                    auto activate = [&](auto gelu) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float2 g = make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                            const float2 u = make_float2(__uint_as_float(v[4 + 2 * j]), __uint_as_float(v[5 + 2 * j]));
                            const float2 w = __fmul2_rn(act_of<decltype(gelu)::value>(g), u);
                            h[j] = pack2_f32<O>(w.x, w.y);
                        }
                    };
                    if (gated.act == MOE_ACT_SILU)
                        activate(std::false_type());
                    else
                        activate(std::true_type());
                    store_transposed(put_h, h[0], h[1]);
                    if (gated.keep != MOE_KEEP_NONE)
                        store_transposed(put_pre, pack2<O>(v[0], v[1]), pack2<O>(v[2], v[3]), pack2<O>(v[4], v[5]), pack2<O>(v[6], v[7]));
                    __syncwarp();
                    const int64_t row0 = (int64_t)t.lo + c;
                    if (lane < 16 && c + hr < t.rows && m + side * 8 < P)
                        *reinterpret_cast<uint4*>(out + (row0 + hr) * P + m + side * 8) =
                            *reinterpret_cast<const uint4*>(hbuf + hr * 32 + ((side ^ ((hr >> 2) & 1)) << 4));
                    if (gated.keep != MOE_KEEP_NONE) {
                        const uint4 w = *reinterpret_cast<const uint4*>(stage + r * 64 + ((piece ^ ((r >> 1) & 3)) << 4));
                        const int j = m + (piece & 1) * 8;
                        const int64_t at = (row0 + r) * P2 + (piece >> 1) * (int64_t)P + j;
                        const bool live = j < P && c + r < t.rows;
                        if (gated.keep == MOE_KEEP_16BIT) {
                            if (live) *reinterpret_cast<uint4*>(static_cast<O*>(gated.pre_out) + at) = w;
                        } else {
                            // two lanes have a group of the 8-bit form, made from the 16-bit values so that it
                            // equals what packing those gives
                            uint32_t byte;
                            const uint2 codes = ckpt_encode8<O>(w, byte);
                            if (live) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(gated.pre_out) + at) = codes;
                            if ((lane & 1) == 0) bytes[(c + r) * 8 + (piece >> 1) * 4 + quarter] = (uint8_t)byte;
                        }
                    }
                }
                __syncwarp();
                if (gated.keep == MOE_KEEP_E4M3) {
                    // The four quarters' bytes of a row lie side by side: the set's warps meet, and each writes every
                    // fourth step's, four bytes in a row (each in a sector of its own, as they come, they cost 14 of
                    // 285 us at 512 rows a group; a word for four is no faster). The next tile but one uses the same
                    // buffer: by then all four have been at the next one's meeting, after they had read this one's.
                    const uint32_t met = ptx::smem_addr(staging + epi_warps<MODE>() * gated_bytes<MODE>() + 2 * kScaleBytes + 8 * set);
                    if (lane == 0) ptx::mbar_arrive(met);
                    if (!__all_sync(0xffffffffu, wait_phase(met, turns & 1, abort))) break;
                    ++turns;
                    const int j = t.m0 + (int)rank * 64, n = min((P - j) / kCkptGroup, 4);
                    for (int c = set * kStep + quarter * (kSets * kStep); c < t.rows; c += 4 * kSets * kStep) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int br = i * 4 + (lane >> 3), q = lane & 3;
                            const int64_t at = (((int64_t)t.lo + c + br) * P2 + ((lane >> 2) & 1) * (int64_t)P + j) / kCkptGroup + q;
                            if (q < n && c + br < t.rows) gated.scale[at] = bytes[c * 8 + i * 32 + lane];
                        }
                    }
                }
            } else if constexpr (MODE == kGatedBwd) {
                // 8 rows x this warp's 32 outputs at a time: gate and up come in as 16-byte pieces of rows, one step
                // ahead, are laid into shared memory (64 bytes a row, swizzled) and read as the accumulator's
                // 8 x 8 fragments; the gradients go back over them and out, h beside them.
                uint8_t* gbuf = staging + (set * 4 + quarter) * gated_bytes<MODE>();
                constexpr int kUp = kStep * 64;  // up's buffer behind gate's, h's behind that
                const uint32_t frag = ptx::smem_addr(gbuf) + (uint32_t)((lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4));
                const int64_t P2 = 2 * (int64_t)P;
                const int r = lane >> 2, piece = lane & 3, j = m + piece * 8;
                uint8_t* own = gbuf + r * 64;
                const int z = (r >> 1) & 3;  // row r's swizzle
                if (set * kStep >= t.rows) release();
#pragma unroll 1
                for (int c = set * kStep; c < t.rows; c += kSets * kStep) {
                    uint32_t v[8], g[4], up[4], h[4];
                    load_fragments(acc + c, v);
                    __syncwarp();
                    if (gated.keep == MOE_KEEP_E4M3) {
                        uint8_t* row = own + (piece >> 1) * kUp;
                        uint4 lo, hi;
                        ckpt_decode16<O>(in[0], sc, lo, hi);
                        *reinterpret_cast<uint4*>(row + (((2 * (piece & 1)) ^ z) << 4)) = lo;
                        *reinterpret_cast<uint4*>(row + (((2 * (piece & 1) + 1) ^ z) << 4)) = hi;
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) *reinterpret_cast<uint4*>(own + i * kUp + ((piece ^ z) << 4)) = in[i];
                    }
                    if (c + kSets * kStep < t.rows) fetch(c + kSets * kStep);
                    __syncwarp();
                    load_transposed(frag, g[0], g[1], g[2], g[3]);
                    load_transposed(frag + kUp, up[0], up[1], up[2], up[3]);
                    wait_columns(v);
                    if (c + kSets * kStep >= t.rows) release();
                    auto gradients = [&](auto gelu) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {  // outputs 8 q .. 8 q + 7; two rows each
                            const float2 uv = unpack2<O>(up[q]), d = make_float2(__uint_as_float(v[2 * q]), __uint_as_float(v[2 * q + 1]));
                            float2 a, slope;
                            act_and_slope<decltype(gelu)::value>(unpack2<O>(g[q]), a, slope);
                            const float2 dg = __fmul2_rn(__fmul2_rn(d, uv), slope), du = __fmul2_rn(d, a), hv = __fmul2_rn(a, uv);
                            g[q] = pack2_f32<O>(dg.x, dg.y);
                            up[q] = pack2_f32<O>(du.x, du.y);
                            h[q] = pack2_f32<O>(hv.x, hv.y);
                        }
                    };
                    if (gated.act == MOE_ACT_SILU)
                        gradients(std::false_type());
                    else
                        gradients(std::true_type());
                    __syncwarp();
                    store_transposed(frag, g[0], g[1], g[2], g[3]);
                    store_transposed(frag + kUp, up[0], up[1], up[2], up[3]);
                    store_transposed(frag + 2 * kUp, h[0], h[1], h[2], h[3]);
                    __syncwarp();
                    if (j < P && c + r < t.rows) {
                        O* grads = static_cast<O*>(gated.pre_out);
                        const uint8_t* from = own + ((piece ^ z) << 4);
                        const int64_t at = (int64_t)t.lo + c + r;
                        *reinterpret_cast<uint4*>(grads + at * P2 + j) = *reinterpret_cast<const uint4*>(from);
                        *reinterpret_cast<uint4*>(grads + at * P2 + P + j) = *reinterpret_cast<const uint4*>(from + kUp);
                        if (out) *reinterpret_cast<uint4*>(out + at * P + j) = *reinterpret_cast<const uint4*>(from + 2 * kUp);
                    }
                }
                __syncwarp();
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
// kGated's weights [El][2][N][K] of 2-byte elements: boxes of 16 outputs' gate rows and up rows, 128 bytes each.
bool make_gated_map(CUtensorMap* m, const void* base, uint64_t K, uint64_t N, uint64_t El) {
    const cuuint64_t size[4] = {K, N, 2, El}, stride[3] = {K * 2, K * N * 2, K * N * 4};
    const cuuint32_t box[4] = {kDepth, 16, 2, 1};
    return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, base, size, stride, box, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// Tensor [z, y, x] (z = 1: two dimensions) of 2- or 4-byte elements, boxes of box_y rows x 128
// bytes with the 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* base, int esize, uint64_t x, uint64_t y, uint64_t z, uint32_t box_y, int dims) {
    const cuuint64_t size[3] = {x, y, z}, stride[2] = {x * esize, x * y * esize};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / esize), box_y, 1};
    return encode_map(m, esize == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, dims, base, size, stride, box,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

template <int MODE, typename O>
int launch_grouped(const void* a, const void* b, const int32_t* off, const int32_t* cnt, int El, int64_t R, int N, int K,
                   int dtype, void* out, int parts, int num_sms, cudaStream_t stream, const Gated& gated = {}) {
    Maps maps{};
    bool ok = true;
    if (MODE == kWgrad) {
        const uint64_t rows = R > 0 ? (uint64_t)R : 1;  // R = 0: nothing is loaded
        const void* any = out;
        ok = make_map(&maps.a, R > 0 ? a : any, 2, N, rows, 1, kDepth, 2) &&
             make_map(&maps.b[0], R > 0 ? b : any, 2, K, rows, 1, kDepth, 2) &&
             make_map(&maps.o, out, sizeof(O), K, N, (uint64_t)El * parts, 32, 3);
    } else {
        ok = MODE == kGated ? make_gated_map(&maps.a, b, K, N, El) : make_map(&maps.a, b, 2, K, N, El, MODE == kFwd ? 128 : kDepth, 3);
        // a CTA has half of a tile's columns, and no group has more than R rows: up to the first box that holds them
        const int half = (int)(R < kMaxN ? (R + 15) / 16 * 8 : kMaxN / 2);
        for (int i = 0; i < kRowBoxes && (i == 0 || (8 << (i - 1)) < half); ++i)
            ok = ok && make_map(&maps.b[i], a, 2, like_fwd(MODE) ? K : N, R, 1, 8u << i, 2);
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
    const int64_t m_tiles = ((int64_t)(like_dgrad(MODE) ? K : N) + tile_outputs<MODE>() - 1) / tile_outputs<MODE>();
    const int64_t part_tiles = m_tiles * (((int64_t)K + kMaxN - 1) / kMaxN), group_tiles = part_tiles * parts;
    // no more pairs than tiles (an upper bound: the groups' sizes are not known here)
    const int64_t most = MODE == kWgrad ? El * group_tiles : (R / kLeastN + (R < El ? R : El)) * m_tiles;
    const int pairs = (int)(most < num_sms / 2 ? most : num_sms / 2);
    const Shape sh{{(int)m_tiles, magic_of(m_tiles)}, {(int)group_tiles, magic_of(group_tiles)},
                   {(int)part_tiles, magic_of(part_tiles)}, parts, like_dgrad(MODE) ? N : K, (float)m_tiles / (float)pairs};
    launch_k(grouped_kernel<MODE, O>, 2 * pairs, threads_of<MODE>(), smem, stream, maps, off, cnt, El, (int)R, N, K,
             sh, idesc_base(MODE, dtype), stages, static_cast<O*>(out), gated);
    note_launches(1);
    return launch_status();
}

// The error word of this file's kernels (see moe_device_error).
int read_error_word(int clear) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_grouped_error, sizeof(int)) != cudaSuccess) return -1;
    if (clear && v) {
        const int z = 0;
        cudaMemcpyToSymbol(g_grouped_error, &z, sizeof(int));
    }
    return v;
}

}  // namespace
}  // namespace moe
