// How many rows of a group a tile of the grouped products gets (forward, dgrad and the gated forms): at most
// kMaxN >> c, c from choose_rows. Every CTA evaluates the rule from the same whole numbers, so that all agree.
#pragma once

#include <math.h>

#ifndef __CUDACC__  // the rule alone, for a host compiler
#define __host__
#define __device__
#define __forceinline__ inline
#endif

namespace moe {

constexpr int kMaxN = 256;  // columns of a tile
constexpr int kRowChoices = 3, kLeastN = kMaxN >> (kRowChoices - 1);

// Of all groups: the parts that their rows are cut into by each choice, their rows in 16s (each group's rounded
// up), the longest group's rows.
struct RowSums {
    unsigned parts[kRowChoices];
    unsigned rows16, longest;
};

// a / b, good to a few ulp.
__host__ __device__ __forceinline__ float quotient(float a, float b) {
#ifdef __CUDA_ARCH__
    return __fdividef(a, b);
#else
    return a / b;
#endif
}

// steps: stages of the reduced index; share: tiles of a part, along the outputs, for each pair of CTAs; kSlope: with the
// activation's gradients in the epilogue. In clocks: a stage of a tile of n rows takes about the time of 256 + n rows on
// their way into the SM (its MMAs that of 2 n at most); its epilogue, under the next tile's stages but for the last
// one's, 1000 and 13 a row (56 with the gradients, each step of which waits for gate and up). The pairs take the tiles in
// rounds, each about as long as the average tile, which has the rows that the groups have and not the most that it
// may; some pair gets more of the long ones (half of what one is longer by), and the last epilogue is under nothing.
// What it decides, in us of 256 / 128 / 64 rows (one GB300, calls back to back):
//   one group of 2048 rows, 512 x 512            gated backward 15.1 / 10.8 / 9.1    dgrad 8.0 / 6.5 / 6.3
//   one group of 8192 rows, 128 outputs of 2048  forward 15.3 / 13.2 / 18.8
//   128 groups of 16384 rows, Zipf 1.2, 768x2048 forward 150 / 159 / 203             gated backward 105 / 102 / 116
//   128 groups of 2048 rows, Zipf 1.2, 768x2048  forward 123 / 127 / 125             dgrad 62 / 67 / 65
//   16 groups of 300 rows, 768 x 2048            forward 33 / 36 / 54                gated backward 30 / 27 / 38
// Over 47 such batches its choice takes 0.2 % longer than the best one (at most 9 %); 256 rows throughout 5.5 % (67 %).
// Tiles are counted in 32 bits, and the entry points refuse sizes whose tiles of 256 rows might be more than 2^30. Fewer rows
// never make more of them: with many rounds the largest tiles win, as each part costs the 256 rows' time of its own.
// (Sizes between, whose halves are no box of the row maps, measured slower: 4096 rows in tiles of 224 instead of 256,
// 2048 x 2048, 41.9 -> 45.3 us.)
template <bool kSlope>
__host__ __device__ __forceinline__ int choose_rows(const RowSums& sums, float steps, float share) {
    int best = 0;
    float least = 0.f;
    const float rows = 16.f * (float)sums.rows16, longest = (float)sums.longest;
#pragma unroll
    for (int c = 0; c < kRowChoices; ++c) {
        const float parts = (float)(sums.parts[c] > 0 ? sums.parts[c] : 1u);
        const float average = quotient(rows, parts), most = fminf((float)(kMaxN >> c), longest);
        const float per_row = kSlope ? 56.f : 13.f;
        const float round = fmaxf(steps * (256.f + average), 1000.f + per_row * average);
        const float stages = steps * (256.f + most), epilogue = 1000.f + per_row * most;
        const float clocks = ceilf(parts * share) * round + 0.5f * (fmaxf(stages, epilogue) - round) + fminf(stages, epilogue);
        if (c == 0 || clocks < least) best = c, least = clocks;
    }
    return best;
}

// Whether groups of several parts and the others are taken by turns: where the parts that find their weights in L2,
// all but the first of each group, are three in sixteen or more. 128 experts, 768 x 2048, three draws each, forward in
// us, in the groups' order / by turns:
//   65536 rows, Zipf 1.2 (three in five)            289, 289, 292 / 291, 278, 279
//   32768 rows, Zipf 1.2 (two in five)              190, 185, 185 / 180, 181, 181
//   16384 rows, Zipf 1.2 (one in five)              152, 150, 151 / 152, 151, 151
//   16384 rows, Zipf 0.6 (one in ten)               151, 150, 150 / 153, 151, 154
//   8192 rows, Zipf 1.2 (one in eleven)             142, 136, 137 / 142, 139, 137
// (a few long parts at equal distances meet the pairs' own distance, and some pairs get several of them).
__host__ __device__ __forceinline__ bool by_turns(unsigned several_parts, unsigned several_groups, unsigned single_parts) {
    return 16.f * (float)(several_parts - several_groups) >= 3.f * ((float)several_parts + (float)single_parts);
}

}  // namespace moe
