// i8_plan.h -- which kernels a call of ep_expert_linear_i8 launches (expert_i8.hip),
// and the loads and waits of its tile kernel, in plain C++ without HIP: a test on the
// CPU checks the wait counts, and those on the GPU ask which way their sizes take.
#pragma once

#include <stdint.h>

namespace ep {

// Token rows of a full tile, and its weight rows.
constexpr int kTileRows8 = 256, kTileWeights8 = 256;

// Rows of an expert up to which its weights are streamed.
constexpr int kFew8 = 16;

// Each launch takes the experts that suit it, as their rows are known on the device
// only; one is left out where it would find none or few.
struct I8Plan {
    int stream_most;                                // experts of up to so many rows (0: no launch)
    int tile_above;                                 // experts of more rows than this (INT32_MAX: no launch)
};
constexpr I8Plan i8_plan(int64_t num_rows, int capacity, int E) {
    const int64_t most = capacity > 0 ? capacity : num_rows, mean = num_rows / E;
    const bool both = capacity > 0 || mean <= 2 * kFew8;
    if (both && most <= kFew8) return {kFew8, INT32_MAX};
    return both ? I8Plan{kFew8, kFew8} : I8Plan{0, 0};
}

// ---- the stages of a tile ------------------------------------------------------------

// A wave's loads of a stage (128 inputs): 0 .. 7 bring token rows, 8 + 2 q and 9 + 2 q
// rows of the weight tiles q.  While a stage is worked off, the loads of the stage after
// next go to its slot, from those whose rows every wave has read.
constexpr int kLoads8 = 16;

// Quarter q of a stage: loads `from` .. `to` - 1 are asked for in it.  Behind it the
// waves wait for what the next quarter reads: behind quarters 0 and 1 weight tiles 2
// and 3 of the same stage, behind 2 the next stage's token tiles and weight tiles 0,
// behind 3 its weight tiles 1; that is until at most `later` accesses are on the way.
// Loads arrive in the order in which they were asked for, and `later` counts those that
// follow: behind quarter 0 tiles 3 (2) and the next stage (16); behind 1 the next stage
// and quarter 1's (6); behind 2 tiles 1, 2 and 3 (6) and quarters 1 and 2 (12); behind 3
// tiles 2 and 3 (4) and quarters 1, 2 and 3 (16).
//
// Between two items' stages a wave stores the first one's results and asks for the
// scales of the second.  Behind quarters of the first `early` stages of an item these
// too follow what is waited for, and may be counted.
struct I8Quarter {
    int from, to, later, early;
};
constexpr I8Quarter i8_quarter(int q) {
    return q == 0 ? I8Quarter{0, 0, 18, 2} : q == 1 ? I8Quarter{0, 6, 22, 2} : q == 2 ? I8Quarter{6, 12, 18, 1}
                                                                                : I8Quarter{12, 16, 20, 1};
}

}  // namespace ep
