// i8_plan.h -- which kernels a call of ep_expert_linear_i8 launches (expert_i8.hip),
// and the loads and waits of its tile kernel, in plain C++ without HIP: a test on the
// CPU checks the wait counts, and those on the GPU ask which way their sizes take.
#pragma once

#include <stdint.h>

namespace ep {

// Token rows of a full tile, and its weight rows.
constexpr int kTileRows8 = 256, kTileWeights8 = 256;

// A call launches one kernel, for all of its experts: streams (16 token rows x 64 weight
// rows a wave or block) where they all find room on the card at once, for tiles have a
// quarter of the items at most and leave CUs without one; but not over few inputs, where
// a tile's time is short.  Streams against tiles (us), by items as counted here: 96,
// 64 experts with 6 rows, 4096 -> 2 x 1024, 14 / 28; 256, 256 with 8, 7168 -> 2 x 2048,
// 46 / 65; 256, 16 with 128, 1024 -> 1024, 9 / 13; 512, 8 with 64, 4096 -> 4096, 28 / 34;
// 576, 256 with 16, 7168 -> 2 x 2048, 82 / 85; but 448, 256 with 8, 2048 -> 7168, 25.4 /
// 24.7; 768, 8 with 128, 4096 -> 4096, 44 / 35; 272, 60 with 64, 512 -> 512, 12 / 11.
// (However few rows the experts have, tiles are as fast where there are enough of them:
// 256 experts of 4 rows, 2048 -> 7168, 655 / 634; of 16, 1074 / 685.)
// The rows of a padded call are those of its buffer, however few are filled.
constexpr int64_t kStreamItems8 = 640;
constexpr int kStreamInputs8 = 1024;
constexpr bool i8_streams(int64_t num_rows, int E, int K, int N, bool silu) {
    const int64_t halves = (num_rows < E ? num_rows : E) / 2;       // of an expert's last tile, on average
    const int64_t columns = (N + (silu ? 31 : 63)) / (silu ? 32 : 64);
    return K >= kStreamInputs8 && (num_rows / 16 + halves) * columns <= kStreamItems8;
}

// ---- the stages of a tile ------------------------------------------------------------

// A wave's loads of a stage (128 inputs): 0 .. 7 bring token rows, 8 + 2 q and 9 + 2 q
// rows of the weight tiles q.  While a stage is worked off, the loads of the stage after
// next go to its slot, from those whose rows every wave has read, and the last four a
// quarter into the next stage, for quarter 3 is busy with reads.
constexpr int kLoads8 = 16;

// Quarter q of a stage: loads `from` .. `to` - 1 are asked for in it, of the stage after
// next, or (quarter 0) of the next.  Behind it the waves wait for what the next quarter
// reads: behind quarters 0 and 1 weight tiles 2 and 3 of the same stage, behind 2 the next
// stage's token tiles and weight tiles 0, behind 3 its weight tiles 1; that is until at
// most `later` accesses are on the way.  Loads arrive in the order in which they were
// asked for, and `later` counts those that follow: behind quarter 0 tiles 3 (2), the last
// stage's quarters 1 and 2 (12) and this one's quarter 0 (4); behind 1 the same 12, and
// quarters 0 and 1 (10); behind 2 tiles 1 (2) and quarters 0, 1 and 2 (16); behind 3
// these 16.
//
// Between two items' stages a wave stores the first one's results and asks for the
// scales of the second.  In an item's first stage these too follow what is waited for,
// and may be counted.
struct I8Quarter {
    int from, to, later;
};
constexpr I8Quarter i8_quarter(int q) {
    return q == 0 ? I8Quarter{12, 16, 18} : q == 1 ? I8Quarter{0, 6, 22} : q == 2 ? I8Quarter{6, 12, 18}
                                                                                  : I8Quarter{0, 0, 16};
}

}  // namespace ep
