// w4_plan.h -- which kernels a call of ep_expert_linear_w4 launches (expert_w4.hip),
// and the loads and waits of its tile kernel, in plain C++ without HIP: a test on the
// CPU checks the wait counts, and those on the GPU ask which way their sizes take.
#pragma once

#include <stdint.h>

namespace ep {

// ---- the launches of a call --------------------------------------------------------
constexpr int kTileRows = 128, kTileWeights = 512;  // token rows and weight rows of a full tile

// The scales of streamed weights: through shared memory, eight at a time, or singly.
enum Scales { kSingle, kEight, kShared };
constexpr int kSharedScales = 8192;
constexpr Scales w4_scales(int K) { return K <= kSharedScales ? kShared : K % 256 == 0 ? kEight : kSingle; }

// Rows of an expert up to which its weights are streamed.  Streams against tiles
// (us), of 4, 8, 12 and 16 rows: 64 experts, 4096 -> 2 x 1024, 61 / 70, 65 / 70,
// 70 / 71, 75 / 71; 256 experts, 2048 -> 7168, 410 / 447, 460 / 453, 493 / 458,
// 531 / 469; 256 experts, 7168 -> 2 x 2048, 697 / 840, 758 / 851, 843 / 868, 905 / 876;
// 60 experts, 2048 -> 2 x 1408, 51 / 64, 54 / 64, 57 / 64, 62 / 64.
constexpr int kFew = 12;

// But where the streams' items (16 rows x 64 weight rows, half a tile an expert
// not full) find room on the card at once, streams take all rows: tiles have an
// eighth of the items, and leave CUs without one.  Streams against tiles (us), by
// items: 60, 8 experts of 16 rows, 3968 -> 432, 15 / 31; 544, one of 128, 4096 ->
// 4096, 26 / 49; 690, 60 of 17, 2048 -> 2 x 256, 22 / 32; 1152, 8 of 64, 7168 -> 2048,
// 57 / 79; 1024, 64 of 24, 512 -> 512, 14.7 / 13.3; but 2048, 8 of 24, 3968 -> 8192,
// 62 / 57; 2176, 8 of 128, 3968 -> 2048, 55 / 38.  Long experts with few outputs
// read more token rows than weights: one of 4000, 1024 -> 72 (502 items) 17 / 10; 16
// of 400, 3968 -> 72, 26 / 22; 16 of 200, 19 / 20.
constexpr int64_t kAllItems = 1280, kAllMean = 256;

// Smaller tiles where they all run at once and those of 128 rows would leave
// CUs without one (half a tile an expert is not full).  In us, 128 against 64
// or 32: 4 experts of 500 rows, 2048 -> 2 x 2048, 45 / 37; 16 of 200, 3968 -> 72,
// 41 / 20; one of 2000, 4096 -> 4096, 80 / 67; 64 of 206, 5760 -> 504, 113 / 86;
// but 16 of 1392, 3968 -> 72, 48 / 54; 64 of 64, 4096 -> 2 x 1024, 86 / 112.
constexpr int64_t kTilesAtOnce = 320;

// Each launch takes the experts that suit it, as their rows are known on the device
// only; one is left out where it would find none or few.  The rows of a padded call are
// those of its buffer, E * capacity, however few are filled; what that costs is the
// second launch, at times: 256 experts with 4 of 128 rows, 2048 -> 7168, 413 + 4.6 us
// (packed 412 + 4.7); 8 with 1 of 512, 4096 -> 2 x 1024, 12.7 + 3.9 (12.5).
struct W4Plan {
    int stream_most;                                // experts of up to so many rows (0: no launch)
    int tile_above;                                 // experts of more rows than this (INT32_MAX: no launch)
    int tile_rows;                                  // 32, 64 or 128
};
constexpr W4Plan w4_plan(int64_t num_rows, int capacity, int E, int N, bool silu) {
    const int64_t halves = (num_rows < E ? num_rows : E) / 2;       // of an expert's last tile, on average
    const int64_t most = capacity > 0 ? capacity : num_rows, mean = num_rows / E;
    const int64_t stream_columns = (N + (silu ? 31 : 63)) / (silu ? 32 : 64);
    if (mean <= kAllMean && (num_rows / 16 + halves) * stream_columns <= kAllItems) return {INT32_MAX, INT32_MAX, 0};
    const bool both = capacity > 0 || mean <= 2 * kFew;
    if (both && most <= kFew) return {kFew, INT32_MAX, 0};
    const int out = silu ? kTileWeights / 2 : kTileWeights;
    const int64_t columns = (N + out - 1) / out;
    int tile_rows = kTileRows;
    while (tile_rows > 32 && (num_rows / (tile_rows / 2) + halves) * columns <= kTilesAtOnce) tile_rows /= 2;
    return both ? W4Plan{kFew, kFew, tile_rows} : W4Plan{0, 0, tile_rows};
}

// ---- the steps of a tile ---------------------------------------------------------------

// One step (128 inputs) of a tile of 32 * `tiles` token rows, as a wave runs it: half
// of its products, in which it asks for `weights` loads into registers (`late`: in the
// other half); the barrier, before which it waits until at most `later` of its loads
// are on the way (`idle_later` in a wave past the last output, which brings token rows
// only); the other half, with `fills` loads of token rows into shared memory.
struct TileStep {
    int weights;
    bool late;
    int fills;
    int later, idle_later;
};

// Step `buf` = 0 .. 3 of the loop over 512 inputs (rest == 0), or one of the up to
// three steps after it (rest = 1 .. 3, buf = rest - 1).
//
// A step's rows are asked for three steps ahead, one load a row tile.  The barrier
// says that the next step's rows have arrived in every wave.  Loads arrive in the
// order in which they were asked for, so `later` may count only loads that surely
// follow those rows.
//
// In the loop these are the rows of the step after (`tiles`) and the weights of two
// steps: 6 loads a step in full tiles; in smaller ones 8 in every other step, and 2 of
// scales in the last.  The loop's code reads them all, so the compiler keeps them.
//
// How many steps come after the loop is not known, and what the last of them asked
// for a further one would be read by no code.  The compiler leaves such loads out,
// and a count that includes them waits for nothing.  So these steps ask only for what
// another of them reads (no token rows: the loop has asked for all), and `later`
// counts no weights:
//   first:  only the rows of the third step surely follow those of the second;
//   second: nothing surely follows those of the third.  (Full tiles: this step's
//           weights were asked for after those rows, and their products have begun,
//           so the rows are in, and the third's weights may be on the way.)
//   third:  waits for nothing that is on the way.  (Its barrier guards nothing, but
//           without it the compiler makes a second loop for the waves past the last
//           output, and spills 400 registers.)
constexpr TileStep tile_step(int tiles, int buf, int rest) {
    const bool lines = tiles < 4;
    return rest == 0   ? lines ? TileStep{buf % 2 == 0 ? 8 : buf == 3 ? 2 : 0, false, tiles,
                                          tiles + (buf == 3 ? 10 : 8), tiles}
                               : TileStep{6, false, tiles, tiles + 6, tiles}
           : rest == 1 ? lines ? TileStep{4, true, 0, tiles, tiles} : TileStep{6, false, 0, tiles, tiles}
           : rest == 2 ? lines ? TileStep{0, false, 0, 0, 0} : TileStep{6, false, 0, 6, 0}
                       : TileStep{0, false, 0, 0, 0};
}

}  // namespace ep
