// w4_plan.h -- the loads and waits of the tile kernel of ep_expert_linear_w4
// (expert_w4.hip), in plain C++ without HIP, so that a test on the CPU can check
// the wait counts.
#pragma once

namespace ep {

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
