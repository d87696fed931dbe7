// i8_plan.h -- which kernels a call of ep_expert_linear_i8 launches (expert_i8.hip), in
// plain C++ without HIP: the tests ask which way their sizes take.
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

}  // namespace ep
