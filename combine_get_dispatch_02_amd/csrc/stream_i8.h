// stream_i8.h -- products of 8-bit integers for up to 16 token rows, bound by reading
// the weights (gfx950).
//
// 64 inputs of 16 weight rows against 16 token rows at a time
// (v_mfma_i32_16x16x64_i8): lane l holds inputs 16 q .. + 15 (q = l / 16) of row
// l % 16 of either operand, and of the product outputs 4 q .. + 3 for token row l % 16.
// The sums are integers, so neither their order nor how they are split changes a result.
#pragma once

#include "expert_rows.h"

namespace ep {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Products of kTiles weight tiles over inputs k .. + 127, k + step .. + 127, ... < K.
// weights(j) is the buffer of weight tile j, and row[j] the lane's offset in it: that of
// its weight row, and 16 q.  tokens(h, at) gives the lane's 16 codes of its token row
// at inputs at + 64 h + 16 q.  K is a multiple of 128, so a step takes whole 128-byte
// lines of each row; kDeep steps are on the way at a time.  The token rows
// are asked for before the weights that they meet, for loads return in order.
template <int kTiles, int kDeep>
struct Stream8 {
    u32x4 w[kDeep][kTiles][2], v[kDeep][2];

    // Every load is made on every way through the loop, past the end the last step's
    // again: a branch around a load makes the compiler wait for all that are on the way.
    template <typename Weights, typename Tokens>
    __device__ __forceinline__ void load(int buf, int at, int K, const uint32_t (&row)[kTiles], Weights weights,
                                         Tokens tokens) {
        at = at < K ? at : K - 128;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int h = 0; h < 2; ++h) v[buf][h] = tokens(h, at);
#pragma unroll
        for (int j = 0; j < kTiles; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) w[buf][j][h] = load16(weights(j), row[j], at + 64 * h);
        __builtin_amdgcn_sched_barrier(0);
    }
    template <typename Weights, typename Tokens>
    __device__ __forceinline__ void start(int k, int step, int K, const uint32_t (&row)[kTiles], Weights weights,
                                          Tokens tokens) {
#pragma unroll
        for (int b = 0; b < kDeep; ++b) load(b, k + b * step, K, row, weights, tokens);
    }
    template <typename Weights, typename Tokens>
    __device__ __forceinline__ void run(int k, int step, int K, const uint32_t (&row)[kTiles], Weights weights,
                                        Tokens tokens, i32x4 (&acc)[kTiles]) {
        for (; k < K; k += kDeep * step)
#pragma unroll
            for (int b = 0; b < kDeep; ++b) {
                const int at = k + b * step;
                if (at < K) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < kTiles; ++j)
                            acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w[b][j][h]),
                                                                           __builtin_bit_cast(i32x4, v[b][h]), acc[j], 0, 0, 0);
                }
                load(b, at + kDeep * step, K, row, weights, tokens);
            }
    }
};

}  // namespace
}  // namespace ep
