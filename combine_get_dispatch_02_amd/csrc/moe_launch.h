// moe_launch.h -- internal kernel launchers of the operators on either side of
// dispatch and combine: routing, gradients, the experts' products (host side).
#pragma once

#include "ep_launch.h"

namespace ep {

// ---- routing ------------------------------------------------------------------
// Score, choice and weights of ep_route; type: EP_TYPE_*.
struct RouteOptions {
    bool sigmoid;        // else softmax
    bool renormalize;
    float scale;
    int num_groups, topk_groups, group_top;
};
hipError_t launch_route(const void* logits, int type, const float* bias, int64_t T, int E, int k,
                        const RouteOptions& opt, int64_t* topk_idx, float* topk_weights,
                        hipStream_t stream);
hipError_t launch_route_backward(const void* logits, int type, const int64_t* topk_idx,
                                 const float* grad_weights, int64_t T, int E, int k, bool sigmoid,
                                 bool renormalize, float scale, void* grad_logits,
                                 hipStream_t stream);

// ---- gradient of combine --------------------------------------------------------
hipError_t launch_combine_backward(const void* grad_out, const void* expert_out, int64_t num_rows,
                                   const int32_t* token_row, const float* topk_weights, int64_t T,
                                   int H, int k, void* grad_expert_out, float* grad_topk_weights,
                                   hipStream_t stream);

// ---- experts' products with 4-bit weights ----------------------------------------
hipError_t launch_expert_linear_w4(const void* x, int64_t num_rows, const int32_t* expert_rows,
                                   int capacity, const uint8_t* w_codes, const uint8_t* w_scales,
                                   int E, int K, int N, bool silu_mul, void* y, hipStream_t stream);

}  // namespace ep
