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


// ---- the experts' layer in 8-bit integers -------------------------------------------
// Tokens cast on their way to their receive rows (cap > 0: to padded slots), and rows
// cast in place.
hipError_t launch_dispatch_i8(const void* x, const int64_t* topk_idx, const float* topk_weights, int64_t T, int H,
                              int k, int E, int R, int cap, int8_t* recv, float* recv_scales, int32_t* recv_src_idx,
                              float* recv_w, int32_t* expert_offset, int32_t* rank_offset, int32_t* recv_count,
                              int32_t* token_row, void* workspace, hipStream_t stream);
hipError_t launch_dispatch_ll_i8(const void* x, const int64_t* topk_idx, const float* topk_weights, int64_t T, int H,
                                 int k, int E, int cap, int8_t* recv, float* recv_scales, int32_t* recv_count,
                                 int32_t* recv_src_idx, float* recv_w, int32_t* token_slot, void* workspace,
                                 hipStream_t stream);
hipError_t launch_dispatch_copy_i8(const void* x, const int32_t* token_row, int8_t* recv, float* recv_scales,
                                   int64_t num_rows, int64_t T, int H, int k, hipStream_t stream);
hipError_t launch_quantize_i8(const void* x, int64_t num_rows, int K, const int32_t* expert_rows, int E, int capacity,
                              int8_t* codes, float* scales, hipStream_t stream);
hipError_t launch_expert_linear_i8(const int8_t* x, const float* x_scales, int64_t num_rows,
                                   const int32_t* expert_rows, int capacity, const int8_t* w, const float* w_scales,
                                   int E, int K, int N, bool silu_mul, void* y, hipStream_t stream);
constexpr int kMoeMaxSlots = 512;                  // T * k
constexpr int kMoeMaxFfn = 1 << 15;                // F
// The whole layer for a few tokens (S = T * k slots).
size_t moe_i8_workspace_bytes(int S, int F);
hipError_t launch_moe_i8(const void* x, const int64_t* topk_idx, const float* topk_weights, int T, int k, int E, int H,
                         int F, const int8_t* up, const float* up_scales, const int8_t* down, const float* down_scales,
                         void* workspace, void* out, hipStream_t stream);

}  // namespace ep
