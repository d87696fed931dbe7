// combine_backward.hip -- ep_combine_backward on gfx950.
//
// out[t] = sum_j w[t,j] y[row(t,j)], so dy[row] = w g[t] and dw[t,j] =
// <g[t], y[row]>.  One wave per slot (t, j): it reads its row of y and the
// token's g once, and the whole dot product stays in the wave, so the sum's
// order is fixed by H alone.
#include "ep_device.h"
#include "ep_launch.h"

namespace ep {
namespace {

template <bool kWithY, bool kWithG>
__global__ __launch_bounds__(256) void combine_backward_kernel(
    const u32x4* __restrict__ g, const u32x4* __restrict__ y, int64_t num_rows,
    const int32_t* __restrict__ token_row, const float* __restrict__ topk_weights, int64_t slots, int V, int k,
    u32x4* __restrict__ dy, float* __restrict__ dw) {
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const int64_t step = static_cast<int64_t>(gridDim.x) * 4;
    for (int64_t s = static_cast<int64_t>(blockIdx.x) * 4 + wave; s < slots; s += step) {
        const int row = token_row[s];
        if (row < 0 || row >= num_rows) {
            if (kWithY && lane == 0) dw[s] = 0.0f;
            continue;
        }
        const float w = topk_weights ? topk_weights[s] : 1.0f;
        const u32x4* gt = g + s / k * V;
        const int64_t at = static_cast<int64_t>(row) * V;
        float acc[8] = {};
        for (int v = lane; v < V; v += kWave) {
            const u32x4 a = gt[v];
            if (kWithY) {
                const u32x4 b = y[at + v];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[2 * i] = __builtin_fmaf(bf16_lo(a[i]), bf16_lo(b[i]), acc[2 * i]);
                    acc[2 * i + 1] = __builtin_fmaf(bf16_hi(a[i]), bf16_hi(b[i]), acc[2 * i + 1]);
                }
            }
            if (kWithG) {
                u32x4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = bf16_rne(w * bf16_lo(a[i])) | (bf16_rne(w * bf16_hi(a[i])) << 16);
                dy[at + v] = o;
            }
        }
        if (kWithY) {
            float sum = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
            if (lane == 0) dw[s] = sum;
        }
    }
}

}  // namespace

hipError_t launch_combine_backward(const void* grad_out, const void* expert_out, int64_t num_rows,
                                   const int32_t* token_row, const float* topk_weights, int64_t T, int H, int k,
                                   void* grad_expert_out, float* grad_topk_weights, hipStream_t stream) {
    const int64_t slots = T * k;
    const int64_t blocks = ceil_div(slots, 4), cap = kMaxLaunchThreads / 256;
    const dim3 grid(static_cast<unsigned>(blocks < cap ? blocks : cap));
    const u32x4* g = static_cast<const u32x4*>(grad_out);
    const u32x4* y = static_cast<const u32x4*>(expert_out);
    u32x4* dy = static_cast<u32x4*>(grad_expert_out);
    if (dy && grad_topk_weights)
        hipLaunchKernelGGL((combine_backward_kernel<true, true>), grid, dim3(256), 0, stream, g, y, num_rows,
                           token_row, topk_weights, slots, H / 8, k, dy, grad_topk_weights);
    else if (dy)
        hipLaunchKernelGGL((combine_backward_kernel<false, true>), grid, dim3(256), 0, stream, g, y, num_rows,
                           token_row, topk_weights, slots, H / 8, k, dy, grad_topk_weights);
    else
        hipLaunchKernelGGL((combine_backward_kernel<true, false>), grid, dim3(256), 0, stream, g, y, num_rows,
                           token_row, topk_weights, slots, H / 8, k, dy, grad_topk_weights);
    return hipGetLastError();
}

}  // namespace ep
