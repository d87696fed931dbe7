// combine_backward.hip -- ep_combine_backward on gfx950.
//
// out[t] = sum_j w[t,j] y[row(t,j)], so dy[row] = w g[t] and dw[t,j] =
// <g[t], y[row]>.  A wave (or four) per slot (t, j): it reads its row of y and the
// token's g once and writes its row of dy; the dot product's order is fixed by
// the launch shape, so results do not change from run to run.
#include "ep_device.h"
#include "moe_launch.h"

namespace ep {
namespace {

// kSplit waves of a block take a slot, kBatch 16-byte vectors a lane at a time:
// all of a batch's loads are asked for before any is used.  Rows are read and
// written once, past the caches (nontemporal), which the tokens' g then has to
// itself.  Bound by HBM: 195 us for 4096 tokens x 7168, top 8 (1.0 GB, 5.1 TB/s;
// a large copy reaches 5.2), against 212 with one vector at a time, 196 with four
// and 208 through the caches (with four).
constexpr int kBatch = 2;

// Few slots leave most of the chip without a wave, so four waves share one: 9.7
// against 12.7 us at 1024 slots of H = 7168, 16.1 against 15.6 at 2048.  A wave's
// quarter has to be a vector a lane at least.
bool split_slots(int64_t slots, int V) { return slots <= 1536 && V >= 4 * kWave; }

template <bool kWithY, bool kWithG, int kSplit>
__global__ __launch_bounds__(256) void combine_backward_kernel(
    const u32x4* __restrict__ g, const u32x4* __restrict__ y, int64_t num_rows,
    const int32_t* __restrict__ token_row, const float* __restrict__ topk_weights, int64_t slots, int V, int k,
    u32x4* __restrict__ dy, float* __restrict__ dw) {
    __shared__ float part[4];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const int share = wave % kSplit;
    constexpr int kSlots = 4 / kSplit;              // of a block
    const int64_t step = static_cast<int64_t>(gridDim.x) * kSlots;
    for (int64_t s = static_cast<int64_t>(blockIdx.x) * kSlots + wave / kSplit; s < slots; s += step) {
        const int row = token_row[s];
        if (row < 0 || row >= num_rows) {
            if (kWithY && lane == 0 && share == 0) dw[s] = 0.0f;
            continue;                               // all kSplit waves of the slot
        }
        const float w = topk_weights ? topk_weights[s] : 1.0f;
        const u32x4* gt = g + s / k * V;
        const int64_t at = static_cast<int64_t>(row) * V;
        float acc[8] = {};
        for (int v0 = share * kWave + lane; v0 < V; v0 += kBatch * kSplit * kWave) {
            u32x4 a[kBatch], b[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {      // past the row's end: its last vector, not used
                const int v = v0 + u * kSplit * kWave < V ? v0 + u * kSplit * kWave : V - 1;
                a[u] = gt[v];
                if (kWithY) b[u] = __builtin_nontemporal_load(y + at + v);
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int v = v0 + u * kSplit * kWave;
                if (v >= V) break;
                u32x4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float lo = bf16_lo(a[u][i]), hi = bf16_hi(a[u][i]);
                    if (kWithY) {
                        acc[2 * i] = __builtin_fmaf(lo, bf16_lo(b[u][i]), acc[2 * i]);
                        acc[2 * i + 1] = __builtin_fmaf(hi, bf16_hi(b[u][i]), acc[2 * i + 1]);
                    }
                    if (kWithG) o[i] = bf16_rne(w * lo) | (bf16_rne(w * hi) << 16);
                }
                if (kWithG) __builtin_nontemporal_store(o, dy + at + v);
            }
        }
        if (kWithY) {
            float sum = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
            if (kSplit == 1) {
                if (lane == 0) dw[s] = sum;
            } else {                                // kSplit == 4: the block's one slot
                if (lane == 0) part[wave] = sum;
                __syncthreads();
                if (threadIdx.x == 0) dw[s] = (part[0] + part[1]) + (part[2] + part[3]);
                __syncthreads();
            }
        }
    }
}

// Rows of at most kLanes vectors: a wave takes 64 / kLanes slots, a vector a lane
// (6893 tokens x 144, top 6: 11.7 us, 16.6 with a wave a slot.  Four sets of slots
// at once took 9.9, and 5.0 instead of 2.9 for 128 tokens x 256, top 2).
template <bool kWithY, bool kWithG, int kLanes>
__global__ __launch_bounds__(256) void combine_backward_short_kernel(
    const u32x4* __restrict__ g, const u32x4* __restrict__ y, int64_t num_rows,
    const int32_t* __restrict__ token_row, const float* __restrict__ topk_weights, int64_t slots, int V, int k,
    u32x4* __restrict__ dy, float* __restrict__ dw) {
    const int v = lane_id() % kLanes;
    const int64_t step = static_cast<int64_t>(gridDim.x) * (256 / kLanes);
    for (int64_t s = static_cast<int64_t>(blockIdx.x) * (256 / kLanes) + threadIdx.x / kLanes; s < slots; s += step) {
        const int row = token_row[s];
        const bool valid = row >= 0 && row < num_rows;
        float sum = 0.0f, odd = 0.0f;
        if (valid && v < V) {
            const u32x4 a = g[s / k * V + v];
            const int64_t at = static_cast<int64_t>(row) * V + v;
            if (kWithY) {
                const u32x4 b = __builtin_nontemporal_load(y + at);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    sum = __builtin_fmaf(bf16_lo(a[i]), bf16_lo(b[i]), sum);
                    odd = __builtin_fmaf(bf16_hi(a[i]), bf16_hi(b[i]), odd);
                }
                sum += odd;
            }
            if (kWithG) {
                const float w = topk_weights ? topk_weights[s] : 1.0f;
                u32x4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = bf16_rne(w * bf16_lo(a[i])) | (bf16_rne(w * bf16_hi(a[i])) << 16);
                __builtin_nontemporal_store(o, dy + at);
            }
        }
        if (kWithY) {
#pragma unroll
            for (int d = kLanes / 2; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
            if (v == 0) dw[s] = sum;                // 0 of an empty slot
        }
    }
}

template <bool kWithY, bool kWithG, int kLanes>
hipError_t launch_short(const u32x4* g, const u32x4* y, int64_t num_rows, const int32_t* token_row, const float* w,
                        int64_t slots, int V, int k, u32x4* dy, float* dw, hipStream_t stream) {
    const int64_t blocks = ceil_div(slots, 256 / kLanes), cap = kMaxLaunchThreads / 256;
    hipLaunchKernelGGL((combine_backward_short_kernel<kWithY, kWithG, kLanes>),
                       dim3(static_cast<unsigned>(blocks < cap ? blocks : cap)), dim3(256), 0, stream, g, y, num_rows,
                       token_row, w, slots, V, k, dy, dw);
    return hipGetLastError();
}

template <bool kWithY, bool kWithG>
hipError_t launch(const u32x4* g, const u32x4* y, int64_t num_rows, const int32_t* token_row, const float* w,
                  int64_t slots, int V, int k, u32x4* dy, float* dw, hipStream_t stream) {
    if (V <= 16) return launch_short<kWithY, kWithG, 16>(g, y, num_rows, token_row, w, slots, V, k, dy, dw, stream);
    if (V <= 32) return launch_short<kWithY, kWithG, 32>(g, y, num_rows, token_row, w, slots, V, k, dy, dw, stream);
    const bool split = split_slots(slots, V);
    const int64_t blocks = split ? slots : ceil_div(slots, 4), cap = kMaxLaunchThreads / 256;
    const dim3 grid(static_cast<unsigned>(blocks < cap ? blocks : cap));
    if (split)
        hipLaunchKernelGGL((combine_backward_kernel<kWithY, kWithG, 4>), grid, dim3(256), 0, stream, g, y, num_rows,
                           token_row, w, slots, V, k, dy, dw);
    else
        hipLaunchKernelGGL((combine_backward_kernel<kWithY, kWithG, 1>), grid, dim3(256), 0, stream, g, y, num_rows,
                           token_row, w, slots, V, k, dy, dw);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_combine_backward(const void* grad_out, const void* expert_out, int64_t num_rows,
                                   const int32_t* token_row, const float* topk_weights, int64_t T, int H, int k,
                                   void* grad_expert_out, float* grad_topk_weights, hipStream_t stream) {
    const u32x4* g = static_cast<const u32x4*>(grad_out);
    const u32x4* y = static_cast<const u32x4*>(expert_out);
    u32x4* dy = static_cast<u32x4*>(grad_expert_out);
    if (dy && grad_topk_weights)
        return launch<true, true>(g, y, num_rows, token_row, topk_weights, T * k, H / 8, k, dy, grad_topk_weights,
                                  stream);
    if (dy)
        return launch<false, true>(g, y, num_rows, token_row, topk_weights, T * k, H / 8, k, dy, nullptr, stream);
    return launch<true, false>(g, y, num_rows, token_row, topk_weights, T * k, H / 8, k, nullptr,
                               grad_topk_weights, stream);
}

}  // namespace ep
