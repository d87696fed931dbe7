// dispatch_i8.hip -- rows cast to 8-bit integers, as ep_dispatch_i8 and its cached and
// padded forms send tokens to their receive rows, and as ep_quantize_i8 leaves them in
// place, on gfx950.
//
// A row is read once and kept in registers while its largest magnitude is found (rows
// of up to 8192 channels; longer ones are read twice).  Bound by HBM: 2 bytes a channel
// in, 1 out for every receive row.  4096 tokens x 7168, top 8: 50.6 us for 295 MB, 5.8
// TB/s of which the reads come out of the last-level cache, where the index kernels
// before it (13.6 us) bring x; 32768 rows x 2048 in place: 35 us for 201 MB, 5.8 TB/s.
#include "moe_launch.h"
#include "quant_i8.h"
#include "small_rows.h"

namespace ep {
namespace {

// ---- tokens to their receive rows --------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kCopyPieces = 2;

// A block a token: its codes are computed once, and go to all its rows from registers.
// Rows outside [0, num_rows) are skipped.
__global__ __launch_bounds__(kCopyThreads) void copy_i8_kernel(const u32x4* __restrict__ x,
                                                               const int32_t* __restrict__ token_row, int64_t T,
                                                               int pieces, int k, int64_t num_rows,
                                                               u32x4* __restrict__ recv, float* __restrict__ scales) {
    __shared__ uint32_t room[1][kCopyThreads / kWave];
    const int lane = lane_id();
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        int mine = -1;
        const u32x4* const row[1] = {x + t * pieces * 2};
        cast_rows<kCopyThreads, kCopyPieces, 1, true>(
            row, pieces, static_cast<int>(threadIdx.x), room,
            [&] {
                const int to = token_row[t * k + (lane < k ? lane : 0)];
                mine = lane < k && to < num_rows ? to : -1;
            },
            [&](int, int p, const u32x4& codes) {
                for (int j = 0; j < k; ++j) {
                    const int r = read_lane(mine, j);
                    if (r >= 0) __builtin_nontemporal_store(codes, recv + static_cast<int64_t>(r) * pieces + p);
                }
            },
            [&](int, float s) {
                if (threadIdx.x < kWave && mine >= 0) scales[mine] = s;
            });
        __syncthreads();                            // `room` is read
    }
}

// Small batches: the rows are derived in the block (small_rows.h), while its token is on
// the way.  128 tokens x 7168, top 8 of 256: 5.4 us, of which the index work is the most.
constexpr int kSmallThreads = 512;

__global__ __launch_bounds__(kSmallThreads) void dispatch_small_i8_kernel(
    const u32x4* __restrict__ x, const int64_t* __restrict__ topk_idx, const float* __restrict__ topk_weights,
    int64_t T, int k, int E, int R, int cap, int pieces, u32x4* __restrict__ recv, float* __restrict__ scales,
    int32_t* __restrict__ token_row, int32_t* __restrict__ recv_src_idx, float* __restrict__ recv_w,
    int32_t* __restrict__ expert_offset, int32_t* __restrict__ rank_offset, int32_t* __restrict__ recv_count) {
    extern __shared__ int32_t lds[];
    __shared__ uint32_t room[1][kSmallThreads / kWave];
    int32_t* rows = lds + 2 * E + 16 + kSmallMaxK;
    const int64_t t = blockIdx.x;
    const u32x4* const row[1] = {x + t * pieces * 2};
    cast_rows<kSmallThreads, 1, 1, true>(
        row, pieces, static_cast<int>(threadIdx.x), room,
        [&] {
            small_token_rows(topk_idx, topk_weights, T, k, E, R, cap, t, true, t == 0, token_row, recv_src_idx, recv_w,
                             expert_offset, rank_offset, recv_count, lds, rows);
        },
        [&](int, int p, const u32x4& codes) {
            for (int j = 0; j < k; ++j)
                if (rows[j] >= 0) __builtin_nontemporal_store(codes, recv + static_cast<int64_t>(rows[j]) * pieces + p);
        },
        [&](int, float s) {
            const int j = static_cast<int>(threadIdx.x);
            if (j < k && rows[j] >= 0) scales[rows[j]] = s;
        });
}

// ---- rows in place -------------------------------------------------------------------
// kRowThreads threads a row, 256 a block: a wave where it can hold a row, so that no
// barrier is met.  expert_rows as ep_expert_linear_i8 takes it,
// or NULL: all rows.
template <int kRowThreads, int kPieces>
__global__ __launch_bounds__(256) void quantize_i8_kernel(const u32x4* __restrict__ x, int64_t num_rows, int pieces,
                                                          const int32_t* __restrict__ expert_rows, int E, int capacity,
                                                          u32x4* __restrict__ codes, float* __restrict__ scales) {
    constexpr int kRows = 256 / kRowThreads;
    __shared__ uint32_t room[1][kRowThreads / kWave];
    const int thread = static_cast<int>(threadIdx.x) % kRowThreads;
    int64_t first = 0, end = num_rows;
    if (expert_rows && capacity == 0) {
        first = expert_rows[0] > 0 ? expert_rows[0] : 0;
        end = expert_rows[E] < num_rows ? expert_rows[E] : num_rows;
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    for (int64_t at = static_cast<int64_t>(blockIdx.x) * kRows; at < num_rows; at += step) {
        const int64_t r = at + __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kRowThreads);
        bool filled = r >= first && r < end;
        if (expert_rows && capacity > 0 && filled) {
            const int e = static_cast<int>(r) / capacity;
            filled = static_cast<int>(r) - e * capacity < expert_rows[e];
        }
        // (Threads of one row agree, and so do those that meet at a barrier.)
        const u32x4* const row[1] = {x + r * pieces * 2};
        if (filled)
            cast_rows<kRowThreads, kPieces, 1, true>(
                row, pieces, thread, room, [] {},
                [&](int, int p, const u32x4& c) { __builtin_nontemporal_store(c, codes + r * pieces + p); },
                [&](int, float s) {
                    if (thread == 0) scales[r] = s;
                });
        if (kRowThreads > kWave) __syncthreads();
    }
}

constexpr int64_t kMaxBlocks = kMaxLaunchThreads / 512;
unsigned at_most(int64_t blocks) { return static_cast<unsigned>(blocks < kMaxBlocks ? blocks : kMaxBlocks); }

}  // namespace

hipError_t launch_dispatch_copy_i8(const void* x, const int32_t* token_row, int8_t* recv, float* recv_scales,
                                   int64_t num_rows, int64_t T, int H, int k, hipStream_t stream) {
    if (T == 0) return hipSuccess;
    hipLaunchKernelGGL(copy_i8_kernel, dim3(at_most(T)), dim3(kCopyThreads), 0, stream, static_cast<const u32x4*>(x),
                       token_row, T, H / 16, k, num_rows, reinterpret_cast<u32x4*>(recv), recv_scales);
    return hipGetLastError();
}

hipError_t launch_dispatch_i8(const void* x, const int64_t* topk_idx, const float* topk_weights, int64_t T, int H,
                              int k, int E, int R, int cap, int8_t* recv, float* recv_scales, int32_t* recv_src_idx,
                              float* recv_w, int32_t* expert_offset, int32_t* rank_offset, int32_t* recv_count,
                              int32_t* token_row, void* workspace, hipStream_t stream) {
    if (dispatch_is_small(T, k)) {
        hipLaunchKernelGGL(dispatch_small_i8_kernel, dim3(static_cast<unsigned>(T)), dim3(kSmallThreads),
                           small_lds_bytes(E), stream, static_cast<const u32x4*>(x), topk_idx,
                           (recv_w ? topk_weights : nullptr), T, k, E, R, cap, H / 16, reinterpret_cast<u32x4*>(recv),
                           recv_scales, token_row, recv_src_idx, (topk_weights ? recv_w : nullptr), expert_offset,
                           rank_offset, recv_count);
        return hipGetLastError();
    }
    const int64_t x_bytes = T * static_cast<int64_t>(H) * 2;
    const hipError_t e = launch_dispatch_index(topk_idx, topk_weights, T, k, E, R, recv_src_idx, recv_w, expert_offset,
                                               rank_offset, token_row, workspace,
                                               prefetch_pays(x_bytes, false) ? x : nullptr, x_bytes, cap, recv_count,
                                               stream);
    if (e != hipSuccess) return e;
    const int64_t rows = cap > 0 ? static_cast<int64_t>(E) * cap : T * k;
    return launch_dispatch_copy_i8(x, token_row, recv, recv_scales, rows, T, H, k, stream);
}

hipError_t launch_quantize_i8(const void* x, int64_t num_rows, int K, const int32_t* expert_rows, int E, int capacity,
                              int8_t* codes, float* scales, hipStream_t stream) {
    const int pieces = K / 16;
    auto go = [&](auto kernel, int rows) {
        hipLaunchKernelGGL(kernel, dim3(at_most(ceil_div(num_rows, rows))), dim3(256), 0, stream,
                           static_cast<const u32x4*>(x), num_rows, pieces, expert_rows, E, capacity,
                           reinterpret_cast<u32x4*>(codes), scales);
        return hipGetLastError();
    };
    if (K <= 1024) return go(quantize_i8_kernel<64, 1>, 4);
    if (K <= 2048) return go(quantize_i8_kernel<64, 2>, 4);
    if (K <= 4096) return go(quantize_i8_kernel<64, 4>, 4);
    return go(quantize_i8_kernel<256, 2>, 1);
}

}  // namespace ep
