// small_rows.h -- the receive order of a small batch, derived inside each block of
// the kernel that moves its rows (gfx950).
#pragma once

#include "ep_device.h"
#include "ep_launch.h"

namespace ep {
namespace {

__device__ __forceinline__ void write_offsets(const int32_t* eoff, int total, int E, int R,
                                              int32_t* __restrict__ expert_offset,
                                              int32_t* __restrict__ rank_offset) {
    const int epr = E / R;
    for (int e = threadIdx.x; e <= E; e += blockDim.x) expert_offset[e] = e < E ? eoff[e] : total;
    if (rank_offset)
        for (int r = threadIdx.x; r <= R; r += blockDim.x) rank_offset[r] = r < R ? eoff[r * epr] : total;
}

// For T*k <= kSmallSlots every copy block derives the rows of its own token:
// it counts all T*k ids in LDS (those before the token, and all), scans the
// totals over experts, and ranks the token's k slots among themselves.  The
// ids are a few KB and L2-resident after the first blocks, so this costs one
// round trip that overlaps the block's x loads, and no index launch precedes
// the copy.  The token's first block writes its token_row / recv_src_idx /
// recv_topk_weights; block 0 writes the offsets.
// With cap > 0 the same blocks fill the padded expert-major layout instead:
// the slot of (t, j) is e*cap + (its position among expert e's slots), or -1
// from position cap on, and block 0 writes recv_count[e] = min(count, cap).
// LDS: cnt_pre[E], cnt_all[E], wave_tot[16], own[EP_MAX_TOPK], rows[EP_MAX_TOPK].
constexpr int kSmallMaxK = 64;
constexpr int kSmallBatch = 4;     // id loads per thread per step of the small-batch sweep

__device__ inline int block_exclusive_scan_rt(int32_t* a, int n, int32_t* wave_tot) {
    const int nthreads = blockDim.x;
    const int ipt = (n + nthreads - 1) / nthreads;
    const int b = threadIdx.x * ipt;
    int sum = 0;
    for (int i = 0; i < ipt; ++i)
        if (b + i < n) sum += a[b + i];
    int incl = sum;
    const int lane = lane_id();
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const int v = __shfl_up(incl, off, kWave);
        if (lane >= off) incl += v;
    }
    const int wave = threadIdx.x / kWave;
    if (lane == kWave - 1) wave_tot[wave] = incl;
    __syncthreads();
    int base = 0, total = 0;
    for (int w = 0; w < nthreads / kWave; ++w) {
        base += (w < wave) ? wave_tot[w] : 0;
        total += wave_tot[w];
    }
    int run = base + incl - sum;
    for (int i = 0; i < ipt; ++i)
        if (b + i < n) {
            const int v = a[b + i];
            a[b + i] = run;
            run += v;
        }
    __syncthreads();
    return total;
}

// Rows of token t into rows_out[0..k) (LDS, -1 for an empty slot).  Called by
// every thread of the block.
__device__ inline void small_token_rows(const int64_t* __restrict__ topk_idx,
                                 const float* __restrict__ topk_weights, int64_t T, int k, int E,
                                 int R, int cap, int64_t t, bool write_maps, bool write_offs,
                                 int32_t* __restrict__ token_row,
                                 int32_t* __restrict__ recv_src_idx, float* __restrict__ recv_w,
                                 int32_t* __restrict__ expert_offset,
                                 int32_t* __restrict__ rank_offset,
                                 int32_t* __restrict__ recv_count, int32_t* lds,
                                 int32_t* rows_out) {
    int32_t* cnt_pre = lds;
    int32_t* cnt_all = lds + E;
    int32_t* wave_tot = lds + 2 * E;
    int32_t* own = wave_tot + 16;
    const int j = threadIdx.x;
    // The token's weights (needed only by its first block) and the first
    // batch of ids are requested before anything waits, so they share one
    // round trip with the caller's x loads: kSmallBatch loads per thread,
    // indices clamped to the last slot (no branch around a load, which would
    // make the compiler wait for it).
    const float wj = (write_maps && recv_w && j < k) ? topk_weights[t * k + j] : 0.0f;
    const int total_slots = static_cast<int>(T * k);
    const int first = static_cast<int>(t * k);
    const int step = kSmallBatch * static_cast<int>(blockDim.x);
    int64_t v[kSmallBatch];
#pragma unroll
    for (int u = 0; u < kSmallBatch; ++u) {
        const int sl = u * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x);
        v[u] = topk_idx[sl < total_slots ? sl : total_slots - 1];
    }
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        cnt_pre[e] = 0;
        cnt_all[e] = 0;
    }
    __syncthreads();
    for (int s0 = 0; s0 < total_slots; s0 += step) {
        if (s0 > 0) {
#pragma unroll
            for (int u = 0; u < kSmallBatch; ++u) {
                const int sl = s0 + u * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x);
                v[u] = topk_idx[sl < total_slots ? sl : total_slots - 1];
            }
        }
#pragma unroll
        for (int u = 0; u < kSmallBatch; ++u) {
            const int sl = s0 + u * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x);
            if (sl >= total_slots) continue;
            const int64_t e = v[u];
            const bool valid = e >= 0 && e < E;
            if (valid) {
                atomicAdd(&cnt_all[e], 1);
                if (sl < first) atomicAdd(&cnt_pre[e], 1);
            }
            if (sl >= first && sl < first + k) own[sl - first] = valid ? static_cast<int32_t>(e) : -1;
        }
    }
    __syncthreads();
    if (cap > 0) {
        if (write_offs)
            for (int e = threadIdx.x; e < E; e += blockDim.x) recv_count[e] = min(cnt_all[e], cap);
    } else {
        const int total = block_exclusive_scan_rt(cnt_all, E, wave_tot);
        if (write_offs) write_offsets(cnt_all, total, E, R, expert_offset, rank_offset);
    }
    if (j < k) {
        const int e = own[j];
        int row = -1;
        if (e >= 0) {
            int before = 0;
            for (int q = 0; q < j; ++q) before += own[q] == e;
            const int pos = cnt_pre[e] + before;
            if (cap <= 0) row = cnt_all[e] + pos;
            else if (pos < cap) row = e * cap + pos;
        }
        rows_out[j] = row;
        if (write_maps) {
            token_row[t * k + j] = row;
            if (row >= 0) {
                recv_src_idx[row] = static_cast<int32_t>(t);
                if (recv_w) recv_w[row] = wj;
            }
        }
    }
    __syncthreads();
}

inline size_t small_lds_bytes(int E) {
    return (2 * static_cast<size_t>(E) + 16 + 2 * kSmallMaxK) * sizeof(int32_t);
}

}  // namespace
}  // namespace ep
