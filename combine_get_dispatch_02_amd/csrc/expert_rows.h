// expert_rows.h -- what the kernels of the experts' products share (gfx950): loads
// through buffer resources, the rows of each expert, and the work items of a launch.
#pragma once

#include "ep_device.h"
#include "ep_launch.h"

namespace ep {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// Loads through a buffer resource: a base and a running offset that are the same
// in all lanes stay in scalar registers, beside one 32-bit offset a lane.  (As
// plain pointers each stream of loads costs a pair of vector registers.)
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer(const void* p, int64_t bytes) {
    const int64_t most = 0x7FFFFFFF;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes < most ? bytes : most),
                                             0x00020000);
}
__device__ __forceinline__ u32x4 load16(Buffer b, uint32_t lane_offset, uint32_t offset) {
    return __builtin_amdgcn_raw_buffer_load_b128(b, lane_offset, __builtin_amdgcn_readfirstlane(offset), 0);
}
__device__ __forceinline__ u32x2 load8(Buffer b, uint32_t lane_offset, uint32_t offset) {
    return __builtin_amdgcn_raw_buffer_load_b64(b, lane_offset, __builtin_amdgcn_readfirstlane(offset), 0);
}
__device__ __forceinline__ uint32_t load4(Buffer b, uint32_t lane_offset, uint32_t offset) {
    return __builtin_amdgcn_raw_buffer_load_b32(b, lane_offset, __builtin_amdgcn_readfirstlane(offset), 0);
}
__device__ __forceinline__ uint32_t load1(Buffer b, uint32_t lane_offset, uint32_t offset) {
    return __builtin_amdgcn_raw_buffer_load_b8(b, lane_offset, __builtin_amdgcn_readfirstlane(offset), 0);
}

// 16 bytes a lane past the registers, to the wave's 1024 bytes of shared memory
// at `to` in lane order.  (The host pass does not know this size.)
__device__ __forceinline__ void load_shared(u32x4* to, Buffer b, uint32_t lane_offset, uint32_t offset) {
#ifdef __HIP_DEVICE_COMPILE__
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void*)to, 16, lane_offset,
                                             __builtin_amdgcn_readfirstlane(offset), 0, 0);
#endif
}

struct Rows {
    int64_t first;
    int count;
};

// Rows of expert e, limited to the buffers whatever the map says.
__device__ __forceinline__ Rows rows_of(const int32_t* __restrict__ expert_rows, int e, int capacity,
                                        int64_t num_rows) {
    if (capacity > 0) {
        const int n = expert_rows[e];
        return {static_cast<int64_t>(e) * capacity, n < 0 ? 0 : n > capacity ? capacity : n};
    }
    int64_t a = expert_rows[e], b = expert_rows[e + 1];
    a = a < 0 ? 0 : a > num_rows ? num_rows : a;
    b = b < a ? a : b > num_rows ? num_rows : b;
    return {a, static_cast<int>(b - a)};
}

// Work items of a launch, numbered on the device (the row counts are known
// there only): the row tiles of every expert with more than `above` and at most
// `most` rows, expert by expert, and for each the column tiles, which run
// fastest.  In shared memory: start[e], the row tiles before expert e (at most
// INT32_MAX), start[E] in all.
struct Table {
    int32_t* start;                                 // [E + 1]
    int32_t* first;                                 // [E] first row
    int32_t* count;                                 // [E] rows
};
inline size_t table_bytes(int E) { return sizeof(int32_t) * (3 * static_cast<size_t>(E) + 1); }

__device__ __forceinline__ uint32_t add_limited(uint32_t a, uint32_t b) {
    const uint32_t c = a + b;                       // both at most INT32_MAX
    return c < INT32_MAX ? c : INT32_MAX;
}

[[maybe_unused]] __device__ Table make_table(int32_t* room, const int32_t* __restrict__ expert_rows, int E, int capacity,
                            int64_t num_rows, int tile_rows, int above, int most) {
    __shared__ uint32_t sums[8];
    __shared__ uint64_t wrong[8];
    const Table t = {room, room + E + 1, room + 2 * E + 1};
    const int lane = lane_id(), wave = static_cast<int>(threadIdx.x) / kWave;
    const int threads = static_cast<int>(blockDim.x), per = (E + threads - 1) / threads;
    const int e0 = static_cast<int>(threadIdx.x) * per;
    for (int pass = 0;; ++pass) {
        uint32_t mine = 0;
        bool bad = false;                           // offsets out of order or range
        for (int i = 0; i < per; ++i) {
            const int e = e0 + i;
            if (e >= E) break;
            if (pass == 0) {
                const Rows r = rows_of(expert_rows, e, capacity, num_rows);
                t.first[e] = static_cast<int32_t>(r.first);
                t.count[e] = r.count;
                bad |= capacity == 0 && (r.first != expert_rows[e] || r.first + r.count != expert_rows[e + 1]);
            }
            const int count = t.count[e], n = count > above && count <= most ? (count - 1) / tile_rows + 1 : 0;
            t.start[e + 1] = n;                     // summed up below
            mine = add_limited(mine, n);
        }
        uint32_t upto = mine;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const uint32_t o = __shfl_up(upto, d);
            if (lane >= d) upto = add_limited(upto, o);
        }
        const uint64_t any = ballot(bad);
        if (lane == kWave - 1) {
            sums[wave] = upto;
            wrong[wave] = any;
        }
        uint32_t before = __shfl_up(upto, 1);
        if (lane == 0) before = 0;
        __syncthreads();
        uint64_t repair = 0;
        for (int w = 0; w < threads / kWave; ++w) {
            if (w < wave) before = add_limited(before, sums[w]);
            repair |= wrong[w];
        }
        if (repair) {
            // A map that no dispatch makes: in order, each expert takes what the
            // ones before it have left, so that no row has two experts and the
            // work stays that of num_rows rows.
            __syncthreads();
            if (threadIdx.x == 0) {
                int64_t at = 0;
                for (int e = 0; e < E; ++e) {
                    const Rows r = rows_of(expert_rows, e, capacity, num_rows);
                    const int64_t end = r.first + r.count;
                    at = r.first > at ? r.first : at;
                    t.first[e] = static_cast<int32_t>(at);
                    t.count[e] = static_cast<int32_t>(end > at ? end - at : 0);
                    at = end > at ? end : at;
                }
            }
            __syncthreads();
            continue;
        }
        if (threadIdx.x == 0) t.start[0] = 0;
        for (int i = 0; i < per; ++i) {
            if (e0 + i >= E) break;
            before = add_limited(before, t.start[e0 + i + 1]);
            t.start[e0 + i + 1] = before;
        }
        __syncthreads();
        return t;
    }
}

// The expert whose row tiles include number `tile` < start[E]: every lane asks
// about one expert in `step`, then about one of those between.
__device__ __forceinline__ int expert_of(const Table& t, int E, int tile) {
    const int step = (E + kWave - 1) / kWave, lane = lane_id();
    const int p = lane * step;
    int e = (__popcll(ballot(p < E && t.start[p < E ? p : 0] <= tile)) - 1) * step;
    if (step > 1) {
        const int o = e + lane;
        e += __popcll(ballot(lane < step && o < E && t.start[o < E ? o : 0] <= tile)) - 1;
    }
    return __builtin_amdgcn_readfirstlane(e);
}

// A launch's share of the items for this block.  Blocks go to the 8 chiplets
// (XCDs) in turn, so each chiplet takes one eighth of the items, in order: what
// neighbouring items share (an expert's weights, a tile's token rows) meets in
// one L2.
struct Share {
    int64_t at, end, step;
};
__device__ __forceinline__ Share share_of(int64_t items) {
    const int64_t xcd = blockIdx.x % 8;
    return {items * xcd / 8 + blockIdx.x / 8, items * (xcd + 1) / 8, static_cast<int64_t>(gridDim.x) / 8};
}

// v / (1 + exp(-v)) by the hardware's 2^x and reciprocal, each off by a step or
// so of fp32: |v| of them in all, where half a step of the result's bf16 is 2^15.
__device__ __forceinline__ float silu(float v) {
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * v));
}

__device__ __forceinline__ u32x2 four_bf16(const f32x4& v) {
    return u32x2{bf16_rne(v[0]) | (bf16_rne(v[1]) << 16), bf16_rne(v[2]) | (bf16_rne(v[3]) << 16)};
}
__device__ __forceinline__ void store4(uint16_t* p, const f32x4& v) { *reinterpret_cast<u32x2*>(p) = four_bf16(v); }

// Blocks for `items` at most, in whole eighths, up to `full`.
inline unsigned blocks_for(int64_t items, int64_t full) {
    const int64_t b = items < full ? items : full;
    return static_cast<unsigned>((b + 7) / 8 * 8);
}

}  // namespace
}  // namespace ep
