// expert_w4.hip -- ep_expert_linear_w4 on gfx950.
//
// y[r] = x[r] . W[e(r)]^T over the rows of each expert, W in E2M1 codes with
// one E8M0 scale per 32 inputs.  The matrix instruction contracts 32 inputs of
// 16 weight rows against 16 token rows (v_mfma_f32_16x16x32_bf16).  A code
// times its scale is exact in bf16, so the only roundings are the fp32
// accumulation and the final one to bf16.
//
// The order of the contraction is free as long as both operands agree, so a
// lane takes 16 consecutive bytes of its weight row: 32 inputs, exactly one
// scale group.  The four lane groups of a wave (lane / 16) hold the four
// groups of a 128-input block, and step s of four contracts inputs
// 32 q + 8 s .. + 7 of every group q.
#include "ep_device.h"
#include "ep_launch.h"

namespace ep {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

// Eight codes of one word, times the scale 2^(b - 127) whose bits are b << 23.
__device__ __forceinline__ bf16x8 decode(uint32_t codes, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

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
__device__ __forceinline__ uint32_t load1(Buffer b, uint32_t lane_offset, uint32_t offset) {
    return __builtin_amdgcn_raw_buffer_load_b8(b, lane_offset, __builtin_amdgcn_readfirstlane(offset), 0);
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
// there only): the row tiles of every expert, expert by expert, and for each
// the column tiles, which run fastest.  start[e] is the number of row tiles
// before expert e, limited to int32 (maps out of order could add up to more).
__device__ void count_tiles(const int32_t* __restrict__ expert_rows, int E, int capacity, int64_t num_rows,
                            int tile_rows, int32_t* __restrict__ start) {
    __shared__ int64_t sums[kThreads / kWave];
    const int lane = lane_id(), wave = static_cast<int>(threadIdx.x) / kWave;
    const int per = (E + kThreads - 1) / kThreads;
    const int e0 = static_cast<int>(threadIdx.x) * per;
    int64_t mine = 0;
    for (int i = 0; i < per; ++i)
        if (e0 + i < E) mine += (rows_of(expert_rows, e0 + i, capacity, num_rows).count + tile_rows - 1) / tile_rows;
    int64_t upto = mine;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int64_t o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == kWave - 1) sums[wave] = upto;
    __syncthreads();
    int64_t before = upto - mine;
    for (int w = 0; w < wave; ++w) before += sums[w];
    for (int i = 0; i < per; ++i) {
        if (e0 + i >= E) break;
        start[e0 + i] = static_cast<int32_t>(before < INT32_MAX ? before : INT32_MAX);
        before += (rows_of(expert_rows, e0 + i, capacity, num_rows).count + tile_rows - 1) / tile_rows;
        if (e0 + i == E - 1) start[E] = static_cast<int32_t>(before < INT32_MAX ? before : INT32_MAX);
    }
    __syncthreads();
}

// The expert whose row tiles include number `tile` < start[E].
__device__ __forceinline__ int expert_of(const int32_t* start, int E, int tile) {
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (start[mid] <= tile) lo = mid;
        else hi = mid;
    }
    return lo;
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

__device__ __forceinline__ float silu(float v) { return v / (1.0f + expf(-v)); }

// ---- few rows per expert: bound by reading the weights ---------------------------
// One item: up to 16 kRowTiles token rows x 64 weight rows (kSilu: 32 gate rows
// and their 32 up rows).  The four waves split the inputs, 128 at a time in
// turn, so that a single token's products still put enough loads in flight, and
// join their sums in shared memory in wave order.
template <bool kSilu, int kRowTiles>
__global__ __launch_bounds__(kThreads, kRowTiles == 1 ? 4 : 2) void stream_w4_kernel(
    const uint16_t* __restrict__ x, int64_t num_rows, const int32_t* __restrict__ expert_rows, int capacity,
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int E, int K, int N,
    uint16_t* __restrict__ y) {
    constexpr int kOut = kSilu ? 32 : 64;           // outputs of an item
    __shared__ f32x4 part[4][4][kWave];             // [wave][weight tile][lane]
    extern __shared__ int32_t start[];              // [E + 1]
    const int lane = lane_id(), q = lane / 16, i16 = lane % 16;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    count_tiles(expert_rows, E, capacity, num_rows, 16 * kRowTiles, start);
    const int columns = (N + kOut - 1) / kOut;
    const Share mine = share_of(static_cast<int64_t>(start[E]) * columns);
    for (int64_t item = mine.at; item < mine.end; item += mine.step) {
        const int tile = static_cast<int>(item / columns);
        const int n0 = static_cast<int>(item - static_cast<int64_t>(tile) * columns) * kOut;
        const int e = expert_of(start, E, tile);
        const Rows rows = rows_of(expert_rows, e, capacity, num_rows);
        const int m0 = (tile - start[e]) * 16 * kRowTiles, left = rows.count - m0;

        // Lanes past the rows or outputs repeat the last one and store nothing.
        // Addresses: the item's first row, the same in all lanes, and offsets.
        const int64_t w0 = static_cast<int64_t>(e) * (kSilu ? 2 * N : N) + n0;
        const int64_t wide = N - n0 < 128 ? N - n0 : 128;
        const Buffer wb[2] = {buffer(codes + w0 * (K / 2), wide * (K / 2)),
                              buffer(codes + (w0 + (kSilu ? N : 0)) * (K / 2), wide * (K / 2))};    // [1]: up rows
        const Buffer sb[2] = {buffer(scales + w0 * (K / 32), wide * (K / 32)),
                              buffer(scales + (w0 + (kSilu ? N : 0)) * (K / 32), wide * (K / 32))};
        const Buffer xb = buffer(x + (rows.first + m0) * K, static_cast<int64_t>(left < 128 ? left : 128) * K * 2);
        uint32_t cr[4], xr[kRowTiles];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            int n = (kSilu ? j % 2 : j) * 16 + i16;
            n = n0 + n < N ? n : N - 1 - n0;
            cr[j] = static_cast<uint32_t>(n) * (K / 2) + q * 16;
        }
#pragma unroll
        for (int i = 0; i < kRowTiles; ++i) {
            const int m = i * 16 + i16 < left ? i * 16 + i16 : left - 1;
            xr[i] = (static_cast<uint32_t>(m) * K + q * 32) * 2;
        }
        const int tiles = left < 16 * kRowTiles ? (left + 15) / 16 : kRowTiles;

        f32x4 acc[kRowTiles][4] = {};
        u32x4 w[2][4];
        uint32_t b[2][4];
        auto load = [&](int buf, int kb) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[buf][j] = load16(wb[kSilu ? j / 2 : 0], cr[j], kb / 2);
                b[buf][j] = load1(sb[kSilu ? j / 2 : 0], cr[j] / 16, kb / 32);
            }
        };
        auto multiply = [&](int buf, int kb) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                bf16x8 a[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) a[j] = decode(w[buf][j][s], __uint_as_float(b[buf][j] << 23));
#pragma unroll
                for (int i = 0; i < kRowTiles; ++i) {
                    if (i >= tiles) break;
                    const bf16x8 v = __builtin_bit_cast(bf16x8, load16(xb, xr[i], (kb + 8 * s) * 2));
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[j], v, acc[i][j], 0, 0, 0);
                }
            }
        };
        int kb = wave * 128;
        if (kb < K) load(0, kb);
        for (; kb < K; kb += 1024) {
            if (kb + 512 < K) load(1, kb + 512);
            multiply(0, kb);
            if (kb + 512 >= K) break;
            if (kb + 1024 < K) load(0, kb + 1024);
            multiply(1, kb + 512);
        }

        // Join: thread t takes outputs 4 (t % 16) .. + 3 of token row t / 16.
        const int m = static_cast<int>(threadIdx.x) / 16, c = static_cast<int>(threadIdx.x) % 16;
#pragma unroll
        for (int i = 0; i < kRowTiles; ++i) {
            if (i >= tiles) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) part[wave][j][lane] = acc[i][j];
            __syncthreads();
            auto sum = [&](int j) {
                const int at = c % 4 * 16 + m;      // the lane that held it
                return (part[0][j][at] + part[1][j][at]) + (part[2][j][at] + part[3][j][at]);
            };
            const int j = c / 4, n = n0 + 4 * c;
            if (i * 16 + m < left && 4 * c < kOut && n < N) {
                f32x4 v = sum(j);
                if (kSilu) {
                    const f32x4 up = sum(j + 2);
#pragma unroll
                    for (int u = 0; u < 4; ++u) v[u] = silu(v[u]) * up[u];
                }
                *reinterpret_cast<u32x2*>(y + (rows.first + m0 + i * 16 + m) * N + n) =
                    u32x2{bf16_rne(v[0]) | (bf16_rne(v[1]) << 16), bf16_rne(v[2]) | (bf16_rne(v[3]) << 16)};
            }
            __syncthreads();
        }
    }
}

// ---- many rows per expert: bound by the matrix unit ------------------------------
// One item: 128 token rows x 128 weight rows (kSilu: 64 gate rows and their 64
// up rows), 64 x 64 to each of the four waves.  The token rows of a 128-input
// step come through shared memory (double buffered, loaded past the registers);
// the codes, an eighth of their bytes per value, straight into the registers of
// the wave that decodes them, a step ahead.
constexpr int kStep = 128;

// The 16-byte chunk of a 256-byte row that holds inputs 8 c .. + 7 of row r:
// rows are read 16 at a time at the same c, which would all meet in one bank.
__device__ __forceinline__ int chunk_of(int r, int c) { return c ^ (r & 15); }

template <bool kSilu>
__global__ __launch_bounds__(kThreads, 2) void tile_w4_kernel(
    const uint16_t* __restrict__ x, int64_t num_rows, const int32_t* __restrict__ expert_rows, int capacity,
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int E, int K, int N,
    uint16_t* __restrict__ y) {
    constexpr int kOut = kSilu ? 64 : 128;
    __shared__ u32x4 even[128 * 16], odd[128 * 16];
    extern __shared__ int32_t start[];
    const int lane = lane_id(), q = lane / 16, i16 = lane % 16;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const int wm = wave / 2 * 64, wn = wave % 2;
    count_tiles(expert_rows, E, capacity, num_rows, 128, start);
    const int columns = (N + kOut - 1) / kOut;
    const Share mine = share_of(static_cast<int64_t>(start[E]) * columns);
    for (int64_t item = mine.at; item < mine.end; item += mine.step) {
        const int tile = static_cast<int>(item / columns);
        const int n0 = static_cast<int>(item - static_cast<int64_t>(tile) * columns) * kOut;
        const int e = expert_of(start, E, tile);
        const Rows rows = rows_of(expert_rows, e, capacity, num_rows);
        const int m0 = (tile - start[e]) * 128, left = rows.count - m0;

        const int64_t w0 = static_cast<int64_t>(e) * (kSilu ? 2 * N : N) + n0;
        const int64_t wide = N - n0 < 128 ? N - n0 : 128;
        const Buffer wb[2] = {buffer(codes + w0 * (K / 2), wide * (K / 2)),
                              buffer(codes + (w0 + (kSilu ? N : 0)) * (K / 2), wide * (K / 2))};    // [1]: up rows
        const Buffer sb[2] = {buffer(scales + w0 * (K / 32), wide * (K / 32)),
                              buffer(scales + (w0 + (kSilu ? N : 0)) * (K / 32), wide * (K / 32))};
        const Buffer xb = buffer(x + (rows.first + m0) * K, static_cast<int64_t>(left < 128 ? left : 128) * K * 2);
        uint32_t cr[4], fill[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            int n = (kSilu ? wn * 32 + j % 2 * 16 : wn * 64 + j * 16) + i16;
            n = n0 + n < N ? n : N - 1 - n0;
            cr[j] = static_cast<uint32_t>(n) * (K / 2) + q * 16;
        }
        // This wave fills rows 32 wave .. + 31, four to a load: lane l writes
        // place l % 16 of row l / 16, so it reads the chunk that belongs there.
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = wave * 32 + i * 4 + q;
            fill[i] = static_cast<uint32_t>(r < left ? r : left - 1) * K * 2 + chunk_of(r, i16) * 16;
        }
        auto stage = [&](u32x4* to, int kb) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    xb, (__attribute__((address_space(3))) void*)(to + (wave * 32 + i * 4) * 16), 16, fill[i],
                    __builtin_amdgcn_readfirstlane(kb * 2), 0, 0);
        };
        u32x4 w[2][4];
        uint32_t b[2][4];
        auto load = [&](int buf, int kb) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[buf][j] = load16(wb[kSilu ? j / 2 : 0], cr[j], kb / 2);
                b[buf][j] = load1(sb[kSilu ? j / 2 : 0], cr[j] / 16, kb / 32);
            }
        };
        f32x4 acc[4][4] = {};
        auto multiply = [&](const u32x4* from, int buf) {
            bf16x8 v[2][4];
            auto read = [&](int s) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = wm + i * 16 + i16;
                    v[s % 2][i] = __builtin_bit_cast(bf16x8, from[r * 16 + chunk_of(r, q * 4 + s)]);
                }
            };
            read(0);
            // The barriers to scheduling keep each step's reads ahead of the
            // products of the step before, and no further: all four in front spill.
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (s < 3) read(s + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bf16x8 a = decode(w[buf][j][s], __uint_as_float(b[buf][j] << 23));
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, v[s % 2][i], acc[i][j], 0, 0, 0);
                }
            }
        };
        // A step's loads have arrived (vmcnt), in every wave (barrier), and every
        // wave is done with the step before, whose buffer the next loads fill.
        auto arrive = [&] {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
        };
        __syncthreads();                            // the last item's reads are done
        stage(even, 0);
        load(0, 0);
        for (int kb = 0; kb < K; kb += 2 * kStep) {
            arrive();
            if (kb + kStep < K) {
                stage(odd, kb + kStep);
                load(1, kb + kStep);
            }
            multiply(even, 0);
            if (kb + kStep >= K) break;
            arrive();
            if (kb + 2 * kStep < K) {
                stage(even, kb + 2 * kStep);
                load(0, kb + 2 * kStep);
            }
            multiply(odd, 1);
        }

        // A lane holds outputs 4 q .. + 3 of token row i16 of each 16 x 16 tile.
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = wm + i * 16 + i16;
            if (m >= left) continue;
            uint16_t* row = y + (rows.first + m0 + m) * N;
#pragma unroll
            for (int j = 0; j < (kSilu ? 2 : 4); ++j) {
                const int n = n0 + (kSilu ? wn * 32 : wn * 64) + j * 16 + 4 * q;
                f32x4 v = acc[i][j];
                if (kSilu) {
#pragma unroll
                    for (int u = 0; u < 4; ++u) v[u] = silu(v[u]) * acc[i][j + 2][u];
                }
                if (n < N)
                    *reinterpret_cast<u32x2*>(row + n) =
                        u32x2{bf16_rne(v[0]) | (bf16_rne(v[1]) << 16), bf16_rne(v[2]) | (bf16_rne(v[3]) << 16)};
            }
        }
    }
}

struct Call {
    const void* x;
    int64_t num_rows;
    const int32_t* expert_rows;
    int capacity;
    const uint8_t* codes;
    const uint8_t* scales;
    int E, K, N;
    void* y;
    hipStream_t stream;
};

// Blocks for `items` at most, in whole eighths, up to `full`.
unsigned blocks_for(int64_t items, int64_t full) {
    const int64_t b = items < full ? items : full;
    return static_cast<unsigned>((b + 7) / 8 * 8);
}

template <bool kSilu, int kRowTiles>
hipError_t launch_stream(const Call& c) {
    const int64_t tiles = c.num_rows / (16 * kRowTiles) + (c.num_rows < c.E ? c.num_rows : c.E);
    hipLaunchKernelGGL((stream_w4_kernel<kSilu, kRowTiles>),
                       dim3(blocks_for(tiles * ceil_div(c.N, kSilu ? 32 : 64), 256 * (kRowTiles == 1 ? 4 : 2))),
                       dim3(kThreads), sizeof(int32_t) * (c.E + 1), c.stream, static_cast<const uint16_t*>(c.x),
                       c.num_rows, c.expert_rows, c.capacity, c.codes, c.scales, c.E, c.K, c.N,
                       static_cast<uint16_t*>(c.y));
    return hipGetLastError();
}

template <bool kSilu>
hipError_t launch_tile(const Call& c) {
    const int64_t tiles = c.num_rows / 128 + (c.num_rows < c.E ? c.num_rows : c.E);
    hipLaunchKernelGGL((tile_w4_kernel<kSilu>), dim3(blocks_for(tiles * ceil_div(c.N, kSilu ? 64 : 128), 256 * 2)),
                       dim3(kThreads), sizeof(int32_t) * (c.E + 1), c.stream, static_cast<const uint16_t*>(c.x),
                       c.num_rows, c.expert_rows, c.capacity, c.codes, c.scales, c.E, c.K, c.N,
                       static_cast<uint16_t*>(c.y));
    return hipGetLastError();
}

template <bool kSilu>
hipError_t launch(const Call& c) {
    const int64_t mean = c.num_rows / c.E;
    if (mean <= 12) return launch_stream<kSilu, 1>(c);
    if (mean <= 64) return launch_stream<kSilu, 4>(c);
    return launch_tile<kSilu>(c);
}

}  // namespace

hipError_t launch_expert_linear_w4(const void* x, int64_t num_rows, const int32_t* expert_rows, int capacity,
                                   const uint8_t* w_codes, const uint8_t* w_scales, int E, int K, int N,
                                   bool silu_mul, void* y, hipStream_t stream) {
    const Call c = {x, num_rows, expert_rows, capacity, w_codes, w_scales, E, K, N, y, stream};
    return silu_mul ? launch<true>(c) : launch<false>(c);
}

}  // namespace ep
