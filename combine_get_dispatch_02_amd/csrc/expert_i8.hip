// expert_i8.hip -- ep_expert_linear_i8 on gfx950.
//
// y[r] = x[r] . W[e(r)]^T over the rows of each expert, both in 8-bit integers, with
// one scale a row of x and one a row of W.  The sums are exact in 32 bits; what is
// rounded is the sum on its way to fp32, its products with the scales and the result.
#include "i8_plan.h"
#include "moe_launch.h"
#include "stream_i8.h"

namespace ep {
namespace {

typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;

struct Call {
    const int8_t* x;
    const float* x_scales;
    int64_t num_rows;
    const int32_t* expert_rows;
    int capacity;
    const int8_t* w;
    const float* w_scales;
    int E, K, N;
    uint16_t* y;
};

// What an item's waves read: weight rows from n0 on (w[1]: the up rows that belong to
// them), their scales, and token rows from row0 on.
struct Operands {
    int64_t row0;
    int n0, left;                                   // first output, token rows left
    Buffer w[2], x;
    const float* w_scales[2];
};
template <bool kSilu>
__device__ __forceinline__ Operands operands(const Call& c, int e, int64_t row0, int left, int n0, int wide, int deep) {
    const int64_t w0 = static_cast<int64_t>(e) * (kSilu ? 2 * c.N : c.N) + n0, up = kSilu ? c.N : 0;
    const int64_t rows = c.N - n0 < wide ? c.N - n0 : wide, tokens = left < deep ? left : deep;
    return {row0, n0, left,
            {buffer(c.w + w0 * c.K, rows * c.K), buffer(c.w + (w0 + up) * c.K, rows * c.K)},
            buffer(c.x + row0 * c.K, tokens * c.K),
            {c.w_scales + w0, c.w_scales + w0 + up}};
}
// Weight row n of an item's; those past the outputs repeat the last one, and what they
// give is not stored.
__device__ __forceinline__ uint32_t weight_row(const Operands& o, int n, int N) {
    return o.n0 + n < N ? n : N - 1 - o.n0;
}

// Four outputs, in fp32.
__device__ __forceinline__ f32x4 scaled(const i32x4& sum, float x_scale, const f32x4& w_scale) {
    f32x4 v;
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = static_cast<float>(sum[c]) * (x_scale * w_scale[c]);
    return v;
}
__device__ __forceinline__ f32x4 silu_mul(const f32x4& gate, const f32x4& up) {
    f32x4 v;
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = silu(gate[c]) * up[c];
    return v;
}
__device__ __forceinline__ f32x4 scales4(const float* scales, int n) {
    return *reinterpret_cast<const f32x4*>(scales + n);
}

// ---- few rows per expert: bound by reading the weights ---------------------------
// A wave takes 64 weight rows (kSilu: 32 gate rows and their 32 up rows) and up to 16
// token rows.  Where there are items for every wave, each takes whole items; where
// there are not, the four waves of a block split an item's inputs, so that every CU has
// loads in flight, and join their sums in shared memory.
template <bool kSilu>
__global__ __launch_bounds__(kThreads, 2) void stream_i8_kernel(Call c, int most) {
    constexpr int kOut = kSilu ? 32 : 64;           // outputs of an item
    constexpr int kDeep = 3;
    __shared__ i32x4 part[16][kWave];
    extern __shared__ int32_t room[];
    const int lane = lane_id(), q = lane / 16, i16 = lane % 16;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const Table t = make_table(room, c.expert_rows, c.E, c.capacity, c.num_rows, 16, 0, most);
    const int columns = (c.N + kOut - 1) / kOut;
    const int64_t items = static_cast<int64_t>(t.start[c.E]) * columns;
    const bool split = 4 * items < 5 * static_cast<int64_t>(gridDim.x);
    Share mine = share_of(items);
    if (!split) {                                   // neighbouring items to the waves of a block
        mine.at += blockIdx.x / 8 * 3 + wave;
        mine.step *= 4;
    }
    for (int64_t item = mine.at; item < mine.end; item += mine.step) {
        const int tile = static_cast<int>(item / columns);
        const int column = static_cast<int>(item - static_cast<int64_t>(tile) * columns);
        const int e = expert_of(t, c.E, tile);
        const int m0 = (tile - t.start[e]) * 16;
        const int left = __builtin_amdgcn_readfirstlane(t.count[e] - m0);
        const int64_t row0 = __builtin_amdgcn_readfirstlane(t.first[e]) + static_cast<int64_t>(m0);
        const Operands o = operands<kSilu>(c, e, row0, left, column * kOut, kOut, 16);
        uint32_t row[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            row[j] = weight_row(o, (kSilu ? j % 2 : j) * 16 + i16, c.N) * static_cast<uint32_t>(c.K) + q * 16;
        const uint32_t mine_x = (i16 < left ? i16 : left - 1) * static_cast<uint32_t>(c.K) + q * 16;
        auto weights = [&](int j) { return o.w[kSilu ? j / 2 : 0]; };
        auto tokens = [&](int h, int at) { return load16(o.x, mine_x, at + 64 * h); };
        i32x4 acc[4] = {};
        Stream8<4, kDeep, true> s;
        const int k = split ? wave * 128 : 0, step = split ? 512 : 128;
        s.start(k, step, c.K, row, weights, tokens);
        s.run(k, step, c.K, row, weights, tokens, acc);

        // Of split items wave w ends up with weight tile w (kSilu: waves 0 and 1 with
        // the gate's and the up rows').
        uint16_t* out = c.y + (row0 + i16) * c.N;
        if (split) {
#pragma unroll
            for (int j = 0; j < 4; ++j) part[wave * 4 + j][lane] = acc[j];
            __syncthreads();
            auto sum = [&](int j) { return part[j][lane] + part[4 + j][lane] + part[8 + j][lane] + part[12 + j][lane]; };
            const int n = wave * 16 + 4 * q;
            if (wave * 16 < kOut && i16 < left && o.n0 + n < c.N) {
                const float xs = c.x_scales[row0 + i16];
                f32x4 v = scaled(sum(wave), xs, scales4(o.w_scales[0], n));
                if (kSilu) v = silu_mul(v, scaled(sum(wave + 2), xs, scales4(o.w_scales[1], n)));
                store4(out + o.n0 + n, v);
            }
            __syncthreads();
        } else if (i16 < left) {
            const float xs = c.x_scales[row0 + i16];
#pragma unroll
            for (int j = 0; j < kOut / 16; ++j) {
                const int n = j * 16 + 4 * q;
                if (o.n0 + n >= c.N) break;
                f32x4 v = scaled(acc[j], xs, scales4(o.w_scales[0], n));
                if (kSilu) v = silu_mul(v, scaled(acc[j + 2], xs, scales4(o.w_scales[1], n)));
                store4(out + o.n0 + n, v);
            }
        }
    }
}

// ---- many rows per expert ----------------------------------------------------------
// One item: up to 64 kT token rows x 256 weight rows (kSilu: 128 gate rows and their
// 128 up rows).  Four waves, one a SIMD, two by two: each has 128 weight rows (kSilu: 64
// of either) and 32 kT token rows, 4 kT products of 32 x 32 (v_mfma_i32_32x32x32_i8) a
// step of 32 inputs.  Both operands come through a ring of stages of 64 inputs in shared
// memory, loaded past the registers.
//
// A row has 64 bytes of a stage, four places of 16; inputs 16 c .. + 15 of row r are at
// place c ^ (r / 4 % 4), so that any 16 neighbouring rows' places c lie in different
// banks.  A lane holds row l % 32 of either operand, and inputs 32 u + 16 (l / 32) .. +
// 15 in step u.

// 16 bytes a lane past the registers to shared memory at byte `to` + 16 lane.  By hand:
// the compiler takes any later read of shared memory for one of what such a load
// writes, and waits for it.  Whoever reads the bytes waits by arrive().
typedef uint32_t Words4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void load_past(uint32_t to, const Words4& from, uint32_t lane_offset, uint32_t offset) {
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(to), "v"(lane_offset), "s"(from), "s"(offset)
                 : "memory");
#endif
}
__device__ __forceinline__ Words4 words(const void* p, int64_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const int64_t most = 0x7FFFFFFF;
    return Words4{static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(a))),
                  static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(a >> 32) & 0xFFFF)),
                  static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(bytes < most ? bytes : most))),
                  0x00020000u};
}

// The loads behind the newest kLater have arrived in every wave, and every wave is done
// with the shared memory it read.
template <int kLater>
__device__ __forceinline__ void arrive() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kLater) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

constexpr int kStage = 64;                          // inputs of a stage
constexpr int kRing = 128 * 1024;                   // bytes of shared memory for the stages

template <bool kSilu, int kT>
__device__ __forceinline__ void tile_item(const Call& c, int e, int64_t row0, int left, int n0, uint8_t* ring) {
    constexpr int kTokens = 64 * kT, kBytes = (kTileWeights8 + kTokens) * kStage;
    constexpr int kDeep = kRing / kBytes < 6 ? kRing / kBytes : 6;
    constexpr int kLoads = 4 + kT;                  // a stage's loads of a wave
    const int lane = lane_id(), h = lane / 32, i32 = lane % 32;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const int wy = wave / 2, wx = wave % 2;
    const uint32_t at_ring = static_cast<uint32_t>(
        reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)ring));

    // This wave fills weight rows 64 wave .. + 63 and token rows 16 kT wave .. on, 16 rows
    // a load: lane l writes place l % 4 of row l / 4.  kSilu: 64 gate rows, 64 up rows, 64
    // gate rows and 64 up rows.
    const int64_t w0 = static_cast<int64_t>(e) * (kSilu ? 2 * c.N : c.N) + n0;
    const bool up = kSilu && wave % 2 == 1;
    const int base = kSilu ? wy * 64 : wave * 64, outs = c.N - n0;      // first output of this wave's weight rows
    const int wide = outs < kTileWeights8 ? outs : kTileWeights8;
    const Words4 wb = words(c.w + (w0 + (up ? c.N : 0)) * c.K, static_cast<int64_t>(wide) * c.K);
    const Words4 xb = words(c.x + row0 * c.K, static_cast<int64_t>(left < kTokens ? left : kTokens) * c.K);
    uint32_t fill[kLoads];
    const uint32_t place = ((lane & 3) ^ (lane >> 4 & 3)) * 16;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int r = (i < 4 ? base + i * 16 : (wave * kT + i - 4) * 16) + lane / 4, most = i < 4 ? wide : left;
        fill[i] = (r < most ? r : most - 1) * static_cast<uint32_t>(c.K) + place;
    }
    const int stages = c.K / kStage;
    auto ask = [&](int i, int stage, uint32_t to) {
        const int at = (stage < stages ? stage : stages - 1) * kStage;
        if (i < 4) load_past(to + (wave * 4 + i) * 1024, wb, fill[i], at);
        else load_past(to + kTileWeights8 * kStage + (wave * kT + i - 4) * 1024, xb, fill[i], at);
    };

    i32x16 acc[kT][4] = {};
    i32x4 a[2][4], b[2][kT];
    // Where the lane finds its inputs of step 0; those of step 1 are 32 bytes on or back.
    const uint32_t first = (h ^ (i32 >> 2 & 1)) * 16 + (i32 >> 3 & 1) * 32 + i32 * 64;
    // Operand g of step u: weight tile g, or token tile g - 4.
    auto read = [&](int g, int u, uint32_t from) {
        const uint8_t* p = ring + from + (first ^ (u * 32));
        if (g < 4) a[u][g] = *reinterpret_cast<const i32x4*>(p + (wy * 128 + g * 32) * kStage);
        else b[u][g - 4] = *reinterpret_cast<const i32x4*>(p + (kTileWeights8 + (wx * kT + g - 4) * 32) * kStage);
    };
    // The products of step u, and between them reads of the other step's operands at
    // `from` and, in step 1, the loads of stage `stage` to `to`.  (In this order: left
    // to itself the compiler reads an operand just before its first product.)
    auto multiply = [&](int u, uint32_t from, int stage, uint32_t to) {
#pragma unroll
        for (int m = 0; m < 4 * kT; ++m) {
            const int i = m / 4, j = m % 4;
            acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[u][j], b[u][i], acc[i][j], 0, 0, 0);
#pragma unroll
            for (int g = m; g < kLoads; g += 4 * kT) {
                read(g, 1 - u, from);
                if (u == 1) ask(g, stage, to);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    arrive<0>();                                    // the last item's loads and reads are done
#pragma unroll
    for (int d = 0; d < kDeep; ++d)
#pragma unroll
        for (int i = 0; i < kLoads; ++i) ask(i, d, at_ring + d * kBytes);
    arrive<(kDeep - 1) * kLoads>();
#pragma unroll
    for (int g = 0; g < kLoads; ++g) read(g, 0, 0);
    uint32_t here = 0;
    for (int s = 0; s < stages; ++s) {
        const uint32_t next = here + kBytes < kDeep * kBytes ? here + kBytes : 0;
        multiply(0, here, 0, 0);
        // The next stage is in, and every wave has read this one.
        arrive<(kDeep - 2) * kLoads>();
        multiply(1, next, s + kDeep, at_ring + here);
        here = next;
    }

    // A lane holds outputs 8 p + 4 h .. + 3 (p = 0 .. 3) of token row i32 of each 32 x 32
    // tile.
#pragma unroll
    for (int i = 0; i < kT; ++i) {
        const int m = (wx * kT + i) * 32 + i32;
        if (m >= left) break;
        const float xs = c.x_scales[row0 + m];
        uint16_t* out = c.y + (row0 + m) * c.N + n0;
#pragma unroll
        for (int j = 0; j < (kSilu ? 2 : 4); ++j)
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int n = wy * (kSilu ? 64 : 128) + j * 32 + 8 * p + 4 * h;
                if (n >= outs) continue;
                auto part = [&](int t) {
                    return i32x4{acc[i][t][4 * p], acc[i][t][4 * p + 1], acc[i][t][4 * p + 2], acc[i][t][4 * p + 3]};
                };
                f32x4 v = scaled(part(j), xs, scales4(c.w_scales + w0, n));
                if (kSilu) v = silu_mul(v, scaled(part(j + 2), xs, scales4(c.w_scales + w0 + c.N, n)));
                store4(out + n, v);
            }
    }
}

template <bool kSilu>
__global__ __launch_bounds__(kThreads, 1) void tile_i8_kernel(Call c, int above) {
    constexpr int kOut = kSilu ? kTileWeights8 / 2 : kTileWeights8;
    __shared__ __align__(1024) uint8_t ring[kRing];
    extern __shared__ int32_t room[];
    const Table t = make_table(room, c.expert_rows, c.E, c.capacity, c.num_rows, kTileRows8, above, INT32_MAX);
    const int columns = (c.N + kOut - 1) / kOut;
    const Share mine = share_of(static_cast<int64_t>(t.start[c.E]) * columns);
    for (int64_t item = mine.at; item < mine.end; item += mine.step) {
        const int tile = static_cast<int>(item / columns);
        const int e = expert_of(t, c.E, tile);
        const int m0 = (tile - t.start[e]) * kTileRows8, rest = t.count[e] - m0;
        const int left = __builtin_amdgcn_readfirstlane(rest < kTileRows8 ? rest : kTileRows8);
        const int64_t row0 = __builtin_amdgcn_readfirstlane(t.first[e]) + static_cast<int64_t>(m0);
        const int n0 = static_cast<int>(item - static_cast<int64_t>(tile) * columns) * kOut;
        // Products of rows that are not there would cost what the others do.
        if (left > 128) tile_item<kSilu, 4>(c, e, row0, left, n0, ring);
        else if (left > 64) tile_item<kSilu, 2>(c, e, row0, left, n0, ring);
        else tile_item<kSilu, 1>(c, e, row0, left, n0, ring);
    }
    arrive<0>();                                    // no load may write shared memory after the block's end
}

// Row tiles of `rows` that a map in order can ask for at most.
int64_t most_tiles(const Call& c, int rows) { return c.num_rows / rows + (c.num_rows < c.E ? c.num_rows : c.E); }

template <bool kSilu>
hipError_t launch(const Call& c, hipStream_t stream) {
    const I8Plan plan = i8_plan(c.num_rows, c.capacity, c.E);
    if (plan.stream_most > 0) {
        const int64_t items = most_tiles(c, 16) * ceil_div(c.N, kSilu ? 32 : 64);
        hipLaunchKernelGGL((stream_i8_kernel<kSilu>), dim3(blocks_for(items, 256 * 2)), dim3(kThreads),
                           table_bytes(c.E), stream, c, plan.stream_most);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (plan.tile_above == INT32_MAX) return hipSuccess;
    const int64_t items = most_tiles(c, kTileRows8) * ceil_div(c.N, kSilu ? kTileWeights8 / 2 : kTileWeights8);
    hipLaunchKernelGGL((tile_i8_kernel<kSilu>), dim3(blocks_for(items, 256)), dim3(kThreads), table_bytes(c.E), stream,
                       c, plan.tile_above);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_linear_i8(const int8_t* x, const float* x_scales, int64_t num_rows,
                                   const int32_t* expert_rows, int capacity, const int8_t* w, const float* w_scales,
                                   int E, int K, int N, bool silu_mul, void* y, hipStream_t stream) {
    const Call c = {x, x_scales, num_rows, expert_rows, capacity, w, w_scales, E, K, N, static_cast<uint16_t*>(y)};
    return silu_mul ? launch<true>(c, stream) : launch<false>(c, stream);
}

}  // namespace ep
