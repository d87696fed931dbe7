// moe_i8.hip -- ep_moe_i8 on gfx950: a whole mixture-of-experts layer for a few tokens
// in two launches.
//
//   up    casts the tokens, multiplies them with the gate and up rows of their
//         experts, and leaves h = silu(gate) * up in the workspace in fp32;
//   down  casts h, multiplies it with the experts' down rows, and adds each token's
//         slots with their weights.
//
// Bound by reading the weights of the experts that some slot chose, once each.  The
// slots are grouped by expert in every block anew (at most kMaxSlots ids), so that
// no launch has to do it before; the casts too are done by every block for what it needs,
// out of the caches.  Sums of products are integers, so no order changes a result;
// each token's slots are added in slot order.
#include "moe_launch.h"
#include "quant_i8.h"
#include "stream_i8.h"

namespace ep {
namespace {

// ---- the slots by expert -------------------------------------------------------------
// Tiles of up to `most` slots of one expert, in order of the experts and then of the
// slots: every block of a launch finds the same.
struct Slots {
    int tiles;
    int32_t* expert;                                // [tiles]
    int32_t* first;                                 // [tiles + 1] first place in `order`
    int32_t* order;                                 // [slots] slot (t * k + j)
};
// An expert's slots are counted by chunks of 64, four to a word.
__host__ __device__ __forceinline__ int count_words(int S) { return (S + 255) / 256; }
size_t slots_bytes(int S, int E) {
    return sizeof(int32_t) * (static_cast<size_t>(count_words(S)) * E + 3 * S + 1);
}
static_assert(kMoeMaxSlots <= 512 && kMoeMaxSlots % 256 == 0, "two words of counts");

// The sum of the bytes of v, plus a.
__device__ __forceinline__ int add_bytes(uint32_t v, int a) {
    return static_cast<int>(__builtin_amdgcn_sad_u8(v, 0u, static_cast<uint32_t>(a)));
}

template <int kThreads>
__device__ __forceinline__ Slots group_slots(const int64_t* __restrict__ topk_idx, int S, int E, int most,
                                             int32_t* room) {
    constexpr int kEach = (kMoeMaxSlots + kThreads - 1) / kThreads;
    __shared__ int32_t sums[kThreads / kWave];
    const int words = count_words(S), nbits = 32 - __builtin_clz(E);
    uint32_t* count = reinterpret_cast<uint32_t*>(room);            // [words][E]
    room += words * E;
    const Slots s = {0, room, room + S, room + 2 * S + 1};
    const int me = static_cast<int>(threadIdx.x), lane = lane_id(), wave = me / kWave;
    int id[kEach], place[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int slot = i * kThreads + me;
        const int64_t e = topk_idx[slot < S ? slot : S - 1];
        id[i] = slot < S && e >= 0 && e < E ? static_cast<int>(e) : -1;
    }
    for (int e = me; e < words * E; e += kThreads) count[e] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const uint64_t peers = match_key(id[i], id[i] >= 0, nbits);
        const int chunk = (i * kThreads + me) / kWave;
        place[i] = __popcll(peers & lanes_below());
        if (id[i] >= 0 && place[i] == 0)
            atomicAdd(&count[chunk / 4 * E + id[i]], static_cast<uint32_t>(__popcll(peers)) << chunk % 4 * 8);
    }
    __syncthreads();
    // Tiles (high half) and slots (low half) before each expert.
    const int per = (E + kThreads - 1) / kThreads, e0 = me * per;
    auto slots_of = [&](int e) { return add_bytes(count[e], words > 1 ? add_bytes(count[E + e], 0) : 0); };
    int mine = 0;
    for (int i = 0; i < per && e0 + i < E; ++i) {
        const int n = slots_of(e0 + i);
        mine += n + ((n + most - 1) / most << 16);
    }
    // The chunks before a slot's.
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int chunk = (i * kThreads + me) / kWave;
        if (id[i] < 0) continue;
        place[i] = add_bytes(count[chunk / 4 * E + id[i]] & ((1u << chunk % 4 * 8) - 1), place[i]);
        if (chunk >= 4) place[i] = add_bytes(count[id[i]], place[i]);
    }
    int upto = mine;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == kWave - 1) sums[wave] = upto;
    __syncthreads();
    int before = upto - mine, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / kWave; ++w) {
        if (w < wave) before += sums[w];
        all += sums[w];
    }
    for (int i = 0; i < per && e0 + i < E; ++i) {
        const int n = slots_of(e0 + i), start = before & 0xFFFF;
        int tile = before >> 16;
        for (int at = 0; at < n; at += most, ++tile) {
            s.expert[tile] = e0 + i;
            s.first[tile] = start + at;
        }
        count[e0 + i] = start;                      // from here on
        before += n + ((n + most - 1) / most << 16);
    }
    if (me == 0) s.first[all >> 16] = all & 0xFFFF;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEach; ++i)
        if (id[i] >= 0) s.order[count[id[i]] + place[i]] = i * kThreads + me;
    __syncthreads();
    return {__builtin_amdgcn_readfirstlane(all >> 16), s.expert, s.first, s.order};
}
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Rows of codes in shared memory are this much longer, so that 16 rows' pieces at one
// place lie in different banks.
constexpr int kPad = 16;

// ---- up ------------------------------------------------------------------------------
// A block takes a run of items: 32 gate rows and their 32 up rows of an expert against
// a tile of its slots.  Its four waves split an item's inputs and join their sums in
// shared memory.  The tokens of a tile are cast into shared memory when its first
// item comes.
constexpr int kUpThreads = 256;
constexpr int kUpCodes = 48 * 1024;                 // bytes of codes: two blocks a CU

int up_rows(int H) { return H + kPad > kUpCodes ? 1 : kUpCodes / (H + kPad) < 16 ? kUpCodes / (H + kPad) : 16; }

__global__ __launch_bounds__(kUpThreads, 2) void moe_up_i8_kernel(const uint16_t* __restrict__ x,
                                                                  const int64_t* __restrict__ topk_idx, int S, int k,
                                                                  int E, int H, int F, const int8_t* __restrict__ up,
                                                                  const float* __restrict__ up_scales, int rows,
                                                                  float* __restrict__ h) {
    __shared__ i32x4 part[16][kWave];
    __shared__ float x_scale[16];
    __shared__ uint32_t most[2][kUpThreads / kWave];
    extern __shared__ __align__(16) uint8_t room[];
    uint8_t* codes = room;                          // [rows][H + kPad]
    const int lane = lane_id(), q = lane / 16, i16 = lane % 16, stride = H + kPad;
    const int wave = uniform(static_cast<int>(threadIdx.x) / kWave);
    const Slots s = group_slots<kUpThreads>(topk_idx, S, E, rows, reinterpret_cast<int32_t*>(room + rows * stride));
    const int columns = (F + 31) / 32;
    const int64_t items = static_cast<int64_t>(s.tiles) * columns;
    // Blocks go to the 8 chiplets in turn: neighbouring runs to the blocks of one.
    const int64_t b = blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8;
    int64_t item = items * b / gridDim.x;
    const int64_t end = items * (b + 1) / gridDim.x;
    if (item == end) return;

    Stream8<4, 3, false> stream;
    uint32_t row[4];
    Buffer w[2];
    const float* w_scales = nullptr;
    int n0 = 0;
    const uint8_t* mine = nullptr;
    auto weights = [&](int j) { return w[j / 2]; };
    auto tokens = [&](int half, int at) { return *reinterpret_cast<const u32x4*>(mine + at + 64 * half); };
    // The item's rows and first loads.
    auto start = [&](int e, int column) {
        n0 = column * 32;
        const int64_t w0 = static_cast<int64_t>(e) * 2 * F + n0;
        const int left = F - n0 < 32 ? F - n0 : 32;
        w[0] = buffer(up + w0 * H, static_cast<int64_t>(left) * H);
        w[1] = buffer(up + (w0 + F) * H, static_cast<int64_t>(left) * H);
        w_scales = up_scales + w0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = j % 2 * 16 + i16;
            row[j] = (n < left ? n : left - 1) * static_cast<uint32_t>(H) + q * 16;
        }
        stream.start(wave * 128, 512, H, row, weights, tokens);
    };
    int tile = -1, count = 0, first = 0;
    for (; item < end; ++item) {
        const int now = static_cast<int>(item / columns), column = static_cast<int>(item - static_cast<int64_t>(now) * columns);
        if (now != tile) {
            tile = now;
            first = uniform(s.first[tile]);
            count = uniform(s.first[tile + 1]) - first;
            const int e = uniform(s.expert[tile]);
            for (int r = 0; r < count; ++r) {
                const int token = uniform(s.order[first + r]) / k;
                cast_row<kUpThreads, 2, false>(
                    reinterpret_cast<const u32x4*>(x + static_cast<int64_t>(token) * H), H / 16,
                    static_cast<int>(threadIdx.x), most[r & 1],
                    [&] {
                        if (r == 0) start(e, column);
                    },
                    [&](int p, const u32x4& v) { *reinterpret_cast<u32x4*>(codes + r * stride + p * 16) = v; },
                    [&](float scale) {
                        if (threadIdx.x == 0) x_scale[r] = scale;
                    });
            }
            mine = codes + (i16 < count ? i16 : count - 1) * stride + q * 16;
            __syncthreads();
        }
        i32x4 acc[4] = {};
        stream.run(wave * 128, 512, H, row, weights, tokens, acc);
        const int n = n0 + wave * 16 + 4 * q;
        const float* ws = w_scales + wave * 16 + 4 * q;
        // The next item's loads go out before this one's sums are joined.
        if (item + 1 < end && column + 1 < columns) start(uniform(s.expert[tile]), column + 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) part[wave * 4 + j][lane] = acc[j];
        __syncthreads();
        if (wave < 2 && i16 < count && n < F) {
            auto sum = [&](int j) { return part[j][lane] + part[4 + j][lane] + part[8 + j][lane] + part[12 + j][lane]; };
            const i32x4 gate = sum(wave), other = sum(wave + 2);
            const f32x4 gs = *reinterpret_cast<const f32x4*>(ws), us = *reinterpret_cast<const f32x4*>(ws + F);
            const float xs = x_scale[i16];
            f32x4 v;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                v[c] = silu(static_cast<float>(gate[c]) * (xs * gs[c])) * (static_cast<float>(other[c]) * (xs * us[c]));
            *reinterpret_cast<f32x4*>(h + static_cast<int64_t>(s.order[first + i16]) * F + n) = v;
        }
        __syncthreads();
    }
}

// ---- down ----------------------------------------------------------------------------
// A block has kRows outputs of every token.  It takes the slots in chunks whose codes fit
// shared memory; a chunk's products, tile after tile and 128 inputs at a time, are
// one row of steps of which each of the eight waves takes an eighth, so that its
// loads run on from one expert to the next.  Sums meet in shared memory by integer
// additions.
constexpr int kDownThreads = 512;
constexpr int kDownCodes = 64 * 1024;

// Four codes a lane and step of a row of h, cast into shared memory by one wave; its
// scale.
__device__ __forceinline__ float cast_h(const float* __restrict__ h, int F, uint8_t* to) {
    constexpr int kKeep = 8;                        // vectors in registers: rows of up to 2048
    const int lane = lane_id(), vectors = F / 4;
    const f32x4* row = reinterpret_cast<const f32x4*>(h);
    f32x4 v[kKeep];
    uint32_t m = 0u;
    for (int base = 0; base < vectors; base += kKeep * kWave) {
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            const int p = base + i * kWave + lane;
            v[i] = row[p < vectors ? p : vectors - 1];
        }
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t bits = __float_as_uint(v[i][c]) & 0x7FFFFFFFu;
                m = m > bits ? m : bits;
            }
    }
    const Cast cast = cast_of(wave_most(m));
    for (int base = 0; base < vectors; base += kKeep * kWave) {
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            const int p = base + i * kWave + lane;
            if (vectors > kKeep * kWave) v[i] = row[p < vectors ? p : vectors - 1];
            if (p < vectors) *reinterpret_cast<uint32_t*>(to + p * 4) = four_codes(cast, v[i][0], v[i][1], v[i][2], v[i][3]);
        }
    }
    return cast.scale;
}

template <int kRows>
__global__ __launch_bounds__(kDownThreads, 2) void moe_down_i8_kernel(
    const float* __restrict__ h, const int64_t* __restrict__ topk_idx, const float* __restrict__ topk_weights, int S,
    int T, int k, int E, int H, int F, const int8_t* __restrict__ down, const float* __restrict__ down_scales,
    int chunk_slots, int tile_slots, uint16_t* __restrict__ out) {
    constexpr int kTiles = kRows / 16, kDeep = 12 / kTiles;
    extern __shared__ __align__(16) uint8_t room[];
    const int lane = lane_id(), q = lane / 16, i16 = lane % 16, stride = F + kPad;
    const int wave = uniform(static_cast<int>(threadIdx.x) / kWave);
    uint8_t* codes = room;                                                  // [chunk_slots][F + kPad]
    int32_t* sums = reinterpret_cast<int32_t*>(room + chunk_slots * stride);    // [S][kRows]
    float* h_scale = reinterpret_cast<float*>(sums + S * kRows);                // [S]
    const Slots s = group_slots<kDownThreads>(topk_idx, S, E, tile_slots, reinterpret_cast<int32_t*>(h_scale + S));
    for (int i = static_cast<int>(threadIdx.x); i < S * kRows; i += kDownThreads) sums[i] = 0;
    const int n0 = static_cast<int>(blockIdx.x) * kRows, left = H - n0 < kRows ? H - n0 : kRows;
    const int steps = F / 128;
    uint32_t row[kTiles];
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
        const int n = j * 16 + i16;
        row[j] = (n < left ? n : left - 1) * static_cast<uint32_t>(F) + q * 16;
    }
    u32x4 w[kDeep][kTiles][2];
    for (int t0 = 0, t1; t0 < s.tiles; t0 = t1) {
        // The tiles of this chunk: at least one, for tile_slots <= chunk_slots.
        const int place0 = uniform(s.first[t0]);
        for (t1 = t0 + 1; t1 < s.tiles && uniform(s.first[t1 + 1]) - place0 <= chunk_slots;) ++t1;
        const int all = (t1 - t0) * steps, begin = all * wave / 8, end = all * (wave + 1) / 8;
        int from = t0 + begin / steps, from_at = begin % steps, to_ask = end - begin;    // the loads' tile and step
        Buffer wb = buffer(down, 0);
        auto aim = [&] {
            const int64_t w0 = static_cast<int64_t>(uniform(s.expert[from])) * H + n0;
            wb = buffer(down + w0 * F, static_cast<int64_t>(left) * F);
        };
        auto load = [&](int buf) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
#pragma unroll
                for (int half = 0; half < 2; ++half) w[buf][j][half] = load16(wb, row[j], from_at * 128 + 64 * half);
            __builtin_amdgcn_sched_barrier(0);
            // Past its end a wave asks for its last step again.
            if (--to_ask > 0 && ++from_at == steps) {
                from_at = 0;
                ++from;
                aim();
            }
        };
        aim();
#pragma unroll
        for (int b = 0; b < kDeep; ++b) load(b);
        for (int p = wave; p < uniform(s.first[t1]) - place0; p += kDownThreads / kWave) {
            const int slot = uniform(s.order[place0 + p]);
            const float scale = cast_h(h + static_cast<int64_t>(slot) * F, F, codes + p * stride);
            if (lane == 0) h_scale[slot] = scale;
        }
        __syncthreads();
        int tile = t0 + begin / steps, at = begin % steps, first = 0, count = 0;
        const uint8_t* mine = codes;
        auto enter = [&] {
            first = uniform(s.first[tile]);
            count = uniform(s.first[tile + 1]) - first;
            mine = codes + (first - place0 + (i16 < count ? i16 : count - 1)) * stride + q * 16;
        };
        i32x4 acc[kTiles] = {};
        if (begin < end) enter();
        for (int g = begin; g < end; g += kDeep)
#pragma unroll
            for (int b = 0; b < kDeep; ++b) {
                if (g + b < end) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const u32x4 t = *reinterpret_cast<const u32x4*>(mine + at * 128 + 64 * half);
#pragma unroll
                        for (int j = 0; j < kTiles; ++j)
                            acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w[b][j][half]),
                                                                           __builtin_bit_cast(i32x4, t), acc[j], 0, 0, 0);
                    }
                    if (++at == steps || g + b + 1 == end) {
                        if (i16 < count) {
                            int32_t* to = sums + s.order[first + i16] * kRows + 4 * q;
#pragma unroll
                            for (int j = 0; j < kTiles; ++j)
#pragma unroll
                                for (int c = 0; c < 4; ++c) atomicAdd(to + j * 16 + c, acc[j][c]);
                        }
#pragma unroll
                        for (int j = 0; j < kTiles; ++j) acc[j] = i32x4{};
                        at = 0;
                        ++tile;
                        if (g + b + 1 < end) enter();
                    }
                }
                load(b);
            }
        __syncthreads();
    }
    __syncthreads();
    for (int i = static_cast<int>(threadIdx.x); i < T * (kRows / 2); i += kDownThreads) {
        const int t = i / (kRows / 2), n = i % (kRows / 2) * 2;
        if (n >= left) continue;
        float a = 0.0f, b = 0.0f;
        for (int j = 0; j < k; ++j) {
            const int slot = t * k + j;
            const int64_t e = topk_idx[slot];
            if (e < 0 || e >= E) continue;
            const float* ws = down_scales + e * H + n0 + n;
            const float hs = h_scale[slot], weight = topk_weights ? topk_weights[slot] : 1.0f;
            a = __builtin_fmaf(weight, static_cast<float>(sums[slot * kRows + n]) * (hs * ws[0]), a);
            b = __builtin_fmaf(weight, static_cast<float>(sums[slot * kRows + n + 1]) * (hs * ws[1]), b);
        }
        *reinterpret_cast<uint32_t*>(out + static_cast<int64_t>(t) * H + n0 + n) = bf16_rne(a) | bf16_rne(b) << 16;
    }
}

template <int kRows>
hipError_t launch_down(const float* h, const int64_t* topk_idx, const float* topk_weights, int T, int k, int E, int H,
                       int F, const int8_t* down, const float* down_scales, void* out, hipStream_t stream) {
    const int S = T * k, stride = F + kPad;
    int chunk = stride > kDownCodes ? 1 : kDownCodes / stride;
    if (chunk > S) chunk = S;
    const size_t lds = static_cast<size_t>(chunk) * stride + sizeof(int32_t) * S * kRows + sizeof(float) * S + slots_bytes(S, E);
    hipLaunchKernelGGL((moe_down_i8_kernel<kRows>), dim3(static_cast<unsigned>(ceil_div(H, kRows))), dim3(kDownThreads),
                       lds, stream, h, topk_idx, topk_weights, S, T, k, E, H, F, down, down_scales, chunk,
                       chunk < 16 ? chunk : 16, static_cast<uint16_t*>(out));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_i8(const void* x, const int64_t* topk_idx, const float* topk_weights, int T, int k, int E, int H,
                         int F, const int8_t* up, const float* up_scales, const int8_t* down, const float* down_scales,
                         float* h, void* out, hipStream_t stream) {
    const int S = T * k, rows = up_rows(H);
    const int64_t items = static_cast<int64_t>(S) * ceil_div(F, 32);
    hipLaunchKernelGGL(moe_up_i8_kernel, dim3(blocks_for(items, 512)), dim3(kUpThreads),
                       static_cast<size_t>(rows) * (H + kPad) + slots_bytes(S, E), stream, static_cast<const uint16_t*>(x),
                       topk_idx, S, k, E, H, F, up, up_scales, rows, h);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (H <= 4096) return launch_down<16>(h, topk_idx, topk_weights, T, k, E, H, F, down, down_scales, out, stream);
    return launch_down<32>(h, topk_idx, topk_weights, T, k, E, H, F, down, down_scales, out, stream);
}

}  // namespace ep
