// moe_i8.hip -- ep_moe_i8 on gfx950: a whole mixture-of-experts layer for a few tokens
// in two launches.
//
//   up    casts the tokens, multiplies them with the gate and up rows of their
//         experts, and leaves h = silu(gate) * up in the workspace in fp32, with the
//         largest magnitudes of every 32 of a row;
//   down  casts h, multiplies it with the experts' down rows, and adds each token's
//         slots with their weights.
//
// Where experts have few slots each, bound by reading the weights of those that some slot
// chose: 16 tokens, 8 of 256 experts, 7168 -> 2048 (4.5 GB) 760-790 us, 5.8 TB/s; one token
// (353 MB) 76 us, 4.6 TB/s (up 46, down 29), of which a launch's start (the slots, the
// casts, the first loads) is 6 us or more.  What is left at 64 tokens, 6 of 64 experts, 4096 ->
// 1024 (805 MB, 184-201 us, 4.0-4.4 TB/s) are the casts of h, 384 rows in every block of down.
//
// Weights are read once for every tile of up to 16 slots of an expert (fewer in up where
// rows are long: 15 at 8192 inputs, 7 at 16384), in down for every part of the tokens too,
// from the second time on mostly out of the caches; and every block of down casts h of
// all its slots.  So many slots an expert cost more than their weights: 64 tokens, 8 of 8
// experts, 2048 -> 1408 (70 MB, 13 us at 5.2 TB/s) 82 us, 8 of 16, 4096 -> 1408 (278 MB, 53 us)
// 169; by dispatch, products, cast, products and combine 54 and 86.
//
// The slots are grouped by expert in every block anew (at most kMoeMaxSlots ids), so that
// no launch has to do it before; the casts too are done by every block for what it needs,
// out of the caches.  Sums of products are integers, so no order changes a result; each
// token's slots are added in slot order.
#include "moe_launch.h"
#include "quant_i8.h"
#include "stream_i8.h"

namespace ep {
namespace {

// ---- the slots by expert -------------------------------------------------------------
// Tiles of up to `most` slots of one expert, an expert's in order of the slots.  Blocks that
// group the same slots find the same places, but the two launches, and parts of the
// tokens, each have their own: what goes from up to down is held by slot.
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

// At most 64 slots, one a lane: without counters, experts in the order in which the
// slots name them first.
__device__ __forceinline__ Slots group_few_slots(const int64_t* __restrict__ topk_idx, int S, int E, int most,
                                                 int32_t* room) {
    const Slots s = {0, room, room + S, room + 2 * S + 1};
    const int lane = lane_id();
    const int64_t e = topk_idx[lane < S ? lane : S - 1];
    const bool valid = lane < S && e >= 0 && e < E;
    const int id = valid ? static_cast<int>(e) : -1;
    const uint64_t peers = match_key(id, valid, 32 - __builtin_clz(E));
    const int count = __popcll(peers), rank = __popcll(peers & lanes_below()), tiles = (count + most - 1) / most;
    // Tiles (high half) and slots (low half) of the experts named before; of an expert's
    // lanes the first one counts.
    const int mine = valid && rank == 0 ? count + (tiles << 16) : 0;
    int upto = mine;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    const int all = read_lane(upto, kWave - 1);
    const int before = __shfl(upto - mine, valid ? __builtin_ctzll(peers) : 0);
    if (threadIdx.x < kWave) {
        if (valid) s.order[(before & 0xFFFF) + rank] = lane;
        if (valid && rank == 0)
            for (int t = 0; t < tiles; ++t) {
                s.expert[(before >> 16) + t] = id;
                s.first[(before >> 16) + t] = (before & 0xFFFF) + t * most;
            }
        if (lane == 0) s.first[all >> 16] = all & 0xFFFF;
    }
    __syncthreads();
    return {__builtin_amdgcn_readfirstlane(all >> 16), s.expert, s.first, s.order};
}

template <int kThreads>
__device__ __forceinline__ Slots group_slots(const int64_t* __restrict__ topk_idx, int S, int E, int most,
                                             int32_t* room) {
    if (S <= kWave) return group_few_slots(topk_idx, S, E, most, room);
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

typedef float f32x2 __attribute__((ext_vector_type(2)));

// ---- up ------------------------------------------------------------------------------
// An item is 32 gate rows and their 32 up rows of an expert against a tile of its slots.
// A block's eight waves take a run of items together, splitting each item's inputs and
// joining their sums in shared memory; or (kAlone), where there are few inputs to split,
// each wave takes a run of its own, and no wave waits for another.  Loads run on from one
// item to the next, one step of a wave's ahead.  (Steps on the way, and both launches for
// one token: one 79 us, two 80, three 83, four 88; 16 tokens: 785, 786, 791, 794.)  The tokens
// of a tile are cast into shared memory when its first item comes.
constexpr int kUpThreads = 512, kUpWaves = kUpThreads / kWave;
constexpr int kUpShared = 126 * 1024;               // bytes of a CU's 160 KB beside what is declared below
constexpr int kUpOut = 32;                          // outputs of an item

// Rows of a tile: as many as find room.
int up_rows(int S, int E, int H, bool alone) {
    const int rows = (kUpShared - static_cast<int>(slots_bytes(S, E))) / (H + kPad) / (alone ? kUpWaves : 1);
    return rows < 16 ? rows : 16;
}

// What a wave wrote to shared memory is there for its other lanes.
__device__ __forceinline__ void settle_wave() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The largest |h| of a slot's outputs of one item, as fp32 bits: at most[slot * (F / 32)
// + column].
template <bool kAlone>
__global__ __launch_bounds__(kUpThreads, 2) void moe_up_i8_kernel(const uint16_t* __restrict__ x,
                                                                  const int64_t* __restrict__ topk_idx, int S, int k,
                                                                  int E, int H, int F, const int8_t* __restrict__ up,
                                                                  const float* __restrict__ up_scales, int rows,
                                                                  float* __restrict__ h, uint32_t* __restrict__ most) {
    constexpr int kTeam = kAlone ? 1 : kUpWaves;    // waves that share an item
    constexpr int kThreads = kTeam * kWave, kBatch = kAlone ? 2 : 4;        // (rows cast at a time)
    constexpr int kSides = kAlone ? 2 : 1;          // groups of 16 outputs that a wave finishes
    __shared__ i32x4 part[kAlone ? 1 : kUpWaves][4][kWave];
    __shared__ float x_scale[kUpWaves / kTeam][16];
    __shared__ uint32_t row_room[2][kBatch][kTeam], h_room[16];
    extern __shared__ __align__(16) uint8_t room[];
    const int lane = lane_id(), q = lane / 16, i16 = lane % 16, stride = H + kPad;
    const int block_wave = uniform(static_cast<int>(threadIdx.x) / kWave), wave = kAlone ? 0 : block_wave;
    const int team = kAlone ? block_wave : 0, me = wave * kWave + lane;
    uint8_t* codes = room + team * rows * stride;   // [rows][H + kPad]
    const Slots s = group_slots<kUpThreads>(topk_idx, S, E, rows,
                                            reinterpret_cast<int32_t*>(room + kUpWaves / kTeam * rows * stride));
    const int columns = F / kUpOut;
    const int64_t items = static_cast<int64_t>(s.tiles) * columns;
    // Blocks go to the 8 chiplets in turn: neighbouring runs to the blocks of one.
    const int64_t b = (blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8) * (kUpWaves / kTeam) + team;
    const int64_t runs = static_cast<int64_t>(gridDim.x) * (kUpWaves / kTeam);
    const int begin = static_cast<int>(items * b / runs), end = static_cast<int>(items * (b + 1) / runs);
    if (begin == end) return;
    // A wave's steps of an item: inputs 128 (wave + kTeam i) .. + 127.
    const int steps = (H / 128 + kTeam - 1) / kTeam;

    // The loading side.  Past its end a wave asks for its last step again.
    u32x4 w[4][2];
    uint32_t row[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) row[j] = (j % 2 * 16 + i16) * static_cast<uint32_t>(H) + q * 16;
    Buffer from[2];
    int tile = begin / columns, column = begin % columns;
    int ask_step = 0, ask_tile = tile, ask_column = column, ask_left = end - begin;
    auto aim = [&] {
        const int8_t* p = up + (static_cast<int64_t>(uniform(s.expert[ask_tile])) * 2 * F + ask_column * kUpOut) * H;
        from[0] = buffer(p, static_cast<int64_t>(kUpOut) * H);
        from[1] = buffer(p + static_cast<int64_t>(F) * H, static_cast<int64_t>(kUpOut) * H);
    };
    auto load = [&] {
        int at = (wave + ask_step * kTeam) * 128;
        at = at < H ? at : H - 128;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int half = 0; half < 2; ++half) w[j][half] = load16(from[j / 2], row[j], at + 64 * half);
        __builtin_amdgcn_sched_barrier(0);
        if (++ask_step == steps) {
            if (--ask_left > 0) {
                ask_step = 0;
                if (++ask_column == columns) {
                    ask_column = 0;
                    ++ask_tile;
                }
                aim();
            } else {
                ask_left = 1;
                --ask_step;
            }
        }
    };

    // The scales of an item's rows, asked for while the item before is finished.
    f32x4 gs[kSides], us[kSides];
    auto ask_scales = [&] {
        const float* ws = up_scales + static_cast<int64_t>(uniform(s.expert[tile])) * 2 * F + column * kUpOut + wave % 2 * 16 + 4 * q;
#pragma unroll
        for (int g = 0; g < kSides; ++g) {
            gs[g] = *reinterpret_cast<const f32x4*>(ws + g * 16);
            us[g] = *reinterpret_cast<const f32x4*>(ws + F + g * 16);
        }
    };
    // The tile at hand, and its slots' tokens from r0 on, cast.  `ready` runs behind the
    // first loads.
    int count = 0, first = 0;
    const uint8_t* mine = nullptr;
    auto enter = [&] {
        first = uniform(s.first[tile]);
        count = uniform(s.first[tile + 1]) - first;
    };
    auto cast_batch = [&](int r0, auto ready) {
        const u32x4* from_x[kBatch];
#pragma unroll
        for (int r = 0; r < kBatch; ++r) {
            const int token = uniform(s.order[first + (r0 + r < count ? r0 + r : count - 1)]) / k;
            from_x[r] = reinterpret_cast<const u32x4*>(x + static_cast<int64_t>(token) * H);
        }
        cast_rows<kThreads, kAlone ? 2 : 1, kBatch, false, kAlone>(
            from_x, H / 16, me, row_room[r0 / kBatch % 2], ready,
            [&](int r, int p, const u32x4& v) {
                if (r0 + r < count) *reinterpret_cast<u32x4*>(codes + (r0 + r) * stride + p * 16) = v;
            },
            [&](int r, float scale) {
                if (me == 0 && r0 + r < count) x_scale[team][r0 + r] = scale;
            });
    };

    i32x4 acc[4] = {};
    // Four outputs of the lane's slot, from n on, and their largest magnitude so far.
    auto result = [&](const i32x4& gate, const i32x4& other, int g, int n, uint32_t m) {
        const float xs = x_scale[team][i16];
        f32x4 v;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            v[c] = silu(static_cast<float>(gate[c]) * (xs * gs[g][c])) * (static_cast<float>(other[c]) * (xs * us[g][c]));
            m = larger(m, __float_as_uint(v[c]) & 0x7FFFFFFFu);
        }
        *reinterpret_cast<f32x4*>(h + static_cast<int64_t>(s.order[first + i16]) * F + n) = v;
        return m;
    };
    // The waves' sums of an item, and its results.
    auto finish = [&] {
        uint32_t m = 0u;
        if constexpr (kAlone) {
            if (i16 < count)
#pragma unroll
                for (int g = 0; g < 2; ++g) m = result(acc[g], acc[g + 2], g, column * kUpOut + g * 16 + 4 * q, m);
            m = across_rows(m);
            if (lane < count) most[static_cast<int64_t>(s.order[first + lane]) * columns + column] = m;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) part[wave][j][lane] = acc[j];
            __syncthreads();
            if (wave < 2 && i16 < count) {
                auto sum = [&](int j) {
                    i32x4 v = part[0][j][lane];
#pragma unroll
                    for (int o = 1; o < kTeam; ++o) v += part[o][j][lane];
                    return v;
                };
                m = result(sum(wave), sum(wave + 2), 0, column * kUpOut + wave * 16 + 4 * q, m);
            }
            m = across_rows(m);
            if (wave == 1 && q == 0) h_room[i16] = m;
            __syncthreads();
            if (wave == 0 && lane < count)
                most[static_cast<int64_t>(s.order[first + lane]) * columns + column] = larger(m, h_room[lane]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = i32x4{};
    };

    aim();
    enter();
    cast_batch(0, [&] {
        ask_scales();
        load();
    });
    // (The code is kept short: it comes from memory anew in every call.  53 KB of it, with two
    // steps and these casts in each, against 21: 1 token, 1 of 16 experts, 2560 -> 384, 25 / 21
    // us; 8 of 256, 7168 -> 2048, 78 / 76; 40 tokens, 7 of 64, 1024 -> 1024, 73 / 70; but 64, 6
    // of 64, 4096 -> 1024, 184 / 186.)
    int r0 = kBatch;                                // of a tile that is entered anew 0
    for (int left = end - begin;;) {
        if (column == 0 || r0 > 0) {
            if (r0 == 0) {
                if constexpr (kAlone) settle_wave();        // the last tile's codes are read
                enter();
            }
            for (; r0 < count; r0 += kBatch) cast_batch(r0, [] {});
            r0 = 0;
            mine = codes + (i16 < count ? i16 : count - 1) * stride + q * 16;
            if constexpr (kAlone) settle_wave();
            else __syncthreads();
        }
        int step = 0;
        do {
            const int at = (wave + step * kTeam) * 128;
            if (at < H) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const u32x4 t = *reinterpret_cast<const u32x4*>(mine + at + 64 * half);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w[j][half]),
                                                                       __builtin_bit_cast(i32x4, t), acc[j], 0, 0, 0);
                }
            }
            load();
        } while (++step < steps);
        finish();
        if (--left == 0) break;
        if (++column == columns) {
            column = 0;
            ++tile;
        }
        ask_scales();
    }
}

// ---- down ----------------------------------------------------------------------------
// A block has kRows outputs of every token, or of a part of the tokens where that leaves
// CUs without a block (the experts that two parts have in common are read twice, but
// mostly out of the caches).  It takes the slots in chunks whose codes fit half of its
// shared memory for them.  Eight waves multiply: a chunk's products, tile
// after tile and 128 inputs at a time, are one row of steps of which each takes an
// eighth; their loads run on from one chunk to the next, and sums meet in shared memory
// by integer additions.  Eight more waves cast the next chunk's h meanwhile.  (Both
// launches for 64 tokens, 6 of 64 experts, 4096 -> 1024: by the same eight waves, between the
// chunks, 270 us; four of them beside eight 199; eight 186.  Of 88 us of down, 30 go if h is
// not read, and 8 if the weights come out of the L2: h and weights share the CU's way in.)
constexpr int kDownWaves = 8, kCastWaves = 8, kDownThreads = (kDownWaves + kCastWaves) * kWave;
constexpr int kDownCodes = 32 * 1024;               // a chunk's codes at most
constexpr int kDownRoom = 34 * 1024;                // and the bytes they take with their padding

// Tiles t0 .. t1 - 1, with places p0 .. p1 - 1.
struct Chunk {
    int t0, t1, p0, p1;
};
// The chunk that begins with tile t0: as many tiles as have at most `slots` places, and
// that is at least one.  Every lane asks about one tile in `step`, then about one of
// those between.
__device__ __forceinline__ Chunk chunk_from(const Slots& s, int t0, int slots) {
    Chunk c = {t0, t0, 0, 0};
    if (t0 >= s.tiles) return c;
    const int step = (kMoeMaxSlots + kWave - 1) / kWave, lane = lane_id();
    c.p0 = uniform(s.first[t0]);
    auto fits = [&](int t) { return t <= s.tiles && s.first[t <= s.tiles ? t : s.tiles] - c.p0 <= slots; };
    const int t = t0 + (__popcll(ballot(fits(t0 + lane * step))) - 1) * step;
    c.t1 = uniform(t + __popcll(ballot(lane < step && fits(t + lane))) - 1);
    c.p1 = uniform(s.first[c.t1]);
    return c;
}

template <int kRows>
__global__ __launch_bounds__(kDownThreads, kDownThreads / 256) void moe_down_i8_kernel(
    const float* __restrict__ h, const uint32_t* __restrict__ most, const int64_t* __restrict__ topk_idx,
    const float* __restrict__ topk_weights, int T, int parts, int k, int E, int H, int F,
    const int8_t* __restrict__ down, const float* __restrict__ down_scales, int chunk_slots, int tile_slots,
    uint16_t* __restrict__ out) {
    // A wave has 4 KB on the way: 2 steps of 16 rows, or one of 32.  (8, 4 and 2 KB, both launches,
    // us: 64 tokens, 8 of 64 experts, 1024 -> 1024, 85, 81, 87; 32, 6 of 64, 4096 -> 1024, 176,
    // 168, 175; 1, 1 of 16, 2560 -> 384, 22, 20, 20; 16, 8 of 256, 7168 -> 2048, 784, 785, -.)
    constexpr int kTiles = kRows / 16, kDeep = 2 / kTiles;
    extern __shared__ __align__(16) uint8_t room[];
    const int lane = lane_id(), q = lane / 16, i16 = lane % 16, stride = F + kPad, me = static_cast<int>(threadIdx.x);
    const int wave = uniform(me / kWave), half = chunk_slots * stride;
    // From here on tokens, slots and what belongs to them are those of the block's part.
    const int part = static_cast<int>(blockIdx.x) / (H / kRows), n0 = static_cast<int>(blockIdx.x) % (H / kRows) * kRows;
    const int token0 = static_cast<int>(static_cast<int64_t>(T) * part / parts);
    T = static_cast<int>(static_cast<int64_t>(T) * (part + 1) / parts) - token0;
    const int S = T * k;
    const int64_t slot0 = static_cast<int64_t>(token0) * k;
    topk_idx += slot0;
    if (topk_weights) topk_weights += slot0;
    h += slot0 * F;
    most += slot0 * (F / kUpOut);
    out += static_cast<int64_t>(token0) * H;
    uint8_t* codes = room;                                                      // [2][chunk_slots][F + kPad]
    int32_t* sums = reinterpret_cast<int32_t*>(room + 2 * half);                // [S][kRows]
    f32x2* casts = reinterpret_cast<f32x2*>(sums + S * kRows);                  // [S] of a place: scale, 127 / a
    const Slots s = group_slots<kDownThreads>(topk_idx, S, E, tile_slots, reinterpret_cast<int32_t*>(casts + S));
    const int places = uniform(s.first[s.tiles]);

    // Every wave meets the others once before the first chunk's cast, once behind it, and
    // once behind each chunk but the last.
    if (wave >= kDownWaves) {
        constexpr int kThreads = kCastWaves * kWave, kKeep = 4;
        const int mine = me - kDownWaves * kWave, vectors = F / 4, pieces = (vectors + kWave - 1) / kWave;
        for (int p = mine; p < places; p += kThreads) {
            const int columns = F / kUpOut / 4;     // in vectors of four
            const u32x4* from = reinterpret_cast<const u32x4*>(most) + static_cast<int64_t>(s.order[p]) * columns;
            u32x4 m = {};
            for (int c = 0; c < columns; c += 16) {
                u32x4 v[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = from[c + e < columns ? c + e : columns - 1];
#pragma unroll
                for (int e = 0; e < 16; ++e)
#pragma unroll
                    for (int x = 0; x < 4; ++x) m[x] = larger(m[x], v[e][x]);
            }
            const uint32_t bits = larger(larger(m[0], m[1]), larger(m[2], m[3]));
            const float a = __uint_as_float(bits);
            const bool none = bits < 0x04000000u || bits >= 0x7F800000u;    // (127 / a stays finite from 2^-119 on)
            // 127 / a; above 2^60 by way of a * 2^-100, for the reciprocal of more than 2^126 is
            // below the normal numbers, where the hardware gives 0.
            const float by = bits > 0x5D800000u ? 0x1p-100f : 1.0f;
            casts[p] = f32x2{a / 127.0f, none ? 0.0f : 127.0f * by * __builtin_amdgcn_rcpf(a * by)};
        }
        __syncthreads();
        // Pieces of 64 vectors of four of a place's h, place by place, every kCastWaves-th
        // of them this wave's.  The next kKeep, of the same chunk or the next one, are asked
        // for before these are cast; in every chunk a wave has at least one such batch,
        // however few pieces there are for it.
        struct Piece {
            int p, i, row;
        };
        f32x4 v[2][kKeep];
        Chunk c = chunk_from(s, 0, chunk_slots), a = c;                         // cast, asked for
        const Buffer from = buffer(h, static_cast<int64_t>(S) * F * 4);
        Piece asked = {};
        bool all = false;                           // of chunk a are asked for
        auto begin = [&](int p) {
            asked = {p, 0, p < a.p1 - a.p0 ? uniform(s.order[a.p0 + p]) : S};
        };
        // (Past a row's end the next row's are read, past the chunk's last row nothing: there
        // the lanes' own offsets, which alone are held against its size for sure, are
        // behind the buffer's end.)
        auto ask = [&](int b) {
            if (all) {
                a = chunk_from(s, a.t1, chunk_slots);
                begin(wave - kDownWaves);
            }
#pragma unroll
            for (int e = 0; e < kKeep; ++e) {
                v[b][e] = __builtin_bit_cast(f32x4, load16(from, asked.row * F * 4 + (asked.i * kWave + lane) * 16, 0));
                if (++asked.i == pieces) begin(asked.p + kCastWaves);
            }
            all = asked.p >= a.p1 - a.p0;
        };
        Piece at = {wave - kDownWaves, 0, 0};
        int odd = 0;
        auto cast = [&](int b) {
#pragma unroll
            for (int e = 0; e < kKeep; ++e) {
                if (at.p >= c.p1 - c.p0) break;
                const float by = casts[c.p0 + at.p][1];
                // 127 h / a by the product with 127 / a: the quotient's own error is that of fp32.
                uint32_t code[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) code[x] = __float_as_uint(__builtin_fmaf(v[b][e][x], by, 12582912.0f));
                const uint32_t lo = __builtin_amdgcn_perm(code[1], code[0], 0x0C0C0400u);
                const uint32_t hi = __builtin_amdgcn_perm(code[3], code[2], 0x04000C0Cu);
                const int vec = at.i * kWave + lane;
                if (vec < vectors)
                    *reinterpret_cast<uint32_t*>(codes + odd * half + at.p * stride + vec * 4) = by == 0.0f ? 0u : lo | hi;
                if (++at.i == pieces) {
                    at.i = 0;
                    at.p += kCastWaves;
                }
            }
        };
        begin(wave - kDownWaves);
        if (places > 0) ask(0);
        while (c.t0 < s.tiles)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (c.t0 >= s.tiles) break;
                ask(1 - b);
                cast(b);
                if (at.p >= c.p1 - c.p0) {          // the chunk is cast, and a the next one
                    __syncthreads();
                    c = a;
                    at = {wave - kDownWaves, 0, 0};
                    odd ^= 1;
                }
            }
    } else {
        const int steps = F / 128;
        for (int i = me; i < S * kRows; i += kDownWaves * kWave) sums[i] = 0;
        uint32_t row[kTiles];
#pragma unroll
        for (int j = 0; j < kTiles; ++j) row[j] = (j * 16 + i16) * static_cast<uint32_t>(F) + q * 16;
        // A wave's steps of a chunk, and where they begin.
        struct Share {
            Chunk c;
            int left, tile, at;
        };
        auto share_from = [&](int t0) {
            Share r = {chunk_from(s, t0, chunk_slots), 0, 0, 0};
            const int all = (r.c.t1 - r.c.t0) * steps, begin = all * wave / kDownWaves;
            r.left = all * (wave + 1) / kDownWaves - begin;
            r.tile = r.c.t0 + begin / steps;
            r.at = begin % steps;
            return r;
        };
        u32x4 w[kDeep][kTiles][2];
        Share ask = share_from(0);
        Buffer from;
        auto aim = [&] {
            const int64_t w0 = static_cast<int64_t>(uniform(s.expert[ask.tile])) * H + n0;
            from = buffer(down + w0 * F, static_cast<int64_t>(kRows) * F);
        };
        // On to the next chunk in which the wave has a step; behind the last one its last
        // step is asked for again.
        auto ahead = [&] {
            for (int t = ask.c.t1; t < s.tiles;) {
                const Share r = share_from(t);
                if (r.left > 0) {
                    ask = r;
                    aim();
                    return;
                }
                t = r.c.t1;
            }
        };
        auto load = [&](int buf) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < kTiles; ++j)
#pragma unroll
                for (int side = 0; side < 2; ++side) w[buf][j][side] = load16(from, row[j], ask.at * 128 + 64 * side);
            __builtin_amdgcn_sched_barrier(0);
            if (ask.left > 1) {
                --ask.left;
                if (++ask.at == steps) {
                    ask.at = 0;
                    ++ask.tile;
                    aim();
                }
            } else {
                ahead();
            }
        };
        Share now = ask;
        if (places > 0) {
            aim();
            if (ask.left == 0) ahead();
#pragma unroll
            for (int d = 0; d < kDeep; ++d) load(d);
        }
        __syncthreads();
        if (places > 0) __syncthreads();
        int odd = 0, first = 0, count = 0;
        const uint8_t* mine = codes;
        auto enter = [&] {
            first = uniform(s.first[now.tile]);
            count = uniform(s.first[now.tile + 1]) - first;
            mine = codes + odd * half + (first - now.c.p0 + (i16 < count ? i16 : count - 1)) * stride + q * 16;
        };
        // To the next chunk in which the wave has a step.
        auto next_chunk = [&] {
            while (now.left == 0 && now.c.t1 < s.tiles) {
                __syncthreads();
                odd ^= 1;
                now = share_from(now.c.t1);
            }
            if (now.left > 0) enter();
        };
        if (places > 0 && now.left > 0) enter();
        else next_chunk();
        i32x4 acc[kTiles] = {};
        while (now.left > 0)
#pragma unroll
            for (int d = 0; d < kDeep; ++d) {
                if (now.left > 0) {
#pragma unroll
                    for (int side = 0; side < 2; ++side) {
                        const u32x4 t = *reinterpret_cast<const u32x4*>(mine + now.at * 128 + 64 * side);
#pragma unroll
                        for (int j = 0; j < kTiles; ++j)
                            acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w[d][j][side]),
                                                                           __builtin_bit_cast(i32x4, t), acc[j], 0, 0, 0);
                    }
                    --now.left;
                    if (++now.at == steps || now.left == 0) {
                        if (i16 < count) {
                            int32_t* to = sums + (first + i16) * kRows + 4 * q;
#pragma unroll
                            for (int j = 0; j < kTiles; ++j)
#pragma unroll
                                for (int c = 0; c < 4; ++c) atomicAdd(to + j * 16 + c, acc[j][c]);
                        }
#pragma unroll
                        for (int j = 0; j < kTiles; ++j) acc[j] = i32x4{};
                        now.at = 0;
                        ++now.tile;
                        if (now.left > 0) enter();
                        else next_chunk();
                    }
                }
                load(d);
            }
    }
    // Places of the slots, and experts of the places (read out of topk_idx again, the scales
    // would be asked for two loads' time later: one token 80 against 78 us).
    int32_t *place = reinterpret_cast<int32_t*>(codes), *expert = place + S;
    __syncthreads();                                // behind the last chunk
    for (int i = me; i < S; i += kDownThreads) place[i] = -1;
    for (int i = me; i < s.tiles * 16; i += kDownThreads) {
        const int at = s.first[i / 16] + i % 16;
        if (at < s.first[i / 16 + 1]) expert[at] = s.expert[i / 16];
    }
    __syncthreads();
    for (int i = me; i < places; i += kDownThreads) place[s.order[i]] = i;
    __syncthreads();
    // (Slots in batches whose loads are on the way together; those of empty slots read
    // the first expert's scales.)
    constexpr int kBatch = 8;
    for (int i = me; i < T * (kRows / 2); i += kDownThreads) {
        const int t = i / (kRows / 2), n = i % (kRows / 2) * 2;
        float a = 0.0f, b = 0.0f;
        for (int j0 = 0; j0 < k; j0 += kBatch) {
            f32x2 ws[kBatch];
            float weight[kBatch];
            int p[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int slot = t * k + (j0 + j < k ? j0 + j : k - 1);
                p[j] = j0 + j < k ? place[slot] : -1;
                const int64_t e = p[j] >= 0 ? expert[p[j]] : 0;
                ws[j] = *reinterpret_cast<const f32x2*>(down_scales + e * H + n0 + n);
                weight[j] = topk_weights ? topk_weights[slot] : 1.0f;
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (p[j] < 0) continue;
                const float hs = casts[p[j]][0];
                a = __builtin_fmaf(weight[j], static_cast<float>(sums[p[j] * kRows + n]) * (hs * ws[j][0]), a);
                b = __builtin_fmaf(weight[j], static_cast<float>(sums[p[j] * kRows + n + 1]) * (hs * ws[j][1]), b);
            }
        }
        *reinterpret_cast<uint32_t*>(out + static_cast<int64_t>(t) * H + n0 + n) = bf16_rne(a) | bf16_rne(b) << 16;
    }
}

struct Call {
    const void* x;
    const int64_t* topk_idx;
    const float* topk_weights;
    int T, k, E, H, F;
    const int8_t* up;
    const float* up_scales;
    const int8_t* down;
    const float* down_scales;
    float* h;
    uint32_t* most;
    void* out;
    hipStream_t stream;
};

// Below so many inputs each wave takes items by itself: an eighth of them is two steps
// at most, and joining eight waves' sums costs more.  Alone against together (us, both
// launches): 1 token, 8 of 256, 1024 -> 2048, 29 / 34; 30 tokens, 6 of 128, 384 -> 1408,
// 54 / 77; 64, 8 of 256, 1792 -> 768, 211 / 220; but 64, 8 of 8, 1024 -> 2048, 85 / 79; 1,
// 8 of 64, 2048 -> 768, 29 / 28; 16, 6 of 64, 2048 -> 1408, 113 / 111; 64, 6 of 64, 4096 ->
// 1024, 300 / 192.
constexpr int kTogether = 2048;

template <bool kAlone>
hipError_t launch_up(const Call& c) {
    const int S = c.T * c.k, rows = up_rows(S, c.E, c.H, kAlone);
    const int64_t items = static_cast<int64_t>(S) * (c.F / kUpOut);
    hipLaunchKernelGGL((moe_up_i8_kernel<kAlone>), dim3(blocks_for(items, 256)), dim3(kUpThreads),
                       static_cast<size_t>(rows) * (c.H + kPad) * (kAlone ? kUpWaves : 1) + slots_bytes(S, c.E), c.stream,
                       static_cast<const uint16_t*>(c.x), c.topk_idx, S, c.k, c.E, c.H, c.F, c.up, c.up_scales, rows, c.h,
                       c.most);
    return hipGetLastError();
}

template <int kRows>
hipError_t launch_down(const Call& c) {
    // Parts of the tokens where a quarter of the CUs or more would have no block.  (Both
    // launches, one part against as many as this: 30 tokens, 6 of 128 experts, 384 -> 1408,
    // 147 / 77 us; 64, 4 of 64, 1024 -> 768, 82 / 63; 64, 8 of 256, 2048 -> 768, 260 / 231.)
    const int blocks = c.H / kRows;
    const int most_parts = blocks >= 192 ? 1 : 256 / blocks, parts = most_parts < c.T ? most_parts : c.T;
    const int S = (c.T + parts - 1) / parts * c.k, stride = c.F + kPad;
    static_assert(kMoeMaxFfn <= kDownCodes, "a slot's codes fit");
    int chunk = kDownCodes / c.F < kDownRoom / stride ? kDownCodes / c.F : kDownRoom / stride;
    if (chunk > S) chunk = S;
    const size_t lds = 2 * static_cast<size_t>(chunk) * stride + sizeof(int32_t) * S * kRows + sizeof(f32x2) * S + slots_bytes(S, c.E);
    hipLaunchKernelGGL((moe_down_i8_kernel<kRows>), dim3(static_cast<unsigned>(blocks * parts)), dim3(kDownThreads), lds,
                       c.stream, c.h, c.most, c.topk_idx, c.topk_weights, c.T, parts, c.k, c.E, c.H, c.F, c.down,
                       c.down_scales, chunk, chunk < 16 ? chunk : 16, static_cast<uint16_t*>(c.out));
    return hipGetLastError();
}

}  // namespace

size_t moe_i8_workspace_bytes(int S, int F) {
    return sizeof(float) * S * static_cast<size_t>(F) + sizeof(uint32_t) * S * static_cast<size_t>((F + kUpOut - 1) / kUpOut);
}

hipError_t launch_moe_i8(const void* x, const int64_t* topk_idx, const float* topk_weights, int T, int k, int E, int H,
                         int F, const int8_t* up, const float* up_scales, const int8_t* down, const float* down_scales,
                         void* workspace, void* out, hipStream_t stream) {
    float* h = static_cast<float*>(workspace);
    const Call c = {x, topk_idx, topk_weights, T, k, E, H, F, up, up_scales, down, down_scales,
                    h, reinterpret_cast<uint32_t*>(h + static_cast<int64_t>(T) * k * F), out, stream};
    const hipError_t e = H < kTogether ? launch_up<true>(c) : launch_up<false>(c);
    if (e != hipSuccess) return e;
    // Outputs of a block of down.  16 where H leaves many a block; but many slots an expert
    // are better split over twice the parts, for then the casts of h are what a block
    // reads most (us, 16 against 32 outputs: 64 tokens, 8 of 16 experts, 4096 -> 1408, 204 / 164;
    // 8 of 32, 4096 -> 1024, 174 / 151; 8 of 8, 2048 -> 1408, 102 / 81; 16, 8 of 8, 4096 -> 2048,
    // 87 / 82; 64, 4 of 16, 2048 -> 2048, 105 / 106; but 8 of 64, 2048 -> 1408, 171 / 180; 6 of
    // 64, 4096 -> 1024, 188 / 192; 1, 8 of 64, 2048 -> 768, 27 / 29).
    const bool wide = H > 4096 || T * k >= 16 * E;
    return wide ? launch_down<32>(c) : launch_down<16>(c);
}

}  // namespace ep
