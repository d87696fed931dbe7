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

// ---- few items: bound by reading the weights -------------------------------------------
// A wave takes 64 weight rows (kSilu: 32 gate rows and their 32 up rows) and up to 16
// token rows.  Where there are items for every wave, each takes whole items; where
// there are not, the four waves of a block split an item's inputs, so that every CU has
// loads in flight, and join their sums in shared memory.  One token's 8 of 256 experts,
// 7168 -> 2 x 2048 (235 MB): 46 us, 5.2 TB/s.  (One step on the way 45, three 49, four 53: past
// its end a wave asks for its last step again.  8 experts of 16 rows, 4096 -> 4096: 34
// with any; by tiles 61.)  Which calls these are: i8_streams().
//
// What an item's waves read: weight rows from n0 on (w[1]: the up rows that belong to
// them), their scales, and token rows from row0 on.
struct Operands {
    int n0;
    Buffer w[2], x;
    const float* w_scales[2];
};
template <bool kSilu>
__device__ __forceinline__ Operands operands(const Call& c, int e, int64_t row0, int left, int n0) {
    constexpr int kWide = kSilu ? 32 : 64;
    const int64_t w0 = static_cast<int64_t>(e) * (kSilu ? 2 * c.N : c.N) + n0, up = kSilu ? c.N : 0;
    const int64_t rows = c.N - n0 < kWide ? c.N - n0 : kWide, tokens = left < 16 ? left : 16;
    return {n0,
            {buffer(c.w + w0 * c.K, rows * c.K), buffer(c.w + (w0 + up) * c.K, rows * c.K)},
            buffer(c.x + row0 * c.K, tokens * c.K),
            {c.w_scales + w0, c.w_scales + w0 + up}};
}
// Weight row n of an item's; those past the outputs repeat the last one, and what they
// give is not stored.
__device__ __forceinline__ uint32_t weight_row(const Operands& o, int n, int N) {
    return o.n0 + n < N ? n : N - 1 - o.n0;
}

template <bool kSilu>
__global__ __launch_bounds__(kThreads, 2) void stream_i8_kernel(Call c) {
    constexpr int kOut = kSilu ? 32 : 64;           // outputs of an item
    constexpr int kDeep = 2;
    __shared__ i32x4 part[16][kWave];
    extern __shared__ int32_t room[];
    const int lane = lane_id(), q = lane / 16, i16 = lane % 16;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const Table t = make_table(room, c.expert_rows, c.E, c.capacity, c.num_rows, 16, 0, INT32_MAX);
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
        const Operands o = operands<kSilu>(c, e, row0, left, column * kOut);
        uint32_t row[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            row[j] = weight_row(o, (kSilu ? j % 2 : j) * 16 + i16, c.N) * static_cast<uint32_t>(c.K) + q * 16;
        const uint32_t mine_x = (i16 < left ? i16 : left - 1) * static_cast<uint32_t>(c.K) + q * 16;
        auto weights = [&](int j) { return o.w[kSilu ? j / 2 : 0]; };
        auto tokens = [&](int h, int at) { return load16(o.x, mine_x, at + 64 * h); };
        i32x4 acc[4] = {};
        Stream8<4, kDeep> s;
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

// ---- tiles: bound by reading the weights, or with many rows by the matrix unit -----------
// One item: up to 256 token rows x 256 weight rows (kSilu: 128 gate rows and their 128
// up rows).  Four waves, one a SIMD, two by two: each has 128 weight rows (kSilu: 64 of
// either) and half of the token rows, in tiles of 32 x 32 (v_mfma_i32_32x32x32_i8).  Both
// operands come through two slots of 128 inputs in shared memory, loaded past the
// registers; the loads run on from an item to the next.
//
// Rows come in whole lines of 128 bytes (64 bytes of twice as many rows take a load
// twice as long: 38 against 19 cycles a KB and CU from the L2), so a slot takes 64 KB and
// there is room for two.  To have more on the way than one stage, a stage is worked off
// by weight tiles: a wave keeps its token tiles of all 128 inputs in registers, and in
// quarter q multiplies them with its weight tile q, while tile q + 1 is read and, in
// the last quarter, the next stage's token tiles.  So a slot's parts are free again
// one after the other, long before the stage ends, and are asked for anew 1.25 to 1.5
// stages before they are read.
//
// A row has eight places of 16 bytes in a slot; inputs 16 c .. + 15 of row r are at place
// c ^ (r / 2 % 8), so that any 16 neighbouring rows' places c lie in different banks.
// A lane holds row l % 32 of either operand, and inputs 32 u + 16 (l / 32) .. + 15 in step
// u of a stage's four.
//
// 256 experts with 128 rows on average, 7168 -> 2 x 2048 (7.9 GB): 1.45-1.51 ms, 5.2-5.4
// TB/s.  64 with 768, 4096 -> 2 x 1024: 420-450 us, 1.8-2.0 POP/s; half of its cycles are
// the matrix unit's, at the 1.5-1.7 GHz that the card's power leaves (a loop of products
// alone runs at 3.0-3.2 POP/s), and what nothing hides are the results (an exponential
// and a reciprocal each: 10 of some 100 thousand cycles an item).  Stages of 64 inputs in
// a ring of four: 506 us for it; 128-byte rows: 461; parts asked for by quarters: 429;
// with the last quarter's loads in the next stage's first, beside fewer reads: 411.

// 16 (or 4) bytes a lane past the registers to shared memory at byte `to` + 16 lane
// (+ 4 lane).  By hand: the compiler takes any later read of shared memory for one of
// what such a load writes, and waits for it.  Whoever reads the bytes waits by arrive().
// The compiler does not see which scalars a load by hand reads, and one that a vector
// instruction wrote (it may keep scalars in vector lanes) may be read five wait states
// later at the earliest: s_mov is one, s_nop 3 four.  (With two in all, which is enough only
// by the order that the compiler happens to choose, the two sizes above take 1 % and 0.3 %
// less: 1491 against 1507 us, 423 against 424.)
typedef uint32_t Words4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void load_past(uint32_t to, const Words4& from, uint32_t lane_offset, uint32_t offset) {
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(to), "v"(lane_offset), "s"(from), "s"(offset)
                 : "memory", "m0");
#endif
}
__device__ __forceinline__ void load_past4(uint32_t to, const Words4& from, uint32_t lane_offset) {
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(to), "v"(lane_offset), "s"(from)
                 : "memory", "m0");
#endif
}
// Where shared memory `p` lies in the block's.
template <typename T>
__device__ __forceinline__ uint32_t shared_at(T* p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) T*)p));
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v)));
}
__device__ __forceinline__ Words4 words(const void* p, int64_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const int64_t most = 0x7FFFFFFF;
    return Words4{uniform(static_cast<uint32_t>(a)), uniform(static_cast<uint32_t>(a >> 32) & 0xFFFFu),
                  uniform(static_cast<uint32_t>(bytes < most ? bytes : most)), 0x00020000u};
}

// The loads behind the newest kLater have arrived in every wave, and every wave is done
// with the shared memory it read.
template <int kLater>
__device__ __forceinline__ void arrive() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kLater) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The same in two steps: the wave's own loads, kMore more of them on the way where `more`;
// and the other waves, (kReads) when this one's reads are done.
template <int kLater, int kMore>
__device__ __forceinline__ void wait(bool more) {
    if (more) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLater + kMore) : "memory");
    else asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLater) : "memory");
}
template <bool kReads = true>
__device__ __forceinline__ void meet() {
    if (kReads) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

constexpr int kStage = 128;                                             // inputs of a stage
constexpr int kTokenPart = kTileWeights8 * kStage;                      // where a slot's token rows begin
constexpr int kSlot = (kTileWeights8 + kTileRows8) * kStage;            // bytes of a slot
constexpr int kLoads = kLoads8;

struct Item {
    int e, left, n0;                                // expert, token rows, first output
    int64_t row0;
};
// A block's items one after the other, by tile and column: `tiles` and `columns` on to
// the next one, without a division.
struct Walk {
    int64_t left;                                   // items, this one among them
    int tile, column;
    int tiles, columns, all;                        // step; columns of a tile
    __device__ __forceinline__ void on() {
        --left;
        tile += tiles;
        column += columns;
        if (column >= all) {
            column -= all;
            ++tile;
        }
    }
};
// An expert's rows go to its tiles in equal parts, of whole 64: four tiles of 192 rows
// end together, three of 256 and one of 10 do not.
__device__ __forceinline__ Item item_of(const Table& t, int E, const Walk& w, int outputs) {
    const int e = expert_of(t, E, w.tile), count = __builtin_amdgcn_readfirstlane(t.count[e]);
    const uint32_t tiles = (count - 1) / kTileRows8 + 1;
    const int rows = (static_cast<uint32_t>(count - 1) / tiles / 64 + 1) * 64;
    const int m0 = (w.tile - __builtin_amdgcn_readfirstlane(t.start[e])) * rows;
    return {e, count - m0 < rows ? count - m0 : rows, w.column * outputs,
            __builtin_amdgcn_readfirstlane(t.first[e]) + static_cast<int64_t>(m0)};
}

// The loading side of a wave: where it reads weight rows and token rows from.  Load i
// brings eight rows.  Of a stage's 16, 0 .. 7 bring token rows 64 wave .. + 63, and 8 + 2 q
// and 9 + 2 q a quarter of the rows of the waves' weight tiles q: rows 32 q + 16 (wave %
// 2) .. + 15 of half wave / 2 of the weight rows.  kSilu: of tiles 0 and 1 gate rows, of 2
// and 3 up rows.  Rows that are not there repeat the last one.
struct Fill {
    Words4 w[2], x;
    uint32_t at[kLoads];
    int stage;
};
// Output (of the item's) of row r of the weight rows, 32-row tile by tile.
template <bool kSilu>
__device__ __forceinline__ int output_of(int r) { return kSilu ? r / 128 * 64 + r % 64 : r; }
// The row in the slot's part that load i begins with.
__device__ __forceinline__ int first_row(int i, int wave) {
    return i < 8 ? wave * 64 + i * 8 : wave / 2 * 128 + (i - 8) / 2 * 32 + wave % 2 * 16 + i % 2 * 8;
}
template <bool kSilu>
__device__ __forceinline__ void aim(Fill& f, const Call& c, const Item& it, int wave) {
    int lane = lane_id();
    asm volatile("" : "+v"(lane));
    const int wide = c.N - it.n0 < kTileWeights8 ? c.N - it.n0 : kTileWeights8;
    const int64_t w0 = static_cast<int64_t>(it.e) * (kSilu ? 2 * c.N : c.N) + it.n0;
    f.w[0] = words(c.w + w0 * c.K, static_cast<int64_t>(wide) * c.K);
    f.w[1] = kSilu ? words(c.w + (w0 + c.N) * c.K, static_cast<int64_t>(wide) * c.K) : f.w[0];
    f.x = words(c.x + it.row0 * c.K, static_cast<int64_t>(it.left) * c.K);
    f.stage = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int slot_row = first_row(i, wave) + lane / 8, r = i < 8 ? slot_row : output_of<kSilu>(slot_row);
        const int most = i < 8 ? it.left : wide;
        const uint32_t place = (lane % 8 ^ (slot_row / 2 % 8)) * 16;
        f.at[i] = (r < most ? r : most - 1) * static_cast<uint32_t>(c.K) + place;
    }
}
// Load i of the stage, to the slot at byte `to`.
template <bool kSilu>
__device__ __forceinline__ void ask(const Fill& f, int i, uint32_t to, int wave) {
    load_past(to + (i < 8 ? kTokenPart : 0) + first_row(i, wave) * kStage, i < 8 ? f.x : f.w[kSilu && i >= 12 ? 1 : 0],
              f.at[i], f.stage * kStage);
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t two_bf16(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}

// One item of up to 64 kT token rows: its stages, of which the first lies in the slot at
// `here`, and its results.  stored: the stores of the item before.  advance() moves the
// loading side on by a stage.
template <bool kSilu, int kT, typename Advance>
__device__ __forceinline__ void tile_item(const Call& c, const Item& it, const Fill& f, Advance advance,
                                          const uint8_t* ring, uint32_t at_ring, const float* scales, uint32_t& here,
                                          int& stored, int wave) {
    // Worked out anew for each item from what the compiler may not see through, or it
    // keeps every offset of every size of tile in registers, and those in memory.
    int lane = lane_id();
    asm volatile("" : "+v"(lane));
    const int h = lane / 32, i32 = lane % 32, wy = wave / 2, wx = wave % 2;
    i32x16 acc[kT][4] = {};
    i32x4 a[2][4], b[4][kT];                        // [quarter % 2][step], [step][token tile]
    // Where the lane finds its inputs of step 0; those of step u are at this ^ 32 u.
    const uint32_t first = (h ^ (i32 >> 1 & 7)) * 16 + i32 * kStage;
    auto read_a = [&](int q, int u, uint32_t from) {
        a[q % 2][u] = *reinterpret_cast<const i32x4*>(ring + (first ^ (u * 32)) + from + (wy * 128 + q * 32) * kStage);
    };
    auto read_b = [&](int u, int i, uint32_t from) {
        b[u][i] = *reinterpret_cast<const i32x4*>(ring + (first ^ (u * 32)) + from + kTokenPart + (wx * kT + i) * 32 * kStage);
    };
    // Quarter q of the stage in the slot at `from` (the next one's at `next`): its
    // products, between them reads, and its loads into this slot or (quarter 0) the
    // next.  (In this order: left to itself the compiler reads an operand just before
    // its first product.)
    auto quarter = [&](int q, uint32_t from, uint32_t next) {
        const int ask0 = i8_quarter(q).from, ask1 = i8_quarter(q).to;
#pragma unroll
        for (int m = 0; m < 4 * kT; ++m) {
            const int u = m / kT, i = m % kT;
            acc[i][q] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[q % 2][u], b[u][i], acc[i][q], 0, 0, 0);
            if (m < 4) read_a((q + 1) % 4, m, q < 3 ? from : next);
            if (q == 3) {                           // the tiles of step u have met their last product
                if (i == kT - 1) {
#pragma unroll
                    for (int t = 0; t < kT; ++t) read_b(u, t, next);
                }
            }
            // One every second product (of 16, behind the four that have reads beside
            // them), or where there are few in turn.
#pragma unroll
            for (int g = ask0; g < ask1; ++g)
                if ((kT > 3 ? (g - ask0) * 2 + 4 : kT > 2 ? (g - ask0) * 2 : (g - ask0) % (4 * kT)) == m)
                    ask<kSilu>(f, g, at_ring + (q == 0 ? next : from), wave);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        read_a(0, u, here);
#pragma unroll
        for (int t = 0; t < kT; ++t) read_b(u, t, here);
    }
    // Behind quarter 3 nobody waits for its own reads of shared memory: what they read is
    // asked for anew behind quarter 0 at the earliest.  kMore: the last item's stores, if
    // there were as many as this one makes, and this one's two loads of scales.
    constexpr int kStores = (kSilu ? 4 : 8) * kT, kMore = kStores + 2;
    const int stages = c.K / kStage;
    bool early = stored == kStores;
    for (int s = 0; s < stages; ++s, early = false) {
        const uint32_t next = here ^ kSlot;
        quarter(0, here, next);
        advance();
        wait<i8_quarter(0).later, kMore>(early);
        meet();
        quarter(1, here, next);
        wait<i8_quarter(1).later, kMore>(early);
        meet();
        quarter(2, here, next);
        wait<i8_quarter(2).later, kMore>(early);
        meet();
        quarter(3, here, next);
        wait<i8_quarter(3).later, kMore>(early);
        meet<false>();
        here = next;
    }
    stored = kStores;
    // The scales are in: the loads of a stage at least came after them.
    arrive<kLoads>();

    // A lane holds outputs 8 p + 4 h .. + 3 (p = 0 .. 3) of token row i32 of each 32 x 32
    // tile.  Halves of the wave exchange what they have of p and p + 1, so that each
    // stores 16 bytes.  What is not there goes past the buffer's end, where nothing is
    // stored, so that every wave makes the same number of stores.
    const int outs = c.N - it.n0;
    int n_row = c.N;
    asm volatile("" : "+s"(n_row));
    const Buffer y = buffer(c.y + it.row0 * c.N + it.n0, ((it.left - 1) * static_cast<int64_t>(c.N) + outs) * 2);
    float xs[kT];
#pragma unroll
    for (int i = 0; i < kT; ++i) xs[i] = scales[kTileWeights8 + (wx * kT + i) * 32 + i32];
#pragma unroll
    for (int j = 0; j < (kSilu ? 2 : 4); ++j)
#pragma unroll
        for (int p = 0; p < 4; p += 2) {
            constexpr int kSides = kSilu ? 2 : 1;   // gate and up
            f32x4 ws[kSides][2];
#pragma unroll
            for (int g = 0; g < kSides; ++g)
#pragma unroll
                for (int d = 0; d < 2; ++d) ws[g][d] = scales4(scales, wy * 128 + (j + 2 * g) * 32 + 8 * (p + d) + 4 * h);
            const int n = wy * (kSilu ? 64 : 128) + j * 32 + 8 * (p + h);
#pragma unroll
            for (int i = 0; i < kT; ++i) {
                u32x2 two[2];
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    auto value = [&](int g) {
                        const i32x16& v = acc[i][j + 2 * g];
                        return scaled(i32x4{v[4 * (p + d)], v[4 * (p + d) + 1], v[4 * (p + d) + 2], v[4 * (p + d) + 3]},
                                      xs[i], ws[g][d]);
                    };
                    f32x4 v = value(0);
                    if constexpr (kSilu) v = silu_mul(v, value(1));
                    two[d] = u32x2{two_bf16(v[0], v[1]), two_bf16(v[2], v[3])};
                }
                const u32x2 lo = __builtin_amdgcn_permlane32_swap(two[0][0], two[1][0], false, false);
                const u32x2 hi = __builtin_amdgcn_permlane32_swap(two[0][1], two[1][1], false, false);
                const int m = (wx * kT + i) * 32 + i32;
                const uint32_t to = m < it.left && n < outs ? (m * static_cast<uint32_t>(n_row) + n) * 2 : 1u << 31;
                __builtin_amdgcn_raw_buffer_store_b128(u32x4{lo[0], hi[0], lo[1], hi[1]}, y, to, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
}

template <bool kSilu>
__global__ __launch_bounds__(kThreads, 1) void tile_i8_kernel(Call c) {
    constexpr int kOut = kSilu ? kTileWeights8 / 2 : kTileWeights8;
    __shared__ __align__(1024) uint8_t ring[2 * kSlot];
    // Of an item's weight rows and token rows; the next item's come to the other.
    __shared__ __align__(16) float scales[2][kTileWeights8 + kTileRows8];
    extern __shared__ int32_t room[];
    const Table t = make_table(room, c.expert_rows, c.E, c.capacity, c.num_rows, kTileRows8, 0, INT32_MAX);
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave), lane = lane_id();
    const int columns = (c.N + kOut - 1) / kOut, stages = c.K / kStage;
    const Share mine = share_of(static_cast<int64_t>(t.start[c.E]) * columns);
    if (mine.at >= mine.end) return;
    const uint32_t at_ring = shared_at(ring);
    const int step = static_cast<int>(mine.step), first = static_cast<int>(mine.at / columns);
    Walk walk = {(mine.end - mine.at - 1) / mine.step + 1, first,
                 static_cast<int>(mine.at - static_cast<int64_t>(first) * columns), step / columns, step % columns, columns};

    Fill f;
    Walk filling = walk;
    aim<kSilu>(f, c, item_of(t, c.E, filling, kOut), wave);
    // Behind the last item its last stage is asked for again.
    auto advance = [&] {
        if (++f.stage < stages) return;
        if (filling.left > 1) {
            filling.on();
            aim<kSilu>(f, c, item_of(t, c.E, filling, kOut), wave);
        } else {
            f.stage = stages - 1;
        }
    };
    // Of the second stage all but what its first quarter asks for.
    constexpr int kRest = i8_quarter(0).from;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) ask<kSilu>(f, i, at_ring, wave);
    advance();
#pragma unroll
    for (int i = 0; i < kRest; ++i) ask<kSilu>(f, i, at_ring + kSlot, wave);
    arrive<kRest>();
    uint32_t here = 0;
    int odd = 0, stored = 0;                        // stores of the last item
    for (; walk.left > 0; walk.on(), odd ^= 1) {
        const Item it = item_of(t, c.E, walk, kOut);
        const int wide = c.N - it.n0 < kTileWeights8 ? c.N - it.n0 : kTileWeights8;
        // Scales in the order of the slot's rows.
        const int64_t w0 = static_cast<int64_t>(it.e) * (kSilu ? 2 * c.N : c.N) + it.n0 + (kSilu && wave % 2 == 1 ? c.N : 0);
        const int n = output_of<kSilu>(wave * 64 + lane), m = wave * 64 + lane;
        const uint32_t to = shared_at(scales[odd]) + wave * 256;
        load_past4(to, words(c.w_scales + w0, static_cast<int64_t>(wide) * 4), (n < wide ? n : wide - 1) * 4);
        load_past4(to + kTileWeights8 * 4, words(c.x_scales + it.row0, static_cast<int64_t>(it.left) * 4),
                   (m < it.left ? m : it.left - 1) * 4);
        // Products of rows that are not there would cost what the others do.
        if (it.left > 192) tile_item<kSilu, 4>(c, it, f, advance, ring, at_ring, scales[odd], here, stored, wave);
        else if (it.left > 128) tile_item<kSilu, 3>(c, it, f, advance, ring, at_ring, scales[odd], here, stored, wave);
        else if (it.left > 64) tile_item<kSilu, 2>(c, it, f, advance, ring, at_ring, scales[odd], here, stored, wave);
        else tile_item<kSilu, 1>(c, it, f, advance, ring, at_ring, scales[odd], here, stored, wave);
    }
    arrive<0>();                                    // no load may write shared memory after the block's end
}

// Row tiles of `rows` that a map in order can ask for at most.
int64_t most_tiles(const Call& c, int rows) { return c.num_rows / rows + (c.num_rows < c.E ? c.num_rows : c.E); }

template <bool kSilu>
hipError_t launch(const Call& c, hipStream_t stream) {
    const bool streams = i8_streams(c.num_rows, c.E, c.K, c.N, kSilu);
    const int64_t items = streams ? most_tiles(c, 16) * ceil_div(c.N, kSilu ? 32 : 64)
                                  : most_tiles(c, kTileRows8) * ceil_div(c.N, kSilu ? kTileWeights8 / 2 : kTileWeights8);
    hipLaunchKernelGGL(streams ? stream_i8_kernel<kSilu> : tile_i8_kernel<kSilu>,
                       dim3(blocks_for(items, streams ? 256 * 2 : 256)), dim3(kThreads), table_bytes(c.E), stream, c);
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
