// expert_w4.hip -- ep_expert_linear_w4 on gfx950.
//
// y[r] = x[r] . W[e(r)]^T over the rows of each expert, W in E2M1 codes with
// one E8M0 scale per 32 inputs.  A code times its scale is exact in bf16, so the
// only roundings are the fp32 accumulation and the final one to bf16.
//
// The order of the contraction is free as long as both operands agree, so a
// lane takes 16 consecutive bytes of its weight row: 32 inputs, exactly one
// scale group.  Streams (few rows) contract 32 inputs of 16 weight rows against 16
// token rows at a time (v_mfma_f32_16x16x32_bf16): the four lane groups of a wave
// (lane / 16) hold the four scale groups of a 128-input block, and step s of four
// contracts inputs 32 q + 8 s .. + 7 of every group q.  Tiles (many rows) take 16
// inputs of 32 rows against 32 (v_mfma_f32_32x32x16_bf16), as written there.
#include "expert_rows.h"
#include "moe_launch.h"
#include "w4_plan.h"

namespace ep {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;
constexpr int kTileThreads = 512;

// Eight codes of one word, times the scale 2^(b - 127) whose bits are b << 23.
__device__ __forceinline__ bf16x8 decode(uint32_t codes, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// What an item's waves read: weight rows from n0 on (wb[1]: the up rows that
// belong to them) and token rows from row0 on.
struct Operands {
    int64_t row0;
    int n0, left;                                   // first output, token rows left
    Buffer wb[2], sb[2], xb;
};
template <bool kSilu>
__device__ __forceinline__ Operands operands(const uint16_t* x, const uint8_t* codes, const uint8_t* scales, int e,
                                             int64_t row0, int left, int n0, int K, int N) {
    const int64_t w0 = static_cast<int64_t>(e) * (kSilu ? 2 * N : N) + n0, up = kSilu ? N : 0;
    const int64_t wide = N - n0 < 512 ? N - n0 : 512, deep = left < 128 ? left : 128;
    return {row0, n0, left,
            {buffer(codes + w0 * (K / 2), wide * (K / 2)), buffer(codes + (w0 + up) * (K / 2), wide * (K / 2))},
            {buffer(scales + w0 * (K / 32), wide * (K / 32)), buffer(scales + (w0 + up) * (K / 32), wide * (K / 32))},
            buffer(x + row0 * K, deep * K * 2)};
}
// Offset of weight row n (of an item's) for a lane of group q.  Rows past the
// outputs repeat the last one; what they give is not stored.
__device__ __forceinline__ uint32_t code_offset(const Operands& o, int n, int N, int K, int q) {
    return __umul24(o.n0 + n < N ? n : N - 1 - o.n0, K / 2) + q * 16;
}

// ---- few rows per expert: bound by reading the weights ---------------------------
// A wave takes 64 weight rows (kSilu: 32 gate rows and their 32 up rows) and up
// to 16 token rows, 256 inputs at a time: whole 128-byte lines of the codes (64
// bytes of twice as many rows is a fifth slower from HBM).  Where there are items
// for every wave, each takes whole items; where there are not (a single token's
// eight experts), the four waves of a block split an item's inputs, so that every
// CU has loads in flight, and join their sums in shared memory in wave order.  No
// codes or token rows are staged: the four waves of a block read the same token
// rows, which the L1 holds, and never wait for each other.
//
// The scales are a sixteenth of the codes' bytes, but 8 bytes of every row a step:
// lines that the codes have driven out of the L1 by the next step.  An item's
// scale rows lie together in memory, so they come into shared memory once, in
// whole loads, where K <= kSharedScales; else each step loads eight of a row
// (K % 256 == 0) or single ones.  (128 experts of one row, 7168 -> 2 x 2048, 2.0
// GB: 345 us, 5.8 TB/s, against 432 with eight a load; 256 experts of 4 rows, 2048
// -> 7168, 2.0 GB: 406 against 446; 60 experts of 2 rows, 5760 -> 2 x 1440: 113
// against 150 with single ones.)

// 16-byte places of an item's block of scale rows, in whole loads of 64.
template <bool kSilu>
__device__ __forceinline__ int scale_slots(int K) {
    return ((kSilu ? 32 : 64) * K / 512 + 63) / 64 * 64;
}

// Register s of the lanes of group q (lane / 16) and register q of group s change
// places: halves of the wave first, then neighbouring groups.
__device__ __forceinline__ void transpose_groups(u32x4 (&v)[4]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const u32x2 a = __builtin_amdgcn_permlane32_swap(v[0][c], v[2][c], false, false);
        const u32x2 b = __builtin_amdgcn_permlane32_swap(v[1][c], v[3][c], false, false);
        const u32x2 even = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
        const u32x2 odd = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
        v[0][c] = even[0];
        v[1][c] = even[1];
        v[2][c] = odd[0];
        v[3][c] = odd[1];
    }
}

// acc += the products over inputs k, k + step, ...  kShared: scale_rows has the
// item's, and is being filled: `join` are the waves that fill it together.
template <bool kSilu, Scales kScales>
__device__ __forceinline__ void stream_products(const Operands& o, int k, int step, int K, int N, int q, int i16,
                                                const uint8_t* scale_rows, bool join, f32x4* acc) {
    uint32_t cr[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) cr[j] = code_offset(o, (kSilu ? j % 2 : j) * 16 + i16, N, K, q);
    const uint32_t xr = __umul24(i16 < o.left ? i16 : o.left - 1, K * 2) + q * 16;
    u32x4 w[2][2][4], v[2][4];                      // [buffer][half][weight tile], [half][..]
    u32x2 b[2][4];
    // Every load below is made on every way through the loop, past the end
    // again from the last block: a branch around a load makes the compiler wait
    // for all that is on the way.
    auto load = [&](int buf, int at) {
        at = at < K ? at : K - 128;
        if (kScales == kEight && at + 128 >= K) at = K - 256;
        const int more = kScales == kEight || at + 128 < K ? 128 : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const Buffer wb = o.wb[kSilu ? j / 2 : 0], sb = o.sb[kSilu ? j / 2 : 0];
            w[buf][0][j] = load16(wb, cr[j], at / 2);
            w[buf][1][j] = load16(wb, cr[j], (at + more) / 2);
            if (kScales == kEight) {
                // A row's scales of this step start where group 0's lane has its own.
                b[buf][j] = load8(sb, cr[j] / 16 - q, at / 32);
            } else if (kScales == kSingle) {
                b[buf][j][0] = load1(sb, cr[j] / 16, at / 32);
                b[buf][j][1] = load1(sb, cr[j] / 16, (at + more) / 32);
            }
        }
    };
    // Load s brings group q inputs 32 s + 8 q .. + 7: 64 bytes in a row of each
    // token row (the inputs 32 q + 8 s .. that step s needs lie 64 bytes apart, and
    // four times the cache lookups made these loads cost what the weights do).
    auto rows = [&](int h, int at) {
        at = at < K ? at : K - 128;
#pragma unroll
        for (int s = 0; s < 4; ++s) v[h][s] = load16(o.xb, xr, (at + 32 * s) * 2);
    };
    auto multiply = [&](int buf, int h) {
        transpose_groups(v[h]);
        float scale[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            scale[j] = __uint_as_float((kScales != kSingle ? b[buf][j][h] >> 8 * q & 0xFF : b[buf][j][h]) << 23);
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode(w[buf][h][j][s], scale[j]),
                                                                 __builtin_bit_cast(bf16x8, v[h][s]), acc[j], 0, 0, 0);
    };
    // Loads return in order: the token rows of a half step are asked for before
    // what may stay on the way while they are waited for.
    auto pass = [&](int buf, int at) {
        if (kScales == kShared) {
            const int here = at < K ? at : 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int up = kSilu && j >= 2 ? scale_slots<kSilu>(K) * 16 : 0;
                const int n = (kSilu ? j % 2 : j) * 16 + i16;
                const uint32_t* four = reinterpret_cast<const uint32_t*>(scale_rows + up + n * (K / 32) + here / 32);
                b[buf][j] = u32x2{four[0], four[1]};    // the second four past the inputs' end are not used
            }
        }
        if (at < K) multiply(buf, 0);
        __builtin_amdgcn_sched_barrier(0);
        rows(0, at + step);
        __builtin_amdgcn_sched_barrier(0);
        if (at + 128 < K) multiply(buf, 1);
        __builtin_amdgcn_sched_barrier(0);
        rows(1, at + step + 128);
        __builtin_amdgcn_sched_barrier(0);
        load(buf, at + 2 * step);
        __builtin_amdgcn_sched_barrier(0);
    };
    load(0, k);
    __builtin_amdgcn_sched_barrier(0);
    rows(0, k);
    rows(1, k + 128);
    __builtin_amdgcn_sched_barrier(0);
    load(1, k + step);
    __builtin_amdgcn_sched_barrier(0);
    if (kScales == kShared) {
        // Behind the scales: two times eight codes and two times four rows.
        asm volatile("s_waitcnt vmcnt(24)" ::: "memory");
        if (join) __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    }
    for (; k < K; k += 2 * step) {
        pass(0, k);
        pass(1, k + step);
    }
}

template <bool kSilu, Scales kScales>
__global__ __launch_bounds__(kThreads, 2) void stream_w4_kernel(
    const uint16_t* __restrict__ x, int64_t num_rows, const int32_t* __restrict__ expert_rows, int capacity,
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int E, int K, int N, int most,
    uint16_t* __restrict__ y) {
    constexpr int kOut = kSilu ? 32 : 64;           // outputs of an item
    constexpr int kRoom = 64 * kSharedScales / 32 / 16;
    __shared__ u32x4 scale_room[kScales == kShared ? 4 : 1][kScales == kShared ? kRoom : 1];     // a wave's
    __shared__ f32x4 part_room[kScales == kShared ? 1 : 16][kWave];
    extern __shared__ int32_t room[];
    const int lane = lane_id(), q = lane / 16, i16 = lane % 16;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const Table t = make_table(room, expert_rows, E, capacity, num_rows, 16, 0, most);
    const int columns = (N + kOut - 1) / kOut;
    const int64_t items = static_cast<int64_t>(t.start[E]) * columns;
    // Whole items from 1.25 a block on: 8 experts (7168 -> 2 x 2048, 1 item a block)
    // split 31 us, whole 40; 24 of 64 (4096 -> 2 x 1024, 1.5) 29.5 both; 8 experts
    // (2048 -> 7168, 1.75) 23 and 17; 16 (7168 -> 2 x 2048, 2) 58 and 48.
    const bool split = 4 * items < 5 * static_cast<int64_t>(gridDim.x);
    // Split items have their scales in the first wave's room, the sums of the
    // waves (16 weight tiles x lanes) in the second's.
    static_assert(sizeof(f32x4) * 16 * kWave <= sizeof(u32x4) * kRoom, "room for the sums");
    f32x4(*part)[kWave] = kScales == kShared ? reinterpret_cast<f32x4(*)[kWave]>(scale_room[kScales == kShared ? 1 : 0])
                                             : part_room;
    u32x4* mine_scales = scale_room[kScales == kShared && !split ? wave : 0];
    Share mine = share_of(items);
    if (!split) {                                   // neighbouring items to the waves of a block
        mine.at += blockIdx.x / 8 * 3 + wave;
        mine.step *= 4;
    }
    for (int64_t item = mine.at; item < mine.end; item += mine.step) {
        const int tile = static_cast<int>(item / columns);
        const int column = static_cast<int>(item - static_cast<int64_t>(tile) * columns);
        const int e = expert_of(t, E, tile);
        const int m0 = (tile - t.start[e]) * 16;
        const int left = __builtin_amdgcn_readfirstlane(t.count[e] - m0);
        const int64_t row0 = __builtin_amdgcn_readfirstlane(t.first[e]) + static_cast<int64_t>(m0);
        const Operands o = operands<kSilu>(x, codes, scales, e, row0, left, column * kOut, K, N);
        if (kScales == kShared) {
            // Scale rows of K / 32 bytes, one after the other in memory as here:
            // one block of 64 rows, or two of 32 (kSilu), of whole pieces of 16
            // bytes (K % 128 == 0, N % 8 == 0).  Past a block's or the outputs'
            // last row its last bytes again.  (The wave's, or
            // behind the barriers below the block's, reads of the item before
            // are done.)
            const int slots = scale_slots<kSilu>(K), last = (N - o.n0 < kOut ? N - o.n0 : kOut) * (K / 128) / 4 - 1;
            for (int g = split ? wave : 0; g * 64 < slots * (kSilu ? 2 : 1); g += split ? 4 : 1) {
                const bool up = kSilu && g * 64 >= slots;
                const int at = g * 64 + lane - (up ? slots : 0);
                load_shared(mine_scales + g * 64, o.sb[up ? 1 : 0], (at < last ? at : last) * 16, 0);
            }
        }
        f32x4 acc[4] = {};
        stream_products<kSilu, kScales>(o, split ? wave * 256 : 0, split ? 1024 : 256, K, N, q, i16,
                                        reinterpret_cast<const uint8_t*>(mine_scales), split, acc);

        // A lane holds outputs 4 q .. + 3 of token row i16 of each 16 x 16 tile; of
        // split items wave w ends up with weight tile w (kSilu: waves 0 and 1
        // with the gate's and the up rows').
        uint16_t* row = y + (row0 + i16) * N;
        if (split) {
#pragma unroll
            for (int j = 0; j < 4; ++j) part[wave * 4 + j][lane] = acc[j];
            __syncthreads();
            auto sum = [&](int j) {
                return (part[j][lane] + part[4 + j][lane]) + (part[8 + j][lane] + part[12 + j][lane]);
            };
            const int n = o.n0 + wave * 16 + 4 * q;
            if (wave * 16 < kOut && i16 < left && n < N) {
                f32x4 u = sum(wave);
                if (kSilu) {
                    const f32x4 up = sum(wave + 2);
#pragma unroll
                    for (int c = 0; c < 4; ++c) u[c] = silu(u[c]) * up[c];
                }
                store4(row + n, u);
            }
            __syncthreads();
        } else if (i16 < left) {
#pragma unroll
            for (int j = 0; j < kOut / 16; ++j) {
                const int n = o.n0 + j * 16 + 4 * q;
                f32x4 u = acc[j];
                if (kSilu) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) u[c] = silu(u[c]) * acc[j + 2][c];
                }
                if (n < N) store4(row + n, u);
            }
        }
    }
}

// ---- many rows per expert: bound by the matrix unit ------------------------------
// One item: 32 kTiles token rows x 512 weight rows (kSilu: 256 gate rows and
// their 256 up rows), 64 of them to each of the block's eight waves, so that no code
// is decoded twice.  The token rows of a 128-input step come through shared memory
// (four buffers, loaded past the registers, asked for three steps ahead); the codes
// go straight into the registers of the wave that decodes them, asked for a step
// ahead or, with up to 96 rows, two steps' at a time.

// Products are 32 x 32 here (v_mfma_f32_32x32x16_bf16): per operation they read
// half the operand registers of the 16 x 16 form, and at these sizes the card's
// power bounds the clock.  A lane holds row lane % 32 of either operand; its half
// h = lane / 32 holds 8 of the 16 inputs.  Two loads bring a lane the codes of
// groups h and 2 + h of a 128-input step; step (u, s) of eight contracts inputs
// 32 (2 u + h) + 8 s .. + 7.

// The loads behind the newest kLater have arrived in every wave, and every wave
// is done with the shared memory it read.
template <int kLater>
__device__ __forceinline__ void arrive() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kLater) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The 16-byte place in a 256-byte row that holds inputs 8 c .. + 7 of row r.
// Shared memory serves 16 lanes at a time, of 16 different rows mod 16.
__device__ __forceinline__ int place_of(int r, int c) { return c ^ (r & 15); }

// arrive<later>() for the counts of tile_step.
template <int kTiles>
__device__ __forceinline__ void arrive_but(int later) {
    if (later == 0) arrive<0>();
    else if (later == kTiles) arrive<kTiles>();
    else if (later == 6) arrive<6>();
    else if (later == kTiles + 6) arrive<kTiles + 6>();
    else if (later == kTiles + 8) arrive<kTiles + 8>();
    else arrive<kTiles + 10>();
}

// One item: up to 32 kTiles token rows.
template <bool kSilu, int kTiles>
__device__ __forceinline__ void tile_item(const Operands& o, int K, int N, uint16_t* __restrict__ y, u32x4* s0,
                                          u32x4* s1, u32x4* s2, u32x4* s3) {
    constexpr int kFill = kTiles;                   // loads of four rows a wave
    const int lane = lane_id(), h = lane / 32, i32 = lane % 32;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    uint32_t cr[2], fill[kFill];
#pragma unroll
    for (int j = 0; j < 2; ++j)
        cr[j] = code_offset(o, kSilu ? wave * 32 + i32 : wave * 64 + j * 32 + i32, N, K, h);
    // This wave fills rows 4 kFill wave .. on, four to a load: lane l writes
    // place l % 16 of row l / 16, so it reads the inputs that belong there.
#pragma unroll
    for (int i = 0; i < kFill; ++i) {
        const int r = (wave * kFill + i) * 4 + lane / 16;
        fill[i] = __umul24(r < o.left ? r : o.left - 1, K * 2) + place_of(r, lane % 16) * 16;
    }
    // With few token rows the loads of the weights are the bound: a line of 128
    // bytes is asked for at once, that is two steps' codes of a weight row, two and
    // three steps ahead (a load for each step finds half of them gone from the L1), and
    // the scales of four steps in one load.  256 experts of 32 rows, 7168 -> 2 x
    // 2048, 4.0 GB: 888 us; a step's codes and scales one step ahead 1310; whole
    // lines, their loads spread over the step 1092; whole lines and single steps'
    // scales 1077.  64 experts of 24 rows, 4096 -> 2 x 1024: 75, 98, 87, 87.
    // (Full tiles are bound by the matrix unit, and have no registers left.)
    constexpr bool kLines = kTiles < 4;
    constexpr int kBuffers = kLines ? 4 : 2;
    u32x4 w[kBuffers][2][2];                    // [buffer][weight tile][u]
    u32x4 b[2], later[2];                       // kLines: the scales of four steps, and the next four's
    uint32_t b1[2][2];                          // else of one: [buffer][weight tile]
    // Past the end the last step is asked for again.
    auto within = [&](int kb) { return kb < K ? kb : K - 128; };
    auto one_scale = [&](int j, int kb) { return load4(o.sb[kSilu ? j : 0], cr[j] / 16 - h, kb / 32); };
    // Four steps' from kb on.  Where a row has fewer left, its last four (past the
    // end of the last row nothing may be read), which from_last moves into place.
    auto four_scales = [&](int j, int kb) {
        return load16(o.sb[kSilu ? j : 0], cr[j] / 16 - h, (kb <= K - 512 ? kb : K - 512) / 32);
    };
    auto from_last = [&](u32x4 v, int kb) {
        const int by = (kb - (K - 512)) / 128;
        const bool one = by > 0 && by & 1, two = by > 0 && by & 2;
        v = u32x4{one ? v[1] : v[0], one ? v[2] : v[1], one ? v[3] : v[2], v[3]};
        return u32x4{two ? v[2] : v[0], two ? v[3] : v[1], v[2], v[3]};
    };
    // Load number g of the six of a step's weights.
    auto ask_weights = [&](int g, int buf, int kb) {
        const int j = g / 3, u = g % 3;
        if (u == 2) b1[buf][j] = one_scale(j, kb);
        else w[buf][j][u] = load16(o.wb[kSilu ? j : 0], cr[j], kb / 2 + 32 * u);
    };
    // The loads of a weight tile's codes for the steps at kb and, of four, kb + 128.
    auto ask_lines = [&](int j, int buf, int kb, int loads) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
            if (g < loads)
                w[(buf + g / 2) % kBuffers][j][g % 2] =
                    load16(o.wb[kSilu ? j : 0], cr[j], within(kb + g / 2 * 128) / 2 + 32 * (g % 2));
    };
    // Load number g of a step's token rows.
    auto ask_rows = [&](int g, u32x4* to, int kb) {
        load_shared(to + (wave * kFill + g) * 64, o.xb, fill[g], kb * 2);
    };
    // Waves past the last output bring token rows only.
    const bool idle = o.n0 + wave * (kSilu ? 32 : 64) >= N;
    f32x16 acc[kTiles][2] = {};
    // Registers for the inputs of two groups of products where there are enough.
    constexpr int kReads = kTiles <= 2 ? 2 : 1;
    bf16x8 v[kReads][kTiles], a[2];
    auto read = [&](const u32x4* from, int first, int i, int us) {
        v[us % kReads][i] = __builtin_bit_cast(bf16x8, from[i * 512 + (first ^ ((us & 4) * 2 + us % 4))]);
    };
    auto decode_tile = [&](int buf, int j, int us) {
        const uint32_t scale = ((kLines ? b[j][buf] : b1[buf % 2][j]) >> (8 * h + 16 * (us / 4)) & 0xFF) << 23;
        return decode(w[buf][j][us / 4][us % 4], __uint_as_float(scale));
    };
    // The products of the step at kb, in 16 groups.  Between the groups its
    // loads are asked for, one at a time (all at once they hold up the
    // wave's products): first the weights of the next step (kLines: at every
    // other step a weight tile's codes of the second and third next together),
    // and in the second half the token rows of the third next.  The barrier in
    // the middle says that the next step's rows, asked for two steps ago, are in
    // (behind them are at most one step's rows and weights: the vmcnt), and
    // that every wave is past the step before, whose rows are overwritten.
    // By these counts no wave would wait for what it needs two steps later; but
    // the compiler takes a read of any of the four buffers for one of what the
    // loads past the registers are still writing, and puts waits of its own before
    // reads: for the rows asked for half a step ago in full tiles, and for all of the
    // codes asked for a step ago in the others.  (They are not needed: the barrier
    // is the wait.)  Each weight tile is decoded
    // beside the products of the one before; the next inputs of a row tile
    // are read when its last product is under way.  The barriers to
    // scheduling keep all that in place.  rest: 0 in the loop, 1 .. 3 the steps
    // after it; the loads and counts of each are tile_step's.
    auto multiply = [&](const u32x4* from, const u32x4* then, u32x4* to, int buf, int rest, int kb) {
        const TileStep step = tile_step(kTiles, buf, rest);     // constants where this is called
        if (idle) {
            arrive_but<kTiles>(step.idle_later);
#pragma unroll
            for (int g = 0; g < kFill; ++g)
                if (g < step.fills) ask_rows(g, to, within(kb + 384));
            return;
        }
        // Place 4 h of row i32, from which the others differ by an exclusive or:
        // worked out anew from one register, which the compiler may not see
        // through, or it keeps one for every place.
        int first = i32 * 16 + place_of(i32, 4 * h);
        asm("" : "+v"(first));
#pragma unroll
        for (int us = 0; us < 8; ++us)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int group = us * 2 + j;
                __builtin_amdgcn_sched_barrier(0);
                if (!kLines && group < step.weights) ask_weights(group, 1 - buf, within(kb + 128));
                // Of two weight tiles, before the barrier or behind it.
                if (kLines && step.weights >= 4 && (group == (step.late ? 9 : 0) || group == (step.late ? 13 : 4)))
                    ask_lines(group % 8 / 4, (buf + 2) % kBuffers, kb + 256, step.weights / 2);
                if (kLines && step.weights == 2 && group < 2) later[group] = four_scales(group, kb + 128);
                if (group == 8) arrive_but<kTiles>(step.later);
                if (group > 8 && group - 9 < step.fills) ask_rows(group - 9, to, within(kb + 384));
                __builtin_amdgcn_sched_barrier(0);
                if (j == 0) a[1] = decode_tile(buf, 1, us);
                else if (us < 7) a[0] = decode_tile(buf, 0, us + 1);
                else {
                    if (kLines && step.weights == 2) {
                        b[0] = from_last(later[0], kb + 128);
                        b[1] = from_last(later[1], kb + 128);
                    }
                    a[0] = decode_tile((buf + 1) % kBuffers, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[j], v[us % kReads][i], acc[i][j], 0, 0, 0);
                    if (j == 1) {
                        if (us + kReads < 8) read(from, first, i, us + kReads);
                        else read(then, first, i, us + kReads - 8);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
    };
    static_assert(kFill <= 7, "rows are asked for in the last seven groups");
    arrive<0>();                                // the last item's loads and reads are done
    if (!idle) {
        if (kLines) {
            ask_lines(0, 0, 0, 4);
            ask_lines(1, 0, 0, 4);
            b[0] = four_scales(0, 0);
            b[1] = four_scales(1, 0);
        } else {
#pragma unroll
            for (int g = 0; g < 6; ++g) ask_weights(g, 0, 0);
        }
    }
#pragma unroll
    for (int g = 0; g < kFill; ++g) ask_rows(g, s0, 0);
#pragma unroll
    for (int g = 0; g < kFill; ++g) ask_rows(g, s1, within(128));
#pragma unroll
    for (int g = 0; g < kFill; ++g) ask_rows(g, s2, within(256));
    arrive<2 * kFill>();
    if (!idle) {
        a[0] = decode_tile(0, 0, 0);
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
            for (int us = 0; us < kReads; ++us) read(s0, i32 * 16 + place_of(i32, 4 * h), i, us);
    }
    int kb = 0;
    for (; kb + 512 <= K; kb += 512) {
        multiply(s0, s1, s3, 0, 0, kb);
        multiply(s1, s2, s0, 1, 0, kb + 128);
        multiply(s2, s3, s1, 2 % kBuffers, 0, kb + 256);
        multiply(s3, s0, s2, 3 % kBuffers, 0, kb + 384);
    }
    if (kb < K) multiply(s0, s1, s3, 0, 1, kb);
    if (kb + 128 < K) multiply(s1, s2, s0, 1, 2, kb + 128);
    if (kb + 256 < K) multiply(s2, s3, s1, 2 % kBuffers, 3, kb + 256);

    // A lane holds outputs 8 p + 4 h .. + 3 (p = 0 .. 3) of token row i32 of
    // each 32 x 32 tile.
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
        const int m = i * 32 + i32;
        if (m >= o.left) break;
        uint16_t* row = y + (o.row0 + m) * N;
#pragma unroll
        for (int j = 0; j < (kSilu ? 1 : 2); ++j)
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int n = o.n0 + wave * (kSilu ? 32 : 64) + j * 32 + 8 * p + 4 * h;
                f32x4 v;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    v[c] = acc[i][j][4 * p + c];
                    if (kSilu) v[c] = silu(v[c]) * acc[i][1][4 * p + c];
                }
                if (n < N) store4(row + n, v);
            }
    }
}

template <bool kSilu>
__global__ __launch_bounds__(kTileThreads, 2) void tile_w4_kernel(
    const uint16_t* __restrict__ x, int64_t num_rows, const int32_t* __restrict__ expert_rows, int capacity,
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int E, int K, int N, int above,
    int tile_rows, uint16_t* __restrict__ y) {
    constexpr int kOut = kSilu ? kTileWeights / 2 : kTileWeights;
    __shared__ u32x4 s0[kTileRows * 16], s1[kTileRows * 16], s2[kTileRows * 16], s3[kTileRows * 16];
    extern __shared__ int32_t room[];
    const Table t = make_table(room, expert_rows, E, capacity, num_rows, tile_rows, above, INT32_MAX);
    const int columns = (N + kOut - 1) / kOut;
    const Share mine = share_of(static_cast<int64_t>(t.start[E]) * columns);
    for (int64_t item = mine.at; item < mine.end; item += mine.step) {
        const int tile = static_cast<int>(item / columns);
        const int e = expert_of(t, E, tile);
        const int m0 = (tile - t.start[e]) * tile_rows, rest = t.count[e] - m0;
        const int left = __builtin_amdgcn_readfirstlane(rest < tile_rows ? rest : tile_rows);
        const int64_t row0 = __builtin_amdgcn_readfirstlane(t.first[e]) + static_cast<int64_t>(m0);
        const Operands o = operands<kSilu>(x, codes, scales, e, row0, left,
                                           static_cast<int>(item - static_cast<int64_t>(tile) * columns) * kOut, K, N);
        // An expert's last tile is not full: products of rows that are not there
        // would cost what the others do.  (The smaller ones load the scales of 512
        // inputs at once.)
        if (left > 96 || K < 512) tile_item<kSilu, 4>(o, K, N, y, s0, s1, s2, s3);
        else if (left > 64) tile_item<kSilu, 3>(o, K, N, y, s0, s1, s2, s3);
        else if (left > 32) tile_item<kSilu, 2>(o, K, N, y, s0, s1, s2, s3);
        else tile_item<kSilu, 1>(o, K, N, y, s0, s1, s2, s3);
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

// Row tiles of `rows` that a map in order can ask for at most.
int64_t most_tiles(const Call& c, int rows) { return c.num_rows / rows + (c.num_rows < c.E ? c.num_rows : c.E); }

template <bool kSilu, Scales kScales>
hipError_t launch_stream(const Call& c, int most) {
    const int64_t items = most_tiles(c, 16) * ceil_div(c.N, kSilu ? 32 : 64);
    hipLaunchKernelGGL((stream_w4_kernel<kSilu, kScales>), dim3(blocks_for(items, 256 * 2)), dim3(kThreads),
                       table_bytes(c.E), c.stream, static_cast<const uint16_t*>(c.x), c.num_rows, c.expert_rows,
                       c.capacity, c.codes, c.scales, c.E, c.K, c.N, most, static_cast<uint16_t*>(c.y));
    return hipGetLastError();
}
template <bool kSilu>
hipError_t launch_stream(const Call& c, int most) {
    switch (w4_scales(c.K)) {
        case kShared: return launch_stream<kSilu, kShared>(c, most);
        case kEight: return launch_stream<kSilu, kEight>(c, most);
        default: return launch_stream<kSilu, kSingle>(c, most);
    }
}

template <bool kSilu>
hipError_t launch_tile(const Call& c, const W4Plan& plan) {
    const int64_t columns = ceil_div(c.N, kSilu ? kTileWeights / 2 : kTileWeights);
    const int64_t items = most_tiles(c, plan.tile_rows) * columns;
    hipLaunchKernelGGL((tile_w4_kernel<kSilu>), dim3(blocks_for(items, 256)), dim3(kTileThreads), table_bytes(c.E),
                       c.stream, static_cast<const uint16_t*>(c.x), c.num_rows, c.expert_rows, c.capacity, c.codes,
                       c.scales, c.E, c.K, c.N, plan.tile_above, plan.tile_rows, static_cast<uint16_t*>(c.y));
    return hipGetLastError();
}

template <bool kSilu>
hipError_t launch(const Call& c) {
    const W4Plan plan = w4_plan(c.num_rows, c.capacity, c.E, c.N, kSilu);
    if (plan.stream_most > 0) {
        const hipError_t e = launch_stream<kSilu>(c, plan.stream_most);
        if (e != hipSuccess) return e;
    }
    return plan.tile_above < INT32_MAX ? launch_tile<kSilu>(c, plan) : hipSuccess;
}

}  // namespace

hipError_t launch_expert_linear_w4(const void* x, int64_t num_rows, const int32_t* expert_rows, int capacity,
                                   const uint8_t* w_codes, const uint8_t* w_scales, int E, int K, int N,
                                   bool silu_mul, void* y, hipStream_t stream) {
    const Call c = {x, num_rows, expert_rows, capacity, w_codes, w_scales, E, K, N, y, stream};
    return silu_mul ? launch<true>(c) : launch<false>(c);
}

}  // namespace ep
