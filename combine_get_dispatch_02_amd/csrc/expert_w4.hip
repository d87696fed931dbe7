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
constexpr int kTileRows = 16;

// Eight codes of one word, times the scale 2^(b - 127) whose bits are b << 23.
__device__ __forceinline__ bf16x8 decode(uint32_t codes, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
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

// The expert and the row tile (of kTileRows rows) that tile number `tile` is,
// counting tiles expert by expert; e == E past the last one.  Called by the
// whole block.
struct Tile {
    int e, index;
};
__device__ Tile find_tile(const int32_t* __restrict__ expert_rows, int E, int capacity, int64_t num_rows,
                          int64_t tile) {
    __shared__ int64_t sums[kThreads / kWave];
    __shared__ Tile found;
    const int lane = lane_id(), wave = static_cast<int>(threadIdx.x) / kWave;
    const int per = (E + kThreads - 1) / kThreads;
    const int e0 = static_cast<int>(threadIdx.x) * per;
    int64_t mine = 0;
    for (int i = 0; i < per; ++i)
        if (e0 + i < E) mine += (rows_of(expert_rows, e0 + i, capacity, num_rows).count + kTileRows - 1) / kTileRows;
    int64_t upto = mine;
    for (int d = 1; d < kWave; d <<= 1) {
        const int64_t o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    __syncthreads();
    if (lane == kWave - 1) sums[wave] = upto;
    if (threadIdx.x == 0) found = {E, 0};
    __syncthreads();
    int64_t before = upto - mine;
    for (int w = 0; w < wave; ++w) before += sums[w];
    if (tile >= before && tile < before + mine)
        for (int i = 0; i < per; ++i) {
            if (e0 + i >= E) break;
            const int n = (rows_of(expert_rows, e0 + i, capacity, num_rows).count + kTileRows - 1) / kTileRows;
            if (tile < before + n) {
                found = {e0 + i, static_cast<int>(tile - before)};
                break;
            }
            before += n;
        }
    __syncthreads();
    return found;
}

__device__ __forceinline__ float silu(float v) { return v / (1.0f + expf(-v)); }

// One block: 16 token rows x 64 outputs, 16 outputs a wave.
template <bool kSilu>
__global__ __launch_bounds__(kThreads) void expert_w4_kernel(
    const uint16_t* __restrict__ x, int64_t num_rows, const int32_t* __restrict__ expert_rows, int capacity,
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int E, int K, int N,
    uint16_t* __restrict__ y) {
    const int lane = lane_id(), q = lane / 16, i16 = lane % 16;
    const int n0 = static_cast<int>(blockIdx.x) * 64 + static_cast<int>(threadIdx.x) / kWave * 16;
    for (int64_t tile = blockIdx.y;; tile += gridDim.y) {
        const Tile at = find_tile(expert_rows, E, capacity, num_rows, tile);
        if (at.e >= E) break;
        const Rows rows = rows_of(expert_rows, at.e, capacity, num_rows);
        const int m0 = at.index * kTileRows, left = rows.count - m0;
        // Lanes past the rows or outputs repeat the last one and store nothing.
        const int m = i16 < left ? i16 : left - 1;
        const int n = n0 + i16 < N ? n0 + i16 : N - 1;
        const uint16_t* xr = x + (rows.first + m0 + m) * K + q * 32;
        f32x4 acc[2] = {};
        for (int half = 0; half < (kSilu ? 2 : 1); ++half) {
            const int64_t wr = static_cast<int64_t>(at.e) * (kSilu ? 2 * N : N) + half * static_cast<int64_t>(N) + n;
            const uint8_t* cr = codes + wr * (K / 2) + q * 16;
            const uint8_t* sr = scales + wr * (K / 32) + q;
            f32x4 c = {};
            for (int kb = 0; kb < K; kb += 128) {
                const u32x4 w = *reinterpret_cast<const u32x4*>(cr + kb / 2);
                const float scale = __uint_as_float(static_cast<uint32_t>(sr[kb / 32]) << 23);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const bf16x8 b = *reinterpret_cast<const bf16x8*>(xr + kb + 8 * s);
                    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(decode(w[s], scale), b, c, 0, 0, 0);
                }
            }
            acc[half] = c;
        }
        // A lane holds outputs n0 + 4 q .. + 3 of token row m0 + i16.
        if (i16 < left && n0 + 4 * q < N) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = bf16_rne(kSilu ? silu(acc[0][i]) * acc[1][i] : acc[0][i]);
            *reinterpret_cast<u32x2*>(y + (rows.first + m0 + i16) * N + n0 + 4 * q) =
                u32x2{o[0] | (o[1] << 16), o[2] | (o[3] << 16)};
        }
    }
}

}  // namespace

hipError_t launch_expert_linear_w4(const void* x, int64_t num_rows, const int32_t* expert_rows, int capacity,
                                   const uint8_t* w_codes, const uint8_t* w_scales, int E, int K, int N,
                                   bool silu_mul, void* y, hipStream_t stream) {
    const int64_t tiles = num_rows / kTileRows + E;
    const dim3 grid(static_cast<unsigned>(ceil_div(N, 64)), static_cast<unsigned>(tiles < 65535 ? tiles : 65535));
    if (silu_mul)
        hipLaunchKernelGGL((expert_w4_kernel<true>), grid, dim3(kThreads), 0, stream,
                           static_cast<const uint16_t*>(x), num_rows, expert_rows, capacity, w_codes, w_scales, E, K,
                           N, static_cast<uint16_t*>(y));
    else
        hipLaunchKernelGGL((expert_w4_kernel<false>), grid, dim3(kThreads), 0, stream,
                           static_cast<const uint16_t*>(x), num_rows, expert_rows, capacity, w_codes, w_scales, E, K,
                           N, static_cast<uint16_t*>(y));
    return hipGetLastError();
}

}  // namespace ep
