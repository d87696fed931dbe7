// quant_i8.h -- rows to 8-bit integers with one scale a row (gfx950).
//
// With a = max |x| of the row: scale = a / 127, code = 127 x / a rounded to the
// nearest integer, halves to even.  A row of zeros has scale 0 and codes 0; a row
// that holds an infinity or a NaN has that scale and codes 0, so that whatever is
// computed from it is NaN.
//
// For bf16 rows the codes are those of the exact quotient.  127 x (15 bits) and a (8
// bits) are exact in fp32, and quotients other than halves stay 2^-16 of their value
// away from a half (with mantissas X, A and d the difference of the exponents, 127 X /
// (A 2^d) differs from m + 1/2 by a multiple of 1 / (2 A 2^d)); so a half has to come
// out exactly and the others to 2^-17.  The quotient is 127 x * (1/a) by the hardware's
// reciprocal, off by 2^-22, corrected by its remainder, which an fma gives exactly.
#pragma once

#include "ep_device.h"

namespace ep {
namespace {

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

// The larger magnitudes, two bf16 in a word: their bits without signs order as
// numbers do, infinity and then NaN last.
__device__ __forceinline__ uint32_t most16(uint32_t m, uint32_t v) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m),
                                                                  __builtin_bit_cast(u16x2, v & 0x7FFF7FFFu)));
}
__device__ __forceinline__ uint32_t most16(uint32_t m, const u32x4& v) {
    return most16(most16(most16(most16(m, v[0]), v[1]), v[2]), v[3]);
}
// The fp32 bits of the larger of the two.
__device__ __forceinline__ uint32_t most_bits(uint32_t m) {
    const uint32_t lo = m << 16, hi = m & 0xFFFF0000u;
    return lo > hi ? lo : hi;
}
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }
// Over the wave: within rows of 16 lanes by lane moves, then across them.
template <int kMove>
__device__ __forceinline__ uint32_t moved(uint32_t m) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), kMove, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t across_rows(uint32_t m) {
    const u32x2 a = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    m = larger(a[0], a[1]);
    const u32x2 b = __builtin_amdgcn_permlane32_swap(m, m, false, false);
    return larger(b[0], b[1]);
}
__device__ __forceinline__ uint32_t wave_most(uint32_t m) {
    m = larger(m, moved<0xB1>(m));                  // neighbours
    m = larger(m, moved<0x4E>(m));                  // pairs
    m = larger(m, moved<0x141>(m));                 // halves of eight, mirrored
    m = larger(m, moved<0x140>(m));                 // halves of sixteen, mirrored
    return across_rows(m);
}

// A row's scale, and what its codes are computed with.
struct Cast {
    float scale;
    float times;    // 127, and a power of two where a's reciprocal or 127 a would leave the normal range
    float a;        // a times that power
    float over;     // 1 / a, roughly; 0 for rows whose codes are 0
};
__device__ __forceinline__ Cast cast_of(uint32_t bits) {
    const float a = __uint_as_float(bits);
    const float by = bits < 0x21800000u ? 0x1p100f : bits > 0x5D800000u ? 0x1p-100f : 1.0f;   // outside 2^-60 .. 2^60
    const float near = a * by;
    const bool none = bits == 0u || bits >= 0x7F800000u;
    return {a / 127.0f, 127.0f * by, none ? 1.0f : near, none ? 0.0f : __builtin_amdgcn_rcpf(near)};
}
// 1.5 * 2^23 plus the code: its low byte is the code.
__device__ __forceinline__ uint32_t code_of(const Cast& c, float x) {
    const float n = x * c.times, q = n * c.over;
    return __float_as_uint(__builtin_fmaf(__builtin_fmaf(-q, c.a, n), c.over, q) + 12582912.0f);
}
// (Rows that hold an infinity or a NaN: n may be one too.)
__device__ __forceinline__ uint32_t four_codes(const Cast& c, float x0, float x1, float x2, float x3) {
    const uint32_t a = __builtin_amdgcn_perm(code_of(c, x1), code_of(c, x0), 0x0C0C0400u);
    const uint32_t b = __builtin_amdgcn_perm(code_of(c, x3), code_of(c, x2), 0x04000C0Cu);
    return c.over == 0.0f ? 0u : a | b;
}
// Codes of 16 bf16.
__device__ __forceinline__ u32x4 cast16(const Cast& c, const u32x4& a, const u32x4& b) {
    return u32x4{four_codes(c, bf16_lo(a[0]), bf16_hi(a[0]), bf16_lo(a[1]), bf16_hi(a[1])),
                 four_codes(c, bf16_lo(a[2]), bf16_hi(a[2]), bf16_lo(a[3]), bf16_hi(a[3])),
                 four_codes(c, bf16_lo(b[0]), bf16_hi(b[0]), bf16_lo(b[1]), bf16_hi(b[1])),
                 four_codes(c, bf16_lo(b[2]), bf16_hi(b[2]), bf16_lo(b[3]), bf16_hi(b[3]))};
}

// Pieces of 16 channels (two vectors in, one out) of a row, kPieces to a thread at a
// time, kThreads threads a row.
template <int kThreads, int kPieces, bool kOnce>
struct RowPieces {
    u32x4 v[kPieces][2];
    // Those from `base` on; past the row's end its last piece again.  kOnce: nobody
    // else reads the row, so it need not stay in the caches.
    __device__ __forceinline__ void load(const u32x4* __restrict__ row, int pieces, int base, int thread) {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int p = base + i * kThreads + thread, at = p < pieces ? p : pieces - 1;
            v[i][0] = kOnce ? __builtin_nontemporal_load(row + 2 * at) : row[2 * at];
            v[i][1] = kOnce ? __builtin_nontemporal_load(row + 2 * at + 1) : row[2 * at + 1];
        }
    }
    __device__ __forceinline__ uint32_t most(uint32_t m) const {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) m = most16(most16(m, v[i][0]), v[i][1]);
        return m;
    }
};

// Codes and scales of kRows rows, handed to to(row, piece, codes) and scale(row, s).
// `ready` runs behind the first loads.  kWhole: a row has kThreads * kPieces pieces at most.
template <int kThreads, int kPieces, int kRows, bool kOnce = false, bool kWhole = false, typename Ready, typename To,
          typename Scale>
__device__ __forceinline__ void cast_rows(const u32x4* const (&rows)[kRows], int pieces, int thread,
                                          uint32_t (&room)[kRows][kThreads / kWave], Ready ready, To to, Scale scale) {
    constexpr int kStep = kThreads * kPieces;
    RowPieces<kThreads, kPieces, kOnce> v[kRows];
    uint32_t m[kRows] = {};
#pragma unroll
    for (int r = 0; r < kRows; ++r) v[r].load(rows[r], pieces, 0, thread);
    ready();
#pragma unroll
    for (int r = 0; r < kRows; ++r) m[r] = v[r].most(m[r]);
    for (int base = kStep; !kWhole && base < pieces; base += kStep)
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            v[r].load(rows[r], pieces, base, thread);
            m[r] = v[r].most(m[r]);
        }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        m[r] = wave_most(most_bits(m[r]));
        if (kThreads > kWave && lane_id() == 0) room[r][threadIdx.x / kWave] = m[r];
    }
    if (kThreads > kWave) {
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int w = 0; w < kThreads / kWave; ++w) m[r] = larger(m[r], room[r][w]);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const Cast c = cast_of(m[r]);
        scale(r, c.scale);
        for (int base = 0; base < (kWhole ? 1 : pieces); base += kStep) {
            if (!kWhole && pieces > kStep) v[r].load(rows[r], pieces, base, thread);
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int p = base + i * kThreads + thread;
                if (p < pieces) to(r, p, cast16(c, v[r].v[i][0], v[r].v[i][1]));
            }
        }
    }
}

}  // namespace
}  // namespace ep
