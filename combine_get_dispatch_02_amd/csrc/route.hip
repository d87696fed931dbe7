// route.hip -- ep_route and ep_route_backward on gfx950.
//
// Router logits [T, E] to the k experts of each token and their weights, and
// the gradient back.
//
// Choosing.  L lanes of a wave hold one token (64 / L tokens a wave), C of its
// experts each.  A choice and its expert make one 64-bit key that is also a positive
// double, so that one instruction (v_max_f64, as fast as an fp32 one here) compares
// both, ties included.  Every lane sorts its keys once (a network of v_max / v_min);
// each of the k rounds is then a maximum over the lanes' first keys, and the lane
// that had it moves up its list.  For 32768 tokens of 256 experts, top 8, by logits,
// that is about 780 vector instructions a wave of four tokens, 530 of them the sort
// and the rounds.  Another 400 before the loop over tokens, most of them the group
// code's, which the compiler takes out of the loop whether there are groups or not,
// are paid by every wave, as the grid has a wave for every four tokens.
#include "../../include/ep.h"
#include "ep_device.h"
#include "moe_launch.h"

namespace ep {
namespace {

constexpr int kWaves = 4;
constexpr float kInf = __builtin_inff();

// ---- logits of the three types ---------------------------------------------------
struct F32 { typedef float raw; };
struct Bf16 { typedef uint16_t raw; };
struct F16 { typedef _Float16 raw; };

__device__ __forceinline__ float to_float(F32, float v) { return v; }
__device__ __forceinline__ float to_float(Bf16, uint16_t v) { return bf16_lo(v); }
__device__ __forceinline__ float to_float(F16, _Float16 v) { return static_cast<float>(v); }
__device__ __forceinline__ float from_float(F32, float v) { return v; }
__device__ __forceinline__ uint16_t from_float(Bf16, float v) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));       // to nearest, ties to even
}
__device__ __forceinline__ _Float16 from_float(F16, float v) { return static_cast<_Float16>(v); }

// An unavailable expert's logit reads as -inf.
template <typename In>
__device__ __forceinline__ float logit(const typename In::raw* p) {
    const float v = to_float(In(), *p);
    return v != v ? -kInf : v;
}

// ---- one token's lanes -----------------------------------------------------------
// v combined over the L lanes of a token, in every lane: by rotations within the
// rows of 16 lanes, then by exchanging rows and halves.
template <int kRotate>
__device__ __forceinline__ uint32_t rotate_row(uint32_t v) {
    return __builtin_amdgcn_update_dpp(0, v, 0x120 + kRotate, 0xF, 0xF, true);  // row_ror
}
template <int kRotate>
__device__ __forceinline__ float rotate_row(float v) {
    return __uint_as_float(rotate_row<kRotate>(__float_as_uint(v)));
}
template <int kRotate>
__device__ __forceinline__ double rotate_row(double v) {
    const u32x2 u = __builtin_bit_cast(u32x2, v);
    return __builtin_bit_cast(double, u32x2{rotate_row<kRotate>(u[0]), rotate_row<kRotate>(u[1])});
}
// The two values that neighbouring rows (kHalf: the halves of the wave) hold.
template <bool kHalf>
__device__ __forceinline__ u32x2 exchange(uint32_t v) {
    return kHalf ? __builtin_amdgcn_permlane32_swap(v, v, false, false)
                 : __builtin_amdgcn_permlane16_swap(v, v, false, false);
}
template <bool kHalf, typename Op>
__device__ __forceinline__ float exchange(float v, Op op) {
    const u32x2 u = exchange<kHalf>(__float_as_uint(v));
    return op(__uint_as_float(u[0]), __uint_as_float(u[1]));
}
template <bool kHalf, typename Op>
__device__ __forceinline__ double exchange(double v, Op op) {
    const u32x2 u = __builtin_bit_cast(u32x2, v);
    const u32x2 lo = exchange<kHalf>(u[0]), hi = exchange<kHalf>(u[1]);
    return op(__builtin_bit_cast(double, u32x2{lo[0], hi[0]}), __builtin_bit_cast(double, u32x2{lo[1], hi[1]}));
}
template <int L, typename F, typename Op>
__device__ __forceinline__ F over_lanes(F v, Op op) {
    static_assert(L == 16 || L == 64, "a row of lanes or the whole wave");
    v = op(v, rotate_row<8>(v));
    v = op(v, rotate_row<4>(v));
    v = op(v, rotate_row<2>(v));
    v = op(v, rotate_row<1>(v));
    if (L == 64) {
        v = exchange<false>(v, op);
        v = exchange<true>(v, op);
    }
    return v;
}
template <int L>
__device__ __forceinline__ float max_over(float v) {
    return over_lanes<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L, typename F>
__device__ __forceinline__ F sum_over(F v) {
    return over_lanes<L>(v, [](F a, F b) { return a + b; });
}

// exp(l - top) as a softmax term: 0 for an unavailable expert, and 1 for each
// +inf logit where there is one (top == +inf), whose finite neighbours get 0.
__device__ __forceinline__ float softmax_term(float l, float top) {
    if (l == top) return l == -kInf ? 0.0f : 1.0f;
    return expf(l - top);
}

// exp(x) to about 2^-50 for |x| <= 700: x = n ln 2 + r with |r| <= ln 2 / 2, the
// Taylor series of exp(r) to r^12 (the next term is below 2^-52), scaled by 2^n.
__device__ __forceinline__ double exp64(double x) {
    const double n = __builtin_rint(x * 1.4426950408889634074);
    double r = __builtin_fma(n, -0.6931471805437468, x);    // ln 2 = its first 34 bits,
    r = __builtin_fma(n, -1.619851018665656e-11, r);        // exact times n, and the rest
    double p = 1.0 / 479001600;
    p = __builtin_fma(p, r, 1.0 / 39916800);
    p = __builtin_fma(p, r, 1.0 / 3628800);
    p = __builtin_fma(p, r, 1.0 / 362880);
    p = __builtin_fma(p, r, 1.0 / 40320);
    p = __builtin_fma(p, r, 1.0 / 5040);
    p = __builtin_fma(p, r, 1.0 / 720);
    p = __builtin_fma(p, r, 1.0 / 120);
    p = __builtin_fma(p, r, 1.0 / 24);
    p = __builtin_fma(p, r, 1.0 / 6);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    return __builtin_amdgcn_ldexp(p, static_cast<int>(n));
}
// 1 / d for d in [1, 2^1011]: the hardware's estimate and two Newton steps.
__device__ __forceinline__ double reciprocal64(double d) {
    double r = __builtin_amdgcn_rcp(d);
    r = __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
    return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}
__device__ __forceinline__ double softmax_term64(float l, float top) {
    if (l == top) return l == -kInf ? 0.0 : 1.0;
    return exp64(fmax(static_cast<double>(l) - static_cast<double>(top), -700.0));
}

// sigmoid(l) * exp(-low), low = min(0, largest chosen logit): numerator and
// denominator stay normal numbers where sigmoid itself would underflow.
__device__ __forceinline__ float sigmoid_over(float l, float low) {
    if (l == -kInf) return 0.0f;
    return expf(fminf(l, 0.0f) - low) / (1.0f + expf(-fabsf(l)));
}
__device__ __forceinline__ float sigmoid(float l) { return sigmoid_over(l, 0.0f); }
__device__ __forceinline__ double sigmoid64(float l) {
    return reciprocal64(1.0 + exp64(fmin(fmax(-static_cast<double>(l), -700.0), 700.0)));
}

// ---- keys ------------------------------------------------------------------------
// Choice and expert in one double: 1 + a fraction of 32 bits that order the choice
// and 16 that order equal choices, the lower expert first.  1: unavailable.  -0
// counts as 0.
constexpr uint64_t kNoKey = 0x3FF0000000000000ull;
__device__ __forceinline__ double make_key(float choice, int e) {
    const uint32_t u = __float_as_uint(choice + 0.0f);
    const uint32_t ordered = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
    const uint64_t key = kNoKey | static_cast<uint64_t>(ordered) << 16 | static_cast<uint64_t>(0xFFFF - e);
    return __builtin_bit_cast(double, choice > -kInf ? key : kNoKey);
}
__device__ __forceinline__ bool is_key(double key) { return __builtin_bit_cast(uint64_t, key) != kNoKey; }
__device__ __forceinline__ int key_expert(double key) {
    return 0xFFFF - static_cast<int>(__builtin_bit_cast(uint64_t, key) & 0xFFFF);
}
__device__ __forceinline__ float key_choice(double key) {
    const uint32_t ordered = static_cast<uint32_t>(__builtin_bit_cast(uint64_t, key) >> 16);
    return __uint_as_float(ordered & 0x80000000u ? ordered ^ 0x80000000u : ~ordered);
}
// (As the builtins these are preceded by one instruction an operand that quiets
// NaNs, which keys never are.)
__device__ __forceinline__ double key_max(double a, double b) {
    double r;
    asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ double key_min(double a, double b) {
    double r;
    asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}

// Largest first: Batcher's odd-even merge sort.
template <int C>
__device__ __forceinline__ void sort_keys(double (&k)[C]) {
#pragma unroll
    for (int p = 1; p < C; p *= 2)
#pragma unroll
        for (int d = p; d > 0; d /= 2)
#pragma unroll
            for (int i = 0; i < C - d; ++i)
                if (i >= d % p && (i - d % p) / d % 2 == 0 && i / (2 * p) == (i + d) / (2 * p)) {
                    const double a = key_max(k[i], k[i + d]), b = key_min(k[i], k[i + d]);
                    k[i] = a;
                    k[i + d] = b;
                }
}

// Which experts a lane holds: pieces of P in a row, 16 bytes where C allows,
// piece i from expert a i + b pos on.  Interleaved, the lanes' pieces lie side by
// side, as loads and stores want them; in order, a lane's pieces do, as groups of
// experts want them.
template <typename In, int L, int C>
struct Layout {
    static constexpr int kFull = 16 / static_cast<int>(sizeof(typename In::raw)), P = C < kFull ? C : kFull;
    // (Elements may lie anywhere: global accesses need no alignment.)
    typedef typename In::raw Vector __attribute__((ext_vector_type(P), aligned(sizeof(typename In::raw))));
    int a, b;
    __device__ __forceinline__ explicit Layout(bool in_order) : a(in_order ? P : L * P), b(in_order ? C : P) {}
    __device__ __forceinline__ int expert(int c, int pos) const { return c / P * a + pos * b + c % P; }

    // A token's logits, -inf for experts that do not exist.
    __device__ __forceinline__ void load(const typename In::raw* in, int pos, int E, float (&l)[C]) const {
#pragma unroll
        for (int i = 0; i < C / P; ++i) {
            const int e = i * a + pos * b;
            if (e + P <= E) {
                const Vector v = *reinterpret_cast<const Vector*>(in + e);
#pragma unroll
                for (int c = 0; c < P; ++c) l[i * P + c] = to_float(In(), v[c]);
            } else {
#pragma unroll
                for (int c = 0; c < P; ++c) l[i * P + c] = e + c < E ? to_float(In(), in[e + c]) : -kInf;
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (l[c] != l[c]) l[c] = -kInf;
    }
    __device__ __forceinline__ void store(typename In::raw* out, int pos, int E, const float (&v)[C]) const {
#pragma unroll
        for (int i = 0; i < C / P; ++i) {
            const int e = i * a + pos * b;
            Vector o;
#pragma unroll
            for (int c = 0; c < P; ++c) o[c] = from_float(In(), v[i * P + c]);
            if (e + P <= E) {
                *reinterpret_cast<Vector*>(out + e) = o;
            } else {
#pragma unroll
                for (int c = 0; c < P; ++c)
                    if (e + c < E) out[e + c] = o[c];
            }
        }
    }
};

// The two best of a group.
struct Best {
    float first, second;                            // -inf: none
};
__device__ __forceinline__ Best best_of(Best a, Best b) {
    return {fmaxf(a.first, b.first), fmaxf(fminf(a.first, b.first), fmaxf(a.second, b.second))};
}
// A group's score; of the two best the second counts only if there is one.
__device__ __forceinline__ float group_score(Best b, int group_top) {
    return group_top == 2 && b.second > -kInf ? b.first + b.second : b.first;
}

// D: how far down a lane's list k rounds can get, min(C, k) or more.  kByChoice:
// by 64-bit scores and bias, else by the logits (a kernel of its own: half the
// registers, so twice the waves; with 16 experts a lane it is held to registers
// for three waves a SIMD: 32768 x 256 with a bias 27.9 us, 31.4 with two).
template <typename In, int L, int C, int D, bool kByChoice>
__global__ __launch_bounds__(kWaves* kWave, kByChoice&& C == 16 ? 3 : 1) void route_kernel(const typename In::raw* __restrict__ logits,
                                                              const float* __restrict__ bias, int64_t T,
                                                              int E, int k, RouteOptions opt,
                                                              int64_t* __restrict__ topk_idx,
                                                              float* __restrict__ topk_weights) {
    constexpr int kTokens = kWave / L;
    extern __shared__ float choices[];              // [kWaves * kTokens][E], groups of other sizes only
    const int lane = lane_id(), pos = lane % L, sub = lane / L;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const int size = E / opt.num_groups;
    const Layout<In, L, C> layout(opt.num_groups > 1);
    float b[C] = {};
    if (kByChoice && bias) {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (layout.expert(c, pos) < E) b[c] = bias[layout.expert(c, pos)];
    }
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWaves * kTokens;
    for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * kTokens; t0 < T; t0 += step) {
        const bool live = t0 + sub < T;
        const int64_t t = live ? t0 + sub : T - 1;  // lanes past the end repeat the last token
        float l[C];
        layout.load(logits + t * E, pos, E, l);
        float top = -kInf;
        if (!opt.sigmoid) {
#pragma unroll
            for (int c = 0; c < C; ++c) top = fmaxf(top, l[c]);
            top = max_over<L>(top);
        }

        float choice[C];
#pragma unroll
        for (int c = 0; c < C; ++c) choice[c] = l[c];
        if (kByChoice) {
            // fl32 of the 64-bit score: an fp32 one is off by a step or two, enough
            // to put neighbours in another order.
            if (opt.sigmoid) {
#pragma unroll
                for (int c = 0; c < C; ++c) choice[c] = static_cast<float>(sigmoid64(l[c]));
            } else {
                double s[C], total = 0.0;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    s[c] = softmax_term64(l[c], top);
                    total += s[c];
                }
                total = sum_over<L>(total);
                const double inverse = reciprocal64(total);     // total >= 1, or none is available
#pragma unroll
                for (int c = 0; c < C; ++c) choice[c] = static_cast<float>(s[c] * inverse);
            }
#pragma unroll
            for (int c = 0; c < C; ++c) choice[c] = l[c] > -kInf ? choice[c] + b[c] : -kInf;
        }

        if (opt.num_groups > 1) {
            const int wide = size / C;              // lanes of a group, if whole and a power of two
            if (E == L * C && wide * C == size && (wide & (wide - 1)) == 0) {
                Best best = {-kInf, -kInf};
#pragma unroll
                for (int c = 0; c < C; ++c) best = best_of(best, {choice[c] == choice[c] ? choice[c] : -kInf, -kInf});
                for (int d = 1; d < wide; d *= 2)
                    best = best_of(best, {__shfl_xor(best.first, d), __shfl_xor(best.second, d)});
                const float mine = group_score(best, opt.group_top);
                const int first = pos & ~(wide - 1);
                int better = 0;
                for (int o = 0; o < L; o += wide) {
                    const float v = __shfl(mine, sub * L + o);
                    better += v > mine || (v == mine && o < first);
                }
                if (better >= opt.topk_groups) {
#pragma unroll
                    for (int c = 0; c < C; ++c) choice[c] = -kInf;
                }
            } else {
                // Any size: through shared memory, a lane to a group, and every lane
                // compares all groups with all (bf16, 160 experts in 8 groups, top 6, by
                // logits: 7.6 us for one token, 11.7 for 4096; fp32, 256 experts in 64
                // groups, top 8, by scores, 4096 tokens: 207).
                float* row = choices + (wave * kTokens + sub) * E;
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (layout.expert(c, pos) < E) row[layout.expert(c, pos)] = choice[c];
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
                float mine[kWave / L];
#pragma unroll
                for (int i = 0; i < kWave / L; ++i) {
                    const int g = i * L + pos;
                    Best best = {-kInf, -kInf};
                    if (g < opt.num_groups)
                        for (int u = 0; u < size; ++u) {
                            const float v = row[g * size + u];
                            best = best_of(best, {v == v ? v : -kInf, -kInf});
                        }
                    mine[i] = group_score(best, opt.group_top);
                }
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int i = 0; i < kWave / L; ++i)
                    if (i * L + pos < opt.num_groups) row[i * L + pos] = mine[i];
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
                uint64_t kept = 0;
                for (int g = 0; g < opt.num_groups; ++g) {
                    const float v = row[g];
                    int better = 0;
                    for (int o = 0; o < opt.num_groups; ++o) better += row[o] > v || (row[o] == v && o < g);
                    if (better < opt.topk_groups) kept |= uint64_t(1) << g;
                }
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (layout.expert(c, pos) < E && !(kept >> (layout.expert(c, pos) / size) & 1)) choice[c] = -kInf;
            }
        }

        double key[C];
#pragma unroll
        for (int c = 0; c < C; ++c) key[c] = make_key(choice[c], layout.expert(c, pos));
        sort_keys<C>(key);
        // k rounds: the largest first key of the token's lanes goes to lane j, and
        // the lane that had it moves up.
        double won = __builtin_bit_cast(double, kNoKey);
        for (int j = 0; j < k; ++j) {
            const double best = over_lanes<L>(key[0], [](double x, double y) { return key_max(x, y); });
            if (pos == j) won = best;
            const bool had = key[0] == best;
#pragma unroll
            for (int i = 0; i < D; ++i) {
                const double next = i + 1 < C ? key[i + 1] : __builtin_bit_cast(double, kNoKey);
                key[i] = had ? next : key[i];
            }
        }

        const bool filled = pos < k && is_key(won);
        const int e = filled ? key_expert(won) : -1;
        float le = -kInf;
        if (filled) le = kByChoice ? logit<In>(logits + t * E + e) : key_choice(won);
        float a, total = 1.0f;
        if (opt.sigmoid) {
            const float low = opt.renormalize ? fminf(max_over<L>(le), 0.0f) : 0.0f;
            a = sigmoid_over(le, low);
        } else {
            const float m = opt.renormalize ? max_over<L>(le) : top;
            a = softmax_term(le, m);
            if (!opt.renormalize) {
                // 2^x of the hardware: off by a step and by 2.5 units of l - top,
                // which is small where a term counts.
                total = 0.0f;
#pragma unroll
                for (int c = 0; c < C; ++c)
                    total += l[c] == top ? (top > -kInf ? 1.0f : 0.0f)
                                         : __builtin_amdgcn_exp2f((l[c] - top) * 1.44269504f);
                total = sum_over<L>(total);
            }
        }
        if (opt.renormalize) total = sum_over<L>(a);
        if (live && pos < k) {
            topk_idx[t * k + pos] = e;
            topk_weights[t * k + pos] = filled ? a / total * opt.scale : 0.0f;
        }
    }
}

// The value of lane i of the token's lanes, in all of them.
template <int L>
__device__ __forceinline__ uint32_t from_lane(uint32_t v, int i) {
    if (L == 64) return __builtin_amdgcn_readlane(v, i);
    switch (i) {                                    // i is a constant where this is called: row_newbcast
#define EP_LANE(n) \
    case n: return __builtin_amdgcn_update_dpp(0, v, 0x150 + n, 0xF, 0xF, true);
        EP_LANE(0) EP_LANE(1) EP_LANE(2) EP_LANE(3) EP_LANE(4) EP_LANE(5) EP_LANE(6) EP_LANE(7)
        EP_LANE(8) EP_LANE(9) EP_LANE(10) EP_LANE(11) EP_LANE(12) EP_LANE(13) EP_LANE(14) EP_LANE(15)
#undef EP_LANE
    }
    return 0;
}

// ---- gradient --------------------------------------------------------------------
// Tokens and experts to lanes as above; lane j also takes slot j.  The slots'
// contributions meet in a row of the block's memory, from which every lane takes
// those of its experts: bound by writing [T, E] (and reading it, kDense: softmax
// not renormalised, where every element has a gradient).
template <typename In, int L, int C, bool kDense>
__global__ __launch_bounds__(kWaves* kWave) void route_backward_kernel(
    const typename In::raw* __restrict__ logits, const int64_t* __restrict__ topk_idx,
    const float* __restrict__ grad_weights, int64_t T, int E, int k, bool is_sigmoid, bool renormalize,
    float scale, typename In::raw* __restrict__ grad_logits) {
    constexpr int kTokens = kWave / L, P = Layout<In, L, C>::P, kPiece = P < 4 ? P : 4;
    typedef float Piece __attribute__((ext_vector_type(kPiece)));
    // [token][piece c / 4 of a lane][lane]: what a lane reads at once lies together.
    __shared__ Piece rows[kWaves * kTokens][C / kPiece][L];
    const int lane = lane_id(), pos = lane % L, sub = lane / L;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const Layout<In, L, C> layout(false);
    Piece(*row)[L] = rows[wave * kTokens + sub];
    float* flat = reinterpret_cast<float*>(row);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWaves * kTokens;
    for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * kTokens; t0 < T; t0 += step) {
        const bool live = t0 + sub < T;
        const int64_t t = live ? t0 + sub : T - 1;  // lanes past the end repeat the last token
        const typename In::raw* in = logits + t * E;
        float l[C];
        if (kDense) layout.load(in, pos, E, l);
        int e = -1;
        float g = 0.0f, le = -kInf;
        if (pos < k) {
            const int64_t id = topk_idx[t * k + pos];
            g = grad_weights[t * k + pos];
            if (id >= 0 && id < E) {
                e = static_cast<int>(id);
                le = logit<In>(in + e);
            }
        }
        if (le == -kInf) {                          // unavailable: no score, no gradient
            g = 0.0f;
            e = -1;
        }
        // This slot's contribution d; kDense: to the sum in s (d - mean), else as it is.
        float d, mean = 0.0f;
        if (kDense) {
            float top = -kInf, total = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c) top = fmaxf(top, l[c]);
            top = max_over<L>(top);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                // 2^x of the hardware: off by a step and by 2.5 units of l - top, and
                // the rounding of the exponent's argument is the larger part of that.
                l[c] = l[c] == top ? (top > -kInf ? 1.0f : 0.0f)
                                   : __builtin_amdgcn_exp2f((l[c] - top) * 1.44269504f);
                total += l[c];
            }
            total = sum_over<L>(total);
            const float inverse = total > 0.0f ? scale / total : 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c) l[c] *= inverse;            // scale * s
            d = g;
            mean = sum_over<L>(e >= 0 ? g * (softmax_term(le, top) / total) : 0.0f);
        } else if (renormalize) {
            const float m = max_over<L>(le);
            const float a = is_sigmoid ? sigmoid_over(le, fminf(m, 0.0f)) : softmax_term(le, m);
            const float sum = sum_over<L>(a);
            const float p = sum > 0.0f ? a / sum : 0.0f;
            d = scale * p * (g - sum_over<L>(g * p));
            if (is_sigmoid) d *= sigmoid(-le);
        } else {
            d = scale * g * sigmoid(le) * sigmoid(-le);
        }
        // Slots of the same expert add in slot order, whichever lane writes.
        float all = 0.0f;
        if (L == 64) {
            for (int j = 0; j < k; ++j)
                if (read_lane(e, j) == e) all += read_lane(d, j);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                if (j >= k) break;
                const int o = static_cast<int>(from_lane<L>(static_cast<uint32_t>(e), j));
                const float v = __uint_as_float(from_lane<L>(__float_as_uint(d), j));
                all += o == e ? v : 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < C / kPiece; ++i) row[i][pos] = Piece{};
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (e >= 0) {
            const int c = e / (L * P) * P + e % P;  // of lane e / P mod L
            flat[(c / kPiece * L + e / P % L) * kPiece + c % kPiece] = all;
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        float out[C];
#pragma unroll
        for (int i = 0; i < C / kPiece; ++i) {
            const Piece v = row[i][pos];
#pragma unroll
            for (int c = 0; c < kPiece; ++c)
                out[i * kPiece + c] = kDense ? l[i * kPiece + c] * (v[c] - mean) : v[c];
        }
        __builtin_amdgcn_wave_barrier();
        if (live) layout.store(grad_logits + t * E, pos, E, out);
    }
}

bool by_choice(const float* bias, const RouteOptions& opt) {
    return bias || (opt.num_groups > 1 && opt.group_top == 2);
}

template <typename In, int L, int C, int D>
hipError_t launch_lanes(const void* logits, const float* bias, int64_t T, int E, int k, const RouteOptions& opt,
                        int64_t* topk_idx, float* topk_weights, hipStream_t stream) {
    const int per_block = kWaves * (kWave / L);
    const int64_t blocks = ceil_div(T, per_block), cap = kMaxLaunchThreads / (kWaves * kWave);
    const dim3 grid(static_cast<unsigned>(blocks < cap ? blocks : cap)), block(kWaves * kWave);
    const size_t lds = opt.num_groups > 1 ? sizeof(float) * per_block * E : 0;
    const typename In::raw* in = static_cast<const typename In::raw*>(logits);
    if (by_choice(bias, opt))
        hipLaunchKernelGGL((route_kernel<In, L, C, D, true>), grid, block, lds, stream, in, bias, T, E, k, opt,
                           topk_idx, topk_weights);
    else
        hipLaunchKernelGGL((route_kernel<In, L, C, D, false>), grid, block, lds, stream, in, bias, T, E, k, opt,
                           topk_idx, topk_weights);
    return hipGetLastError();
}

// Tokens from which a row of 16 lanes takes one: it has a quarter of the
// instructions a token, 64 lanes the shorter way through one.  Measured by logits,
// and taken for scores too, 64 lanes against 16 (us): 256 experts, top 8, 4.1 / 5.3 at 2048 tokens, 5.7 / 5.5 at 4096,
// 27.6 / 18.6 at 32768; 128 experts, top 4, 3.6 / 3.7 at 2048, 4.9 / 3.8 at 4096;
// 64 experts, top 6, 2.9 / 3.1 at 1024, 3.3 / 3.1 at 2048.  The gradient has fewer
// instructions to save: 256 experts 5.3 / 5.5 at 8192, 13.6 / 11.7 at 32768 (fp32,
// softmax), 16.4 / 13.2 (bf16, every logit); 64 experts 3.2 / 3.5 at 4096, 4.2 / 3.7
// at 8192.
int64_t row_tokens(int E) { return E > 128 ? 4096 : 2048; }
int64_t row_tokens_back(int E) { return E > 128 ? 12288 : 6144; }

template <typename In>
hipError_t launch_type(const void* logits, const float* bias, int64_t T, int E, int k, const RouteOptions& opt,
                       int64_t* topk_idx, float* topk_weights, hipStream_t stream) {
#define EP_ROUTE(L, C, D) launch_lanes<In, L, C, D>(logits, bias, T, E, k, opt, topk_idx, topk_weights, stream)
    if (T >= row_tokens(E) && k <= 16) {
        if (E <= 64) return EP_ROUTE(16, 4, 4);
        if (E <= 128) return EP_ROUTE(16, 8, 8);
        if (E <= 256) return k <= 8 ? EP_ROUTE(16, 16, 8) : EP_ROUTE(16, 16, 16);
        // (By 64-bit scores 32 of them a lane leave a wave alone on its SIMD: 16384 x
        // 512 takes 47 us, 38 with 64 lanes a token.  By logits it is 17 and 21.)
        if (E <= 512 && k <= 8 && !by_choice(bias, opt)) return EP_ROUTE(16, 32, 8);
    }
    if (E <= 64) return EP_ROUTE(64, 1, 1);
    if (E <= 256) return EP_ROUTE(64, 4, 4);
    if (E <= 512) return EP_ROUTE(64, 8, 8);
    if (E <= 1024) return EP_ROUTE(64, 16, 16);
    return EP_ROUTE(64, 32, 32);
#undef EP_ROUTE
}

template <typename In, int L, int C>
hipError_t launch_back_lanes(const void* logits, const int64_t* topk_idx, const float* grad_weights, int64_t T,
                             int E, int k, bool is_sigmoid, bool renormalize, float scale, void* grad_logits,
                             hipStream_t stream) {
    const int64_t blocks = ceil_div(T, kWaves * (kWave / L)), cap = kMaxLaunchThreads / (kWaves * kWave);
    const dim3 grid(static_cast<unsigned>(blocks < cap ? blocks : cap)), block(kWaves * kWave);
    const typename In::raw* in = static_cast<const typename In::raw*>(logits);
    typename In::raw* out = static_cast<typename In::raw*>(grad_logits);
    if (!is_sigmoid && !renormalize)
        hipLaunchKernelGGL((route_backward_kernel<In, L, C, true>), grid, block, 0, stream, in, topk_idx,
                           grad_weights, T, E, k, is_sigmoid, renormalize, scale, out);
    else
        hipLaunchKernelGGL((route_backward_kernel<In, L, C, false>), grid, block, 0, stream, in, topk_idx,
                           grad_weights, T, E, k, is_sigmoid, renormalize, scale, out);
    return hipGetLastError();
}

template <typename In>
hipError_t launch_back(const void* logits, const int64_t* topk_idx, const float* grad_weights, int64_t T, int E,
                       int k, bool is_sigmoid, bool renormalize, float scale, void* grad_logits,
                       hipStream_t stream) {
#define EP_BACK(L, C)                                                                                        \
    launch_back_lanes<In, L, C>(logits, topk_idx, grad_weights, T, E, k, is_sigmoid, renormalize, scale,     \
                                grad_logits, stream)
    if (T >= row_tokens_back(E) && k <= 16) {
        if (E <= 64) return EP_BACK(16, 4);
        if (E <= 128) return EP_BACK(16, 8);
        if (E <= 256) return EP_BACK(16, 16);
    }
    if (E <= 64) return EP_BACK(64, 1);
    if (E <= 256) return EP_BACK(64, 4);
    if (E <= 512) return EP_BACK(64, 8);
    if (E <= 1024) return EP_BACK(64, 16);
    return EP_BACK(64, 32);
#undef EP_BACK
}

}  // namespace

hipError_t launch_route(const void* logits, int type, const float* bias, int64_t T, int E, int k,
                        const RouteOptions& opt, int64_t* topk_idx, float* topk_weights, hipStream_t stream) {
    if (type == EP_TYPE_F32) return launch_type<F32>(logits, bias, T, E, k, opt, topk_idx, topk_weights, stream);
    if (type == EP_TYPE_BF16) return launch_type<Bf16>(logits, bias, T, E, k, opt, topk_idx, topk_weights, stream);
    return launch_type<F16>(logits, bias, T, E, k, opt, topk_idx, topk_weights, stream);
}

hipError_t launch_route_backward(const void* logits, int type, const int64_t* topk_idx,
                                 const float* grad_weights, int64_t T, int E, int k, bool is_sigmoid,
                                 bool renormalize, float scale, void* grad_logits, hipStream_t stream) {
    if (type == EP_TYPE_F32)
        return launch_back<F32>(logits, topk_idx, grad_weights, T, E, k, is_sigmoid, renormalize, scale,
                                grad_logits, stream);
    if (type == EP_TYPE_BF16)
        return launch_back<Bf16>(logits, topk_idx, grad_weights, T, E, k, is_sigmoid, renormalize, scale,
                                 grad_logits, stream);
    return launch_back<F16>(logits, topk_idx, grad_weights, T, E, k, is_sigmoid, renormalize, scale, grad_logits,
                            stream);
}

}  // namespace ep
