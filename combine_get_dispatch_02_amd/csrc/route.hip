// route.hip -- ep_route and ep_route_backward on gfx950.
//
// Router logits [T, E] to the k experts of each token and their weights, and
// the gradient back.  L lanes of a wave hold one token (64 / L tokens per
// wave), C of its experts each: expert e = c * L + lane.
#include "../../include/ep.h"
#include "ep_device.h"
#include "ep_launch.h"

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
__device__ __forceinline__ uint16_t from_float(Bf16, float v) { return static_cast<uint16_t>(bf16_rne(v)); }
__device__ __forceinline__ _Float16 from_float(F16, float v) { return static_cast<_Float16>(v); }

// An unavailable expert's logit reads as -inf.
template <typename In>
__device__ __forceinline__ float logit(const typename In::raw* p) {
    const float v = to_float(In(), *p);
    return v != v ? -kInf : v;
}

template <int L>
__device__ __forceinline__ float max_over(float v) {
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}
template <int L, typename F>
__device__ __forceinline__ F sum_over(F v) {
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// exp(l - top) as a softmax term: 0 for an unavailable expert, and 1 for each
// +inf logit where there is one (top == +inf), whose finite neighbours get 0.
__device__ __forceinline__ float softmax_term(float l, float top) {
    if (l == top) return l == -kInf ? 0.0f : 1.0f;
    return expf(l - top);
}
__device__ __forceinline__ double softmax_term64(float l, float top) {
    if (l == top) return l == -kInf ? 0.0 : 1.0;
    return exp(static_cast<double>(l) - static_cast<double>(top));
}

// sigmoid(l) * exp(-low), low = min(0, largest chosen logit): numerator and
// denominator stay normal numbers where sigmoid itself would underflow.
__device__ __forceinline__ float sigmoid_over(float l, float low) {
    if (l == -kInf) return 0.0f;
    return expf(fminf(l, 0.0f) - low) / (1.0f + expf(-fabsf(l)));
}
__device__ __forceinline__ float sigmoid(float l) { return sigmoid_over(l, 0.0f); }
__device__ __forceinline__ double sigmoid64(float l) {
    return 1.0 / (1.0 + exp(-static_cast<double>(l)));
}

// Choice and expert in one 64-bit key: larger choices first, and of equal
// choices the lower expert.  0: unavailable.  -0 counts as 0.
__device__ __forceinline__ uint64_t make_key(float choice, int e) {
    if (!(choice > -kInf)) return 0;
    const uint32_t u = __float_as_uint(choice + 0.0f);
    const uint32_t ordered = u & 0x80000000u ? ~u : u | 0x80000000u;
    return static_cast<uint64_t>(ordered) << 16 | static_cast<uint64_t>(0xFFFF - e);
}
__device__ __forceinline__ int key_expert(uint64_t key) { return 0xFFFF - static_cast<int>(key & 0xFFFF); }

template <int L>
__device__ __forceinline__ uint64_t max_key_over(uint64_t v) {
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) {
        const uint64_t o = static_cast<uint64_t>(__shfl_xor(static_cast<unsigned long long>(v), d));
        v = o > v ? o : v;
    }
    return v;
}

template <typename In, int L, int C>
__global__ __launch_bounds__(kWaves* kWave) void route_kernel(const typename In::raw* __restrict__ logits,
                                                              const float* __restrict__ bias, int64_t T,
                                                              int E, int k, RouteOptions opt,
                                                              int64_t* __restrict__ topk_idx,
                                                              float* __restrict__ topk_weights) {
    constexpr int kTokens = kWave / L;
    extern __shared__ float choices[];              // [kWaves * kTokens][E], groups only
    const int lane = lane_id(), pos = lane % L, sub = lane / L;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    const bool by_choice = bias || (opt.num_groups > 1 && opt.group_top == 2);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWaves * kTokens;
    for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * kTokens; t0 < T; t0 += step) {
        const bool live = t0 + sub < T;
        const int64_t t = live ? t0 + sub : T - 1;  // lanes past the end repeat the last token
        float l[C];
        float top = -kInf;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = c * L + pos;
            l[c] = e < E ? logit<In>(logits + t * E + e) : -kInf;
            top = fmaxf(top, l[c]);
        }
        top = max_over<L>(top);

        float choice[C];
        if (by_choice) {
            double total = 1.0;
            if (!opt.sigmoid) {
                total = 0.0;
#pragma unroll
                for (int c = 0; c < C; ++c) total += softmax_term64(l[c], top);
                total = sum_over<L>(total);
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int e = c * L + pos;
                const double s = opt.sigmoid ? sigmoid64(l[c]) : softmax_term64(l[c], top) / total;
                const float b = bias && e < E ? bias[e] : 0.0f;
                choice[c] = l[c] > -kInf ? static_cast<float>(s) + b : -kInf;
            }
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) choice[c] = l[c];
        }

        uint64_t kept = ~uint64_t(0);
        if (opt.num_groups > 1) {
            float* row = choices + (wave * kTokens + sub) * E;
            const int size = E / opt.num_groups;
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (c * L + pos < E) row[c * L + pos] = choice[c];
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            // Every lane scores the groups g = pos, pos + L, ...; of two NaN-free
            // bests the second counts only if it is available.
            float* score = row;                     // overwritten below, group by group
            kept = 0;
            float mine[kWave / L];
#pragma unroll
            for (int i = 0; i < kWave / L; ++i) {
                const int g = i * L + pos;
                float first = -kInf, second = -kInf;
                if (g < opt.num_groups)
                    for (int u = 0; u < size; ++u) {
                        const float v = row[g * size + u];
                        if (v > first) {
                            second = first;
                            first = v;
                        } else if (v > second) {
                            second = v;
                        }
                    }
                mine[i] = first;
                if (opt.group_top == 2 && second > -kInf) mine[i] = first + second;
            }
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < kWave / L; ++i)
                if (i * L + pos < opt.num_groups) score[i * L + pos] = mine[i];
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            for (int g = 0; g < opt.num_groups; ++g) {
                const float v = score[g];
                int better = 0;
                for (int o = 0; o < opt.num_groups; ++o)
                    better += score[o] > v || (score[o] == v && o < g);
                if (better < opt.topk_groups) kept |= uint64_t(1) << g;
            }
            __builtin_amdgcn_wave_barrier();
        }

        uint64_t key[C];
        const int size = E / opt.num_groups;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = c * L + pos;
            key[c] = e < E && (kept >> (e / size) & 1) ? make_key(choice[c], e) : 0;
        }
        // k rounds: the largest key of the token's lanes goes to lane j.
        uint64_t won = 0;
        for (int j = 0; j < k; ++j) {
            uint64_t best = 0;
#pragma unroll
            for (int c = 0; c < C; ++c) best = key[c] > best ? key[c] : best;
            best = max_key_over<L>(best);
            if (pos == j) won = best;
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (key[c] == best) key[c] = 0;
        }

        const bool filled = pos < k && won != 0;
        const int e = filled ? key_expert(won) : -1;
        const float le = filled ? logit<In>(logits + t * E + e) : -kInf;
        float a, total = 1.0f;
        if (opt.sigmoid) {
            const float low = opt.renormalize ? fminf(max_over<L>(le), 0.0f) : 0.0f;
            a = sigmoid_over(le, low);
        } else {
            const float m = opt.renormalize ? max_over<L>(le) : top;
            a = softmax_term(le, m);
            if (!opt.renormalize) {
                total = 0.0f;
#pragma unroll
                for (int c = 0; c < C; ++c) total += softmax_term(l[c], top);
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

// One wave per token: lane j takes slot j, the slots' contributions meet in a
// row of the block's memory, and the whole wave writes the row out.
template <typename In>
__global__ __launch_bounds__(kWaves* kWave) void route_backward_kernel(
    const typename In::raw* __restrict__ logits, const int64_t* __restrict__ topk_idx,
    const float* __restrict__ grad_weights, int64_t T, int E, int k, bool is_sigmoid, bool renormalize,
    float scale, typename In::raw* __restrict__ grad_logits) {
    extern __shared__ float rows[];                 // [kWaves][E]
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
    float* row = rows + wave * E;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWaves;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWaves + wave; t < T; t += step) {
        const typename In::raw* in = logits + t * E;
        int e = -1;
        float g = 0.0f, l = -kInf;
        if (lane < k) {
            const int64_t id = topk_idx[t * k + lane];
            if (id >= 0 && id < E) {
                e = static_cast<int>(id);
                g = grad_weights[t * k + lane];
                l = logit<In>(in + e);
            }
        }
        const bool dense = !is_sigmoid && !renormalize;
        float top = -kInf, total = 0.0f;
        if (dense) {
            for (int i = lane; i < E; i += kWave) top = fmaxf(top, logit<In>(in + i));
            top = max_over<kWave>(top);
            for (int i = lane; i < E; i += kWave) total += softmax_term(logit<In>(in + i), top);
            total = sum_over<kWave>(total);
        }
        float d, mean = 0.0f;                       // this slot's contribution
        if (l == -kInf) g = 0.0f;                   // unavailable: no score, no gradient
        if (dense) {
            const float s = total > 0.0f ? softmax_term(l, top) / total : 0.0f;
            mean = sum_over<kWave>(g * s);
            d = g;
        } else if (renormalize) {
            const float m = max_over<kWave>(l);
            const float a = is_sigmoid ? sigmoid_over(l, fminf(m, 0.0f)) : softmax_term(l, m);
            const float sum = sum_over<kWave>(a);
            const float p = sum > 0.0f ? a / sum : 0.0f;
            mean = sum_over<kWave>(g * p);
            d = p * (g - mean);
            if (is_sigmoid) d *= sigmoid(-l);
        } else {
            d = g * sigmoid(l) * sigmoid(-l);
        }
        // Slots of the same expert add in slot order, whichever lane writes.
        float all = 0.0f;
        for (int j = 0; j < k; ++j)
            if (read_lane(e, j) == e) all += read_lane(d, j);
        for (int i = lane; i < E; i += kWave) row[i] = 0.0f;
        __builtin_amdgcn_wave_barrier();
        if (e >= 0 && l > -kInf) row[e] = all;
        __builtin_amdgcn_wave_barrier();
        for (int i = lane; i < E; i += kWave) {
            float v = row[i];
            if (dense) {
                const float s = total > 0.0f ? softmax_term(logit<In>(in + i), top) / total : 0.0f;
                v = s * (v - mean);
            }
            grad_logits[t * E + i] = from_float(In(), scale * v);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <typename In, int L, int C>
hipError_t launch_lc(const void* logits, const float* bias, int64_t T, int E, int k, const RouteOptions& opt,
                     int64_t* topk_idx, float* topk_weights, hipStream_t stream) {
    const int per_block = kWaves * (kWave / L);
    const int64_t blocks = ceil_div(T, per_block), cap = kMaxLaunchThreads / (kWaves * kWave);
    const size_t lds = opt.num_groups > 1 ? sizeof(float) * per_block * E : 0;
    hipLaunchKernelGGL((route_kernel<In, L, C>), dim3(static_cast<unsigned>(blocks < cap ? blocks : cap)),
                       dim3(kWaves * kWave), lds, stream, static_cast<const typename In::raw*>(logits), bias, T, E,
                       k, opt, topk_idx, topk_weights);
    return hipGetLastError();
}

template <typename In>
hipError_t launch_type(const void* logits, const float* bias, int64_t T, int E, int k, const RouteOptions& opt,
                       int64_t* topk_idx, float* topk_weights, hipStream_t stream) {
    if (E <= 64) return launch_lc<In, 64, 1>(logits, bias, T, E, k, opt, topk_idx, topk_weights, stream);
    if (E <= 256) return launch_lc<In, 64, 4>(logits, bias, T, E, k, opt, topk_idx, topk_weights, stream);
    if (E <= 512) return launch_lc<In, 64, 8>(logits, bias, T, E, k, opt, topk_idx, topk_weights, stream);
    return launch_lc<In, 64, 32>(logits, bias, T, E, k, opt, topk_idx, topk_weights, stream);
}

template <typename In>
hipError_t launch_back(const void* logits, const int64_t* topk_idx, const float* grad_weights, int64_t T, int E,
                       int k, bool is_sigmoid, bool renormalize, float scale, void* grad_logits,
                       hipStream_t stream) {
    const int64_t blocks = ceil_div(T, kWaves), cap = kMaxLaunchThreads / (kWaves * kWave);
    hipLaunchKernelGGL((route_backward_kernel<In>), dim3(static_cast<unsigned>(blocks < cap ? blocks : cap)),
                       dim3(kWaves * kWave), sizeof(float) * kWaves * E, stream,
                       static_cast<const typename In::raw*>(logits), topk_idx, grad_weights, T, E, k, is_sigmoid,
                       renormalize, scale, static_cast<typename In::raw*>(grad_logits));
    return hipGetLastError();
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
