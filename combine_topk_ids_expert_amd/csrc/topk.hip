// Top-k gating: from a token's router logits l [E] to its k experts and their
// weights, and the gradient of the weights.
//
//   key_e   = l_e, or sigmoid(l_e) + bias_e in float64 (only the selection
//             sees the bias, and two experts' keys may lie closer than
//             float32 resolves)
//   ids     = the k largest keys, largest first, equal ones by lower index;
//             experts whose key is NaN or -inf are never chosen, and the
//             places left over hold -1 and weight 0
//   softmax: p = exp(l - max l) / sum, over the chosen (renormalize) or all
//            experts that could be chosen
//   sigmoid: p = sigmoid(l), divided by the chosen ones' sum (renormalize)
//   weights = scale * p
//
// Gradient for given ids, g = dL/dweights, per chosen pick j (an id outside
// [0, E) is left out; an id given twice counts as two picks):
//   softmax, renormalized:  dl_{id_j} += scale p_j (g_j - sum_i p_i g_i)
//   softmax over all:       dl_e = scale p_e ([e chosen] g_e - sum_i p_i g_i)
//   sigmoid, renormalized:  ds_j = scale (g_j - sum_i w_i g_i) / sum s
//   sigmoid:                ds_j = scale g_j;   dl = ds s (1 - s)
#include "device_common.h"
#include "launch.h"

namespace mxmoe {
namespace {

constexpr int kThreads = 256;                 // one wave per token
constexpr int kTokens = kThreads / kWave;
// Tokens of one launch: 2^31 work-items at most.
constexpr int64_t kTokensPerLaunch = (int64_t)1 << 25;
constexpr float kInf = __builtin_inff();

template <typename T>
__device__ __forceinline__ float logit(const void* p, int64_t at) {
    const typename T::storage* q = static_cast<const typename T::storage*>(p) + at;
    if (!MX_CAN_LOAD(q, sizeof(*q), kSiteTopkLoad)) return -kInf;
    return to_f32(T{}, *q);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
    return v;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) v = fmaxf(v, __shfl_xor(v, d, kWave));
    return v;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// exp(x - m), 1 where both are the same infinity.
__device__ __forceinline__ float exp_below(float x, float m) {
    return x == m ? 1.0f : expf(x - m);
}

// Lane l holds experts l, l + 64, ...: PER of them.
template <typename T, int PER>
__global__ __launch_bounds__(kThreads) void topk_gating_kernel(GatingArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * kTokens + (threadIdx.x >> 6);
    if (t >= a.num_tokens) return;
    const int E = a.num_experts;
    float x[PER];
    double key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * kWave + lane;
        x[i] = e < E ? logit<T>(a.logits, t * E + e) : -kInf;
        if (x[i] != x[i]) x[i] = -kInf;
        key[i] = (double)x[i];
        if (a.bias != nullptr && x[i] > -kInf) {
            const float b = MX_CAN_LOAD(a.bias + e, 4, kSiteTopkLoad) ? a.bias[e] : 0.0f;
            key[i] = 1.0 / (1.0 + exp(-(double)x[i])) + (double)b;
            if (!(key[i] > -(double)kInf)) {
                key[i] = -(double)kInf;
                x[i] = -kInf;
            }
        }
    }
    float all_max = -kInf;
#pragma unroll
    for (int i = 0; i < PER; ++i) all_max = fmaxf(all_max, x[i]);
    all_max = wave_max(all_max);
    float all_sum = 0.0f;
    if (!a.sigmoid && !a.renormalize) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (x[i] > -kInf) all_sum += exp_below(x[i], all_max);
        all_sum = wave_sum(all_sum);
    }
    int my_id = -1;                            // lane j keeps pick j
    float my_x = -kInf;
    for (int j = 0; j < a.topk; ++j) {
        double best = -(double)kInf;
        int at = 0x7fffffff;
        float bx = -kInf;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i * kWave + lane;
                bx = x[i];
            }
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const double ob = __shfl_xor(best, d, kWave);
            const int oa = __shfl_xor(at, d, kWave);
            const float ox = __shfl_xor(bx, d, kWave);
            if (ob > best || (ob == best && oa < at)) {
                best = ob;
                at = oa;
                bx = ox;
            }
        }
        if (!(best > -(double)kInf)) break;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (at == i * kWave + lane) key[i] = -(double)kInf;
        if (lane == j) {
            my_id = at;
            my_x = bx;
        }
    }
    float p = 0.0f;
    if (my_id >= 0) p = a.sigmoid ? sigmoid(my_x) : exp_below(my_x, all_max);
    float total = 1.0f;
    if (a.renormalize) total = wave_sum(p);
    else if (!a.sigmoid) total = all_sum;
    if (lane < a.topk) {
        int32_t* id = a.ids + t * a.topk + lane;
        float* w = a.weights + t * a.topk + lane;
        if (MX_CAN_STORE(id, 4, kSiteTopkOut)) *id = my_id;
        if (MX_CAN_STORE(w, 4, kSiteTopkOut)) *w = total > 0.0f ? a.scale * (p / total) : 0.0f;
    }
}

template <typename T, int PER>
__global__ __launch_bounds__(kThreads) void topk_gating_backward_kernel(GatingArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * kTokens + (threadIdx.x >> 6);
    if (t >= a.num_tokens) return;
    const int E = a.num_experts;
    float x[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * kWave + lane;
        x[i] = e < E ? logit<T>(a.logits, t * E + e) : -kInf;
        if (x[i] != x[i]) x[i] = -kInf;
    }
    // lane j holds pick j
    int id = -1;
    float g = 0.0f, px = -kInf;
    if (lane < a.topk) {
        const int32_t* ip = a.ids + t * a.topk + lane;
        const float* gp = a.weights + t * a.topk + lane;
        if (MX_CAN_LOAD(ip, 4, kSiteTopkLoad)) id = *ip;
        if (MX_CAN_LOAD(gp, 4, kSiteTopkLoad)) g = *gp;
        if (id < 0 || id >= E) id = -1;
        if (id >= 0) {
            px = logit<T>(a.logits, t * E + id);
            if (!(px > -kInf)) id = -1;
        }
        if (id < 0) g = 0.0f;
    }
    const bool live = id >= 0;
    float d = 0.0f, dot = 0.0f, all_max = -kInf, all_sum = 0.0f;
    if (a.sigmoid) {
        const float s = live ? sigmoid(px) : 0.0f;
        float ds = g;
        if (a.renormalize) {
            const float total = wave_sum(s);
            dot = wave_sum(total > 0.0f ? s / total * g : 0.0f);
            ds = total > 0.0f ? (g - dot) / total : 0.0f;
        }
        d = live ? a.scale * ds * s * (1.0f - s) : 0.0f;
    } else {
        if (a.renormalize) {
            all_max = wave_max(live ? px : -kInf);
            all_sum = wave_sum(live ? exp_below(px, all_max) : 0.0f);
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) all_max = fmaxf(all_max, x[i]);
            all_max = wave_max(all_max);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (x[i] > -kInf) all_sum += exp_below(x[i], all_max);
            all_sum = wave_sum(all_sum);
        }
        const float p = live ? exp_below(px, all_max) / all_sum : 0.0f;
        dot = wave_sum(p * g);
        d = live ? a.scale * p * (a.renormalize ? g - dot : g) : 0.0f;
    }
    const bool rest = !a.sigmoid && !a.renormalize;
    float out[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        out[i] = rest && x[i] > -kInf
                     ? -a.scale * (exp_below(x[i], all_max) / all_sum) * dot : 0.0f;
    for (int j = 0; j < a.topk; ++j) {
        const int at = __builtin_amdgcn_readlane(id, j);
        const float v = __uint_as_float(
            (uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(d), j));
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (at == i * kWave + lane) out[i] += v;
    }
    typename T::storage* row = static_cast<typename T::storage*>(a.grad_logits) + t * E;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * kWave + lane;
        if (e < E && MX_CAN_STORE(row + e, sizeof(*row), kSiteTopkOut))
            row[e] = from_f32(T{}, out[i]);
    }
}

template <typename T, bool Backward>
hipError_t start(const GatingArgs& a, hipStream_t stream) {
    auto go = [&](auto kernel) {
        for (int64_t t0 = 0; t0 < a.num_tokens; t0 += kTokensPerLaunch) {
            GatingArgs b = a;
            b.num_tokens = a.num_tokens - t0 < kTokensPerLaunch ? a.num_tokens - t0 : kTokensPerLaunch;
            const int64_t row = t0 * a.num_experts * (int64_t)sizeof(typename T::storage);
            b.logits = static_cast<const uint8_t*>(a.logits) + row;
            if (Backward) b.grad_logits = static_cast<uint8_t*>(a.grad_logits) + row;
            b.ids = a.ids + t0 * a.topk;
            b.weights = a.weights + t0 * a.topk;
            const dim3 grid((unsigned)((b.num_tokens + kTokens - 1) / kTokens));
            launch_kernel(kernel, grid, dim3(kThreads), 0, stream, nullptr, nullptr, b);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        return hipSuccess;
    };
    const int per = (a.num_experts + kWave - 1) / kWave;
#define MX_PER(n) \
    if (per <= n) return Backward ? go(topk_gating_backward_kernel<T, n>) : go(topk_gating_kernel<T, n>);
    MX_PER(1) MX_PER(2) MX_PER(4) MX_PER(5) MX_PER(8) MX_PER(16)
#undef MX_PER
    return hipErrorInvalidValue;
}

template <bool Backward>
hipError_t start(const GatingArgs& a, hipStream_t stream) {
    if (a.dtype == 0) return start<F32, Backward>(a, stream);
    if (a.dtype == 1) return start<F16, Backward>(a, stream);
    return start<BF16, Backward>(a, stream);
}

}  // namespace

hipError_t launch_topk_gating(const GatingArgs& a, hipStream_t stream) {
    return start<false>(a, stream);
}

hipError_t launch_topk_gating_backward(const GatingArgs& a, hipStream_t stream) {
    return start<true>(a, stream);
}

}  // namespace mxmoe
