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
//
// The launch bounds small calls, instructions the large ones.  Up to 12 picks
// four tokens share a wave, 16 lanes each: the k-th largest of the lanes' maxima
// bounds the k-th largest key from below, so the keys from there on are a short
// list, and an expert's place is the number of listed keys before it.  With a
// wave to a token and one reduction to a pick, 65536 tokens x 288 experts (float32,
// sigmoid with a bias) took 140 us; this form takes 36: 80 MB, 2.2 TB/s (288
// sigmoids a token, and keys in 64 bits for those listed).  32 tokens x 256
// experts: 7 us a call, of which 4 to 5 in the kernel.  Gradient, 16384 tokens x
// 128 experts, bf16: 5.4 us in the kernel, 9.4 MB.
#include <type_traits>

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

// One token with a whole wave, one pick after the other: the form that takes
// any k and any number of equal keys.  Lane l holds experts l, l + 64, ...: PER
// of them.
template <typename T, int PER>
__device__ __forceinline__ void gate_token(const GatingArgs& a, int64_t t) {
    const int lane = threadIdx.x & 63;
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
__global__ __launch_bounds__(kThreads) void topk_gating_wave_kernel(GatingArgs a) {
    const int64_t t = (int64_t)blockIdx.x * kTokens + (threadIdx.x >> 6);
    if (t < a.num_tokens) gate_token<T, PER>(a, t);
}

// ---- four tokens to a wave, for few picks ------------------------------------
// 16 lanes hold a token's logits, 4 NC each.  The k-th largest of their 16
// maxima is a bound that at least k experts reach, and few more do: about 16 (1/16
// + ... + 1/(17 - k)), 13 of 288 for k = 8.  Those are put into a list in LDS,
// and each counts the list's larger keys, which is its place.  So no pick waits
// for the one before, and with a bias only the listed keys are computed in
// float64.  A list of more than kList goes through gate_token.
constexpr int kRowTopk = 12;
constexpr int kList = 32;

template <int Ctrl>
__device__ __forceinline__ float dpp_f(float v) {
    return __int_as_float(dpp<Ctrl>(__float_as_int(v)));
}
__device__ __forceinline__ float row_max(float v) {
    v = fmaxf(v, dpp_f<0xb1>(v));
    v = fmaxf(v, dpp_f<0x4e>(v));
    v = fmaxf(v, dpp_f<0x141>(v));
    return fmaxf(v, dpp_f<0x140>(v));
}
__device__ __forceinline__ float row_min(float v) { return -row_max(-v); }
__device__ __forceinline__ float row_sum(float v) {
    v += dpp_f<0xb1>(v);
    v += dpp_f<0x4e>(v);
    v += dpp_f<0x141>(v);
    return v + dpp_f<0x140>(v);
}
// How many of a row's 16 values are larger than the lane's.
template <int N = 15>
__device__ __forceinline__ int row_larger(float v) {
    const int here = dpp_f<0x120 + N>(v) > v ? 1 : 0;       // row_ror:N
    if constexpr (N > 1) return here + row_larger<N - 1>(v);
    return here;
}
// Sum of the lanes below in the row.
__device__ __forceinline__ int row_before(int v) {
    int s = v;
    s += dpp<0x111>(s);
    s += dpp<0x112>(s);
    s += dpp<0x114>(s);
    s += dpp<0x118>(s);
    return s - v;
}

template <typename T, int NC>
__global__ __launch_bounds__(kThreads, NC <= 5 ? 4 : NC <= 8 ? 3 : 2) void topk_gating_kernel(
    GatingArgs a, bool vec, bool vec_bias) {
    struct Entry { float x; int32_t id; };
    __shared__ Entry list[kThreads / 16][kList];
    __shared__ double keys[kThreads / 16][kList];
    const int lane = threadIdx.x & 63, l = lane & 15, row = threadIdx.x >> 4;
    const int64_t t = (int64_t)blockIdx.x * (kThreads / 16) + row;
    const bool live = t < a.num_tokens;
    const int E = a.num_experts;
    using S = typename T::storage;
    struct alignas(4 * sizeof(S)) Four { S v[4]; };
    // Keys in float32 of experts (16 c + l) 4 + i: the logits, or with a bias
    // values within 2^-21 max(1, |key|) of the float64 ones (the exponential's and
    // the quotient's few roundings).
    float key[NC][4], mine = -kInf, all_sum = 0.0f;
    const S* logits = static_cast<const S*>(a.logits) + t * E;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int e = (c * 16 + l) * 4;
        if (vec && live && e < E && MX_CAN_LOAD(logits + e, sizeof(Four), kSiteTopkLoad)) {
            const Four f = *reinterpret_cast<const Four*>(logits + e);
#pragma unroll
            for (int i = 0; i < 4; ++i) key[c][i] = to_f32(T{}, f.v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                key[c][i] = !vec && live && e + i < E ? logit<T>(a.logits, t * E + e + i) : -kInf;
        }
    }
    if (a.bias != nullptr) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int e = (c * 16 + l) * 4;
            struct alignas(16) Four32 { float v[4]; };
            Four32 b{};
            if (vec_bias) {
                if (e < E && MX_CAN_LOAD(a.bias + e, 16, kSiteTopkLoad))
                    b = *reinterpret_cast<const Four32*>(a.bias + e);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (e + i < E && MX_CAN_LOAD(a.bias + e + i, 4, kSiteTopkLoad))
                        b.v[i] = a.bias[e + i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = key[c][i], k = __builtin_amdgcn_rcpf(1.0f + __expf(-x)) + b.v[i];
                key[c][i] = x > -kInf ? k : -kInf;
            }
        }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            key[c][i] = fmaxf(key[c][i], -kInf);               // NaN becomes -inf
            mine = fmaxf(mine, key[c][i]);
        }
    const float most = row_max(mine);
    if (!a.sigmoid && !a.renormalize) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (key[c][i] > -kInf) all_sum += exp_below(key[c][i], most);
        all_sum = row_sum(all_sum);
    }
    float bound = row_min(row_larger(mine) < a.topk ? mine : kInf);
    if (a.bias != nullptr && bound > -kInf && bound < kInf)
        bound -= 0x1p-19f * fmaxf(1.0f, fabsf(bound));      // twice the keys' error, and more
    bound = fmaxf(bound, -3.402823466e38f);                 // of finite keys the lowest
    int n = 0;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) n += key[c][i] >= bound ? 1 : 0;
    int at = row_before(n);
    const int count = __builtin_amdgcn_ds_bpermute((lane | 15) * 4, at + n);
    if (__ballot(count > kList) != 0) {
        const int64_t t0 = t - (lane >> 4);
        for (int r = 0; r < 4; ++r)
            if (t0 + r < a.num_tokens) gate_token<T, NC>(a, t0 + r);
        return;
    }
    // unused entries lose against every other
    list[row][l] = list[row][l + 16] = Entry{-kInf, 0x7fffffff};
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (key[c][i] >= bound)
                list[row][at++] = Entry{key[c][i], (c * 16 + l) * 4 + i};
    // lane l takes entries l and l + 16
    const bool two = __ballot(count > 16) != 0;
    Entry my[2] = {list[row][l], list[row][l + 16]};
    int rank[2] = {0, 0};
    if (a.bias != nullptr) {
        double exact[2] = {-(double)kInf, -(double)kInf};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h == 1 && !two) break;
            if (l + 16 * h < count) {
                const float b = MX_CAN_LOAD(a.bias + my[h].id, 4, kSiteTopkLoad)
                                    ? a.bias[my[h].id] : 0.0f;
                my[h].x = logit<T>(a.logits, t * E + my[h].id);
                exact[h] = 1.0 / (1.0 + exp(-(double)my[h].x)) + (double)b;
            }
            keys[row][l + 16 * h] = exact[h];
        }
        auto count_larger = [&](int h, int first) {
#pragma unroll
            for (int j = first; j < first + 16; ++j) {
                const double k = keys[row][j];
                rank[h] += k > exact[h] || (k == exact[h] && list[row][j].id < my[h].id) ? 1 : 0;
            }
        };
        count_larger(0, 0);
        if (two) {
            count_larger(0, 16);
            count_larger(1, 0);
            count_larger(1, 16);
        }
    } else {
        auto count_larger = [&](int h, int first) {
#pragma unroll
            for (int j = first; j < first + 16; ++j) {
                const Entry o = list[row][j];
                rank[h] += o.x > my[h].x || (o.x == my[h].x && o.id < my[h].id) ? 1 : 0;
            }
        };
        count_larger(0, 0);
        if (two) {
            count_larger(0, 16);
            count_larger(1, 0);
            count_larger(1, 16);
        }
    }
    float p[2], total = 0.0f;
    bool chosen[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        chosen[h] = l + 16 * h < count && rank[h] < a.topk;
        p[h] = !chosen[h] ? 0.0f : a.sigmoid ? sigmoid(my[h].x) : exp_below(my[h].x, most);
        total += p[h];
    }
    total = row_sum(total);
    if (!a.renormalize) total = a.sigmoid ? 1.0f : all_sum;
    if (!live) return;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (chosen[h]) {
            int32_t* id = a.ids + t * a.topk + rank[h];
            float* w = a.weights + t * a.topk + rank[h];
            if (MX_CAN_STORE(id, 4, kSiteTopkOut)) *id = my[h].id;
            if (MX_CAN_STORE(w, 4, kSiteTopkOut))
                *w = total > 0.0f ? a.scale * (p[h] / total) : 0.0f;
        }
    if (l >= count && l < a.topk) {
        int32_t* id = a.ids + t * a.topk + l;
        float* w = a.weights + t * a.topk + l;
        if (MX_CAN_STORE(id, 4, kSiteTopkOut)) *id = -1;
        if (MX_CAN_STORE(w, 4, kSiteTopkOut)) *w = 0.0f;
    }
}

// One token with a whole wave, for any k.
template <typename T, int PER>
__global__ __launch_bounds__(kThreads) void topk_gating_backward_wave_kernel(GatingArgs a) {
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

// The gradient with four tokens to a wave, for up to 16 picks: lane l of a
// token's 16 holds pick l and writes experts (16 c + l) 4 + i.
template <int J, int N, typename F>
__device__ __forceinline__ void for_each_pick(F&& f) {
    if constexpr (J < N) {
        f(std::integral_constant<int, J>{});
        for_each_pick<J + 1, N>(f);
    }
}

template <typename T, int NC>
__global__ __launch_bounds__(kThreads) void topk_gating_backward_kernel(GatingArgs a, bool vec) {
    const int l = threadIdx.x & 15;
    const int64_t t = (int64_t)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);
    const bool here = t < a.num_tokens;
    const int E = a.num_experts;
    using S = typename T::storage;
    struct alignas(4 * sizeof(S)) Four { S v[4]; };
    int id = -1;
    float g = 0.0f, px = -kInf;
    if (here && l < a.topk) {
        const int32_t* ip = a.ids + t * a.topk + l;
        const float* gp = a.weights + t * a.topk + l;
        if (MX_CAN_LOAD(ip, 4, kSiteTopkLoad)) id = *ip;
        if (MX_CAN_LOAD(gp, 4, kSiteTopkLoad)) g = *gp;
        if (id >= 0 && id < E) px = logit<T>(a.logits, t * E + id);
    }
    const bool live = px > -kInf;                           // not NaN either
    if (!live) {
        id = -1;
        g = 0.0f;
        px = -kInf;
    }
    const bool rest = !a.sigmoid && !a.renormalize;         // every expert has a gradient
    float x[NC][4], most = px, sum, d;
    if (rest) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = (c * 16 + l) * 4 + i;
                x[c][i] = here && e < E ? logit<T>(a.logits, t * E + e) : -kInf;
                x[c][i] = fmaxf(x[c][i], -kInf);            // NaN becomes -inf
                most = fmaxf(most, x[c][i]);
            }
    }
    most = row_max(most);
    if (a.sigmoid) {
        const float s = live ? sigmoid(px) : 0.0f;
        float ds = g;
        if (a.renormalize) {
            const float total = row_sum(s);
            const float dot = row_sum(total > 0.0f ? s / total * g : 0.0f);
            ds = total > 0.0f ? (g - dot) / total : 0.0f;
        }
        d = live ? a.scale * ds * s * (1.0f - s) : 0.0f;
        sum = 0.0f;
    } else {
        sum = live ? exp_below(px, most) : 0.0f;
        if (rest) {
            sum = 0.0f;
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) sum += x[c][i] > -kInf ? exp_below(x[c][i], most) : 0.0f;
        }
        sum = row_sum(sum);
        const float p = live ? exp_below(px, most) / sum : 0.0f;
        const float dot = row_sum(p * g);
        d = live ? a.scale * p * (rest ? g : g - dot) : 0.0f;
        if (rest) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[c][i] = x[c][i] > -kInf
                                  ? -a.scale * (exp_below(x[c][i], most) / sum) * dot : 0.0f;
        }
    }
    if (!rest) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[c][i] = 0.0f;
    }
    // one pick after the other, in order: row_newbcast gives the row its lane
    for_each_pick<0, 16>([&](auto j) {
        if (decltype(j)::value >= a.topk) return;
        const int at = dpp<0x150 + decltype(j)::value>(id);
        const float v = dpp_f<0x150 + decltype(j)::value>(d);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (at == (c * 16 + l) * 4 + i) x[c][i] += v;
    });
    if (!here) return;
    S* row = static_cast<S*>(a.grad_logits) + t * E;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int e = (c * 16 + l) * 4;
        if (vec) {
            Four f;
#pragma unroll
            for (int i = 0; i < 4; ++i) f.v[i] = from_f32(T{}, x[c][i]);
            if (e < E && MX_CAN_STORE(row + e, sizeof(Four), kSiteTopkOut))
                *reinterpret_cast<Four*>(row + e) = f;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (e + i < E && MX_CAN_STORE(row + e + i, sizeof(S), kSiteTopkOut))
                    row[e + i] = from_f32(T{}, x[c][i]);
        }
    }
}

// go(arguments, workgroups) for batches of tokens, `per_group` to a workgroup.
template <typename T, typename F>
hipError_t for_token_batches(const GatingArgs& a, int per_group, F&& go) {
    for (int64_t t0 = 0; t0 < a.num_tokens; t0 += kTokensPerLaunch) {
        GatingArgs b = a;
        b.num_tokens = a.num_tokens - t0 < kTokensPerLaunch ? a.num_tokens - t0 : kTokensPerLaunch;
        const int64_t row = t0 * a.num_experts * (int64_t)sizeof(typename T::storage);
        b.logits = static_cast<const uint8_t*>(a.logits) + row;
        if (a.grad_logits != nullptr) b.grad_logits = static_cast<uint8_t*>(a.grad_logits) + row;
        b.ids = a.ids + t0 * a.topk;
        b.weights = a.weights + t0 * a.topk;
        go(b, dim3((unsigned)((b.num_tokens + per_group - 1) / per_group)));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// The kernel for lanes that hold n = 1, 2, ... 64ths of the experts.
#define MX_PER_LANE(go) \
    if (per <= 1) return go(std::integral_constant<int, 1>{}); \
    if (per <= 2) return go(std::integral_constant<int, 2>{}); \
    if (per <= 4) return go(std::integral_constant<int, 4>{}); \
    if (per <= 5) return go(std::integral_constant<int, 5>{}); \
    if (per <= 8) return go(std::integral_constant<int, 8>{}); \
    return go(std::integral_constant<int, 16>{});

template <typename T>
hipError_t start(const GatingArgs& a, hipStream_t stream) {
    const int per = (a.num_experts + kWave - 1) / kWave;
    const bool rows = a.topk <= kRowTopk;
    const bool vec = a.num_experts % 4 == 0 &&
                     (uintptr_t)a.logits % (4 * sizeof(typename T::storage)) == 0;
    auto go = [&](auto n) {
        return for_token_batches<T>(a, rows ? kThreads / 16 : kTokens, [&](const GatingArgs& b,
                                                                         dim3 grid) {
            if (rows)
                launch_kernel(topk_gating_kernel<T, decltype(n)::value>, grid, dim3(kThreads), 0,
                              stream, nullptr, nullptr, b, vec, vec && (uintptr_t)a.bias % 16 == 0);
            else
                launch_kernel(topk_gating_wave_kernel<T, decltype(n)::value>, grid,
                              dim3(kThreads), 0, stream, nullptr, nullptr, b);
        });
    };
    MX_PER_LANE(go)
}

template <typename T>
hipError_t start_backward(const GatingArgs& a, hipStream_t stream) {
    const int per = (a.num_experts + kWave - 1) / kWave;
    const bool rows = a.topk <= 16;
    const bool vec = a.num_experts % 4 == 0 &&
                     (uintptr_t)a.grad_logits % (4 * sizeof(typename T::storage)) == 0;
    auto go = [&](auto n) {
        return for_token_batches<T>(a, rows ? kThreads / 16 : kTokens, [&](const GatingArgs& b,
                                                                         dim3 grid) {
            if (rows)
                launch_kernel(topk_gating_backward_kernel<T, decltype(n)::value>, grid,
                              dim3(kThreads), 0, stream, nullptr, nullptr, b, vec);
            else
                launch_kernel(topk_gating_backward_wave_kernel<T, decltype(n)::value>, grid,
                              dim3(kThreads), 0, stream, nullptr, nullptr, b);
        });
    };
    MX_PER_LANE(go)
}

}  // namespace

hipError_t launch_topk_gating(const GatingArgs& a, hipStream_t stream) {
    if (a.dtype == 0) return start<F32>(a, stream);
    if (a.dtype == 1) return start<F16>(a, stream);
    return start<BF16>(a, stream);
}

hipError_t launch_topk_gating_backward(const GatingArgs& a, hipStream_t stream) {
    if (a.dtype == 0) return start_backward<F32>(a, stream);
    if (a.dtype == 1) return start_backward<F16>(a, stream);
    return start_backward<BF16>(a, stream);
}

}  // namespace mxmoe
