// Products of few rows with their expert's weights, for decoding: the weights
// pass once from HBM through registers to the matrix cores, with nothing in
// between, so that their bytes are the time.
//
//   out[r][n] = sum_k x[r][k] w[e][n][k]
//
// with w either of x's 16-bit type or 4 bits with one scale (and zero point)
// per `group` positions:  w = (q - z) s.  For those,
//
//   sum_{k in G} (q - z) x = sum_k (B + q) x - (B + z) sum_k x,
//
// where B + q is the 16-bit number whose low mantissa bits are q (B = 128 in
// bf16, 1024 in fp16): one AND-OR makes two of them, every B + q is exact,
// and the sum of x comes from one more matrix instruction against ones.  Both
// sums and their difference are float32: the difference loses log2(B / 4)
// bits, 2^-19 (bf16) or 2^-16 (fp16) of sum |q x|, far below the output's
// rounding.
#include "device_common.h"
#include "gemm_common.h"
#include "launch.h"

namespace mxmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kRows = 64;          // rows of x in one tile, 16 MT of them at a time
constexpr int kCols = 64;          // rows of w in one tile: 4 blocks of 16
constexpr int kUnit = 128;         // contraction positions of one wave's turn
constexpr int kXcds = 8;

enum Weights { kW16, kW4 };

template <typename T> struct Bias;
template <> struct Bias<BF16> { static constexpr uint32_t bits = 0x43004300u, one = 0x3f803f80u;
                                static constexpr float value = 128.0f; };
template <> struct Bias<F16> { static constexpr uint32_t bits = 0x64006400u, one = 0x3c003c00u;
                               static constexpr float value = 1024.0f; };

__device__ __forceinline__ u32x4 load16(const uint8_t* p, bool in, int site) {
    if (!in || !MX_CAN_LOAD(p, 16, site)) return u32x4{0u, 0u, 0u, 0u};
    return *reinterpret_cast<const u32x4*>(p);
}

// Positions of x in the order in which pairs come out of eight nibbles:
// (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ u32x4 nibble_order(u32x4 v) {
    return u32x4{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u),
                 __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
                 __builtin_amdgcn_perm(v[3], v[1], 0x05040100u),
                 __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
}

// Eight nibbles as B + q.
template <typename T>
__device__ __forceinline__ u32x4 widen4(uint32_t q) {
    constexpr uint32_t m = 0x000f000fu, b = Bias<T>::bits;
    return u32x4{(q & m) | b, ((q >> 4) & m) | b, ((q >> 8) & m) | b, ((q >> 12) & m) | b};
}

// Lane group g (16 lanes) holds words 4 g .. 4 g + 3 of 16; afterwards word i
// of group g is word 4 i + g: a 4 x 4 transpose between lane groups.
__device__ __forceinline__ void transpose_groups(uint32_t (&d)[4]) {
    auto s02 = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
    auto s13 = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
    auto lo = __builtin_amdgcn_permlane16_swap(s02[0], s13[0], false, false);
    auto hi = __builtin_amdgcn_permlane16_swap(s02[1], s13[1], false, false);
    d[0] = lo[0];
    d[1] = lo[1];
    d[2] = hi[0];
    d[3] = hi[1];
}

template <typename T, Weights W, bool Gated, int MT>
__device__ __forceinline__ void run_tile(const GemmArgs& a, int e, int64_t row0, int rows,
                                         int32_t n0, float* lds) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int g = lane >> 4, r16 = lane & 15;
    const int32_t cols = (int32_t)a.out_cols;
    // rows of w: block j of the tile; gated tiles alternate gate and up blocks
    const uint8_t* wp[4];
    int64_t wrow[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        int32_t c = n0 + (Gated ? (j >> 1) * 16 : j * 16) + r16;
        c = c < cols ? c : cols - 1;
        wrow[j] = (int64_t)c + (Gated ? (j & 1) * a.out_cols : 0);
        wp[j] = a.w + (int64_t)e * a.w_expert_bytes + wrow[j] * a.w_row_bytes;
    }
    const uint8_t* xp[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int r = i * 16 + r16 < rows ? i * 16 + r16 : rows - 1;
        xp[i] = a.x + (row0 + r) * a.x_row_bytes;
    }
    f32x4 acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t len = a.len;
    const int64_t w_rows = Gated ? 2 * a.out_cols : a.out_cols;
    for (int64_t k0 = (int64_t)wave * kUnit; k0 < len; k0 += kWaves * kUnit) {
        if constexpr (W == kW16) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int64_t k = k0 + t * 32 + g * 8;
                const bool in = k < len;
                u32x4 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = load16(wp[j] + k * 2, in, kSiteGemmLoad);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const u32x4 x = load16(xp[i] + k * 2, in, kSiteGemmLoad);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = mfma_16(T{}, x, w[j], acc[i][j]);
                }
            }
        } else {
            uint32_t q[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t k = k0 + g * 32;
                const u32x4 v = load16(wp[j] + k / 2, k < len, kSiteGemmLoad);
#pragma unroll
                for (int t = 0; t < 4; ++t) q[j][t] = v[t];
                transpose_groups(q[j]);
            }
            f32x4 part[MT][4], sx[MT];
            const u32x4 ones = {Bias<T>::one, Bias<T>::one, Bias<T>::one, Bias<T>::one};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int64_t kt = k0 + t * 32;
                const bool first = (kt & (a.group - 1)) == 0 || t == 0;
                if (first) {
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        sx[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int j = 0; j < 4; ++j) part[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                    }
                }
                u32x4 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = widen4<T>(q[j][t]);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const u32x4 x = nibble_order(
                        load16(xp[i] + (kt + g * 8) * 2, kt < len, kSiteGemmLoad));
                    sx[i] = mfma_16(T{}, x, ones, sx[i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) part[i][j] = mfma_16(T{}, x, w[j], part[i][j]);
                }
                if (kt < len && (t == 3 || ((kt + 32) & (a.group - 1)) == 0)) {
                    const int64_t at = kt / a.group;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int64_t si =
                            ((int64_t)e * w_rows + wrow[j]) * (len / a.group) + at;
                        const uint16_t* sp = static_cast<const uint16_t*>(a.w_scales) + si;
                        const float s =
                            MX_CAN_LOAD(sp, 2, kSiteGemmScale) ? to_f32(T{}, *sp) : 0.0f;
                        float z = 8.0f;
                        if (a.w_zeros != nullptr && MX_CAN_LOAD(a.w_zeros + si, 1, kSiteGemmScale))
                            z = (float)a.w_zeros[si];
                        z += Bias<T>::value;
#pragma unroll
                        for (int i = 0; i < MT; ++i)
#pragma unroll
                            for (int d = 0; d < 4; ++d)
                                acc[i][j][d] =
                                    fmaf(s, fmaf(-z, sx[i][d], part[i][j][d]), acc[i][j][d]);
                    }
                }
            }
        }
    }
    // The waves' sums are added in order through LDS: [wave][row][column].
    const int out_cols = Gated ? kCols / 2 : kCols;
    for (int i = 0; i < MT; ++i) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int d = 0; d < 4; ++d)
                lds[(wave * 16 + g * 4 + d) * (kCols + 1) + j * 16 + r16] = acc[i][j][d];
        __syncthreads();
        for (int at = threadIdx.x; at < 16 * out_cols; at += kThreads) {
            const int m = at / out_cols, c = at - m * out_cols;
            const int r = i * 16 + m;
            if (r >= rows || n0 + c >= cols) continue;
            auto total = [&](int col) {
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) v += lds[(w * 16 + m) * (kCols + 1) + col];
                return v;
            };
            const int64_t row = row0 + r;
            if constexpr (Gated) {
                const int col = (c >> 4) * 32 + (c & 15);
                const float gate = total(col), up = total(col + 16);
                store1(a.out, a.out_dtype, row * a.out_cols + n0 + c, silu_mul(gate, up));
                if (a.gate_up != nullptr) {
                    store1(a.gate_up, a.out_dtype, row * 2 * a.out_cols + n0 + c, gate);
                    store1(a.gate_up, a.out_dtype, (row * 2 + 1) * a.out_cols + n0 + c, up);
                }
            } else {
                store1(a.out, a.out_dtype, row * a.out_cols + n0 + c, total(c));
            }
        }
    }
}

__device__ __forceinline__ int32_t row_tiles(int32_t rows) { return (rows + kRows - 1) / kRows; }

template <typename T, Weights W, bool Gated>
__global__ __launch_bounds__(kThreads) void skinny_kernel(GemmArgs a) {
    __shared__ float lds[kWaves * 16 * (kCols + 1)];
    __shared__ int32_t first_tile[kMaxExperts + 1];
    __shared__ int32_t wave_total[kWaves];
    count_row_tiles<kThreads>(a, first_tile, wave_total, row_tiles);
    const int32_t cols_per_tile = Gated ? kCols / 2 : kCols;
    const int32_t n_tiles = (int32_t)((a.out_cols + cols_per_tile - 1) / cols_per_tile);
    const int64_t total = (int64_t)uniform(first_tile[a.num_experts]) * n_tiles;
    const int64_t per = (total + kXcds - 1) / kXcds;
    const int64_t begin = per * (blockIdx.x % kXcds);
    const int64_t end = begin + per < total ? begin + per : total;
    int e = 0;
    for (int64_t t = begin + blockIdx.x / kXcds; t < end; t += gridDim.x / kXcds) {
        e = expert_of_tile(first_tile, a.num_experts, n_tiles, t, e);
        const Segment sg = uniform_segment(a, e);
        const int32_t mt = row_tiles(sg.count);
        const int64_t r = t - (int64_t)uniform(first_tile[e]) * n_tiles;
        const int32_t n_tile = (int32_t)(r / mt), m_tile = (int32_t)(r - (int64_t)n_tile * mt);
        const int64_t row0 = sg.begin + (int64_t)m_tile * kRows;
        const int rows = sg.count - m_tile * kRows < kRows ? sg.count - m_tile * kRows : kRows;
        if (rows <= 0) continue;
        const int32_t n0 = n_tile * cols_per_tile;
        if (rows <= 16) run_tile<T, W, Gated, 1>(a, e, row0, rows, n0, lds);
        else if (rows <= 32) run_tile<T, W, Gated, 2>(a, e, row0, rows, n0, lds);
        else run_tile<T, W, Gated, 4>(a, e, row0, rows, n0, lds);
    }
}

// Workgroups of the persistent grid.
#ifndef MXMOE_SKINNY_GROUPS
#define MXMOE_SKINNY_GROUPS 1024
#endif
static_assert(MXMOE_SKINNY_GROUPS % kXcds == 0, "every XCD has the same number of workgroups");

template <typename... KArgs>
hipError_t start(void (*kernel)(KArgs...), const GemmArgs& a, hipStream_t stream) {
    launch_kernel(kernel, dim3(MXMOE_SKINNY_GROUPS), dim3(kThreads), 0, stream, nullptr, nullptr,
                  a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_w4(const GemmArgs& a, hipStream_t stream) {
    if (a.dtype == 1)
        return a.gated ? start(skinny_kernel<F16, kW4, true>, a, stream)
                       : start(skinny_kernel<F16, kW4, false>, a, stream);
    return a.gated ? start(skinny_kernel<BF16, kW4, true>, a, stream)
                   : start(skinny_kernel<BF16, kW4, false>, a, stream);
}

}  // namespace mxmoe
