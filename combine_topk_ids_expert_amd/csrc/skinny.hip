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
// Rows of x in one tile, the columns of a matrix instruction.  More of them
// would take the registers that keep loads under way; an expert with more rows
// has its weights' tiles repeated, next to each other in the same L2.
constexpr int kRows = 16;
constexpr int kCols = 64;          // rows of w in one tile: 4 blocks of 16
constexpr int kUnit = 128;         // contraction positions of one wave's turn
constexpr int kXcds = 8;

template <typename T> struct Bias;
template <> struct Bias<BF16> { static constexpr uint32_t bits = 0x43004300u, one = 0x3f803f80u;
                                static constexpr float value = 128.0f; };
template <> struct Bias<F16> { static constexpr uint32_t bits = 0x64006400u, one = 0x3c003c00u;
                               static constexpr float value = 1024.0f; };

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

// One tile: `rows` rows of x from row0 on, 64 rows of expert e's weights, which
// give the output columns from n0 on.
struct Tile {
    int32_t e, rows, n0;
    int64_t row0;
};

// One unit's weights of a lane: of each 16-row block, 32 positions of row
// l & 15 and the scales and zero points of the unit's 128 / Group groups.
template <int Group>
struct Unit {
    static constexpr int kScales = kUnit / Group;
    u32x4 w[4];
    uint32_t s[4][(kScales + 1) / 2];
    uint32_t z[4];
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, -1, 0x00020000);
}

// Where a lane's weights lie: uniform bases of the tile's gate (or only) and up
// rows, and the lane's row below them for each block.
template <typename T, bool Gated, int Group>
struct Weights {
    const uint8_t* base[2];
    const uint16_t* scales[2];
    const uint8_t* zeros[2];
    uint32_t row[4];

    __device__ __forceinline__ void init(const GemmArgs& a, const Tile& t) {
        const int64_t groups = a.len / Group;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t at = t.e * (Gated ? 2 * a.out_cols : a.out_cols) + t.n0 +
                               (Gated ? h * a.out_cols : 0);
            base[h] = a.w + at * a.w_row_bytes;
            scales[h] = static_cast<const uint16_t*>(a.w_scales) + at * groups;
            zeros[h] = a.w_zeros + at * groups;
        }
        const int last = (int)a.out_cols - 1 - t.n0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // gated tiles alternate gate and up blocks
            const int r = (Gated ? (j >> 1) * 16 : j * 16) + (int)(threadIdx.x & 15);
            row[j] = (uint32_t)(r < last ? r : last);
        }
    }
    // The unit from position k0 on; positions past the end read the last ones
    // there are (x is zero there).
    __device__ __forceinline__ void load(const GemmArgs& a, int64_t k0, Unit<Group>& u) const {
        constexpr int kScales = Unit<Group>::kScales;
        int32_t k = (int32_t)k0 + ((threadIdx.x & 63) >> 4) * 32;
        k = k < a.len ? k : (int32_t)a.len - 32;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint8_t* b = base[Gated ? j & 1 : 0];
            const uint32_t at = row[j] * (uint32_t)a.w_row_bytes + (uint32_t)(k / 2);
            u.w[j] = u32x4{0u, 0u, 0u, 0u};
            if (MX_CAN_LOAD(b + at, 16, kSiteGemmLoad))
                u.w[j] = __builtin_amdgcn_raw_buffer_load_b128(buffer(b), at, 0, 0);
        }
        const uint32_t groups = (uint32_t)(a.len / Group), g0 = (uint32_t)(k0 / Group);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint16_t* b = scales[Gated ? j & 1 : 0];
            const uint8_t* zb = zeros[Gated ? j & 1 : 0];
            const uint32_t at = row[j] * groups + g0;
            if (a.whole_units) {
                uint32_t s[2] = {0u, 0u}, z = 0u;
                if (MX_CAN_LOAD(b + at, 2 * kScales, kSiteGemmScale)) {
                    if constexpr (kScales == 4) {
                        const u32x2 v =
                            __builtin_amdgcn_raw_buffer_load_b64(buffer(b), at * 2, 0, 0);
                        s[0] = v[0];
                        s[1] = v[1];
                    } else if constexpr (kScales == 2) {
                        s[0] = __builtin_amdgcn_raw_buffer_load_b32(buffer(b), at * 2, 0, 0);
                    } else {
                        s[0] = __builtin_amdgcn_raw_buffer_load_b16(buffer(b), at * 2, 0, 0);
                    }
                }
                if (a.w_zeros != nullptr && MX_CAN_LOAD(zb + at, kScales, kSiteGemmScale)) {
                    if constexpr (kScales == 4)
                        z = __builtin_amdgcn_raw_buffer_load_b32(buffer(zb), at, 0, 0);
                    else if constexpr (kScales == 2)
                        z = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(buffer(zb), at, 0, 0);
                    else
                        z = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(buffer(zb), at, 0, 0);
                }
                u.s[j][0] = s[0];
                if constexpr (kScales == 4) u.s[j][1] = s[1];
                u.z[j] = z;
            } else {
                u.z[j] = 0;
#pragma unroll
                for (int g = 0; g < kScales; ++g) {
                    const uint32_t i = at + (g0 + g < groups ? g : groups - 1 - g0);
                    const uint32_t v = MX_CAN_LOAD(b + i, 2, kSiteGemmScale) ? b[i] : 0;
                    u.s[j][g / 2] = g % 2 ? u.s[j][g / 2] | v << 16 : v;
                    if (a.w_zeros != nullptr && MX_CAN_LOAD(zb + i, 1, kSiteGemmScale))
                        u.z[j] |= (uint32_t)zb[i] << (8 * g);
                }
            }
        }
    }
};

// The wave's share of a tile's sums: units wave, wave + 4, ... of the
// contraction, the first of them in `u`, each unit's weights loaded while the
// one before is multiplied.
template <typename T, bool Gated, int Group>
__device__ __forceinline__ void multiply(const GemmArgs& a, const Tile& t,
                                         const Weights<T, Gated, Group>& weights, Unit<Group> u,
                                         f32x4 (&acc)[4]) {
    constexpr int kScales = Unit<Group>::kScales, kSteps = Group / 32;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int g = lane >> 4, r16 = lane & 15;
    const uint8_t* xb = a.x + t.row0 * a.x_row_bytes;
    const uint32_t x_at =
        (uint32_t)(r16 < t.rows ? r16 : t.rows - 1) * (uint32_t)a.x_row_bytes + g * 16;
    for (int64_t k0 = (int64_t)wave * kUnit; k0 < a.len; k0 += kWaves * kUnit) {
        u32x4 x[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            x[q] = u32x4{0u, 0u, 0u, 0u};
            const uint32_t k = (uint32_t)k0 + q * 32;
            if (k < a.len && MX_CAN_LOAD(xb + x_at + k * 2, 16, kSiteGemmLoad))
                x[q] = __builtin_amdgcn_raw_buffer_load_b128(buffer(xb), x_at, k * 2, 0);
        }
        Unit<Group> next = u;
        if (k0 + kWaves * kUnit < a.len) weights.load(a, k0 + kWaves * kUnit, next);
        uint32_t w[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int q = 0; q < 4; ++q) w[j][q] = u.w[j][q];
            transpose_groups(w[j]);
        }
        const u32x4 ones = {Bias<T>::one, Bias<T>::one, Bias<T>::one, Bias<T>::one};
#pragma unroll
        for (int gr = 0; gr < kScales; ++gr) {
            if (k0 + gr * Group >= a.len) break;
            f32x4 part[4], sx = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < 4; ++j) part[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
                const int q = gr * kSteps + st;
                const u32x4 xo = nibble_order(x[q]);
                sx = mfma_16(T{}, xo, ones, sx);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    part[j] = mfma_16(T{}, xo, widen4<T>(w[j][q]), part[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float s = to_f32(T{}, (uint16_t)(u.s[j][gr / 2] >> (16 * (gr % 2))));
                const float z = Bias<T>::value + (a.w_zeros != nullptr
                                                      ? (float)((u.z[j] >> (8 * gr)) & 0xffu)
                                                      : 8.0f);
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    acc[j][d] = fmaf(s, fmaf(-z, sx[d], part[j][d]), acc[j][d]);
            }
        }
        u = next;
    }
}

// The waves' sums added in order through LDS, [wave][row][column], and written.
template <bool Gated>
__device__ __forceinline__ void finish(const GemmArgs& a, const Tile& t,
                                       const f32x4 (&acc)[4], float* lds) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int g = lane >> 4, r16 = lane & 15;
    constexpr int kOut = Gated ? kCols / 2 : kCols;
    const int32_t cols = (int32_t)a.out_cols;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int d = 0; d < 4; ++d)
            lds[(wave * 16 + g * 4 + d) * (kCols + 1) + j * 16 + r16] = acc[j][d];
    __syncthreads();
    for (int at = threadIdx.x; at < t.rows * kOut; at += kThreads) {
        const int m = at / kOut, c = at % kOut;
        if (t.n0 + c >= cols) continue;
        auto total = [&](int col) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) v += lds[(w * 16 + m) * (kCols + 1) + col];
            return v;
        };
        const int64_t out = (t.row0 + m) * a.out_cols + t.n0 + c;
        if constexpr (Gated) {
            const int col = (c >> 4) * 32 + (c & 15);
            store1(a.out, a.out_dtype, out, silu_mul(total(col), total(col + 16)));
        } else {
            store1(a.out, a.out_dtype, out, total(c));
        }
    }
}

__device__ __forceinline__ int32_t row_tiles(int32_t rows) { return (rows + kRows - 1) / kRows; }

// 3 waves per SIMD (at most 168 registers), each with 4 KiB of weights under way.
template <typename T, bool Gated, int Group>
__global__ __launch_bounds__(kThreads, 3) void w4_kernel(GemmArgs a) {
    __shared__ float lds[kWaves * 16 * (kCols + 1)];
    __shared__ int32_t first_tile[kMaxExperts + 1];
    __shared__ int32_t wave_total[kWaves];
    count_row_tiles<kThreads>(a, first_tile, wave_total, row_tiles);
    const int32_t cols_per_tile = Gated ? kCols / 2 : kCols;
    const int32_t n_tiles = (int32_t)((a.out_cols + cols_per_tile - 1) / cols_per_tile);
    const int64_t total = (int64_t)uniform(first_tile[a.num_experts]) * n_tiles;
    // each XCD takes a contiguous eighth of the tiles
    const int64_t per = (total + kXcds - 1) / kXcds;
    const int64_t begin = per * (blockIdx.x % kXcds);
    const int64_t end = begin + per < total ? begin + per : total;
    int e = 0;
    auto tile_of = [&](int64_t t) {
        e = expert_of_tile(first_tile, a.num_experts, n_tiles, t, e);
        const Segment sg = uniform_segment(a, e);
        const int32_t mt = row_tiles(sg.count);
        const int64_t r = t - (int64_t)uniform(first_tile[e]) * n_tiles;
        const int32_t n_tile = (int32_t)(r / mt), m_tile = (int32_t)(r - (int64_t)n_tile * mt);
        Tile tile;
        tile.e = e;
        tile.rows = sg.count - m_tile * kRows < kRows ? sg.count - m_tile * kRows : kRows;
        tile.n0 = n_tile * cols_per_tile;
        tile.row0 = sg.begin + (int64_t)m_tile * kRows;
        return tile;
    };
    int64_t t = begin + blockIdx.x / kXcds;
    if (t >= end) return;
    const int64_t k0 = (int64_t)(threadIdx.x >> 6) * kUnit;
    Weights<T, Gated, Group> weights;
    Unit<Group> u;
    Tile tile = tile_of(t);
    weights.init(a, tile);
    if (k0 < a.len) weights.load(a, k0, u);
    while (true) {
        f32x4 acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        multiply<T, Gated, Group>(a, tile, weights, u, acc);
        // the next tile's first unit is loaded under this one's sums
        const Tile done = tile;
        t += gridDim.x / kXcds;
        if (t < end) {
            tile = tile_of(t);
            weights.init(a, tile);
            if (k0 < a.len) weights.load(a, k0, u);
        }
        finish<Gated>(a, done, acc, lds);
        if (t >= end) return;
    }
}

// Workgroups of the persistent grid.
#ifndef MXMOE_SKINNY_GROUPS
#define MXMOE_SKINNY_GROUPS 768
#endif
static_assert(MXMOE_SKINNY_GROUPS % kXcds == 0, "every XCD has the same number of workgroups");

template <typename... KArgs>
hipError_t start(void (*kernel)(KArgs...), const GemmArgs& a, hipStream_t stream) {
    launch_kernel(kernel, dim3(MXMOE_SKINNY_GROUPS), dim3(kThreads), 0, stream, nullptr, nullptr,
                  a);
    return hipGetLastError();
}

template <typename T, bool Gated>
hipError_t start(const GemmArgs& a, hipStream_t stream) {
    if (a.group == 32) return start(w4_kernel<T, Gated, 32>, a, stream);
    if (a.group == 64) return start(w4_kernel<T, Gated, 64>, a, stream);
    return start(w4_kernel<T, Gated, 128>, a, stream);
}

}  // namespace

hipError_t launch_grouped_w4(const GemmArgs& a, hipStream_t stream) {
    if (a.dtype == 1) return a.gated ? start<F16, true>(a, stream) : start<F16, false>(a, stream);
    return a.gated ? start<BF16, true>(a, stream) : start<BF16, false>(a, stream);
}

}  // namespace mxmoe
