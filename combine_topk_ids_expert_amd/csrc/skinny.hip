// Products of few rows with their expert's 4-bit weights, for decoding: the
// weights pass once from HBM through registers to the matrix cores, with
// nothing in between, so that their bytes are the time.
//
//   out[r][n] = sum_k x[r][k] w[e][n][k],   w = (q - z) s
//
// with one scale s (and zero point z, or 8) per group G of positions:
//
//   sum_{k in G} (q - z) x = -(B + z) sum_k x + sum_k (B + q) x,
//
// where B + q is the 16-bit number whose low mantissa bits are q (B = 128 in
// bf16, 1024 in fp16): one AND-OR makes two of them, every B + q is exact,
// and the sum of x comes from one more matrix instruction against ones.  Both
// sums and their difference are float32: the difference loses log2(B / 4)
// bits, 2^-19 (bf16) or 2^-16 (fp16) of sum |q x|, far below the output's
// rounding.
//
// A workgroup takes 64 rows of w and at most 16 of x; its four waves split the
// contraction in turns of 128 positions and their sums are added in LDS in a
// fixed order.  Three workgroups to a CU (168 registers a lane) measured best:
// 2 to a CU with x loaded ahead 218 us, 8 waves to a workgroup slower than 4, at
// 256 rows x 2048 -> 7168 over 64 experts with zero points, where this form takes
// 128 us (518 MB, 4.0 TB/s; a copy reaches 4.9, reads alone 6.2).  One token's 8
// picks of 256 experts, 4096 -> 2 x 2048 gated: 22 us (69 MB, 3.2 TB/s): short
// enough that the launch, the search of the offsets and the last sums show.
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

// kPlain: len is a multiple of 128 and holds 8 groups or more, no zero points;
// kZeros: the same with them; kAny: any.
enum Form { kPlain, kZeros, kAny };

// One unit's weights of a lane: of each 16-row block, 32 positions of row
// l & 15 and the scales and zero points of the unit's 128 / Group groups.
template <int Group>
struct Unit {
    static constexpr int kScales = kUnit / Group;
    u32x4 w[4];
    uint32_t s[4][(kScales + 1) / 2];
    uint32_t z[4];
};

// The scales and zero points of 8 groups in a row, of row `lane` of the tile: a
// load for all 64 rows.  (Loads by the unit, 2 to 8 bytes from each of 16 rows
// four times over, cost the L1 cache twice what the weights do.)
struct Scales {
    uint32_t s[4], z[2];
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, -1, 0x00020000);
}

// Where a lane's weights lie: uniform bases of the tile's gate (or only) and up
// rows, and the byte and scale offsets of the lane's row of each block.
template <bool Gated, int Group, Form F>
struct Weights {
    static constexpr int kScales = Unit<Group>::kScales;
    const uint8_t* base[2];
    const uint16_t* scales[2];
    const uint8_t* zeros[2];
    uint32_t w_at[4], s_at[4];
    uint32_t row;                 // the tile's row `lane`, for the scales

    __device__ __forceinline__ void init(const GemmArgs& a, const Tile& t) {
        const int lane = threadIdx.x & 63;
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
            const int r = (Gated ? (j >> 1) * 16 : j * 16) + (lane & 15);
            const uint32_t at = (uint32_t)(r < last ? r : last);
            w_at[j] = at * (uint32_t)a.w_row_bytes + (lane >> 4) * 16;
            s_at[j] = at * (uint32_t)groups;
        }
        const int r = (Gated ? (lane >> 5) * 16 : (lane >> 4) * 16) + (lane & 15);
        row = (uint32_t)(r < last ? r : last);
    }
    // The unit's words; its scales come from `scales`.
    __device__ __forceinline__ void load_words(uint32_t k0, Unit<Group>& u) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint8_t* b = base[Gated ? j & 1 : 0];
            u.w[j] = u32x4{0u, 0u, 0u, 0u};
            if (MX_CAN_LOAD(b + w_at[j] + k0 / 2, 16, kSiteGemmLoad))
                u.w[j] = __builtin_amdgcn_raw_buffer_load_b128(buffer(b), w_at[j], k0 / 2, 0);
        }
    }
    // Groups g0 .. + 8 of the tile's row `lane`; of the last ones, what there is.
    __device__ __forceinline__ void load_scales(const GemmArgs& a, uint32_t g0, Scales& v) const {
        const uint32_t groups = (uint32_t)a.len / Group;
        const uint32_t from = g0 + 8 <= groups ? g0 : groups - 8, skip = g0 - from;
        const int lane = threadIdx.x & 63, half = Gated ? (lane >> 4) & 1 : 0;
        const uint32_t at = row * groups + from;
        const uint16_t* sp = scales[half] + at;
        uint64_t lo = 0, hi = 0;
        struct __attribute__((packed, aligned(2))) Eight { uint64_t v[2]; };
        struct __attribute__((packed, aligned(1))) Bytes { uint64_t v; };
        if (MX_CAN_LOAD(sp, 16, kSiteGemmScale)) {
            const Eight e = *reinterpret_cast<const Eight*>(sp);
            lo = e.v[0];
            hi = e.v[1];
        }
        uint64_t zv = 0;
        if (F == kZeros && MX_CAN_LOAD(zeros[half] + at, 8, kSiteGemmScale))
            zv = reinterpret_cast<const Bytes*>(zeros[half] + at)->v;
        if (skip != 0) {
            const uint32_t bits = skip * 16;
            lo = bits < 64 ? lo >> bits | hi << (64 - bits) : hi >> (bits - 64);
            hi = bits < 64 ? hi >> bits : 0;
            zv >>= skip * 8;
        }
        v.s[0] = (uint32_t)lo;
        v.s[1] = (uint32_t)(lo >> 32);
        v.s[2] = (uint32_t)hi;
        v.s[3] = (uint32_t)(hi >> 32);
        v.z[0] = (uint32_t)zv;
        v.z[1] = (uint32_t)(zv >> 32);
    }
    // Unit i of the 8 groups' to the lanes that hold its weights.
    __device__ __forceinline__ static void take(const Scales& v, int i, Unit<Group>& u) {
        const int r16 = threadIdx.x & 15;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int from = (j * 16 + r16) * 4;
            auto get = [&](uint32_t x) {
                return (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)x);
            };
            if constexpr (kScales == 4) {
                u.s[j][0] = get(v.s[2 * i]);
                u.s[j][1] = get(v.s[2 * i + 1]);
                if (F == kZeros) u.z[j] = get(v.z[i]);
            } else if constexpr (kScales == 2) {
                u.s[j][0] = get(v.s[i]);
                if (F == kZeros) u.z[j] = get(v.z[i / 2] >> (16 * (i % 2)));
            } else {
                u.s[j][0] = get(v.s[i / 2] >> (16 * (i % 2))) & 0xffffu;
                if (F == kZeros) u.z[j] = get(v.z[i / 4] >> (8 * (i % 4)));
            }
        }
    }
    // A unit that may be cut short, or whose scales are not aligned: positions
    // and groups past the end read the last ones there are.
    __device__ __forceinline__ void load_any(const GemmArgs& a, uint32_t k0, Unit<Group>& u) const {
        const uint32_t len = (uint32_t)a.len, own = ((threadIdx.x & 63) >> 4) * 32;
        const uint32_t k = k0 + own < len ? k0 : len - 32 - own;    // may wrap, own is added back
        const uint32_t groups = len / Group, g0 = k0 / Group;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint8_t* b = base[Gated ? j & 1 : 0];
            const uint32_t at = w_at[j] - own / 2 + (k + own) / 2;
            u.w[j] = u32x4{0u, 0u, 0u, 0u};
            if (MX_CAN_LOAD(b + at, 16, kSiteGemmLoad))
                u.w[j] = *reinterpret_cast<const u32x4*>(b + at);
            u.z[j] = 0;
#pragma unroll
            for (int g = 0; g < kScales; ++g) {
                const uint32_t i = s_at[j] + (g0 + g < groups ? g0 + g : groups - 1);
                const uint16_t* sb = scales[Gated ? j & 1 : 0];
                const uint32_t v = MX_CAN_LOAD(sb + i, 2, kSiteGemmScale) ? sb[i] : 0;
                u.s[j][g / 2] = g % 2 ? u.s[j][g / 2] | v << 16 : v;
                const uint8_t* zb = zeros[Gated ? j & 1 : 0];
                if (a.w_zeros != nullptr && MX_CAN_LOAD(zb + i, 1, kSiteGemmScale))
                    u.z[j] |= (uint32_t)zb[i] << (8 * g);
            }
        }
    }
};

// A lane's share of x in a unit: positions 8 (l >> 4) .. + 8 of each 32 of row
// l & 15; zeros past the end.
struct Rows {
    const uint8_t* base;
    uint32_t at;

    __device__ __forceinline__ void init(const GemmArgs& a, const Tile& t) {
        const int lane = threadIdx.x & 63, r = lane & 15;
        base = a.x + t.row0 * a.x_row_bytes;
        at = (uint32_t)(r < t.rows ? r : t.rows - 1) * (uint32_t)a.x_row_bytes + (lane >> 4) * 16;
    }
    template <Form F>
    __device__ __forceinline__ void load(const GemmArgs& a, uint32_t k0, u32x4 (&x)[4]) const {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t k = k0 + q * 32;
            x[q] = u32x4{0u, 0u, 0u, 0u};
            if ((F != kAny || k < a.len) && MX_CAN_LOAD(base + at + k * 2, 16, kSiteGemmLoad))
                x[q] = __builtin_amdgcn_raw_buffer_load_b128(buffer(base), at, k * 2, 0);
        }
    }
};

// Adds one unit's products to the sums: per group the sum of (B + q) x, which
// starts from -(B + z) sum x, times the scale.
template <typename T, int Group, Form F>
__device__ __forceinline__ void add_unit(const GemmArgs& a, const Unit<Group>& u,
                                         const u32x4 (&x)[4], f32x4 (&acc)[4]) {
    constexpr int kScales = Unit<Group>::kScales, kSteps = Group / 32;
    const u32x4 ones = {Bias<T>::one, Bias<T>::one, Bias<T>::one, Bias<T>::one};
    u32x4 xo[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) xo[q] = nibble_order(x[q]);
    f32x4 start[kScales];                               // -(B + 8) sum x, or sum x
#pragma unroll
    for (int gr = 0; gr < kScales; ++gr) {
        start[gr] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int st = 0; st < kSteps; ++st)
            start[gr] = mfma_16(T{}, xo[gr * kSteps + st], ones, start[gr]);
    }
    const bool zeros = F == kZeros || (F == kAny && a.w_zeros != nullptr);
    if (!zeros) {
#pragma unroll
        for (int gr = 0; gr < kScales; ++gr)
#pragma unroll
            for (int d = 0; d < 4; ++d) start[gr][d] *= -(Bias<T>::value + 8.0f);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = u.w[j][q];
        transpose_groups(w);
#pragma unroll
        for (int gr = 0; gr < kScales; ++gr) {
            f32x4 part = start[gr];
            if (zeros) {
                const float z = -(Bias<T>::value + (float)((u.z[j] >> (8 * gr)) & 0xffu));
#pragma unroll
                for (int d = 0; d < 4; ++d) part[d] *= z;
            }
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
                const int q = gr * kSteps + st;
                part = mfma_16(T{}, xo[q], widen4<T>(w[q]), part);
            }
            const float s = to_f32(T{}, (uint16_t)(u.s[j][gr / 2] >> (16 * (gr % 2))));
#pragma unroll
            for (int d = 0; d < 4; ++d) acc[j][d] = fmaf(s, part[d], acc[j][d]);
        }
        __builtin_amdgcn_sched_barrier(0);              // one block's words at a time
    }
}

// What one unit takes from memory.
template <int Group>
struct Stage {
    Unit<Group> u;
    u32x4 x[4];
};

// The wave's share of a tile: a quarter of the contraction's units, in a row.
template <typename T, bool Gated, int Group, Form F>
struct Tiling {
    static constexpr int kBatch = 8 / Unit<Group>::kScales;     // units of 8 groups
    Weights<Gated, Group, F> weights;
    Rows rows;
    uint32_t k0, end;             // positions

    __device__ __forceinline__ void init(const GemmArgs& a, const Tile& t) {
        weights.init(a, t);
        rows.init(a, t);
        const uint32_t units = ((uint32_t)a.len + kUnit - 1) / kUnit;
        const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        k0 = units * wave / kWaves * kUnit;
        end = units * (wave + 1) / kWaves * kUnit;
    }
    // Sets off the loads of the first unit.
    __device__ __forceinline__ void start(const GemmArgs& a, Stage<Group>& s, Scales& v) const {
        if (k0 >= end) return;
        load(a, k0, s);
        if (F != kAny) weights.load_scales(a, k0 / Group, v);
    }
    __device__ __forceinline__ void load(const GemmArgs& a, uint32_t k, Stage<Group>& s) const {
        if (k >= end) return;
        if constexpr (F == kAny) weights.load_any(a, k, s.u);
        else weights.load_words(k, s.u);
        rows.template load<F>(a, k, s.x);
    }
    // The sums over the wave's units, each loaded while the one before is
    // multiplied; the scales are loaded 8 groups ahead.
    __device__ __forceinline__ void multiply(const GemmArgs& a, Stage<Group> (&s)[2], Scales v,
                                             f32x4 (&acc)[4]) const {
        for (uint32_t k = k0; k < end;) {
            Scales next = v;
            if (F != kAny && k + kBatch * kUnit < end)
                weights.load_scales(a, (k + kBatch * kUnit) / Group, next);
#pragma unroll
            for (int i = 0; i < kBatch; ++i, k += kUnit) {
                if (k >= end) break;
                load(a, k + kUnit, s[(i + 1) & 1]);
                if (F != kAny) weights.take(v, i, s[i & 1].u);
                add_unit<T, Group, F>(a, s[i & 1].u, s[i & 1].x, acc);
            }
            v = next;
        }
    }
};

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
template <typename T, bool Gated, int Group, Form F>
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
    Tiling<T, Gated, Group, F> tiling;
    Stage<Group> stages[2];
    Scales scales;
    Tile tile = tile_of(t);
    tiling.init(a, tile);
    tiling.start(a, stages[0], scales);
    while (true) {
        f32x4 acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        tiling.multiply(a, stages, scales, acc);
        // the next tile's first unit is loaded under this one's sums
        const Tile done = tile;
        t += gridDim.x / kXcds;
        if (t < end) {
            tile = tile_of(t);
            tiling.init(a, tile);
            tiling.start(a, stages[0], scales);
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

template <typename T, bool Gated, int Group>
hipError_t start(const GemmArgs& a, hipStream_t stream) {
    if (!a.whole_units) return start(w4_kernel<T, Gated, Group, kAny>, a, stream);
    if (a.w_zeros != nullptr) return start(w4_kernel<T, Gated, Group, kZeros>, a, stream);
    return start(w4_kernel<T, Gated, Group, kPlain>, a, stream);
}

template <typename T, bool Gated>
hipError_t start(const GemmArgs& a, hipStream_t stream) {
    if (a.group == 32) return start<T, Gated, 32>(a, stream);
    if (a.group == 64) return start<T, Gated, 64>(a, stream);
    return start<T, Gated, 128>(a, stream);
}

}  // namespace

hipError_t launch_grouped_w4(const GemmArgs& a, hipStream_t stream) {
    if (a.dtype == 1) return a.gated ? start<F16, true>(a, stream) : start<F16, false>(a, stream);
    return a.gated ? start<BF16, true>(a, stream) : start<BF16, false>(a, stream);
}

}  // namespace mxmoe
