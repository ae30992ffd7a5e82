// Matrix products grouped by expert, over the ragged row segments that routing
// and dispatch leave behind:
//
//   kForward   out[r][n] = sum_k x[r][k] w[e][n][k]     w [E][N][K]
//   kRowGrad   out[r][j] = sum_c x[r][c] w[e][c][j]     w [E][C][J] (the rows'
//              gradient through the weights of a forward product)
//   kWeightGrad out[e][n][k] = sum_{r in segment e} dy[r][n] x[r][k]
//
// Segment e is the rows b = offsets[e] .. b + c, c = offsets[e+1] - b, or
// sizes[e][0] where that is smaller; both are clipped to the arrays, so no
// value of them makes an access leave the arrays.  Rows outside the segments
// are neither read nor written.
#include "device_common.h"
#include "gemm_common.h"
#include "launch.h"

namespace mxmoe {
namespace {

constexpr int kThreads = 512;             // 8 waves: 2 along m, 4 along n
constexpr int kTileM = 256, kTileN = 256;
constexpr int kStepBytes = 128;           // contraction bytes of one step, a tile row in LDS
constexpr int kTileBytes = 256 * kStepBytes;
constexpr int kXcds = 8;

enum Mode { kForward, kRowGrad, kWeightGrad };

// How an operand's tile lies in memory: with the contraction contiguous (one
// tile row of 128 bytes per output row), or with the contraction across rows
// (64 tile rows of 256 elements).
enum Kind { kAlong, kAcross };

// One operand of a tile.
struct Operand {
    const uint8_t* base;     // kAlong: row 0 of the matrix; kAcross: contraction row 0
    int64_t row_bytes;
    int32_t first;           // first row (kAlong) / column (kAcross) of the tile
    int32_t limit;           // rows / columns there are
    int32_t half;            // gated: row of the first up row (the tile alternates 16
                             // gate rows and 16 up rows), else 0
};

// The loads to LDS that this wave has issued are done; a barrier by itself
// does not wait for them.
__device__ __forceinline__ void wait_for_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Matrix row of row `r` of a tile.
template <bool Gated>
__device__ __forceinline__ int32_t tile_row(const Operand& o, int r) {
    if (Gated) {
        const int32_t c = o.first + (r >> 5) * 16 + (r & 15);
        return (c < o.limit ? c : o.limit - 1) + ((r >> 4) & 1) * o.half;
    }
    const int32_t c = o.first + r;
    return c < o.limit ? c : o.limit - 1;
}

// Swizzles: 16-byte chunk c of tile row r lies at chunk position c ^ swizzle,
// so that the 16-byte (kAlong) and transposing 8-byte (kAcross) fragment
// reads of one cycle fall on different banks.
__device__ __forceinline__ int swizzle_across(int kk) {
    return ((kk & 3) | (((kk >> 3) & 1) << 2)) << 1;
}

// Brings contraction step `step` of an operand into its LDS tile: 32 loads of
// 1 KiB, four per wave, straight to LDS.  Lane l of a load fills the 16 bytes
// at position l, so the swizzle is applied to the address it reads.
// `len`: contraction length in elements; rows, columns and (in the last step)
// contraction positions past the end read the last ones there are, which
// zero_tail and the epilogue leave out.
template <Kind K, bool Gated, int ElemBytes>
__device__ __forceinline__ void stage(const Operand& o, uint8_t* tile, int64_t step, int64_t len,
                                      int rows_needed) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int piece = wave * 4 + i;
        const uint8_t* p;
        if constexpr (K == kAlong) {
            if (piece * 8 >= rows_needed) continue;
            const int r = piece * 8 + (lane >> 3);
            const int chunk = (lane & 7) ^ (lane >> 3);
            int64_t at = step * kStepBytes + chunk * 16;
            const int64_t last = len * ElemBytes - 16;
            at = at < last ? at : last;
            p = o.base + tile_row<Gated>(o, r) * o.row_bytes + at;
        } else {
            const int kk = piece * 2 + (lane >> 5);
            const int chunk = (lane & 31) ^ swizzle_across(kk);
            int64_t row = step * 64 + kk;
            row = row < len ? row : len - 1;
            int32_t col = o.first + chunk * 8;
            col = col < o.limit ? col : o.limit - 8;
            p = o.base + row * o.row_bytes + (int64_t)col * 2;
        }
        if (!MX_CAN_LOAD(p, 16, kSiteGemmLoad)) continue;
        __builtin_amdgcn_global_load_lds(
            (const __attribute__((address_space(1))) void*)p,
            (__attribute__((address_space(3))) void*)(tile + piece * 1024), 16, 0, 0);
    }
}

// The same for rows that are not 16-byte aligned, element by element, with
// zeros past every end.
template <Kind K, bool Gated>
__device__ __forceinline__ void stage_elements(const Operand& o, uint8_t* tile, int64_t step,
                                               int64_t len) {
    for (int i = 0; i < 4; ++i) {
        const int piece = i * 512 + threadIdx.x;            // 16 bytes of the tile
        uint32_t v[4];
        for (int d = 0; d < 4; ++d) {
            uint32_t word = 0;
            for (int h = 0; h < 2; ++h) {
                const int e = d * 2 + h;
                const uint8_t* p;
                bool in;
                if constexpr (K == kAlong) {
                    const int r = piece >> 3, chunk = (piece & 7) ^ (r & 7);
                    const int64_t k = step * 64 + chunk * 8 + e;
                    in = k < len;
                    p = o.base + tile_row<Gated>(o, r) * o.row_bytes + k * 2;
                } else {
                    const int kk = piece >> 5, chunk = (piece & 31) ^ swizzle_across(kk);
                    const int64_t row = step * 64 + kk;
                    const int32_t col = o.first + chunk * 8 + e;
                    in = row < len && col < o.limit;
                    p = o.base + row * o.row_bytes + (int64_t)col * 2;
                }
                if (in && MX_CAN_LOAD(p, 2, kSiteGemmLoad))
                    word |= (uint32_t)*reinterpret_cast<const uint16_t*>(p) << (16 * h);
            }
            v[d] = word;
        }
        *reinterpret_cast<u32x4*>(tile + piece * 16) = u32x4{v[0], v[1], v[2], v[3]};
    }
}

// Zeros at the contraction positions past `valid` (< 64) of a staged tile.
template <Kind K>
__device__ __forceinline__ void zero_tail(uint8_t* tile, int valid) {
    for (int i = 0; i < 4; ++i) {
        const int piece = i * 512 + threadIdx.x;
        bool past;
        if constexpr (K == kAlong) past = ((piece & 7) ^ ((piece >> 3) & 7)) * 8 >= valid;
        else past = (piece >> 5) >= valid;
        if (past) *reinterpret_cast<u32x4*>(tile + piece * 16) = u32x4{0u, 0u, 0u, 0u};
    }
}

// Fragment of 16 rows x 32 contraction positions (16-bit types) of a staged
// tile: lane l holds row l & 15, positions 8 (l >> 4) .. + 8 of half `ks`.
template <Kind K>
__device__ __forceinline__ u32x4 fragment(const uint8_t* tile, int sub, int ks) {
    const int lane = threadIdx.x & 63;
    if constexpr (K == kAlong) {
        const int chunk = (ks * 4 + (lane >> 4)) ^ (lane & 7);
        return *reinterpret_cast<const u32x4*>(tile + (sub * 16 + (lane & 15)) * kStepBytes +
                                               chunk * 16);
    } else {
        // ds_read_b64_tr_b16: the 16 lanes of a group read four rows of 16
        // elements, and lane i gets column i of them.
        const int g = lane >> 4, j = lane & 15;
        const int kk = ks * 32 + g * 8 + (j >> 2);
        const int chunk = (sub * 2 + ((j & 3) >> 1)) ^ swizzle_across(kk);
        const uint8_t* p = tile + kk * 512 + chunk * 16 + (j & 1) * 8;
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * 512));
        u32x4 r;
        __builtin_memcpy(&r, &lo, 8);
        __builtin_memcpy(reinterpret_cast<char*>(&r) + 8, &hi, 8);
        return r;
    }
}

// FP8: 16 rows x 128 positions, lane l holds row l & 15, 32 (l >> 4) .. + 32.
__device__ __forceinline__ i32x8 fragment_fp8(const uint8_t* tile, int sub) {
    const int lane = threadIdx.x & 63;
    const uint8_t* row = tile + (sub * 16 + (lane & 15)) * kStepBytes;
    const int c = (lane >> 4) * 2;
    i32x8 r;
    __builtin_memcpy(&r, row + ((c ^ (lane & 7)) << 4), 16);
    __builtin_memcpy(reinterpret_cast<char*>(&r) + 16, row + (((c + 1) ^ (lane & 7)) << 4), 16);
    return r;
}

template <typename T>
constexpr bool is_fp8() { return __is_same(T, FP8); }

template <typename T, Mode M, bool Gated>
struct Tiles {
    static constexpr Kind kP = M == kWeightGrad ? kAcross : kAlong;   // m side
    static constexpr Kind kQ = M == kForward ? kAlong : kAcross;      // n side
    static constexpr int kElem = is_fp8<T>() ? 1 : 2;
    static constexpr int kStep = kStepBytes / kElem;                  // contraction per step
};

// One output tile: rows 0 .. m_rows of the m operand, columns of the n
// operand.  Row m of the tile goes to output row out_row0 + m.
struct TileJob {
    Operand p, q;
    int64_t len;             // contraction length
    int32_t m_rows;
    int64_t out_row0;
    const float* p_scales;   // fp8: scales of the tile's first row / of the expert
    const float* q_scales;
};

template <typename T, Mode M, bool Gated, int MI>
__device__ __forceinline__ void run_tile(const GemmArgs& a, const TileJob& job, uint8_t* lds) {
    using S = Tiles<T, M, Gated>;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int wm = wave & 1, wn = wave >> 1;
    f32x4 acc[MI][4];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t steps = (job.len + S::kStep - 1) / S::kStep;
    uint8_t* tp = lds;                                  // two tiles of the m operand,
    uint8_t* tq = lds + 2 * kTileBytes;                 // two of the n operand
    const int p_rows = MI * 32;
    auto bring = [&](int64_t s) {
        const int b = (int)(s & 1) * kTileBytes;
        if (a.aligned || is_fp8<T>()) {
            stage<S::kP, false, S::kElem>(job.p, tp + b, s, job.len, p_rows);
            stage<S::kQ, Gated, S::kElem>(job.q, tq + b, s, job.len, kTileN);
        } else if constexpr (!is_fp8<T>()) {
            stage_elements<S::kP, false>(job.p, tp + b, s, job.len);
            stage_elements<S::kQ, Gated>(job.q, tq + b, s, job.len);
        }
    };
    if (steps > 0) bring(0);
    for (int64_t s = 0; s < steps; ++s) {
        wait_for_loads();
        __syncthreads();                                // tile s is there, tile s - 1 is read
        const int b = (int)(s & 1) * kTileBytes;
        const int64_t rest = job.len - s * S::kStep;
        if (!is_fp8<T>() && rest < S::kStep && a.aligned) {
            zero_tail<S::kP>(tp + b, (int)rest);
            zero_tail<S::kQ>(tq + b, (int)rest);
            __syncthreads();
        }
        if (s + 1 < steps) bring(s + 1);
        if constexpr (is_fp8<T>()) {
            // one step is one scale block: its product, unscaled, then a
            // float32 multiply-add with both scales
            float sq[Gated ? 4 : 1];
            const int64_t kb = job.len / 128;
#pragma unroll
            for (int h = 0; h < (Gated ? 4 : 1); ++h) {
                const int32_t row = tile_row<Gated>(job.q, wn * 64 + h * 16);
                const float* p = job.q_scales + (int64_t)(row >> 7) * kb + s;
                sq[h] = MX_CAN_LOAD(p, 4, kSiteGemmScale) ? *p : 0.0f;
            }
            i32x8 q[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = fragment_fp8(tq + b, wn * 4 + j);
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const int32_t m = (i * 2 + wm) * 16 + (lane & 15);
                const int32_t mc = m < job.m_rows ? m : job.m_rows - 1;
                const float* ps = job.p_scales + (int64_t)mc * kb + s;
                const float sp = MX_CAN_LOAD(ps, 4, kSiteGemmScale) ? *ps : 0.0f;
                const i32x8 p = fragment_fp8(tp + b, i * 2 + wm);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x4 part = mfma_fp8(q[j], p, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
                    const float sc = sp * sq[Gated ? j : 0];
#pragma unroll
                    for (int d = 0; d < 4; ++d) acc[i][j][d] = fmaf(part[d], sc, acc[i][j][d]);
                }
            }
        } else {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                u32x4 q[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) q[j] = fragment<S::kQ>(tq + b, wn * 4 + j, ks);
#pragma unroll
                for (int i = 0; i < MI; ++i) {
                    const u32x4 p = fragment<S::kP>(tp + b, i * 2 + wm, ks);
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = mfma_16(T{}, q[j], p, acc[i][j]);
                }
            }
        }
    }
    __syncthreads();                                    // the next tile's loads may begin
    // Lane l holds columns 4 (l >> 4) .. + 4 of row l & 15 of each 16 x 16 block.
    const int64_t n = a.out_cols;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int32_t m = (i * 2 + wm) * 16 + (lane & 15);
        if (m >= job.m_rows) continue;
        const int64_t row = job.out_row0 + m;
        if constexpr (Gated) {
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const int64_t col = job.q.first + wn * 32 + (j / 2) * 16 + (lane >> 4) * 4;
                f32x4 v;
#pragma unroll
                for (int d = 0; d < 4; ++d) v[d] = silu_mul(acc[i][j][d], acc[i][j + 1][d]);
                store4(a.out, a.out_dtype, a.vector_store, row * n, col, n, v, false);
                if (a.gate_up != nullptr) {
                    store4(a.gate_up, a.out_dtype, a.vector_store, row * 2 * n, col, n, acc[i][j],
                           false);
                    store4(a.gate_up, a.out_dtype, a.vector_store, row * 2 * n + n, col, n,
                           acc[i][j + 1], false);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t col = job.q.first + wn * 64 + j * 16 + (lane >> 4) * 4;
                store4(a.out, a.out_dtype, a.vector_store, row * n, col, n, acc[i][j],
                       M == kWeightGrad && a.accumulate);
            }
        }
    }
}

__device__ __forceinline__ int32_t m_tiles(int32_t rows) { return (rows + kTileM - 1) / kTileM; }

// Forward and row-gradient products: a persistent grid walks the tiles of all
// segments, whose number only the device knows.
template <typename T, Mode M, bool Gated>
__global__ __launch_bounds__(kThreads, 2) void gemm_rows_kernel(GemmArgs a) {
    __shared__ __align__(16) uint8_t lds[4 * kTileBytes];
    __shared__ int32_t first_tile[kMaxExperts + 1];
    __shared__ int32_t wave_total[kThreads / kWave];
    count_row_tiles<kThreads>(a, first_tile, wave_total, m_tiles);
    const int32_t cols_per_tile = Gated ? kTileN / 2 : kTileN;
    const int32_t n_tiles = (int32_t)((a.out_cols + cols_per_tile - 1) / cols_per_tile);
    const int64_t total = (int64_t)first_tile[a.num_experts] * n_tiles;
    // Workgroup b runs on XCD b % 8: each XCD takes a contiguous eighth of the tiles.
    const int64_t per = (total + kXcds - 1) / kXcds;
    const int64_t begin = per * (blockIdx.x % kXcds);
    const int64_t end = begin + per < total ? begin + per : total;
    int e = 0;
    for (int64_t t = begin + blockIdx.x / kXcds; t < end; t += gridDim.x / kXcds) {
        e = expert_of_tile(first_tile, a.num_experts, n_tiles, t, e);
        const Segment sg = segment(a, e);
        const int32_t mt = m_tiles(sg.count);
        const int64_t r = t - (int64_t)first_tile[e] * n_tiles;
        // groups of at most 8 row tiles, rows fastest inside a group
        const int32_t per_group = 8 * n_tiles;
        const int32_t group = (int32_t)(r / per_group);
        const int32_t in_group = (int32_t)(r - (int64_t)group * per_group);
        const int32_t rows_in_group = mt - group * 8 < 8 ? mt - group * 8 : 8;
        const int32_t n_tile = in_group / rows_in_group;
        const int32_t m_tile = group * 8 + in_group - n_tile * rows_in_group;
        // the segment's rows are spread over its tiles in multiples of 64
        const int32_t step = ((sg.count + mt - 1) / mt + 63) / 64 * 64;
        const int64_t m0 = (int64_t)m_tile * step;
        const int32_t rows = (int32_t)(sg.count - m0 < step ? sg.count - m0 : step);
        if (rows <= 0) continue;
        TileJob job;
        job.p = Operand{a.x + (sg.begin + m0) * a.x_row_bytes, a.x_row_bytes, 0, rows, 0};
        job.q = Operand{a.w + (int64_t)e * a.w_expert_bytes, a.w_row_bytes,
                        n_tile * cols_per_tile, (int32_t)a.out_cols,
                        Gated ? (int32_t)a.out_cols : 0};
        job.len = a.len;
        job.m_rows = rows;
        job.out_row0 = sg.begin + m0;
        if constexpr (is_fp8<T>()) {
            job.p_scales = a.x_scales + (sg.begin + m0) * (a.len / 128);
            job.q_scales = static_cast<const float*>(a.w_scales) + (int64_t)e * a.w_scale_rows * (a.len / 128);
        }
        if (rows <= 64) run_tile<T, M, Gated, 2>(a, job, lds);
        else if (rows <= 128) run_tile<T, M, Gated, 4>(a, job, lds);
        else if (rows <= 192) run_tile<T, M, Gated, 6>(a, job, lds);
        else run_tile<T, M, Gated, 8>(a, job, lds);
    }
}

// Weight gradients: E x (n tiles x k tiles) output tiles, each over the rows
// of its expert's segment.
template <typename T>
__global__ __launch_bounds__(kThreads, 2) void gemm_weight_grad_kernel(GemmArgs a) {
    __shared__ __align__(16) uint8_t lds[4 * kTileBytes];
    const int32_t mt = (int32_t)((a.out_rows + kTileM - 1) / kTileM);
    const int32_t nt = (int32_t)((a.out_cols + kTileN - 1) / kTileN);
    const int32_t tiles = mt * nt;
    const int xcd = blockIdx.x % kXcds;
    const int64_t per = (tiles + kXcds - 1) / kXcds;    // each XCD: the same tiles of every expert
    const int64_t total = per * a.num_experts;
    for (int64_t t = blockIdx.x / kXcds; t < total; t += gridDim.x / kXcds) {
        const int32_t e = (int32_t)(t / per);
        const int64_t at = xcd * per + (t - e * per);
        if (at >= tiles) continue;
        const int32_t n_tile = (int32_t)(at / mt), m_tile = (int32_t)(at - (int64_t)n_tile * mt);
        const Segment sg = segment(a, e);
        if (sg.count == 0 && a.accumulate) continue;
        TileJob job;
        job.p = Operand{a.x + sg.begin * a.x_row_bytes, a.x_row_bytes, m_tile * kTileM,
                        (int32_t)a.out_rows, 0};
        job.q = Operand{a.w + sg.begin * a.w_row_bytes, a.w_row_bytes, n_tile * kTileN,
                        (int32_t)a.out_cols, 0};
        job.len = sg.count;
        job.m_rows = (int32_t)(a.out_rows - (int64_t)m_tile * kTileM < kTileM
                                   ? a.out_rows - (int64_t)m_tile * kTileM : kTileM);
        job.out_row0 = (int64_t)e * a.out_rows + (int64_t)m_tile * kTileM;
        job.p_scales = job.q_scales = nullptr;
        run_tile<T, kWeightGrad, false, 8>(a, job, lds);
    }
}

// Workgroups of a persistent grid: one per CU (their LDS fills one).
#ifndef MXMOE_GEMM_GROUPS
#define MXMOE_GEMM_GROUPS 256
#endif
static_assert(MXMOE_GEMM_GROUPS % kXcds == 0, "every XCD has the same number of workgroups");

template <typename... KArgs>
hipError_t start(void (*kernel)(KArgs...), const GemmArgs& a, hipStream_t stream) {
    launch_kernel(kernel, dim3(MXMOE_GEMM_GROUPS), dim3(kThreads), 0, stream, nullptr, nullptr, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_gemm(const GemmArgs& a, hipStream_t stream) {
    if (a.dtype == 3)
        return a.gated ? start(gemm_rows_kernel<FP8, kForward, true>, a, stream)
                       : start(gemm_rows_kernel<FP8, kForward, false>, a, stream);
    if (a.dtype == 1) {
        if (a.transposed) return start(gemm_rows_kernel<F16, kRowGrad, false>, a, stream);
        return a.gated ? start(gemm_rows_kernel<F16, kForward, true>, a, stream)
                       : start(gemm_rows_kernel<F16, kForward, false>, a, stream);
    }
    if (a.transposed) return start(gemm_rows_kernel<BF16, kRowGrad, false>, a, stream);
    return a.gated ? start(gemm_rows_kernel<BF16, kForward, true>, a, stream)
                   : start(gemm_rows_kernel<BF16, kForward, false>, a, stream);
}

hipError_t launch_grouped_wgrad(const GemmArgs& a, hipStream_t stream) {
    return a.dtype == 1 ? start(gemm_weight_grad_kernel<F16>, a, stream)
                        : start(gemm_weight_grad_kernel<BF16>, a, stream);
}

}  // namespace mxmoe
