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
#include <type_traits>

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

// Loads straight to LDS: lane l's 16 bytes at base + soffset + voffset go to LDS
// address `lds` + 16 l.  Written as assembly because the compiler, which cannot tell
// the tile being filled from the tile being read, would wait for the loads
// before the next LDS read; wait_for_loads and a barrier stand where the
// filled tile is first read.
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t rs, uint32_t voffset,
                                            uint32_t soffset, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %3\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                 :: "v"(voffset), "s"(rs), "s"(soffset), "s"(lds) : "memory");
}

// The loads to LDS that this wave has issued are done; a barrier by itself
// does not wait for them.
__device__ __forceinline__ void wait_for_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ uint32_t lds_address(const uint8_t* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)p;
}

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

// An operand's loads: one step is 32 loads of 1 KiB, four per wave.  Lane l of a
// load fills the 16 bytes at position l of its KiB, so the swizzle is applied
// to the address it reads.  Rows, columns and (in the last step) contraction
// positions past the end read the last ones there are, which zero_tail and the
// epilogue leave out.
template <Kind K, bool Gated, int ElemBytes>
struct Loader {
    // kAcross: loads 2 and 3 are 4 rows below loads 0 and 1, with their swizzle
    static constexpr int kOffsets = K == kAlong ? 4 : 2;
    uint32_t voffset[kOffsets];
    const uint8_t* base;          // of the next step
    int64_t step_bytes;

    // Contraction positions `valid` (of a step) exist.
    __device__ __forceinline__ uint32_t offset(const Operand& o, int i, int64_t valid) const {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
        const int piece = wave * 4 + i;
        if constexpr (K == kAlong) {
            const int r = piece * 8 + (lane >> 3);
            int32_t at = ((lane & 7) ^ (lane >> 3)) * 16;
            const int32_t last = (int32_t)valid * ElemBytes - 16;
            at = at < last ? at : last;
            return (uint32_t)(tile_row<Gated>(o, r) - o.first) * (uint32_t)o.row_bytes + at;
        } else {
            int kk = piece * 2 + (lane >> 5);
            const int chunk = (lane & 31) ^ swizzle_across(kk);
            kk = kk < valid ? kk : (int)valid - 1;
            int32_t col = o.first + chunk * 8;
            col = col < o.limit ? col : o.limit - 8;
            return (uint32_t)kk * (uint32_t)o.row_bytes + (uint32_t)(col - o.first) * 2;
        }
    }
    __device__ __forceinline__ void init(const Operand& o) {
        if constexpr (K == kAlong) {
            base = o.base + (int64_t)o.first * o.row_bytes;
            step_bytes = kStepBytes;
        } else {
            base = o.base + (int64_t)o.first * 2;
            step_bytes = 64 * o.row_bytes;
        }
#pragma unroll
        for (int i = 0; i < kOffsets; ++i) voffset[i] = offset(o, i, 1 << 20);
    }
    // Load i of the next step, whose `valid` positions exist, into `tile`.
    template <bool Whole>
    __device__ __forceinline__ void piece(const Operand& o, const uint8_t* tile, int i,
                                          int64_t valid) const {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<uint8_t*>(base), (short)0, -1, 0x00020000);
        const uint32_t v = Whole ? voffset[i % kOffsets] : offset(o, i, valid);
        const uint32_t down = Whole && i >= kOffsets ? 4 * (uint32_t)o.row_bytes : 0u;
        if (!MX_CAN_LOAD(base + down + v, 16, kSiteGemmLoad)) return;
        load_to_lds(rs, v, (uint32_t)uniform((int32_t)down), lds_address(tile) + (wave * 4 + i) * 1024);
    }
    __device__ __forceinline__ void next() { base += step_bytes; }
};

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

typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;

// Fragments of 16 rows x 128 contraction bytes of a staged tile, of the 16-row
// blocks first + Step i.  Lane l holds row l & 15 of a block: for 16-bit types
// positions 8 (l >> 4) .. + 8 of each half `ks`, for FP8 positions 32 (l >> 4)
// .. + 32.  What depends on the lane and not on the block alone is kept in a few
// LDS addresses (the swizzle's share of a block index is its low three bits);
// the rest are offsets in the instruction.
template <Kind K, int Step>
struct Fragments {
    uint32_t at[4];

    __device__ __forceinline__ void init(const uint8_t* tile, int first, bool fp8) {
        const int lane = threadIdx.x & 63, g = lane >> 4, j = lane & 15;
        const uint32_t base = lds_address(tile);
        if constexpr (K == kAlong) {
            const uint32_t row = base + first * 2048 + j * kStepBytes;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                at[i] = row + (((fp8 ? g * 2 + i : i * 4 + g) ^ (lane & 7)) << 4);
        } else {
            const int kk = g * 8 + (j >> 2), sw = swizzle_across(kk) >> 1;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                at[i] = base + kk * 512 + (((first + Step * i) ^ sw) << 5) + (j & 3) * 8;
        }
    }
    // The other of the two tiles.
    __device__ __forceinline__ void move(int bytes) {
#pragma unroll
        for (int i = 0; i < (K == kAlong ? 2 : 4); ++i) at[i] += bytes;
    }
    __device__ __forceinline__ u32x4 get(int i, int ks) const {
        if constexpr (K == kAlong) {
            return *(lds_u32x4*)(at[ks] + i * Step * 2048);
        } else {
            // ds_read_b64_tr_b16: the 16 lanes of a group read four rows of 16
            // elements, and lane i gets column i of them.
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
            const uint32_t p = at[i & 3] + (i >> 2) * 4 * Step * 32 + ks * 32 * 512;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * 512));
            u32x4 r;
            __builtin_memcpy(&r, &lo, 8);
            __builtin_memcpy(reinterpret_cast<char*>(&r) + 8, &hi, 8);
            return r;
        }
    }
    __device__ __forceinline__ i32x8 get_fp8(int i) const {
        const u32x4 lo = get(i, 0), hi = get(i, 1);
        i32x8 r;
        __builtin_memcpy(&r, &lo, 16);
        __builtin_memcpy(reinterpret_cast<char*>(&r) + 16, &hi, 16);
        return r;
    }
};

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

template <typename T, Mode M, bool Gated>
struct Loaders {
    using S = Tiles<T, M, Gated>;
    Loader<S::kP, false, S::kElem> p;
    Loader<S::kQ, Gated, S::kElem> q;

    // Readies the loads of a tile and, where its rows are aligned, sets off
    // those of the first step.
    __device__ __forceinline__ void start(const GemmArgs& a, const TileJob& job, uint8_t* lds) {
        if (!a.aligned || job.len <= 0) return;
        p.init(job.p);
        q.init(job.q);
        all<8>(job, lds, 0);
    }
    // Load i of 8 of step s.  A wave's four loads of the m operand are 32 rows:
    // those past a smaller tile's MI x 32 are left out.
    template <bool Whole, int MI>
    __device__ __forceinline__ void piece(const TileJob& job, uint8_t* lds, int64_t s, int i) {
        const int64_t valid = job.len - s * S::kStep;
        uint8_t* tile = lds + (s & 1) * kTileBytes;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        if (i >= 4) q.template piece<Whole>(job.q, tile + 2 * kTileBytes, i - 4, valid);
        else if (MI == 8 || S::kP == kAcross || wave < MI)
            p.template piece<Whole>(job.p, tile, i, valid);
    }
    template <int MI>
    __device__ __forceinline__ void all(const TileJob& job, uint8_t* lds, int64_t s) {
        if (job.len - s * S::kStep >= S::kStep) {
#pragma unroll
            for (int i = 0; i < 8; ++i) piece<true, MI>(job, lds, s, i);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) piece<false, MI>(job, lds, s, i);
        }
        next();
    }
    __device__ __forceinline__ void next() {
        p.next();
        q.next();
    }
};

// One tile; its first step's loads are under way.  `advance` sets off the next
// tile's, between the sums and the stores.
template <typename T, Mode M, bool Gated, int MI, typename F>
__device__ __forceinline__ void run_tile(const GemmArgs& a, const TileJob& job, uint8_t* lds,
                                         Loaders<T, M, Gated>& loads, F&& advance) {
    using S = Tiles<T, M, Gated>;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int wm = wave & 1, wn = wave >> 1;
    f32x4 acc[MI][4];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t steps = (job.len + S::kStep - 1) / S::kStep;
    const bool aligned = a.aligned || is_fp8<T>();
    Fragments<S::kP, 2> fp;
    Fragments<S::kQ, 1> fq;
    fp.init(lds, wm, is_fp8<T>());
    fq.init(lds + 2 * kTileBytes, wn * 4, is_fp8<T>());
    // The products of one step from its tiles; Load: with the loads of step
    // s + 1 (a whole one) in between.
    auto multiply = [&](int64_t s, auto load) {
        constexpr bool kLoad = decltype(load)::value;
        if constexpr (is_fp8<T>()) {
            if (kLoad) {
#pragma unroll
                for (int i = 0; i < 8; ++i) loads.template piece<true, MI>(job, lds, s + 1, i);
            }
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
            for (int j = 0; j < 4; ++j) q[j] = fq.get_fp8(j);
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const int32_t m = (i * 2 + wm) * 16 + (lane & 15);
                const int32_t mc = m < job.m_rows ? m : job.m_rows - 1;
                const float* ps = job.p_scales + (int64_t)mc * kb + s;
                const float sp = MX_CAN_LOAD(ps, 4, kSiteGemmScale) ? *ps : 0.0f;
                const i32x8 p = fp.get_fp8(i);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f32x4 part = mfma_fp8(q[j], p, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
                    const float sc = sp * sq[Gated ? j : 0];
#pragma unroll
                    for (int d = 0; d < 4; ++d) acc[i][j][d] = fmaf(part[d], sc, acc[i][j][d]);
                }
            }
        } else {
            // 2 MI turns of one m fragment and four matrix instructions: the
            // fragment two turns ahead, the n fragments of the second half and
            // the next step's loads are issued in between, in this order.
            u32x4 q[2][4], p[3];
#pragma unroll
            for (int j = 0; j < 4; ++j) q[0][j] = fq.get(j, 0);
            p[0] = fp.get(0, 0);
            p[1] = fp.get(1 % MI, 1 / MI);
#pragma unroll
            for (int t = 0; t < 2 * MI; ++t) {
                if (t + 2 < 2 * MI) p[(t + 2) % 3] = fp.get((t + 2) % MI, (t + 2) / MI);
                if (t < MI) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j * MI / 4 == t) q[1][j] = fq.get(j, 1);
                }
                if (kLoad) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i * MI / 8 == t) loads.template piece<true, MI>(job, lds, s + 1, i);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[t % MI][j] = mfma_16(T{}, q[t / MI][j], p[t % 3], acc[t % MI][j]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        if (kLoad) loads.next();
        if (aligned) {
            const int other = (s & 1) ? -kTileBytes : kTileBytes;
            fp.move(other);
            fq.move(other);
        }
    };
    if (aligned) {
        const int64_t whole = job.len / S::kStep;
        int64_t s = 0;
        for (; s + 1 < whole; ++s) {
            wait_for_loads();
            __syncthreads();                            // step s is there, step s - 1 is read
            multiply(s, std::true_type{});
        }
        for (; s < steps; ++s) {                        // the last whole step and a partial one
            wait_for_loads();
            __syncthreads();
            if (s == whole) {
                zero_tail<S::kP>(lds + (s & 1) * kTileBytes, (int)(job.len - s * S::kStep));
                zero_tail<S::kQ>(lds + (2 + (s & 1)) * kTileBytes, (int)(job.len - s * S::kStep));
                __syncthreads();
            }
            if (s + 1 < steps) loads.template all<MI>(job, lds, s + 1);
            multiply(s, std::false_type{});
        }
    } else if constexpr (!is_fp8<T>()) {
        for (int64_t s = 0; s < steps; ++s) {
            __syncthreads();
            stage_elements<S::kP, false>(job.p, lds, s, job.len);
            stage_elements<S::kQ, Gated>(job.q, lds + 2 * kTileBytes, s, job.len);
            __syncthreads();
            multiply(0, std::false_type{});
        }
    }
    __syncthreads();                                    // the tiles are read
    advance();
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
    const int64_t total = (int64_t)uniform(first_tile[a.num_experts]) * n_tiles;
    // Workgroup b runs on XCD b % 8: each XCD takes a contiguous eighth of the tiles.
    const int64_t per = (total + kXcds - 1) / kXcds;
    const int64_t begin = per * (blockIdx.x % kXcds);
    const int64_t end = begin + per < total ? begin + per : total;
    int e = 0;
    auto job_of = [&](int64_t t) {
        e = expert_of_tile(first_tile, a.num_experts, n_tiles, t, e);
        const Segment sg = uniform_segment(a, e);
        const int32_t mt = m_tiles(sg.count);
        const int64_t r = t - (int64_t)uniform(first_tile[e]) * n_tiles;
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
        TileJob job;
        job.m_rows = (int32_t)(sg.count - m0 < step ? sg.count - m0 : step);
        job.p = Operand{a.x + (sg.begin + m0) * a.x_row_bytes, a.x_row_bytes, 0, job.m_rows, 0};
        job.q = Operand{a.w + (int64_t)e * a.w_expert_bytes, a.w_row_bytes,
                        n_tile * cols_per_tile, (int32_t)a.out_cols,
                        Gated ? (int32_t)a.out_cols : 0};
        job.len = a.len;
        job.out_row0 = sg.begin + m0;
        if constexpr (is_fp8<T>()) {
            job.p_scales = a.x_scales + (sg.begin + m0) * (a.len / 128);
            job.q_scales = static_cast<const float*>(a.w_scales) +
                           (int64_t)e * a.w_scale_rows * (a.len / 128);
        }
        return job;
    };
    int64_t t = begin + blockIdx.x / kXcds;
    if (t >= end) return;
    Loaders<T, M, Gated> loads;
    TileJob job = job_of(t);
    loads.start(a, job, lds);
    while (true) {
        const int64_t next = t + gridDim.x / kXcds;
        TileJob next_job;
        auto advance = [&]() {
            if (next >= end) return;
            next_job = job_of(next);
            loads.start(a, next_job, lds);
        };
        if (job.m_rows <= 64) run_tile<T, M, Gated, 2>(a, job, lds, loads, advance);
        else if (job.m_rows <= 128) run_tile<T, M, Gated, 4>(a, job, lds, loads, advance);
        else if (job.m_rows <= 192) run_tile<T, M, Gated, 6>(a, job, lds, loads, advance);
        else run_tile<T, M, Gated, 8>(a, job, lds, loads, advance);
        if (next >= end) return;
        t = next;
        job = next_job;
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
    int64_t t = blockIdx.x / kXcds;
    // the next tile of this workgroup, from t on; false: none
    auto find = [&](TileJob& job) {
        for (; t < total; t += gridDim.x / kXcds) {
            const int32_t e = (int32_t)(t / per);
            const int64_t at = xcd * per + (t - e * per);
            const Segment sg = uniform_segment(a, e);
            if (at >= tiles || (sg.count == 0 && a.accumulate)) continue;
            const int32_t n_tile = (int32_t)(at / mt), m_tile = (int32_t)(at - (int64_t)n_tile * mt);
            job.p = Operand{a.x + sg.begin * a.x_row_bytes, a.x_row_bytes, m_tile * kTileM,
                            (int32_t)a.out_rows, 0};
            job.q = Operand{a.w + sg.begin * a.w_row_bytes, a.w_row_bytes, n_tile * kTileN,
                            (int32_t)a.out_cols, 0};
            job.len = sg.count;
            job.m_rows = (int32_t)(a.out_rows - (int64_t)m_tile * kTileM < kTileM
                                       ? a.out_rows - (int64_t)m_tile * kTileM : kTileM);
            job.out_row0 = (int64_t)e * a.out_rows + (int64_t)m_tile * kTileM;
            return true;
        }
        return false;
    };
    Loaders<T, kWeightGrad, false> loads;
    TileJob job;
    if (!find(job)) return;
    loads.start(a, job, lds);
    while (true) {
        TileJob next_job;
        bool more = false;
        run_tile<T, kWeightGrad, false, 8>(a, job, lds, loads, [&]() {
            t += gridDim.x / kXcds;
            more = find(next_job);
            if (more) loads.start(a, next_job, lds);
        });
        if (!more) return;
        job = next_job;
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
