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
//
// What bounds them.  With many rows to an expert the matrix cores do, with few
// the bytes of the weights, once each; a weight gradient in float32 writes more
// than it reads.  A workgroup per CU keeps the sums of one output tile in
// registers and walks the contraction in steps of 128 bytes per row, which
// loads put straight into LDS.  It walks the tiles too (persistent): the first
// step of the next tile is under way while this one is stored.
//
// Measured on one MI355X, where a large copy moves 4.9 TB/s, weights alone
// stream at up to 6.2 TB/s and the library's dense products of 8192^3 and 16384^3
// reach 1300 and 1560 TFLOP/s in bf16:
//   32768 rows x 2048 -> 7168, 32 experts, bf16     900 us   1070 TFLOP/s
//   4096 rows x 7168 -> 2 x 2048 gated, 32 experts  405 us   4.8 TB/s, 590 TFLOP/s
//   256 rows x 4096 -> 2 x 2048 gated, 256 experts (162 with rows)
//                                                   950 us   5.7 TB/s
//   row gradient, 16384 rows x 4096 x 4096, f16     562 us   978 TFLOP/s
//   weight gradient, the same in bf16 -> float32    743 us   740 TFLOP/s, of which
//                                                   200 us write 1.07 GB
//   FP8 16384 rows x 4096 -> 4096, 128 experts      595 us   920 TFLOP/s, 3.9 TB/s
// Ragged segments cost the large cases their last tiles: 8192^3 with one expert
// runs at 1310-1370 TFLOP/s.  Tried and slower: the weight gradient's experts
// turned from XCD to XCD, non-temporal stores, a wait past the stores in flight.
#include <type_traits>

#include "device_common.h"
#include "gemm_common.h"
#include "launch.h"

namespace mxmoe {
namespace {

// Four waves, 2 x 2, of up to 128 x 128 results each.  A wave of that size
// reads 32 KiB of fragments from LDS per step; eight waves of 128 x 64 would
// read 192 KiB together in place of 128, as long as their matrix instructions
// take.
constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int kTileM = 256;               // of the wide tiles
constexpr int kStepBytes = 128;           // contraction bytes of one step, a tile row in LDS
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

// The same with 4 bytes a lane.
__device__ __forceinline__ void load4_to_lds(__amdgpu_buffer_rsrc_t rs, uint32_t voffset,
                                             uint32_t soffset, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %3\n\tbuffer_load_dword %0, %1, %2 offen lds"
                 :: "v"(voffset), "s"(rs), "s"(soffset), "s"(lds) : "memory");
}

// The loads to LDS that this wave has issued are done; a barrier by itself
// does not wait for them.
__device__ __forceinline__ void wait_for_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// All but the `N` memory operations issued last are done.
template <int N>
__device__ __forceinline__ void wait_for_all_but() {
    asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}

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

// An operand's loads: one step of a tile of 256 rows (or columns) is 32 loads of
// 1 KiB, eight per wave, and load i of wave w is KiB 4 i + w of the tile.  Lane l
// of a load fills the 16 bytes at position l of its KiB, so the swizzle is applied
// to the address it reads.
// Rows, columns and (in the last step) contraction positions past the end read
// the last ones there are, which zero_tail and the epilogue leave out.
template <Kind K, bool Gated, int ElemBytes, int Size>
struct Loader {
    static constexpr int kLoads = Size / 32;
    // kAcross: tile rows in a KiB; loads i + kOffsets, ... are 16 rows below load i,
    // with its swizzle
    static constexpr int kRowsPerKib = 512 / Size, kRowLanes = kWave / kRowsPerKib;
    static constexpr int kOffsets = K == kAlong ? kLoads : 4 / kRowsPerKib;
    uint32_t voffset[kOffsets];
    const uint8_t* base;          // of the next step
    int64_t step_bytes;

    // Contraction positions `valid` (of a step) exist.
    __device__ __forceinline__ uint32_t offset(const Operand& o, int i, int64_t valid) const {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
        const int kib = i * kWaves + wave;
        if constexpr (K == kAlong) {
            const int r = kib * 8 + (lane >> 3);
            int32_t at = ((lane & 7) ^ (lane >> 3)) * 16;
            const int32_t last = (int32_t)valid * ElemBytes - 16;
            at = at < last ? at : last;
            return (uint32_t)(tile_row<Gated>(o, r) - o.first) * (uint32_t)o.row_bytes + at;
        } else {
            int kk = kib * kRowsPerKib + lane / kRowLanes;
            const int chunk = lane % kRowLanes ^ swizzle_across(kk);
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
        const uint32_t down = Whole ? i / kOffsets * 16 * (uint32_t)o.row_bytes : 0u;
        if (!MX_CAN_LOAD(base + down + v, 16, kSiteGemmLoad)) return;
        load_to_lds(rs, v, (uint32_t)uniform((int32_t)down),
                    lds_address(tile) + (i * kWaves + wave) * 1024);
    }
    __device__ __forceinline__ void next() { base += step_bytes; }
};

// The same for rows that are not 16-byte aligned, through registers, with zeros
// past every end.  A piece of 16 bytes comes by one load from where it lies; one
// that crosses the end of its row is the row's last 16 bytes, shifted down on the
// way to LDS.  (Its elements one by one would be a chain of loads in every step
// of the tiles at the edge: 8 experts, 2000 rows x 2047 transposed 140 us.)
template <Kind K, bool Gated, int Rows>
struct Pieces {
    static constexpr int kPieces = Rows * kStepBytes / 16 / kThreads;
    static constexpr int kChunks = K == kAlong ? 8 : Rows / 8;      // of a tile row
    u32x4 v[kPieces];

    // Tile row of the thread's piece i, and its first element in the matrix' row.
    __device__ __forceinline__ static int row(int i) {
        return (i * kThreads + (int)threadIdx.x) / kChunks;
    }
    __device__ __forceinline__ static int64_t element(const Operand& o, int64_t step, int i) {
        const int r = row(i);
        const int chunk = (int)threadIdx.x % kChunks ^ (K == kAlong ? r & 7 : swizzle_across(r));
        return (K == kAlong ? step * 64 : (int64_t)o.first) + chunk * 8;
    }
    __device__ __forceinline__ static int64_t row_length(const Operand& o, int64_t len) {
        return K == kAlong ? len : o.limit;
    }
    __device__ __forceinline__ void load(const Operand& o, int64_t step, int64_t len) {
        const int64_t n = row_length(o, len);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const uint8_t* line;
            if constexpr (K == kAlong) {
                line = o.base + tile_row<Gated>(o, row(i)) * o.row_bytes;
            } else {
                const int64_t r = step * 64 + row(i);
                line = o.base + (r < len ? r : len - 1) * o.row_bytes;
            }
            const int64_t e = element(o, step, i);
            v[i] = u32x4{0u, 0u, 0u, 0u};
            if (n >= 8) {
                const uint8_t* p = line + (e < n - 8 ? e : n - 8) * 2;
                if (MX_CAN_LOAD(p, 16, kSiteGemmLoad)) __builtin_memcpy(&v[i], p, 16);
            } else {
                // as the last 8 elements of a row, the lower of which do not exist
#pragma unroll 1
                for (int j = 0; j < n; ++j) {
                    const uint16_t* p = reinterpret_cast<const uint16_t*>(line) + j;
                    if (!MX_CAN_LOAD(p, 2, kSiteGemmLoad)) continue;
                    const int at = 8 - (int)n + j;
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        if (at >> 1 == d) v[i][d] |= (uint32_t)*p << (16 * (at & 1));
                }
            }
        }
    }
    __device__ __forceinline__ void store(const Operand& o, uint8_t* tile, int64_t step,
                                          int64_t len) const {
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            int64_t here = row_length(o, len) - element(o, step, i);    // elements that exist
            if (K == kAcross && step * 64 + row(i) >= len) here = 0;
            uint64_t lo = v[i][0] | (uint64_t)v[i][1] << 32, hi = v[i][2] | (uint64_t)v[i][3] << 32;
            if (here < 8) {
                const int bits = here > 0 ? (8 - (int)here) * 16 : 0;
                if (bits >= 64) {
                    lo = hi >> (bits - 64);
                    hi = 0;
                } else if (bits > 0) {
                    lo = lo >> bits | hi << (64 - bits);
                    hi >>= bits;
                }
                if (here <= 0) lo = hi = 0;
            }
            *reinterpret_cast<u32x4*>(tile + (i * kThreads + threadIdx.x) * 16) =
                u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
        }
    }
};

// Zeros at the contraction positions past `valid` (< 64) of a staged tile.
template <Kind K, int Rows>
__device__ __forceinline__ void zero_tail(uint8_t* tile, int valid) {
#pragma unroll 1
    for (int i = 0; i < Rows * kStepBytes / 16 / kThreads; ++i) {
        const int piece = i * kThreads + threadIdx.x;
        bool past;
        if constexpr (K == kAlong) past = ((piece & 7) ^ ((piece >> 3) & 7)) * 8 >= valid;
        else past = piece / (Rows / 8) >= valid;
        if (past) *reinterpret_cast<u32x4*>(tile + piece * 16) = u32x4{0u, 0u, 0u, 0u};
    }
}

typedef __attribute__((address_space(3))) const uint8_t lds_byte;
typedef __attribute__((address_space(3))) const u32x4 lds_u32x4;

// Fragments of 16 rows x 128 contraction bytes of a staged tile, of the 16-row
// blocks first + Step i.  Lane l holds row l & 15 of a block: for 16-bit types
// positions 8 (l >> 4) .. + 8 of each half `ks`, for FP8 positions 32 (l >> 4)
// .. + 32.  What depends on the lane and not on the block alone is kept in a few
// LDS addresses (the swizzle's share of a block index is its low three bits);
// the rest are offsets in the instruction.
template <Kind K, int Step, int Size>
struct Fragments {
    static constexpr int kRowBytes = Size * 2;          // kAcross: of a tile row
    // blocks whose index differs in its low three bits alone
    static constexpr int kAt = K == kAlong ? 2 : 8 / Step;
    lds_byte* at[kAt];

    __device__ __forceinline__ void init(const uint8_t* tile, int first, bool fp8) {
        const int lane = threadIdx.x & 63, g = lane >> 4, j = lane & 15;
        lds_byte* const base = (lds_byte*)tile;
        if constexpr (K == kAlong) {
            lds_byte* const row = base + first * 2048 + j * kStepBytes;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                at[i] = row + (((fp8 ? g * 2 + i : i * 4 + g) ^ (lane & 7)) << 4);
        } else {
            const int kk = g * 8 + (j >> 2), sw = swizzle_across(kk) >> 1;
#pragma unroll
            for (int i = 0; i < kAt; ++i)
                at[i] = base + kk * kRowBytes + (((first + Step * i) ^ sw) << 5) + (j & 3) * 8;
        }
    }
    // On to another slot.
    __device__ __forceinline__ void move(int bytes) {
#pragma unroll
        for (int i = 0; i < kAt; ++i) at[i] += bytes;
    }
    __device__ __forceinline__ u32x4 get(int i, int ks) const {
        if constexpr (K == kAlong) {
            return *(lds_u32x4*)(at[ks] + i * Step * 2048);
        } else {
            // ds_read_b64_tr_b16: the 16 lanes of a group read four rows of 16
            // elements, and lane i gets column i of them.
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
            lds_byte* const p = at[i % kAt] + i / kAt * 8 * 32 + ks * 32 * kRowBytes;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
            const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 4 * kRowBytes));
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

// Tiles of the m and the n operand for one step make a slot of LDS.  kWide: 256
// rows x 256 columns, two slots, for the matrix cores.  kNarrow: 128 rows and
// three slots, two steps of loads under way, for experts with so few rows that
// their weights' bytes are the time, and for FP8, whose float32 sums are made by
// vector instructions and so have to fit half the registers.  kSmall: 128 rows x
// 128 columns and four slots, for calls with few tiles.
enum Shape { kWide, kNarrow, kSmall };

template <typename T, Mode M, bool Gated, Shape H>
struct Tiles {
    static constexpr bool kIsWide = H == kWide;
    static constexpr Kind kP = M == kWeightGrad ? kAcross : kAlong;   // m side
    static constexpr Kind kQ = M == kForward ? kAlong : kAcross;      // n side
    static constexpr int kElem = is_fp8<T>() ? 1 : 2;
    static constexpr int kStep = kStepBytes / kElem;                  // contraction per step
    static constexpr int kRows = kIsWide ? kTileM : kTileM / 2;
    static constexpr int NI = H == kSmall ? 4 : 8;                    // 16-column blocks of a wave
    static constexpr int kTileN = 2 * NI * 16;
    static constexpr int kSlots = kIsWide ? 2 : H == kNarrow ? 3 : 4;
    static constexpr int kPBytes = kRows * kStepBytes, kQBytes = kTileN * kStepBytes;
    static constexpr int kScaleBytes = is_fp8<T>() ? 768 : 0;         // 128 rows, 16 blocks
    static constexpr int kSlot = kPBytes + kQBytes + kScaleBytes;
    // Results pass through LDS 16 rows x kStageCols columns of a wave at a time.
    static constexpr int kStageCols = kIsWide ? 64 : 32;
    static constexpr int kStageRow = kStageCols + 4;  // floats; the rest spreads the banks
    static constexpr int kLds = kSlots * kSlot + kWaves * 16 * kStageRow * 4;
    static constexpr int next(int slot) { return slot + 1 == kSlots ? 0 : slot + 1; }
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

template <typename T, Mode M, bool Gated, Shape H>
struct Loaders {
    using S = Tiles<T, M, Gated, H>;
    static constexpr int kNLoads = S::kTileN / 32;
    Loader<S::kP, false, S::kElem, S::kRows> p;
    Loader<S::kQ, Gated, S::kElem, S::kTileN> q;
    uint32_t scale_offset;        // fp8: of the lane's row (waves 0, 1) or block (wave 2)

    // Loads of the m operand of a tile of 32 MI rows.
    static constexpr int m_loads(int MI) { return S::kP == kAlong ? MI : S::kRows / 32; }

    // Readies the loads of a tile and, where its rows are aligned, sets off
    // those of its first step and, as far as there are whole ones, of the steps
    // after it that have a slot (with two slots the second, else all but one).
    __device__ __forceinline__ void start(const GemmArgs& a, const TileJob& job, uint8_t* lds) {
        if (!a.aligned || job.len <= 0) return;
        p.init(job.p);
        q.init(job.q);
        if constexpr (is_fp8<T>()) {
            const uint32_t row_bytes = (uint32_t)(job.len / 128) * 4;
            const int row = threadIdx.x & 127, block = threadIdx.x & 15;
            scale_offset = threadIdx.x < 128
                               ? (uint32_t)(row < job.m_rows ? row : job.m_rows - 1) * row_bytes
                               : (uint32_t)(tile_row<Gated>(job.q, block * 16) >> 7) * row_bytes;
        }
        step(job, lds, 0, 0);
#pragma unroll
        for (int s = 1; s < (S::kIsWide ? 2 : S::kSlots - 1); ++s)
            if (job.len >= (s + 1) * S::kStep) step(job, lds, s, s);
    }
    // Load i of step s into a slot: first the m operand's, then the n operand's.
    template <bool Whole>
    __device__ __forceinline__ void piece(const TileJob& job, const uint8_t* slot, int64_t s,
                                          int i, int m_loads) {
        const int64_t valid = job.len - s * S::kStep;
        if (i >= m_loads) q.template piece<Whole>(job.q, slot + S::kPBytes, i - m_loads, valid);
        else p.template piece<Whole>(job.p, slot, i, valid);
    }
    // fp8: the scales of step s, 64 per wave: of the rows, then of the blocks.
    __device__ __forceinline__ void scales(const TileJob& job, const uint8_t* slot, int64_t s) {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        if (wave == 3) return;
        const float* base = wave < 2 ? job.p_scales : job.q_scales;
        const __amdgpu_buffer_rsrc_t rs =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(base), (short)0, -1, 0x00020000);
        if (!MX_CAN_LOAD(reinterpret_cast<const uint8_t*>(base) + scale_offset + s * 4, 4,
                         kSiteGemmScale))
            return;
        load4_to_lds(rs, scale_offset, (uint32_t)uniform((int32_t)s * 4),
                     lds_address(slot + S::kPBytes + S::kQBytes) + wave * 256);
    }
    // All loads of step s, the next one, into slot number `at`.
    __device__ __forceinline__ void step(const TileJob& job, uint8_t* lds, int64_t s, int at) {
        const bool whole = job.len - s * S::kStep >= S::kStep;
        const int rows = (job.m_rows + 63) / 64 * 64;
        const uint8_t* slot = lds + at * S::kSlot;
        constexpr int kM = S::kRows / 32;
        if constexpr (is_fp8<T>()) scales(job, slot, s);
        if (whole) {
#pragma unroll
            for (int i = 0; i < kM + kNLoads; ++i)
                if (i >= kM || S::kP == kAcross || i * 32 < rows)
                    piece<true>(job, slot, s, i, kM);
        } else {
#pragma unroll 1
            for (int i = 0; i < kM + kNLoads; ++i)
                if (i >= kM || S::kP == kAcross || i * 32 < rows)
                    piece<false>(job, slot, s, i, kM);
        }
        next();
    }
    __device__ __forceinline__ void next() {
        p.next();
        q.next();
    }
};

// Writes a tile's results.  They pass through LDS, 16 rows x StageCols columns
// of a wave at a time, so that each row is written in pieces of 64 to 256 bytes.
// Lane l of a result holds columns 4 (l >> 4) .. + 4 of row l & 15 of a block.
template <typename OT, Mode M, bool Gated, int StageCols, int MI, int NI>
__device__ __forceinline__ void store_tile(const GemmArgs& a, const TileJob& job,
                                           const f32x4 (&acc)[MI][NI], float* stage, int wm,
                                           int wn) {
    using E = typename OT::storage;
    constexpr int kChunk = 16 / (int)sizeof(E);         // elements of a 16-byte store
    constexpr int kStageRow = StageCols + 4, kBlocks = StageCols / 16;
    const int lane = threadIdx.x & 63;
    const int64_t n = a.out_cols;
    // 16 rows (of which `rows` exist) x kCols staged columns to row0, col0 of a
    // matrix `width` wide whose columns end at `limit`
    auto put = [&](void* base, int64_t width, int64_t row0, int64_t col0, int64_t limit, int rows,
                   auto cols, auto value) {
        constexpr int kCols = decltype(cols)::value;
        constexpr int kPerRow = kCols / kChunk;             // stores of a row
        constexpr int kStores = (16 * kPerRow + kWave - 1) / kWave;
        E* const corner = static_cast<E*>(base) + row0 * width + col0;
        if (a.vector_store && col0 + kCols <= limit) {
            // neighbouring lanes write neighbouring 16 bytes of a row
            const __amdgpu_buffer_rsrc_t rs =
                __builtin_amdgcn_make_buffer_rsrc(corner, (short)0, -1, 0x00020000);
            const int r0 = lane / kPerRow < 16 ? lane / kPerRow : 15;
            const int c = lane % kPerRow * kChunk;
            const uint32_t voffset = (uint32_t)(r0 * width + c) * (uint32_t)sizeof(E);
            const uint32_t down = kWave / kPerRow * (uint32_t)width * (uint32_t)sizeof(E);
            union Store { u32x4 raw; E e[kChunk]; };
            Store v[kStores];
            const bool add = M == kWeightGrad && a.accumulate;
            if (add) {
#pragma unroll
                for (int k = 0; k < kStores; ++k)
                    if (r0 + k * (kWave / kPerRow) < rows)
                        v[k].raw = __builtin_amdgcn_raw_buffer_load_b128(rs, voffset, k * down, 0);
            }
#pragma unroll
            for (int k = 0; k < kStores; ++k)
#pragma unroll
                for (int d = 0; d < kChunk; ++d) {
                    const float f = value(r0 + k * (kWave / kPerRow), c + d);
                    v[k].e[d] = from_f32(OT{}, add ? f + to_f32(OT{}, v[k].e[d]) : f);
                }
#pragma unroll
            for (int k = 0; k < kStores; ++k) {
                const int r = r0 + k * (kWave / kPerRow);
                if (r < rows && lane / kPerRow < 16 && MX_CAN_STORE(corner + r * width + c, 16, kSiteGemmOut))
                    __builtin_amdgcn_raw_buffer_store_b128(v[k].raw, rs, voffset, k * down, 0);
            }
        } else {
            const int here = rows < 16 ? rows : 16;
#pragma unroll 1
            for (int at = lane; at < here * kCols; at += kWave) {
                const int r = at / kCols, c = at % kCols;
                E* p = corner + r * width + c;
                if (col0 + c >= limit || !MX_CAN_STORE(p, sizeof(E), kSiteGemmOut)) continue;
                float f = value(r, c);
                if (M == kWeightGrad && a.accumulate) f += to_f32(OT{}, *p);
                *p = from_f32(OT{}, f);
            }
        }
    };
#pragma unroll
    for (int i = 0; i < MI; ++i) {
        const int m0 = (i * 2 + wm) * 16;
        const int rows = job.m_rows - m0;
        if (rows > 0) {
#pragma unroll
            for (int h = 0; h < NI / kBlocks; ++h) {
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int j = 0; j < kBlocks; ++j)
                    *reinterpret_cast<f32x4*>(stage + (lane & 15) * kStageRow + j * 16 +
                                              (lane >> 4) * 4) = acc[i][h * kBlocks + j];
                __builtin_amdgcn_wave_barrier();
                const int64_t row0 = job.out_row0 + m0;
                if constexpr (Gated) {
                    // blocks 0 and 2 are gates, 1 and 3 their ups
                    const int64_t col0 = job.q.first + (wn * NI + h * kBlocks) * 8;
                    auto gate = [&](int r, int c) {
                        return stage[r * kStageRow + (c >> 4) * 32 + (c & 15)];
                    };
                    auto up = [&](int r, int c) {
                        return stage[r * kStageRow + (c >> 4) * 32 + (c & 15) + 16];
                    };
                    auto both = [&](int r, int c) { return silu_mul(gate(r, c), up(r, c)); };
                    const std::integral_constant<int, StageCols / 2> cols;
                    put(a.out, n, row0, col0, n, rows, cols, both);
                    if (a.gate_up != nullptr) {
                        put(a.gate_up, 2 * n, row0, col0, n, rows, cols, gate);
                        put(static_cast<E*>(a.gate_up) + n, 2 * n, row0, col0, n, rows, cols, up);
                    }
                } else {
                    const int64_t col0 = job.q.first + (wn * NI + h * kBlocks) * 16;
                    put(a.out, n, row0, col0, n, rows, std::integral_constant<int, StageCols>{},
                        [&](int r, int c) { return stage[r * kStageRow + c]; });
                }
            }
        }
    }
}

// One tile, whose first loads are under way (Loaders::start).  `advance` sets off
// the next tile's, between the sums and the stores.
template <typename T, Mode M, bool Gated, Shape H, int MI, typename F>
__device__ __forceinline__ void run_tile(const GemmArgs& a, const TileJob& job, uint8_t* lds,
                                         Loaders<T, M, Gated, H>& loads, F&& advance) {
    using S = Tiles<T, M, Gated, H>;
    constexpr int NI = S::NI, kTileN = S::kTileN;
    constexpr bool Wide = S::kIsWide;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int wm = wave & 1, wn = wave >> 1;
    f32x4 acc[MI][NI];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t steps = (job.len + S::kStep - 1) / S::kStep;
    const int64_t whole = job.len / S::kStep;
    constexpr int kMLoads = Loaders<T, M, Gated, H>::m_loads(MI);
    constexpr int kLoads = kMLoads + Loaders<T, M, Gated, H>::kNLoads;
    Fragments<S::kP, 2, S::kRows> fp;
    Fragments<S::kQ, 1, kTileN> fq;
    fp.init(lds, wm, is_fp8<T>());
    fq.init(lds + S::kPBytes, wn * NI, is_fp8<T>());
    int at = 0;                                         // the slot of the step at hand
    auto next_slot = [&]() {
        const int bytes = at + 1 == S::kSlots ? -at * S::kSlot : S::kSlot;
        fp.move(bytes);
        fq.move(bytes);
        at = S::next(at);
    };
    // Other than wide tiles: the loads of the step that comes kSlots - 1 after the
    // one at hand go into the slot before it, which is free.
    constexpr int kAhead = S::kSlots - 1;
    auto free_slot = [&]() { return lds + (at == 0 ? kAhead : at - 1) * S::kSlot; };
    auto load_ahead = [&](int64_t s, int first, int last) {
        const uint8_t* slot = free_slot();
#pragma unroll
        for (int i = first; i < last; ++i)
            if (i < kLoads) loads.template piece<true>(job, slot, s + kAhead, i, kMLoads);
    };
    // Step s + 1 is there; up to kAhead - 1 whole steps after it are under way.
    auto wait_for_next = [&](int64_t s) {
        const int64_t under_way = whole - (s + 2);
        if (kAhead >= 3 && under_way >= 2) wait_for_all_but<2 * kLoads>();
        else if (kAhead >= 2 && under_way >= 1) wait_for_all_but<kLoads>();
        else wait_for_loads();
    };
    if constexpr (is_fp8<T>()) {
        // A step is one scale block.  Each product of 128 positions starts from
        // zero and is added to the sums with its two scales by vector
        // instructions, three products later, so that they run beside the
        // matrix instructions.  A turn is one m fragment.
        constexpr int kFree = MI - 1, kPerTurn = (kLoads + kFree - 1) / kFree;
        constexpr int kAll = MI * NI, kScales = Gated ? NI : 1;
        i32x8 q[NI], p[2];
        float sp[2], sq[kScales], sc[4];
        f32x4 part[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            part[r] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            sc[r] = 0.0f;
        }
        auto scale = [&](int i) {                       // of row (16-row block i's) or column block
            return *reinterpret_cast<const float*>(lds + at * S::kSlot + S::kPBytes + S::kQBytes +
                                                   i * 4);
        };
        auto row_scale = [&](int i) { return scale((i * 2 + wm) * 16 + (lane & 15)); };
        auto add = [&](int n) {                         // product n - 3
            const int m = (n + kAll - 3) % kAll;
#pragma unroll
            for (int d = 0; d < 4; ++d)
                acc[m / NI][m % NI][d] =
                    fmaf(part[(n + 1) & 3][d], sc[(n + 1) & 3], acc[m / NI][m % NI][d]);
        };
        auto multiply = [&](int64_t s, auto next, bool more) {
            constexpr bool kNext = decltype(next)::value;
            float sq_next[kScales];
#pragma unroll
            for (int t = 0; t < MI; ++t) {
                if (t < kFree) {
                    p[(t + 1) & 1] = fp.get_fp8(t + 1);
                    sp[(t + 1) & 1] = row_scale(t + 1);
                    if (more) {
                        if (t == 0) loads.scales(job, free_slot(), s + kAhead);
                        load_ahead(s, t * kPerTurn, (t + 1) * kPerTurn);
                    }
                }
                if (kNext && t == kFree) {
                    wait_for_next(s);
                    __syncthreads();                    // step s + 1 is there, step s is read
                    next_slot();
                    if (more) loads.next();
                    p[(t + 1) & 1] = fp.get_fp8(0);
                    sp[(t + 1) & 1] = row_scale(0);
#pragma unroll
                    for (int h = 0; h < kScales; ++h) sq_next[h] = scale(128 + wn * NI + h);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < NI; ++j) {
                    const int n = t * NI + j;
                    add(n);
                    part[n & 3] = mfma_fp8(q[j], p[t & 1], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
                    sc[n & 3] = sp[t & 1] * sq[Gated ? j : 0];
                    if (kNext && t == kFree) q[j] = fq.get_fp8(j);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            if (kNext) {
#pragma unroll
                for (int h = 0; h < kScales; ++h) sq[h] = sq_next[h];
            }
        };
        wait_for_loads();
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NI; ++j) q[j] = fq.get_fp8(j);
        p[0] = fp.get_fp8(0);
        sp[0] = row_scale(0);
#pragma unroll
        for (int h = 0; h < kScales; ++h) sq[h] = scale(128 + wn * NI + h);
        int64_t s = 0;
        for (; s + 1 < whole; ++s) multiply(s, std::true_type{}, s + kAhead < whole);
        multiply(s, std::false_type{}, false);
#pragma unroll
        for (int n = 0; n < 3; ++n) add(n);
    } else {
        // A step is 2 MI turns of one m fragment and eight matrix instructions.
        // Fragments are read three turns ahead, those of the next step's first
        // turns in the last three; so the barrier between two steps stands
        // before these, and the matrix instructions run across it.  The loads
        // of a tile begin when the barrier frees its memory, a few per turn:
        // with two slots those of step s + 1, most of them in step s, with more
        // those of step s + kAhead.
        constexpr int kTurns = 2 * MI, kFree = kTurns - 3;
        constexpr int kPerTurn = Wide ? (2 * kLoads + kTurns - 1) / kTurns
                                      : (kLoads + kFree - 1) / kFree;
        constexpr int kSecond = MI < kFree ? MI : kFree;  // turns that read the second half of q
        u32x4 q[2][NI], p[4];
        // turns after kFree that still read the first half of q
        constexpr int kFirst = MI > kFree ? MI - kFree : 0;
        auto first_fragments = [&](int t) {             // of the next step, in turn kFree + t
#pragma unroll
            for (int j = 0; j < NI; ++j)
                if (t < 0 || j * 2 / NI + kFirst == t) q[0][j] = fq.get(j, 0);
            if (t < 0 || t == 1) p[0] = fp.get(0, 0);
            if (t < 0 || t == 2) {
                p[1] = fp.get(1 % MI, 1 / MI);
                p[2] = fp.get(2 % MI, 2 / MI);
            }
        };
        // Next: step s + 1 is whole and follows.  more: the step to load is whole.
        // rest (wide): of the loads of step s + 1, those after the first three
        // turns' are still to be set off.
        auto multiply = [&](int64_t s, auto next, bool rest, bool more) {
            constexpr bool kNext = decltype(next)::value;
#pragma unroll
            for (int t = 0; t < kTurns; ++t) {
                if (t < kFree) p[(t + 3) & 3] = fp.get((t + 3) % MI, (t + 3) / MI);
                if (t < kSecond) {
#pragma unroll
                    for (int j = 0; j < NI; ++j)
                        if (j * kSecond / NI == t) q[1][j] = fq.get(j, 1);
                }
                if (!Wide && kNext && t < kFree && more)
                    load_ahead(s, t * kPerTurn, (t + 1) * kPerTurn);
                if (kNext && t == kFree) {
                    if (Wide) wait_for_loads();
                    else wait_for_next(s);
                    __syncthreads();                    // step s + 1 is there, step s is read
                    next_slot();
                    if (Wide ? rest : more) loads.next();
                }
                if (kNext && t >= kFree) first_fragments(t - kFree);
                if (Wide && kNext && (t < kFree ? rest : more)) {
                    const int turn = t < kFree ? t + 3 : t - kFree;
                    const uint8_t* slot = lds + S::next(at) * S::kSlot;
#pragma unroll
                    for (int i = turn * kPerTurn; i < (turn + 1) * kPerTurn; ++i)
                        if (i < kLoads)
                            loads.template piece<true>(job, slot, t < kFree ? s + 1 : s + 2, i,
                                                       kMLoads);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < NI; ++j)
                    acc[t % MI][j] = mfma_16(T{}, q[t / MI][j], p[t & 3], acc[t % MI][j]);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        auto tail = [&](int slot) {                     // zeros past the end of the last step
            const int valid = (int)(job.len - whole * S::kStep);
            zero_tail<S::kP, S::kRows>(lds + slot * S::kSlot, valid);
            zero_tail<S::kQ, kTileN>(lds + slot * S::kSlot + S::kPBytes, valid);
            __syncthreads();
        };
        if (a.aligned && steps > 0) {
            wait_for_loads();
            __syncthreads();
            if (whole == 0) tail(0);
            first_fragments(-1);
            int64_t s = 0;
            for (; s + 1 < whole; ++s)
                multiply(s, std::true_type{}, s > 0, s + (Wide ? 2 : kAhead) < whole);
            const bool ragged = steps > whole && whole > 0;
            if (ragged) loads.step(job, lds, whole, S::next(at));
            multiply(s, std::false_type{}, false, false);
            if (ragged) {
                wait_for_loads();
                __syncthreads();
                next_slot();
                tail(at);
                first_fragments(-1);
                multiply(whole, std::false_type{}, false, false);
            }
        } else if constexpr (!Wide) {
            // not aligned: the next step is loaded beside this one's products
            Pieces<S::kP, false, S::kRows> pp;
            Pieces<S::kQ, Gated, kTileN> pq;
            auto load = [&](int64_t s) {
                pp.load(job.p, s, job.len);
                pq.load(job.q, s, job.len);
            };
            auto store = [&](uint8_t* slot, int64_t s) {
                pp.store(job.p, slot, s, job.len);
                pq.store(job.q, slot + S::kPBytes, s, job.len);
                __syncthreads();
            };
            if (steps > 0) {
                load(0);
                store(lds, 0);
            }
            for (int64_t s = 0; s < steps; ++s) {
                const bool more = s + 1 < steps;
                if (more) load(s + 1);
                first_fragments(-1);
                multiply(s, std::false_type{}, false, false);
                if (more) {
                    store(lds + S::next(at) * S::kSlot, s + 1);
                    next_slot();
                }
            }
        }
    }
    __syncthreads();                                    // the tiles are read
    advance();
    float* stage = reinterpret_cast<float*>(lds + S::kSlots * S::kSlot) + wave * 16 * S::kStageRow;
    constexpr int kCols = S::kStageCols;
    if (a.out_dtype == 2) store_tile<BF16, M, Gated, kCols>(a, job, acc, stage, wm, wn);
    else if (a.out_dtype == 1) store_tile<F16, M, Gated, kCols>(a, job, acc, stage, wm, wn);
    else store_tile<F32, M, Gated, kCols>(a, job, acc, stage, wm, wn);
}

// Forward and row-gradient products: a persistent grid walks the tiles of all
// segments, whose number only the device knows.
template <typename T, Mode M, bool Gated, Shape H>
__global__ __launch_bounds__(kThreads, 1) void gemm_rows_kernel(GemmArgs a) {
    using S = Tiles<T, M, Gated, H>;
    constexpr bool Wide = S::kIsWide;
    __shared__ __align__(16) uint8_t lds[S::kLds];
    __shared__ int32_t first_tile[kMaxExperts + 1];
    __shared__ int32_t wave_total[kWaves];
    auto m_tiles = [](int32_t rows) { return (rows + S::kRows - 1) / S::kRows; };
    count_row_tiles<kThreads>(a, first_tile, wave_total, m_tiles);
    const int32_t cols_per_tile = Gated ? S::kTileN / 2 : S::kTileN;
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
    Loaders<T, M, Gated, H> loads;
    TileJob job = job_of(t);
    loads.start(a, job, lds);
    while (true) {
        const int64_t next = t + gridDim.x / kXcds;
        TileJob next_job;
        // narrow: looked up ahead, their tiles are short and registers are free
        if (!Wide && next < end) next_job = job_of(next);
        auto advance = [&]() {
            if (next >= end) return;
            if (Wide) next_job = job_of(next);
            loads.start(a, next_job, lds);
        };
        if (job.m_rows <= 64) run_tile<T, M, Gated, H, 2>(a, job, lds, loads, advance);
        else if (!Wide || job.m_rows <= 128)
            run_tile<T, M, Gated, H, 4>(a, job, lds, loads, advance);
        else if constexpr (Wide) {
            if (job.m_rows <= 192) run_tile<T, M, Gated, H, 6>(a, job, lds, loads, advance);
            else run_tile<T, M, Gated, H, 8>(a, job, lds, loads, advance);
        }
        if (next >= end) return;
        t = next;
        job = next_job;
    }
}

// Weight gradients: E x (n tiles x k tiles) output tiles, each over the rows
// of its expert's segment.
template <typename T, Shape H>
__global__ __launch_bounds__(kThreads, 1) void gemm_weight_grad_kernel(GemmArgs a) {
    using S = Tiles<T, kWeightGrad, false, H>;
    __shared__ __align__(16) uint8_t lds[S::kLds];
    const int32_t mt = (int32_t)((a.out_rows + S::kRows - 1) / S::kRows);
    const int32_t nt = (int32_t)((a.out_cols + S::kTileN - 1) / S::kTileN);
    const int64_t tiles = (int64_t)mt * nt;
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
            job.p = Operand{a.x + sg.begin * a.x_row_bytes, a.x_row_bytes, m_tile * S::kRows,
                            (int32_t)a.out_rows, 0};
            job.q = Operand{a.w + sg.begin * a.w_row_bytes, a.w_row_bytes, n_tile * S::kTileN,
                            (int32_t)a.out_cols, 0};
            job.len = sg.count;
            const int64_t rows = a.out_rows - (int64_t)m_tile * S::kRows;
            job.m_rows = (int32_t)(rows < S::kRows ? rows : S::kRows);
            job.out_row0 = (int64_t)e * a.out_rows + (int64_t)m_tile * S::kRows;
            return true;
        }
        return false;
    };
    Loaders<T, kWeightGrad, false, H> loads;
    TileJob job;
    if (!find(job)) return;
    loads.start(a, job, lds);
    while (true) {
        TileJob next_job;
        bool more = false;
        run_tile<T, kWeightGrad, false, H, S::kRows / 32>(a, job, lds, loads, [&]() {
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

// Rows per expert (of the array, the counts are on the device) up to which the
// narrow tiles run.  32 experts, 7168 -> 2 x 2048 gated, narrow against wide:
// 16 rows each 314 and 356 us, 96 rows 334 and 384, 128 rows 343 and 396, 192
// rows 537 and 437: they win as long as an expert's rows make one tile, and
// where the average is 96, ragged counts stay below 128.
#ifndef MXMOE_GEMM_NARROW_ROWS
#define MXMOE_GEMM_NARROW_ROWS 96
#endif
constexpr int64_t kNarrowRows = MXMOE_GEMM_NARROW_ROWS;
// Tiles (of 128 rows x 256 columns, as many as the sizes allow) below which the
// small ones run: two for each CU.  1 expert, 2000 rows x 4096 -> 2048: 44 us
// with them and 91 without; 16 experts, 100 rows x 2704 -> 1304: 36 and 55.  Above,
// they read more than they spread: FP8 16384 rows 737 us with them, 628 without.
#ifndef MXMOE_GEMM_SMALL_TILES
#define MXMOE_GEMM_SMALL_TILES 512
#endif
constexpr int64_t kSmallTiles = MXMOE_GEMM_SMALL_TILES;
// Weight gradient: tiles of 256 x 256 below which the small ones run.  1 expert,
// 2000 rows, 512 x 512: 27 us with them and 63 without; 8 experts, 40 rows, 2048 x
// 4096 (1024 tiles) 81 and 65; 16 experts, 16384 rows, 4096 x 4096: 1181 and 743.
#ifndef MXMOE_WGRAD_SMALL_TILES
#define MXMOE_WGRAD_SMALL_TILES 512
#endif
constexpr int64_t kSmallGradTiles = MXMOE_WGRAD_SMALL_TILES;

template <typename... KArgs>
hipError_t start(void (*kernel)(KArgs...), const GemmArgs& a, hipStream_t stream) {
    launch_kernel(kernel, dim3(MXMOE_GEMM_GROUPS), dim3(kThreads), 0, stream, nullptr, nullptr, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_gemm(const GemmArgs& a, hipStream_t stream) {
    // tiles of 128 rows x 256 columns there can be
    const int64_t cols = a.gated ? 2 * a.out_cols : a.out_cols;
    const int64_t row_tiles = a.num_rows / 128 + (a.num_rows < a.num_experts ? a.num_rows
                                                                             : a.num_experts);
    const bool small = row_tiles * ((cols + 255) / 256) < kSmallTiles;
    auto go = [&](auto type, auto mode, auto gated) {
        using T = decltype(type);
        constexpr Mode M = decltype(mode)::value;
        constexpr bool G = decltype(gated)::value;
        if (small) return start(gemm_rows_kernel<T, M, G, kSmall>, a, stream);
        if constexpr (!is_fp8<T>())
            if (a.aligned && a.num_rows > kNarrowRows * a.num_experts)
                return start(gemm_rows_kernel<T, M, G, kWide>, a, stream);
        return start(gemm_rows_kernel<T, M, G, kNarrow>, a, stream);
    };
    const std::integral_constant<Mode, kForward> forward;
    const std::integral_constant<Mode, kRowGrad> row_grad;
    auto of_type = [&](auto type) {
        if (a.gated) return go(type, forward, std::true_type{});
        if constexpr (!is_fp8<decltype(type)>())
            if (a.transposed) return go(type, row_grad, std::false_type{});
        return go(type, forward, std::false_type{});
    };
    return a.dtype == 3 ? of_type(FP8{}) : a.dtype == 1 ? of_type(F16{}) : of_type(BF16{});
}

hipError_t launch_grouped_wgrad(const GemmArgs& a, hipStream_t stream) {
    const int64_t tiles = ((a.out_rows + 255) / 256) * ((a.out_cols + 255) / 256) * a.num_experts;
    auto go = [&](auto type) {
        using T = decltype(type);
        return tiles < kSmallGradTiles || !a.aligned
                   ? start(gemm_weight_grad_kernel<T, kSmall>, a, stream)
                   : start(gemm_weight_grad_kernel<T, kWide>, a, stream);
    };
    return a.dtype == 1 ? go(F16{}) : go(BF16{});
}

}  // namespace mxmoe
