// What the grouped product kernels share: segments, matrix instructions,
// the gated activation and the output stores.
#pragma once

#include "device_common.h"
#include "launch.h"

namespace mxmoe {

constexpr int kMaxExperts = 1024;

struct FP8 { using storage = uint8_t; };

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// A wave-uniform value, kept in scalar registers.
__device__ __forceinline__ int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }

struct Segment {
    int64_t begin;
    int32_t count;
};

// Rows of expert e, clipped to the array.
__device__ __forceinline__ Segment segment(const int32_t* offsets, const int32_t* sizes,
                                           int64_t num_rows, int e) {
    int64_t b = 0, t = 0, c = num_rows;
    if (MX_CAN_LOAD(offsets + e, 8, kSiteGemmMeta)) {
        b = offsets[e];
        t = offsets[e + 1];
    }
    if (sizes != nullptr && MX_CAN_LOAD(sizes + 3 * e, 4, kSiteGemmMeta)) c = sizes[3 * e];
    b = b < 0 ? 0 : b > num_rows ? num_rows : b;
    t = t < 0 ? 0 : t > num_rows ? num_rows : t;
    c = c < t - b ? c : t - b;
    return Segment{b, (int32_t)(c > 0 ? c : 0)};
}

__device__ __forceinline__ Segment segment(const GemmArgs& a, int e) {
    return segment(a.offsets, a.sizes, a.num_rows, e);
}

// The same for an expert that is the same in the whole wave (rows are below 2^31).
__device__ __forceinline__ Segment uniform_segment(const GemmArgs& a, int e) {
    const Segment s = segment(a, e);
    return Segment{(int64_t)uniform((int32_t)s.begin), uniform(s.count)};
}

// D = A x B + C for A, B of 16 rows x 32 positions; lane l of the result holds
// rows 4 (l >> 4) .. + 4 (A's) of column l & 15 (B's).
__device__ __forceinline__ f32x4 mfma_16(BF16, u32x4 a, u32x4 b, f32x4 c) {
    bf16x8 x, y;
    __builtin_memcpy(&x, &a, 16);
    __builtin_memcpy(&y, &b, 16);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_16(F16, u32x4 a, u32x4 b, f32x4 c) {
    f16x8 x, y;
    __builtin_memcpy(&x, &a, 16);
    __builtin_memcpy(&y, &b, 16);
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(x, y, c, 0, 0, 0);
}

// The same for 16 rows x 128 positions of e4m3, unit block scales.
__device__ __forceinline__ f32x4 mfma_fp8(i32x8 a, i32x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0x7f7f7f7f, 0,
                                                            0x7f7f7f7f);
}

// A float32 result that is rounded here and not together with the conversion
// that follows: the compiler joins a product and its conversion to fp16
// (v_fma_mixlo_f16) in code for single elements and not in code for vectors, and
// the two would differ in the last bit.
__device__ __forceinline__ float rounded(float v) {
    asm("" : "+v"(v));
    return v;
}

__device__ __forceinline__ float silu_mul(float g, float u) {
    return rounded(g / (1.0f + __expf(-g)) * u);
}

__device__ __forceinline__ void store1(void* out, int dtype, int64_t at, float v) {
    if (dtype == 0) {
        float* p = static_cast<float*>(out) + at;
        if (MX_CAN_STORE(p, 4, kSiteGemmOut)) *p = v;
        return;
    }
    uint16_t* p = static_cast<uint16_t*>(out) + at;
    if (MX_CAN_STORE(p, 2, kSiteGemmOut)) *p = dtype == 2 ? from_f32(BF16{}, v) : from_f32(F16{}, v);
}

// Whether the bounds of segment e, clipped to the array, are the wrong way round.
__device__ __forceinline__ bool descends(const GemmArgs& a, int e) {
    if (!MX_CAN_LOAD(a.offsets + e, 8, kSiteGemmMeta)) return false;
    const int64_t b = a.offsets[e], t = a.offsets[e + 1];
    return t < b && t < a.num_rows && b > 0;
}

// Row tiles before each expert, first[0 .. E], for tiles(count) tiles of an
// expert with count rows.  For workgroups of `Threads`; `totals` has one
// element per wave.  Ascending offsets make disjoint segments, so that the
// tiles are fewer than num_rows + E; of others, which may hold every row many
// times over, no tile is counted.
template <int Threads, typename F>
__device__ __forceinline__ void count_row_tiles(const GemmArgs& a, int32_t* first, int32_t* totals,
                                                F&& tiles) {
    constexpr int kPer = kMaxExperts / Threads;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int c[kPer], sum = 0;
    bool unordered = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = tid * kPer + i;
        c[i] = e < a.num_experts ? tiles(segment(a, e).count) : 0;
        unordered |= e < a.num_experts && descends(a, e);
        sum += c[i];
    }
    const int upto = wave_inclusive_sum(sum);
    if (lane == 63) totals[wave] = upto;
    const bool none = __syncthreads_or(unordered);
    int before = upto - sum;
    for (int w = 0; w < wave; ++w) before += totals[w];
    if (none) before = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = tid * kPer + i;
        if (none) c[i] = 0;
        if (e <= a.num_experts) first[e] = before;
        before += c[i];
    }
    if (tid == Threads - 1 && a.num_experts == kMaxExperts) first[kMaxExperts] = before;
    __syncthreads();
}

// The expert e' >= e whose tiles, `n_tiles` to a row tile, hold tile t.
__device__ __forceinline__ int expert_of_tile(const int32_t* first, int num_experts,
                                              int32_t n_tiles, int64_t t, int e) {
    const int lane = threadIdx.x & 63;
    for (;; e += kWave) {
        const int at = e + lane + 1;
        const uint64_t hit =
            __ballot(at >= num_experts || (int64_t)first[at] * n_tiles > t);
        if (hit) return e + __builtin_ctzll(hit);
    }
}

}  // namespace mxmoe
