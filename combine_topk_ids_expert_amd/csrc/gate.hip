// Gradient of the gated activation h = silu(g) * u between the two expert
// products, on the rows of the segments:
//
//   s = sigmoid(g);   dg = dh u s (1 + g (1 - s));   du = dh g s
//
// gate_up and its gradient hold a row's n gates, then its n ups.
//
// Bytes bound it: three 16-bit values read and two written for each h.  A
// thread takes 8 columns; whether its row is in a segment comes from one ballot
// over 64 offsets, so padding is not touched.  16384 rows x 2048, bf16: 61 us,
// 335 MB, 5.5 TB/s.
#include "device_common.h"
#include "gemm_common.h"
#include "launch.h"

namespace mxmoe {
namespace {

constexpr int kThreads = 256;

// Whether row r lies in a segment: offsets ascend, so the last segment that
// begins at or before r is the one (64 of them at a time).
__device__ __forceinline__ bool row_in_segment(const int32_t* offsets, const int32_t* sizes,
                                               int num_experts, int64_t num_rows, int64_t r) {
    const int lane = threadIdx.x & 63;
    int begun = 0;
    for (int e0 = 0; e0 < num_experts; e0 += kWave) {
        const int e = e0 + lane;
        const bool before = e < num_experts && MX_CAN_LOAD(offsets + e, 4, kSiteGemmMeta) &&
                            offsets[e] <= r;
        begun += __popcll(__ballot(before));
    }
    if (begun == 0) return false;
    const Segment s = segment(offsets, sizes, num_rows, begun - 1);
    return r >= s.begin && r < s.begin + s.count;
}

__device__ __forceinline__ void silu_mul_grad(float d, float g, float u, float& dg, float& du) {
    const float s = 1.0f / (1.0f + __expf(-g));
    dg = rounded(d * u * s * (1.0f + g * (1.0f - s)));
    du = rounded(d * g * s);
}

// Vec: 8 columns per thread with 16-byte accesses, else one.
template <typename T, bool Vec>
__global__ __launch_bounds__(kThreads) void silu_mul_backward_kernel(
    const uint16_t* grad, const uint16_t* gate_up, uint16_t* grad_gate_up, int64_t n,
    const int32_t* offsets, const int32_t* sizes, int num_experts, int64_t num_rows,
    int64_t row0, int32_t chunks) {
    constexpr int W = Vec ? 8 : 1;
    int64_t chunk;
    const int64_t r = row0 + chunk_row(chunks, chunk);
    const int64_t c = (chunk * blockDim.x + threadIdx.x) * W;
    if (!row_in_segment(offsets, sizes, num_experts, num_rows, r) || c >= n) return;
    const uint16_t* pd = grad + r * n + c;
    const uint16_t* pg = gate_up + r * 2 * n + c;
    uint16_t* og = grad_gate_up + r * 2 * n + c;
    if (!MX_CAN_LOAD(pd, 2 * W, kSiteGateLoad) || !MX_CAN_LOAD(pg, 2 * W, kSiteGateLoad) ||
        !MX_CAN_LOAD(pg + n, 2 * W, kSiteGateLoad))
        return;
    struct alignas(2 * W) Vals { uint16_t v[W]; };
    const Vals d = *reinterpret_cast<const Vals*>(pd), g = *reinterpret_cast<const Vals*>(pg),
               u = *reinterpret_cast<const Vals*>(pg + n);
    Vals dg, du;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        float a, b;
        silu_mul_grad(to_f32(T{}, d.v[i]), to_f32(T{}, g.v[i]), to_f32(T{}, u.v[i]), a, b);
        dg.v[i] = from_f32(T{}, a);
        du.v[i] = from_f32(T{}, b);
    }
    if (MX_CAN_STORE(og, 2 * W, kSiteGateOut)) *reinterpret_cast<Vals*>(og) = dg;
    if (MX_CAN_STORE(og + n, 2 * W, kSiteGateOut)) *reinterpret_cast<Vals*>(og + n) = du;
}

}  // namespace

hipError_t launch_silu_mul_backward(const void* grad, const void* gate_up, void* grad_gate_up,
                                    int dtype, int64_t num_rows, int64_t n,
                                    const int32_t* offsets, const int32_t* sizes,
                                    int32_t num_experts, hipStream_t stream) {
    const bool vec = n % 8 == 0 && ((uintptr_t)grad | (uintptr_t)gate_up |
                                    (uintptr_t)grad_gate_up) % 16 == 0;
    const RowShape sh = row_shape(vec ? n / 8 : n, kThreads);
    return for_row_batches(num_rows, sh, [&](int64_t r0, int64_t, dim3 grid, dim3 block,
                                             hipEvent_t e0, hipEvent_t e1) {
        auto go = [&](auto kernel) {
            launch_kernel(kernel, grid, block, 0, stream, e0, e1,
                          static_cast<const uint16_t*>(grad),
                          static_cast<const uint16_t*>(gate_up),
                          static_cast<uint16_t*>(grad_gate_up), n, offsets, sizes, num_experts,
                          num_rows, r0, sh.chunks);
        };
        if (dtype == 1) vec ? go(silu_mul_backward_kernel<F16, true>)
                            : go(silu_mul_backward_kernel<F16, false>);
        else vec ? go(silu_mul_backward_kernel<BF16, true>)
                 : go(silu_mul_backward_kernel<BF16, false>);
    });
}

}  // namespace mxmoe
