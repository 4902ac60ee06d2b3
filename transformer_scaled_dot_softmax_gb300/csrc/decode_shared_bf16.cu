// decode_shared_bf16.cu -- a decoding step of a batch whose requests share a
// prefix, last launch: the partial sums of all key ranges, the prefix's and
// the caches' (attn_scored_bf16.cuh), merged into the output:
//
//   o = (sum_s w_s O_s) / (sum_s w_s l_s),  w_s = 2^(m_s - M),  M = max_s m_s,
//
// each range with its own reference m_s, sum l_s and unnormalised O_s: exact
// for any division into ranges, and in a fixed order.  Bound by latency: the
// partial sums (256 bytes per row and range) come from L2.
#include <cuda_bf16.h>

#include "kernels.h"
#include "sm103_ptx.cuh"

namespace mha {
namespace {

constexpr int kWarps = 8;
constexpr int HD = kAttnHeadDim;

// kPer warps per row, each taking every kPer-th range; a lane two features.
template <int kPer>
__global__ void __launch_bounds__(32 * kWarps) decode_merge(const float *__restrict__ part_o,
                                                            const float2 *__restrict__ part_ml,
                                                            __nv_bfloat16 *__restrict__ o, int parts, long long rows) {
    __shared__ float sm_o[kWarps][HD];
    __shared__ float sm_m[kWarps], sm_l[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * (kWarps / kPer) + warp / kPer;
    const int first = warp % kPer;
    pdl_wait();
    float m = -INFINITY, l = 0.f;
    float2 acc = make_float2(0.f, 0.f);
    if (row < rows) {
        // 32 of the warp's ranges at a time, a lane each for (m, l)
        for (int s0 = first; s0 < parts; s0 += 32 * kPer) {
            const int s = s0 + lane * kPer;
            const float2 ml = s < parts ? part_ml[s * rows + row] : make_float2(-INFINITY, 0.f);
            float mm = ml.x;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, x));
            const float m_new = fmaxf(m, mm);
            if (m_new == -INFINITY) continue;
            const float keep = m == -INFINITY ? 0.f : ex2_approx(m - m_new);
            const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m_new);
            float fl = f * ml.y;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) fl += __shfl_xor_sync(0xffffffffu, fl, x);
            m = m_new;
            l = l * keep + fl;
            acc.x *= keep;
            acc.y *= keep;
            const int n = min(32, (parts - s0 + kPer - 1) / kPer);
#pragma unroll 4
            for (int i = 0; i < n; ++i) {
                const float fi = __shfl_sync(0xffffffffu, f, i);
                // a range without a visible key left its sums unwritten
                if (fi != 0.f) {
                    const float2 v = reinterpret_cast<const float2 *>(part_o + ((s0 + i * kPer) * rows + row) * HD)[lane];
                    acc.x = fmaf(fi, v.x, acc.x);
                    acc.y = fmaf(fi, v.y, acc.y);
                }
            }
        }
    }
    if (kPer > 1) {
        sm_o[warp][2 * lane] = acc.x;
        sm_o[warp][2 * lane + 1] = acc.y;
        if (lane == 0) {
            sm_m[warp] = m;
            sm_l[warp] = l;
        }
        __syncthreads();
        if (first != 0) return;
        float M = -INFINITY;
        for (int w = 0; w < kPer; ++w) M = fmaxf(M, sm_m[warp + w]);
        l = 0.f;
        acc = make_float2(0.f, 0.f);
        for (int w = 0; w < kPer; ++w) {
            const float f = sm_m[warp + w] == -INFINITY ? 0.f : ex2_approx(sm_m[warp + w] - M);
            l = fmaf(f, sm_l[warp + w], l);
            acc.x = fmaf(f, sm_o[warp + w][2 * lane], acc.x);
            acc.y = fmaf(f, sm_o[warp + w][2 * lane + 1], acc.y);
        }
    }
    if (row >= rows) return;
    const float inv = l > 0.f ? 1.f / l : 0.f;
    reinterpret_cast<uint32_t *>(o + row * HD)[lane] = pack_bf16x2(acc.x * inv, acc.y * inv);
}

template <int kPer>
cudaError_t launch(const float *part_o, const float2 *part_ml, __nv_bfloat16 *o, int parts, long long rows,
                   cudaStream_t stream) {
    constexpr int kRows = kWarps / kPer;
    return launch_kernel(decode_merge<kPer>, dim3(static_cast<unsigned>((rows + kRows - 1) / kRows)), dim3(32 * kWarps), 0,
                         stream, true, 1, part_o, part_ml, o, parts, rows);
}

}  // namespace

cudaError_t launch_decode_merge(const float *part_o, const float2 *part_ml, __nv_bfloat16 *o, int parts, long long rows,
                                cudaStream_t stream) {
    // a warp per row while it has few ranges; otherwise the block's warps share them
    if (parts > 8) return launch<8>(part_o, part_ml, o, parts, rows, stream);
    return launch<1>(part_o, part_ml, o, parts, rows, stream);
}

}  // namespace mha
