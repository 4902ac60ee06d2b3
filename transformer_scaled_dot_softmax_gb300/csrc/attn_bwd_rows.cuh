// attn_bwd_rows.cuh -- the per-row work around the attention backward's main
// kernel, shared by attn_bwd_bf16.cu and the scored backward: the softmax
// Jacobian's row terms before it, the dQ conversion after it.
#pragma once

#include <cuda_bf16.h>

#include "kernels.h"
#include "sm103_ptx.cuh"

namespace mha {

// One thread (t) per 8 features of a row, the heads padded to Tq_pad rows:
// D = rowsum(dO O), -lse in log2 units and a zeroed fp32 dQ accumulator; rows
// past Tq (padding up to a whole query block) get lse = +inf, D = 0.  o_lo:
// null, or what rounding took from o.  Every thread of a warp calls it.
__device__ __forceinline__ void bwd_row_terms(long long t, const __nv_bfloat16 *__restrict__ o,
                                              const __nv_bfloat16 *__restrict__ o_lo,
                                              const __nv_bfloat16 *__restrict__ dout, const float *__restrict__ lse,
                                              float *__restrict__ nlse2, float *__restrict__ dvec,
                                              float *__restrict__ dq_acc, long long BH, int Tq, int Tq_pad) {
    constexpr int HD = kAttnHeadDim;
    constexpr float kLog2e = 1.4426950408889634f;
    const long long row = t >> 3;  // over BH * Tq_pad
    const int part = static_cast<int>(t & 7);
    // no early return: the row sum below is a full-warp shuffle
    const bool valid = row < BH * Tq_pad;
    const long long bh = valid ? row / Tq_pad : 0;
    const int i = valid ? static_cast<int>(row - bh * Tq_pad) : Tq;
    float acc = 0.f;
    if (i < Tq) {
        const long long src = (bh * Tq + i) * HD + part * 8;
        const uint4 a = *reinterpret_cast<const uint4 *>(o + src);
        const uint4 g = *reinterpret_cast<const uint4 *>(dout + src);
        const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            acc = fmaf(__uint_as_float(aw[e] << 16), __uint_as_float(gw[e] << 16), acc);
            acc = fmaf(__uint_as_float(aw[e] & 0xffff0000u), __uint_as_float(gw[e] & 0xffff0000u), acc);
        }
        if (o_lo) {
            const uint4 b = *reinterpret_cast<const uint4 *>(o_lo + src);
            const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc = fmaf(__uint_as_float(bw[e] << 16), __uint_as_float(gw[e] << 16), acc);
                acc = fmaf(__uint_as_float(bw[e] & 0xffff0000u), __uint_as_float(gw[e] & 0xffff0000u), acc);
            }
        }
    }
    // reduce over the 8 threads of the row (consecutive lanes)
    acc += __shfl_xor_sync(0xffffffffu, acc, 1);
    acc += __shfl_xor_sync(0xffffffffu, acc, 2);
    acc += __shfl_xor_sync(0xffffffffu, acc, 4);
    if (!valid) return;
    float4 *z = reinterpret_cast<float4 *>(dq_acc + row * HD + part * 8);
    z[0] = make_float4(0.f, 0.f, 0.f, 0.f);
    z[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (part == 0) {
        dvec[row] = acc;
        float l = -INFINITY;
        if (i < Tq) {
            const float x = lse[bh * Tq + i];
            l = x == -INFINITY ? -INFINITY : -x * kLog2e;
        }
        nlse2[row] = l;
    }
}

// The dQ accumulator of a query block j of head bh is 128 rows x 64 fp32 at
// (bh Tq_pad + 128 j) 64, stored as four 8 KiB quarters (rows 32w .. 32w+31),
// each ordered [16-byte chunk x of the row][row within the quarter][4 floats]:
// the order in which a dQ warp stages its rows without shared-memory bank
// conflicts, so that one untiled bulk reduction adds the whole quarter.
__device__ __forceinline__ long long dq_acc_index(long long bh, int Tq_pad, int i, int chunk) {
    return (bh * Tq_pad + (i & ~31)) * kAttnHeadDim + chunk * 128 + (i & 31) * 4;
}

// dQ = bf16(scale * accumulator): one thread (t) per 8 features of a row; a
// warp takes 32 consecutive rows of one feature group (coalesced accumulator
// reads).
__device__ __forceinline__ void bwd_convert_dq(long long t, const float *__restrict__ dq_acc,
                                               __nv_bfloat16 *__restrict__ dq, long long BH, int Tq, int Tq_pad,
                                               float scale) {
    constexpr int HD = kAttnHeadDim;
    const long long grp = t >> 8;  // 32-row group over BH * Tq_pad / 32
    const int part = static_cast<int>((t >> 5) & 7);
    const int groups = Tq_pad >> 5;
    if (grp >= BH * groups) return;
    const long long bh = grp / groups;
    const int i = static_cast<int>(grp - bh * groups) * 32 + static_cast<int>(t & 31);
    if (i >= Tq) return;
    const float4 a = *reinterpret_cast<const float4 *>(dq_acc + dq_acc_index(bh, Tq_pad, i, 2 * part));
    const float4 b = *reinterpret_cast<const float4 *>(dq_acc + dq_acc_index(bh, Tq_pad, i, 2 * part + 1));
    const uint4 w = make_uint4(pack_bf16x2(a.x * scale, a.y * scale), pack_bf16x2(a.z * scale, a.w * scale),
                               pack_bf16x2(b.x * scale, b.y * scale), pack_bf16x2(b.z * scale, b.w * scale));
    *reinterpret_cast<uint4 *>(dq + (bh * Tq + i) * HD + part * 8) = w;
}

}  // namespace mha
