// decode_shared_bf16.cu -- a decoding step of a batch whose requests share a
// prefix, second launch: each request's own cache, merged with the prefix's
// partial sums (attn_scored_bf16.cuh) into the output.
//
//   o = (sum_i w_i O_i) / (sum_i w_i l_i),  w_i = 2^(m_i - M),  M = max_i m_i
//
// over the prefix's key ranges and the cache's, each part with its own
// reference m_i, sum l_i and unnormalised output O_i: exact, whatever the
// split.
//
// Bound by the cache's bytes (256 per key and K/V head).  One CTA (or a
// cluster of them that splits the keys) serves up to 8 query rows of one
// (batch entry, K/V head), so a group of query heads reads its K/V once; 8
// lanes read one 128-byte key row, a warp 4 consecutive rows per load, 6 rows
// per lane in flight, as in decode_bf16.cu.
#include <cuda_bf16.h>

#include "kernels.h"
#include "scores.cuh"
#include "sm103_ptx.cuh"

namespace mha {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnroll = 6;
constexpr int kKeysPerStep = kWarps * 4 * kUnroll;
constexpr int HD = kAttnHeadDim;

template <int NQ>
struct Smem {
    float w_m[kWarps][NQ];
    float w_l[kWarps][NQ];
    float w_o[kWarps][NQ][HD];
    float c_m[NQ];
    float c_l[NQ];
    float c_o[NQ][HD];
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float dsmem_ld(const void *p, uint32_t rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void bf16x8_to_f32(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ float merge_weight(float m, float M) {
    return m == -INFINITY ? 0.f : ex2_approx(m - M);
}

template <int NQ, int kBias>
__global__ void __launch_bounds__(kThreads) decode_shared_kernel(const __grid_constant__ DecodeSharedParams p) {
    __shared__ Smem<NQ> sm;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int slot = lane >> 3;
    const int part = lane & 7;
    const int splits = static_cast<int>(cluster_size());
    const int split = static_cast<int>(cluster_rank());
    const int bkv = static_cast<int>(blockIdx.x) / splits;
    const int b = bkv / p.Hkv, kvh = bkv - b * p.Hkv;
    const int g = p.H / p.Hkv;
    const int row0 = static_cast<int>(blockIdx.y) * NQ;  // of the g Tq rows of this K/V head
    const int rows = min(NQ, g * p.Tq - row0);
    const long long out0 = (static_cast<long long>(b) * p.H + kvh * g) * p.Tq + row0;

    int len = p.Tk;
    if (p.cache_lens) len = min(max(p.cache_lens[b], 0), p.Tk);
    const int per = ((len + splits - 1) / splits + kKeysPerStep - 1) / kKeysPerStep * kKeysPerStep;
    const int k_begin = min(len, split * per);
    const int k_end = min(len, k_begin + per);

    float qf[NQ][8], m_run[NQ], l_run[NQ], acc[NQ][8];
    float slope2[NQ];
    const float *vec[NQ];
    int pos[NQ], see[NQ];  // position among the cache's keys; keys seen
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        const int row = min(row0 + i, g * p.Tq - 1);
        bf16x8_to_f32(*reinterpret_cast<const uint4 *>(p.q + ((static_cast<long long>(b) * p.H + kvh * g) * p.Tq + row) * HD +
                                                       part * 8),
                      qf[i]);
        const int t = row % p.Tq;
        pos[i] = len - p.Tq + t;
        see[i] = p.causal ? pos[i] + 1 : len;
        const int head = kvh * g + row / p.Tq;
        slope2[i] = kBias == kBiasSlopes ? p.f.slopes[head] * kLog2E : 0.f;
        vec[i] = kBias == kBiasBuckets ? p.f.vec + static_cast<long long>(head) * (2 * p.f.mid + 1) + p.f.mid : nullptr;
        m_run[i] = -INFINITY;
        l_run[i] = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[i][c] = 0.f;
    }

    const __nv_bfloat16 *kb = p.k + static_cast<long long>(bkv) * p.Tk * HD + part * 8;
    const __nv_bfloat16 *vb = p.v + static_cast<long long>(bkv) * p.Tk * HD + part * 8;
    for (int base = k_begin; base < k_end; base += kKeysPerStep) {
        uint4 ku[kUnroll], vu[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int key = base + (u * kWarps + warp) * 4 + slot;
            ku[u] = vu[u] = make_uint4(0u, 0u, 0u, 0u);
            if (key < k_end) {
                ku[u] = __ldcs(reinterpret_cast<const uint4 *>(kb + static_cast<long long>(key) * HD));
                vu[u] = __ldcs(reinterpret_cast<const uint4 *>(vb + static_cast<long long>(key) * HD));
            }
        }
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            float s[kUnroll];
            float smax = -INFINITY;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                float kf[8];
                bf16x8_to_f32(ku[u], kf);
                float d = 0.f;
#pragma unroll
                for (int c = 0; c < 8; ++c) d = fmaf(qf[i][c], kf[c], d);
                d += __shfl_xor_sync(0xffffffffu, d, 1);
                d += __shfl_xor_sync(0xffffffffu, d, 2);
                d += __shfl_xor_sync(0xffffffffu, d, 4);
                const int key = base + (u * kWarps + warp) * 4 + slot;
                const int dist = key - pos[i];
                if (p.capped) d = tanh_any(d * p.f.cap_in);
                float y = d * p.f.mul;
                if (kBias == kBiasSlopes) y = fmaf(-slope2[i], fabsf(static_cast<float>(dist)), y);
                // vec may come from the launch two before this one: read past L1
                if (kBias == kBiasBuckets) y += __ldcg(vec[i] + min(max(dist, -p.f.mid), p.f.mid));
                s[u] = key < k_end && key < see[i] ? y : -INFINITY;
                smax = fmaxf(smax, s[u]);
            }
            smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, 8));
            smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, 16));
            const float m_new = fmaxf(m_run[i], smax);
            if (m_new == -INFINITY) continue;
            const float alpha = m_run[i] == -INFINITY ? 0.f : ex2_approx(m_run[i] - m_new);
            m_run[i] = m_new;
            l_run[i] *= alpha;
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[i][c] *= alpha;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const float pu = ex2_approx(s[u] - m_new);
                l_run[i] += pu;
                float vf[8];
                bf16x8_to_f32(vu[u], vf);
#pragma unroll
                for (int c = 0; c < 8; ++c) acc[i][c] = fmaf(pu, vf[c], acc[i][c]);
            }
        }
    }

#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        float l = l_run[i];
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            float a = acc[i][c];
            a += __shfl_xor_sync(0xffffffffu, a, 8);
            a += __shfl_xor_sync(0xffffffffu, a, 16);
            acc[i][c] = a;
        }
        if (lane < 8) {
#pragma unroll
            for (int c = 0; c < 8; ++c) sm.w_o[warp][i][part * 8 + c] = acc[i][c];
        }
        if (lane == 0) {
            sm.w_m[warp][i] = m_run[i];
            sm.w_l[warp][i] = l;
        }
    }
    __syncthreads();
    for (int idx = threadIdx.x; idx < NQ * HD; idx += kThreads) {
        const int i = idx / HD, c = idx - i * HD;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.w_m[w][i]);
        float L = 0.f, O = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = merge_weight(sm.w_m[w][i], M);
            L += f * sm.w_l[w][i];
            O += f * sm.w_o[w][i][c];
        }
        sm.c_o[i][c] = O;
        if (c == 0) {
            sm.c_m[i] = M;
            sm.c_l[i] = L;
        }
    }
    cluster_sync();
    if (split == 0) {
        // the prefix's partial sums are complete once the launch before this one is
        pdl_wait();
        const long long n_rows = static_cast<long long>(p.B) * p.H * p.Tq;
        for (int idx = threadIdx.x; idx < rows * HD; idx += kThreads) {
            const int i = idx / HD, c = idx - i * HD;
            const long long row = out0 + i;
            float M = -INFINITY;
            for (int r = 0; r < splits; ++r) M = fmaxf(M, dsmem_ld(&sm.c_m[i], r));
            for (int r = 0; r < p.prefix_splits; ++r) M = fmaxf(M, p.part_ml[r * n_rows + row].x);
            float L = 0.f, O = 0.f;
            for (int r = 0; r < splits; ++r) {
                const float f = merge_weight(dsmem_ld(&sm.c_m[i], r), M);
                L += f * dsmem_ld(&sm.c_l[i], r);
                O += f * dsmem_ld(&sm.c_o[i][c], r);
            }
#pragma unroll 4
            for (int r = 0; r < p.prefix_splits; ++r) {
                const float2 ml = p.part_ml[r * n_rows + row];
                const float f = merge_weight(ml.x, M);
                L += f * ml.y;
                O += f * p.part_o[(r * n_rows + row) * HD + c];
            }
            p.o[row * HD + c] = __float2bfloat16_rn(L > 0.f ? O / L : 0.f);
        }
    }
    cluster_sync();
}

template <int NQ, int kBias>
cudaError_t launch(const DecodeSharedParams &p, int cluster, cudaStream_t stream) {
    const int rows = p.H / p.Hkv * p.Tq;
    dim3 grid(static_cast<unsigned>(p.B * p.Hkv * cluster), static_cast<unsigned>((rows + NQ - 1) / NQ));
    return launch_kernel(decode_shared_kernel<NQ, kBias>, grid, dim3(kThreads), 0, stream, p.prefix_splits > 0,
                         static_cast<unsigned>(cluster), p);
}

template <int NQ>
cudaError_t launch_nq(const DecodeSharedParams &p, int bias, int cluster, cudaStream_t stream) {
    if (bias == kBiasSlopes) return launch<NQ, kBiasSlopes>(p, cluster, stream);
    if (bias == kBiasBuckets) return launch<NQ, kBiasBuckets>(p, cluster, stream);
    return launch<NQ, kBiasNone>(p, cluster, stream);
}

}  // namespace

cudaError_t launch_decode_shared(const DecodeSharedParams &p, int bias, cudaStream_t stream) {
    const int rows = p.H / p.Hkv * p.Tq;
    // Keys split over a cluster until there are CTAs for every SM, as long as
    // each still has a step of its own.
    const long long ctas = static_cast<long long>(p.B) * p.Hkv * ((rows + 7) / 8);
    int cluster = 1;
    while (cluster < 8 && ctas * cluster < 4 * kSmsPerGpu && p.Tk > kKeysPerStep * cluster) cluster *= 2;
    if (rows <= 1) return launch_nq<1>(p, bias, cluster, stream);
    if (rows <= 2) return launch_nq<2>(p, bias, cluster, stream);
    if (rows <= 4) return launch_nq<4>(p, bias, cluster, stream);
    return launch_nq<8>(p, bias, cluster, stream);
}

}  // namespace mha
