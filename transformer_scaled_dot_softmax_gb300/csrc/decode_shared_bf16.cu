// decode_shared_bf16.cu -- a decoding step of a batch whose requests share a
// prefix, last launch: the partial sums of all key ranges (the prefix's, and
// the caches' where attn_scored_bf16.cuh took them) merged into the output:
//
//   o = (sum_s w_s O_s) / (sum_s w_s l_s),  w_s = 2^(m_s - M),  M = max_s m_s,
//
// each range with its own reference m_s, sum l_s and unnormalised O_s: exact
// for any division into ranges, and in a fixed order.
//
// Two forms.  decode_merge only merges: bound by latency, the partial sums (256
// bytes per row and range) come from L2.  decode_row_kernel first goes through
// the caches itself, where each K/V head has a single query row: that row is
// one lane in 128 of a tensor-core tile, whose softmax takes as long as a full
// one's, while on the SIMT cores a key costs little more than its 256 bytes
// (caches of up to 1,024 keys, 64 x 16 heads: 28 us against 54; with two rows
// per K/V head 45 against 36, the other way round).  Where the lengths of the
// batch fit the CTA's threads, CTAs take them longest first, and where each has a
// long cache to itself four of them share an SM.  Both, with the limit alone, with
// the order alone, with neither (64 x 16 heads, caches to 1,024, us):
//   random lengths, prefix 8,192  42.5  51.2  45.3  50.3    none  26.4  30.8  27.1  28.6
//   all of 1,024, prefix 8,192    72.8  71.6  70.8  69.0    none  49.3  48.2  50.6  49.5
// (lengths are on the device: no rule on the host can look at them).  The order's
// own registers, 96 where the kernel without it took 80, leave five CTAs an SM
// instead of six: behind a prefix full caches took 60 us then, without one 54.
// 8 lanes read one 128-byte key row, a warp 4 consecutive rows per load, 6 rows per
// lane group in flight (as decode_bf16.cu); a CTA, or a cluster of them that splits
// the keys, serves one head of one batch entry.
#include <cuda_bf16.h>

#include "kernels.h"
#include "scores.cuh"
#include "sm103_ptx.cuh"

namespace mha {
namespace {

constexpr int HD = kAttnHeadDim;

// ------------------------------------------------------------ one row per K/V head
constexpr int kRowWarps = 4;
constexpr int kRowThreads = 32 * kRowWarps;
constexpr int kUnroll = 6;                            // key rows in flight per lane group
constexpr int kKeysPerStep = kRowWarps * 4 * kUnroll;

struct SmemRow {
    float w_m[kRowWarps], w_l[kRowWarps], w_o[kRowWarps][HD];  // a warp's sums
    float c_m, c_l, c_o[HD];                                   // the CTA's, read by the cluster's rank 0
    int len[kRowThreads], b;                                   // the batch's lengths, this CTA's entry
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

template <int kBias>
__global__ void __launch_bounds__(kRowThreads) decode_row_kernel(const __grid_constant__ DecodeRowParams p) {
    __shared__ SmemRow sm;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int slot = lane >> 3;  // which of the warp's 4 consecutive key rows
    const int part = lane & 7;   // which 8 of the 64 features
    const int splits = static_cast<int>(cluster_size());
    const int split = static_cast<int>(cluster_rank());
    long long row = blockIdx.x / splits;  // b H + head: query row, output row and K/V head in one
    int b = static_cast<int>(row / p.H);
    const int head = static_cast<int>(row - static_cast<long long>(b) * p.H);

    int len = p.Tk;
    if (p.cache_lens && p.B <= kRowThreads) {
        // the longest caches first: they would end alone otherwise
        if (threadIdx.x < p.B) sm.len[threadIdx.x] = min(max(p.cache_lens[threadIdx.x], 0), p.Tk);
        __syncthreads();
        if (threadIdx.x < p.B) {
            const int mine = sm.len[threadIdx.x];
            int rank = 0;
            for (int i = 0; i < p.B; ++i) rank += sm.len[i] > mine || (sm.len[i] == mine && i < static_cast<int>(threadIdx.x));
            if (rank == b) sm.b = threadIdx.x;
        }
        __syncthreads();
        b = sm.b;
        len = sm.len[b];
        row = static_cast<long long>(b) * p.H + head;
    } else if (p.cache_lens) {
        len = min(max(p.cache_lens[b], 0), p.Tk);
    }
    const int per = ((len + splits - 1) / splits + kKeysPerStep - 1) / kKeysPerStep * kKeysPerStep;
    const int k_begin = min(len, split * per);
    const int k_end = min(len, k_begin + per);

    float qf[8], acc[8] = {};
    bf16x8_to_f32(*reinterpret_cast<const uint4 *>(p.q + row * HD + part * 8), qf);
    const float slope2 = kBias == kBiasSlopes ? p.f.slopes[head] * kLog2E : 0.f;
    const float *vec = kBias == kBiasBuckets ? bias_vec(p.f, head) : nullptr;
    float m = -INFINITY, l = 0.f;

    const __nv_bfloat16 *kb = p.k + row * p.Tk * HD + part * 8;
    const __nv_bfloat16 *vb = p.v + row * p.Tk * HD + part * 8;
    for (int base = k_begin; base < k_end; base += kKeysPerStep) {
        uint4 ku[kUnroll], vu[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int key = base + (u * kRowWarps + warp) * 4 + slot;
            ku[u] = vu[u] = make_uint4(0u, 0u, 0u, 0u);
            if (key < k_end) {
                ku[u] = __ldcs(reinterpret_cast<const uint4 *>(kb + static_cast<long long>(key) * HD));
                vu[u] = __ldcs(reinterpret_cast<const uint4 *>(vb + static_cast<long long>(key) * HD));
            }
        }
        float s[kUnroll], smax = -INFINITY;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            float kf[8], d = 0.f;
            bf16x8_to_f32(ku[u], kf);
#pragma unroll
            for (int c = 0; c < 8; ++c) d = fmaf(qf[c], kf[c], d);
            d += __shfl_xor_sync(0xffffffffu, d, 1);
            d += __shfl_xor_sync(0xffffffffu, d, 2);
            d += __shfl_xor_sync(0xffffffffu, d, 4);
            const int key = base + (u * kRowWarps + warp) * 4 + slot;
            const int dist = key - (len - 1);  // the query is the cache's last row
            float y = p.capped ? cap_any(d, p.f) : d * p.f.mul;
            if (kBias == kBiasSlopes) y = fmaf(-slope2, fabsf(static_cast<float>(dist)), y);
            // vec may come from the launch two before this one: read past L1
            if (kBias == kBiasBuckets) y += __ldcg(vec + max(min(dist, 0), -p.f.mid));
            s[u] = key < k_end ? y : -INFINITY;
            smax = fmaxf(smax, s[u]);
        }
        smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, 8));
        smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, 16));
        const float m_new = fmaxf(m, smax);
        // without a key to count, or with NaN alone, which has to reach the sums
        const float ref = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = m == -INFINITY ? 0.f : ex2_approx(m - m_new);
        m = m_new;
        l *= alpha;
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] *= alpha;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const float w = ex2_approx(s[u] - ref);
            l += w;
            float vf[8];
            bf16x8_to_f32(vu[u], vf);
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[c] = fmaf(w, vf[c], acc[c]);
        }
    }

    // the warp's 4 key slots hold disjoint keys of the same features
    l += __shfl_xor_sync(0xffffffffu, l, 8);
    l += __shfl_xor_sync(0xffffffffu, l, 16);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        acc[c] += __shfl_xor_sync(0xffffffffu, acc[c], 8);
        acc[c] += __shfl_xor_sync(0xffffffffu, acc[c], 16);
        if (lane < 8) sm.w_o[warp][part * 8 + c] = acc[c];
    }
    if (lane == 0) {
        sm.w_m[warp] = m;
        sm.w_l[warp] = l;
    }
    __syncthreads();
    const int c = threadIdx.x;
    if (c < HD) {
        float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) M = fmaxf(M, sm.w_m[w]);
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
            const float f = merge_weight(sm.w_m[w], M);
            L += f * sm.w_l[w];
            O += f * sm.w_o[w][c];
        }
        sm.c_o[c] = O;
        if (c == 0) {
            sm.c_m = M;
            sm.c_l = L;
        }
    }
    cluster_sync();
    if (split == 0 && c < HD) {
        // the prefix's partial sums are complete once the launch before this one is
        pdl_wait();
        const long long rows = static_cast<long long>(p.B) * p.H;
        float M = -INFINITY, L = 0.f, O = 0.f;
        for (int r = 0; r < splits; ++r) M = fmaxf(M, dsmem_ld(&sm.c_m, r));
        for (int r = 0; r < p.prefix_splits; ++r) M = fmaxf(M, p.part_ml[r * rows + row].x);
        for (int r = 0; r < splits; ++r) {
            const float f = merge_weight(dsmem_ld(&sm.c_m, r), M);
            L += f * dsmem_ld(&sm.c_l, r);
            O += f * dsmem_ld(&sm.c_o[c], r);
        }
#pragma unroll 4
        for (int r = 0; r < p.prefix_splits; ++r) {
            const float2 ml = p.part_ml[r * rows + row];
            const float f = merge_weight(ml.x, M);
            L += f * ml.y;
            O += f * p.part_o[(r * rows + row) * HD + c];
        }
        p.o[row * HD + c] = __float2bfloat16_rn(L != 0.f ? O / L : 0.f);
    }
    // keep every CTA's shared memory alive until rank 0 has read it
    cluster_sync();
}

template <int kBias>
cudaError_t launch_row(const DecodeRowParams &p, int cluster, cudaStream_t stream) {
    // Four CTAs on an SM at a time (by their shared memory) where each has a long
    // cache to itself: those that start later even out what the first had (figures
    // at the top; 40 x 16, all of 1,000 behind 4,096: 41 us against 45 with five,
    // 200 x 16: 158 against 154; 128 x 8, caches to 512: 29 and 27).
    const size_t smem = cluster == 1 && p.Tk > 512 ? 46 * 1024 : 0;
    return launch_kernel(decode_row_kernel<kBias>, dim3(static_cast<unsigned>(p.B * p.H * cluster)), dim3(kRowThreads), smem,
                         stream, p.prefix_splits > 0, static_cast<unsigned>(cluster), p);
}

// ------------------------------------------------------------ merge alone
constexpr int kWarps = 8;

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
    const float inv = l != 0.f ? 1.f / l : 0.f;
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

cudaError_t launch_decode_row(const DecodeRowParams &p, int bias, cudaStream_t stream) {
    // Keys split over a cluster until there are four CTAs for every SM and none
    // has more than 1,024 keys, as long as each still has a step of its own
    // (64 x 16 heads, caches of 1,024: one CTA per head 28 us, two 29, four 38;
    // 16 x 16, caches of 8,192: one 95 us, eight 57).
    const long long heads = static_cast<long long>(p.B) * p.H;
    int cluster = 1;
    while (cluster < 8 && (heads * cluster < 4 * kSmsPerGpu || p.Tk > 1024 * cluster) && p.Tk > kKeysPerStep * cluster)
        cluster *= 2;
    if (bias == kBiasSlopes) return launch_row<kBiasSlopes>(p, cluster, stream);
    if (bias == kBiasBuckets) return launch_row<kBiasBuckets>(p, cluster, stream);
    return launch_row<kBiasNone>(p, cluster, stream);
}

}  // namespace mha
