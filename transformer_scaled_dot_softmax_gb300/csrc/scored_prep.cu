// scored_prep.cu -- the small launches around scored attention: the expanded
// bucket bias and the document ranges before it (with the row terms, before
// the backward), and after the backward dQ, dK, dV and dtable from the sums
// that it left.  Bound by latency where they are small (the preparation
// 4 to 5 us), by their bytes where they are not (2 x 16 heads x 4,096: before
// 15 us for 84 MB, after 12 us for 50).
#include <cuda_bf16.h>

#include <algorithm>

#include "attn_bwd_rows.cuh"
#include "kernels.h"
#include "scores.cuh"
#include "sm103_ptx.cuh"

namespace mha {
namespace {

constexpr int kThreads = 256;

// Bucket of a distance (key minus query position).
__device__ __forceinline__ int bucket_of(const BucketParams &bk, int d) {
    const int away = bk.both ? abs(d) : max(-d, 0);
    int u = 0;
    for (int x = 1; x < bk.num; ++x) u += away >= bk.starts[x] ? 1 : 0;
    return u + (bk.both && d > 0 ? bk.num : 0);
}

struct PrepParams {
    float *vec;    // (H, vec_stride(mid)), or null
    uint8_t *idx;  // (vec_stride(mid)), or null
    int mid, H;
    BucketParams bk;
    int2 *doc_range;  // (B, T), or null
    const int32_t *doc_ids;
    int B, T;
    long long vec_entries() const { return vec ? static_cast<long long>(H) * vec_stride(mid) : 0; }
    long long entries() const { return vec_entries() + (doc_range ? static_cast<long long>(B) * T : 0); }
};

// Entry i: one of vec, then one document range -- the first position of the
// entry's document and the one past its last, both by bisection at once (the
// ids do not decrease).  Latency-bound: log2 T dependent loads.
__device__ __forceinline__ void prep_entry(const PrepParams &p, long long n_vec, long long i) {
    if (i < n_vec) {
        const int len = vec_stride(p.mid);
        const int h = static_cast<int>(i / len);
        const int d = static_cast<int>(i - static_cast<long long>(h) * len) - p.mid;
        const int u = bucket_of(p.bk, d);
        p.vec[i] = __bfloat162float(p.bk.table[u * p.H + h]) * kLog2E;
        if (p.idx && h == 0) p.idx[i] = static_cast<uint8_t>(u);
        return;
    }
    const long long x = i - n_vec;
    if (!p.doc_range || x >= static_cast<long long>(p.B) * p.T) return;
    const int t = static_cast<int>(x % p.T);
    const int32_t *ids = p.doc_ids + (x - t);
    const int32_t id = ids[t];
    int lo = 0, hi = t;       // first position with ids >= id is in [lo, hi]
    int a = t + 1, z = p.T;   // first position past t with ids > id is in [a, z]
    while (lo < hi || a < z) {
        const int m0 = (lo + hi) >> 1, m1 = (a + z) >> 1;
        const int32_t v0 = ids[min(m0, p.T - 1)], v1 = ids[min(m1, p.T - 1)];
        if (lo < hi) {
            if (v0 < id)
                lo = m0 + 1;
            else
                hi = m0;
        }
        if (a < z) {
            if (v1 > id)
                z = m1;
            else
                a = m1 + 1;
        }
    }
    p.doc_range[x] = make_int2(lo, a);
}

// It may begin while the launch before it ends, as the attention kernels do
// after it.  (The attention may not begin before this has passed its wait: its
// CTAs would sit on the SMs, 3 to 5 % slower.  The backward's first launch does
// not begin early, nor does anything beside its last: row terms that start
// while the forward or another conversion ends slow the products that follow,
// 2 x 16 x 8,192 documents 388 to 397 us, causal 805 to 844.)
__global__ void __launch_bounds__(kThreads) scored_prep(const __grid_constant__ PrepParams p, long long n_vec) {
    pdl_wait();
    pdl_launch_dependents();
    prep_entry(p, n_vec, static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x);
}

// Blocks [0, row_blocks): row terms; the others: preparation.
__global__ void __launch_bounds__(kThreads)
    scored_bwd_pre(const __nv_bfloat16 *__restrict__ o, const __nv_bfloat16 *__restrict__ o_lo,
                   const __nv_bfloat16 *__restrict__ dout, const float *__restrict__ lse, float *__restrict__ nlse2,
                   float *__restrict__ dvec, float *__restrict__ dq_acc, long long BH, int Tq, int Tq_pad,
                   unsigned row_blocks, const __grid_constant__ PrepParams p, long long n_vec,
                   unsigned *__restrict__ next_item) {
    pdl_launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0) *next_item = 0u;
    if (blockIdx.x < row_blocks)
        bwd_row_terms(static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x, o, o_lo, dout, lse, nlse2, dvec, dq_acc,
                      BH, Tq, Tq_pad);
    else
        prep_entry(p, n_vec, static_cast<long long>(blockIdx.x - row_blocks) * kThreads + threadIdx.x);
}

// Blocks [0, table_blocks), first because they take longest: 32 buckets of one
// head each, a lane one bucket, the 8 warps every eighth (batch entry, key
// block) each, all added in a fixed order.  The next kv_blocks: dK (times scale)
// and dV from their partial sums, a thread 8 features of a row.  The others: dQ
// to bf16.
__global__ void __launch_bounds__(kThreads)
    scored_bwd_post(const __grid_constant__ ScoredBwdParams p, __nv_bfloat16 *__restrict__ dq,
                    __nv_bfloat16 *__restrict__ dtable, unsigned table_blocks, unsigned kv_blocks, int n_kb) {
    __shared__ float part[kThreads / 32][32];
    pdl_wait();
    if (blockIdx.x < table_blocks) {
        const int total = p.bk.num * (p.bk.both ? 2 : 1), per_head = (total + 31) / 32;
        const int x = static_cast<int>(blockIdx.x);
        const int h = x / per_head, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const int u = (x - h * per_head) * 32 + lane;
        float sum = 0.f;
        if (u < total)
#pragma unroll 8
            for (int i = warp; i < p.B * n_kb; i += kThreads / 32) {
                const int b = i / n_kb, kb = i - b * n_kb;
                sum += p.bucket_part[((static_cast<long long>(b) * p.H + h) * n_kb + kb) * total + u];
            }
        part[warp][lane] = sum;
        __syncthreads();
        if (warp == 0 && u < total) {
            for (int w = 1; w < kThreads / 32; ++w) sum += part[w][lane];
            dtable[u * p.H + h] = __float2bfloat16_rn(sum);
        }
    } else if (blockIdx.x < table_blocks + kv_blocks) {
        const long long n = static_cast<long long>(p.B) * p.Hkv * p.Tk * 8;  // of one tensor
        long long t = static_cast<long long>(blockIdx.x - table_blocks) * kThreads + threadIdx.x;
        if (t >= 2 * n) return;
        const bool is_dv = t >= n;
        if (is_dv) t -= n;
        const float f = is_dv ? 1.f : p.scale;
        float s[8] = {};
        for (int x = 0; x < p.splits; ++x) {
            const float4 *src = reinterpret_cast<const float4 *>((is_dv ? p.part_dv : p.part_dk) + (x * n + t) * 8);
            const float4 a = src[0], b = src[1];
            s[0] += a.x, s[1] += a.y, s[2] += a.z, s[3] += a.w;
            s[4] += b.x, s[5] += b.y, s[6] += b.z, s[7] += b.w;
        }
        reinterpret_cast<uint4 *>(is_dv ? p.dv : p.dk)[t] =
            make_uint4(pack_bf16x2(s[0] * f, s[1] * f), pack_bf16x2(s[2] * f, s[3] * f), pack_bf16x2(s[4] * f, s[5] * f),
                       pack_bf16x2(s[6] * f, s[7] * f));
    } else {
        bwd_convert_dq(static_cast<long long>(blockIdx.x - table_blocks - kv_blocks) * kThreads + threadIdx.x, p.dq_acc, dq,
                       static_cast<long long>(p.B) * p.H, p.Tq, p.Tq_pad, p.scale);
    }
}

unsigned blocks_of(long long threads) { return static_cast<unsigned>((threads + kThreads - 1) / kThreads); }

}  // namespace

cudaError_t launch_scored_prep(float *vec, int far, int H, const BucketParams &bk, int2 *doc_range,
                               const int32_t *doc_ids, int B, int T, cudaStream_t stream) {
    const PrepParams p{vec, nullptr, vec_mid(far), H, bk, doc_range, doc_ids, B, T};
    if (p.entries() == 0) return cudaSuccess;
    return launch_kernel(scored_prep, dim3(blocks_of(p.entries())), dim3(kThreads), 0, stream, true, 1, p, p.vec_entries());
}

cudaError_t launch_scored_bwd_pre(const __nv_bfloat16 *o, const __nv_bfloat16 *o_lo, const __nv_bfloat16 *dout,
                                  const float *lse, float *nlse2, float *dvec, const ScoredBwdParams &p, float *vec,
                                  uint8_t *idx, int2 *doc_range, const int32_t *doc_ids, cudaStream_t stream) {
    const long long BH = static_cast<long long>(p.B) * p.H;
    const PrepParams pp{vec, idx, p.f.mid, p.H, p.bk, doc_range, doc_ids, p.B, p.Tk};
    const unsigned rows = blocks_of(BH * p.Tq_pad * 8), prep = blocks_of(pp.entries());
    return launch_kernel(scored_bwd_pre, dim3(std::max(rows + prep, 1u)), dim3(kThreads), 0, stream, false, 1, o, o_lo, dout, lse,
                         nlse2, dvec, p.dq_acc, BH, p.Tq, p.Tq_pad, rows, pp, pp.vec_entries(), p.next_item);
}

cudaError_t launch_scored_bwd_post(const ScoredBwdParams &p, __nv_bfloat16 *dq, __nv_bfloat16 *dtable,
                                   cudaStream_t stream) {
    const unsigned dq_blocks = p.Tq > 0 ? blocks_of(static_cast<long long>(p.B) * p.H * p.Tq_pad * 8) : 0;
    const unsigned kv_blocks = p.splits > 1 ? blocks_of(static_cast<long long>(p.B) * p.Hkv * p.Tk * 16) : 0;
    const unsigned table_blocks = dtable ? p.H * ((p.bk.num * (p.bk.both ? 2 : 1) + 31) / 32) : 0;
    const unsigned n = dq_blocks + kv_blocks + table_blocks;
    if (n == 0) return cudaSuccess;
    return launch_kernel(scored_bwd_post, dim3(n), dim3(kThreads), 0, stream, true, 1, p, dq, dtable, table_blocks, kv_blocks,
                         p.Tq > 0 ? (p.Tk + 127) / 128 : 0);
}

}  // namespace mha
