// scored_prep.cu -- the small launches around scored attention: before it the
// expanded bucket bias and the document ranges, after the backward the bias
// table's gradient.
#include <cuda_bf16.h>

#include <algorithm>

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

// Threads [0, n_vec) each write one entry of vec, the next B T one document
// range: the first position of the thread's document and the one past its
// last, by bisection (the ids do not decrease).  Latency-bound: log2 T
// dependent loads.
__global__ void scored_prep(float *__restrict__ vec, int mid, long long n_vec, int H,
                            const __grid_constant__ BucketParams bk, int2 *__restrict__ doc_range,
                            const int32_t *__restrict__ doc_ids, int B, int T) {
    pdl_launch_dependents();
    const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    if (i < n_vec) {
        const int len = 2 * mid + 1;
        const int h = static_cast<int>(i / len);
        const int d = static_cast<int>(i - static_cast<long long>(h) * len) - mid;
        vec[i] = __bfloat162float(bk.table[bucket_of(bk, d) * H + h]) * kLog2E;
        return;
    }
    const long long x = i - n_vec;
    if (!doc_range || x >= static_cast<long long>(B) * T) return;
    const int t = static_cast<int>(x % T);
    const int32_t *ids = doc_ids + (x - t);
    const int32_t id = ids[t];
    int lo = 0, hi = t;  // first position with ids >= id
    while (lo < hi) {
        const int m = (lo + hi) >> 1;
        if (ids[m] < id)
            lo = m + 1;
        else
            hi = m;
    }
    int a = t + 1, z = T;  // first position past t with ids > id
    while (a < z) {
        const int m = (a + z) >> 1;
        if (ids[m] > id)
            z = m;
        else
            a = m + 1;
    }
    doc_range[x] = make_int2(lo, a);
}

// Sums of dS over equal distances, all blocks together: block (h, x) adds the
// slots of the block pairs with kb - j = x - near over batch and key blocks, in
// that order (four interleaved chains).  sums: (H, 2 near + 1, 256).
__global__ void __launch_bounds__(1024) sum_diagonals(const float *__restrict__ diag, float *__restrict__ sums, int B,
                                                      int H, int n_kb, int n_qb, int near, int near_slots) {
    __shared__ float part[4][256];
    pdl_launch_dependents();
    pdl_wait();
    const int h = blockIdx.x, off = static_cast<int>(blockIdx.y) - near;  // kb - j
    const int id = threadIdx.x & 255, chain = threadIdx.x >> 8;
    const int kb0 = max(0, off), kb1 = min(n_kb, n_qb + off);  // j = kb - off in [0, n_qb)
    float sum = 0.f;
    for (int b = 0; b < B; ++b) {
        const float *head = diag + (static_cast<long long>(b) * H + h) * n_kb * near_slots * 256 + id;
#pragma unroll 4
        for (int kb = kb0 + chain; kb < kb1; kb += 4) {
            const int slot = kb - off - max(0, kb - near);
            sum += head[(static_cast<long long>(kb) * near_slots + slot) * 256];
        }
    }
    part[chain][id] = sum;
    __syncthreads();
    if (chain == 0)
        sums[(static_cast<long long>(h) * gridDim.y + blockIdx.y) * 256 + id] =
            (part[0][id] + part[1][id]) + (part[2][id] + part[3][id]);
}

// dtable[u, h] from the distance sums and the far sums: block (u, h) adds the
// distances of bucket u (and the far sums of its direction, if it is the one
// that holds them), threads in a fixed order.
__global__ void __launch_bounds__(kThreads) sum_buckets(const float *__restrict__ sums, const float *__restrict__ far_sum,
                                                        __nv_bfloat16 *__restrict__ dtable, int B, int H, int n_kb,
                                                        int near, const __grid_constant__ BucketParams bk) {
    __shared__ float part[kThreads / 32];
    pdl_wait();
    const int u = blockIdx.x, h = blockIdx.y;
    const int rows = 2 * near + 1;
    float sum = 0.f;
    if (sums) {
        for (int x = threadIdx.x; x < rows * 256; x += kThreads) {
            const int id = x & 255, off = (x >> 8) - near;
            if (id < 255 && bucket_of(bk, 128 * off + id - 127) == u)
                sum += sums[(static_cast<long long>(h) * rows + (x >> 8)) * 256 + id];
        }
        // far past: the last bucket; far future: the last of the other
        // direction, or, with one direction, bucket 0
        const bool past = u == bk.num - 1, future = u == (bk.both ? 2 * bk.num - 1 : 0);
        if (past || future)
            for (int x = threadIdx.x; x < B * n_kb; x += kThreads) {
                const int b = x / n_kb, kb = x - b * n_kb;
                const float *f = far_sum + ((static_cast<long long>(b) * H + h) * n_kb + kb) * 2;
                if (past) sum += f[0];
                if (future) sum += f[1];
            }
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        float s = 0.f;
        for (int x = 0; x < kThreads / 32; ++x) s += part[x];
        dtable[u * H + h] = __float2bfloat16_rn(s);
    }
}

}  // namespace

cudaError_t launch_scored_prep(float *vec, int far, int H, const BucketParams &bk, int2 *doc_range,
                               const int32_t *doc_ids, int B, int T, cudaStream_t stream) {
    const int mid = far + 64;
    const long long n_vec = vec ? static_cast<long long>(H) * (2 * mid + 1) : 0;
    const long long n = n_vec + (doc_range ? static_cast<long long>(B) * T : 0);
    if (n == 0) return cudaSuccess;
    scored_prep<<<static_cast<unsigned>((n + kThreads - 1) / kThreads), kThreads, 0, stream>>>(vec, mid, n_vec, H, bk,
                                                                                               doc_range, doc_ids, B, T);
    return cudaGetLastError();
}

cudaError_t launch_scored_dtable(const float *diag, const float *far_sum, float *sums, __nv_bfloat16 *dtable, int B, int H,
                                 int n_kb, int n_qb, int near, int near_slots, const BucketParams &bk,
                                 cudaStream_t stream) {
    const int total = bk.num * (bk.both ? 2 : 1);
    const bool any = B > 0 && n_kb > 0 && n_qb > 0;
    cudaError_t e;
    if (any && (e = launch_kernel(sum_diagonals, dim3(H, 2 * near + 1), dim3(1024), 0, stream, true, 1, diag, sums, B, H,
                                  n_kb, n_qb, near, near_slots)) != cudaSuccess)
        return e;
    return launch_kernel(sum_buckets, dim3(total, H), dim3(kThreads), 0, stream, any, 1,
                         any ? static_cast<const float *>(sums) : nullptr, far_sum, dtable, B, H, n_kb, near, bk);
}

}  // namespace mha
