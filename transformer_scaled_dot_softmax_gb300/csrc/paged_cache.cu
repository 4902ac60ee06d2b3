// paged_cache.cu -- writing new rows into a paged K/V cache and reading cached
// rows back.
//
// An int8 cache keeps a row x of 64 (one token, one head) as whole numbers
// n_i = rint(x_i 2^-e), ties to even, and the exponent e, the least from -126 up
// with max |x_i| <= 127 2^e.  A power of two instead of max / 127: the product
// and its rounding are exact, so the stored row does not depend on how it is
// computed, and n_i 2^e (8 significant bits) is a bf16 number: reading back
// rounds nothing, and attention over the cache is attention over bf16 rows.
// It costs half a bit on average.  In bf16's bits: with max = m 2^k, 1 <= m < 2,
// e is k - 6, or k - 5 where m is past 127/64, which of bf16's mantissas only the
// last one, 255/128, is.  The largest finite numbers, 255 2^120, would become 2^128;
// they are kept as 63 2^122, so that no finite row reads as infinite.
//
// Bound by memory.  8 lanes take one row, 16 bytes each, K and V together; a
// block takes 32 consecutive tokens (or cached rows) of one head, which lie
// together in pages as in head-major rows.  Measured on a GB300: append, 2 x 8,192 tokens
// x 16 heads, bf16 20.0 us (6.7 TB/s of its copy; 20.6 with a row loaded only once its
// page is known), 16 tokens 2.6 us (a launch); read, 16
// sequences of up to 7,936 int8 rows x 16 heads 113 us (204 MB read, 469 MB written, the
// zeros behind shorter sequences among them: 5.9 TB/s).  16-byte loads of int8 rows, 4
// lanes each, take 129: a lane's two stores then lie 32 bytes apart.  8 rows a thread
// instead of 4 take 140, stores that bypass L2 121.
#include <cuda_bf16.h>

#include "kernels.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace mha {
namespace {

constexpr int HD = kAttnHeadDim;
constexpr int kThreads = 256;
constexpr int kRows = kThreads / 8;  // rows of a block at a time
constexpr int kReadRows = 4;         // rows of a thread, reading

// Largest magnitude of a row's bf16 bits, over the row's 8 lanes.
__device__ __forceinline__ uint32_t row_top(const uint4 &u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
#pragma unroll
    for (int d = 1; d < 8; d *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    return top;
}

// The row's stored exponent, and this lane's 8 whole numbers.
__device__ __forceinline__ uint32_t quantise(const uint4 &u, uint2 &out) {
    const uint32_t top = row_top(u);
    out = make_uint2(0u, 0u);
    if (top >= 0x7f80u) return 255u;
    const int biased = static_cast<int>(top >> 7), last = (top & 127u) == 127u ? 1 : 0;
    const uint32_t stored = static_cast<uint32_t>(max(biased - 6 + last, 1));
    const float down = __uint_as_float((254u - stored) << 23);
    const int most = stored == 249u ? 63 : 127;
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t n[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
        n[i] = static_cast<uint32_t>(min(max(__float2int_rn(x * down), -most), most)) & 255u;
    }
    out.x = n[0] | n[1] << 8 | n[2] << 16 | n[3] << 24;
    out.y = n[4] | n[5] << 8 | n[6] << 16 | n[7] << 24;
    return stored;
}

// Values of 8 whole numbers; exact in bf16.
__device__ __forceinline__ uint4 values(const uint2 &n, float power) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int32_t x = static_cast<int32_t>(i < 2 ? n.x : n.y);
        const int lo = i & 1 ? x << 8 >> 24 : x << 24 >> 24, hi = i & 1 ? x >> 24 : x << 16 >> 24;
        w[i] = pack_bf16x2(static_cast<float>(lo) * power, static_cast<float>(hi) * power);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(kThreads) paged_append_kernel(const PagedCache c, const PagedRows k, const PagedRows v) {
    const int token = blockIdx.x * kRows + threadIdx.x / 8, head = blockIdx.y, lane = threadIdx.x & 7;
    pdl_wait();
    pdl_launch_dependents();
    // the last sequence that starts at or before the token, if it reaches it
    int lo = 0, hi = c.B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (c.starts[mid] <= token)
            lo = mid;
        else
            hi = mid;
    }
    const PagedSeq s = paged_seq(c, lo);
    const int pos = s.len - s.n + token - s.row0;
    bool ok = token < c.N && token >= s.row0 && token < s.row0 + s.n && pos >= 0;
    int page = -1;
    uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
    if (ok) {
        x = *reinterpret_cast<const uint4 *>(k.x + head * k.stride_h + token * k.stride_t + 8 * lane);
        y = *reinterpret_cast<const uint4 *>(v.x + head * v.stride_h + token * v.stride_t + 8 * lane);
        page = paged_page(c, lo, pos / c.page);
    }
    ok = page >= 0;
    const int row = head * c.page + pos % c.page;
    const long long at = page * c.stride + row * static_cast<long long>(HD) + 8 * lane;
    if (!c.int8) {
        if (!ok) return;
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(c.k) + at) = x;
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(c.v) + at) = y;
        return;
    }
    uint2 nx, ny;
    const uint32_t ex = quantise(x, nx), ey = quantise(y, ny);
    if (!ok) return;
    *reinterpret_cast<uint2 *>(static_cast<int8_t *>(c.k) + at) = nx;
    *reinterpret_cast<uint2 *>(static_cast<int8_t *>(c.v) + at) = ny;
    if (lane == 0) {
        const long long sat = static_cast<long long>(page) * c.Hkv * c.page + row;
        c.k_scales[sat] = static_cast<uint8_t>(ex);
        c.v_scales[sat] = static_cast<uint8_t>(ey);
    }
}

// 128 rows from `first` on (those before `len`) of a head of sequence b into k, v, at
// row first + i; zeros for pages that are not there and, with kTail, for rows from
// `len` to T.  Called by a whole block.
template <bool kInt8, bool kTail>
__device__ __forceinline__ void copy_rows(const PagedCache &c, int b, int head, int first, int len, int T, __nv_bfloat16 *k,
                                          __nv_bfloat16 *v) {
    const int lane = threadIdx.x & 7, row0 = first + threadIdx.x / 8;
    uint4 x[kReadRows], y[kReadRows];
    uint2 nx[kReadRows], ny[kReadRows];
    uint32_t ex[kReadRows], ey[kReadRows];
    int page[kReadRows];
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
        const int row = row0 + i * kRows;
        page[i] = row < len ? paged_page(c, b, row / c.page) : -1;
    }
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
        const int in = head * c.page + (row0 + i * kRows) % c.page;
        const long long at = page[i] * c.stride + in * static_cast<long long>(HD) + 8 * lane;
        x[i] = y[i] = make_uint4(0u, 0u, 0u, 0u);
        if (kInt8) {
            nx[i] = ny[i] = make_uint2(0u, 0u);
            ex[i] = ey[i] = 127u;
            if (page[i] >= 0) {
                const long long sat = static_cast<long long>(page[i]) * c.Hkv * c.page + in;
                nx[i] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const int8_t *>(c.k) + at));
                ny[i] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const int8_t *>(c.v) + at));
                ex[i] = __ldg(c.k_scales + sat);
                ey[i] = __ldg(c.v_scales + sat);
            }
        } else if (page[i] >= 0) {
            x[i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(c.k) + at));
            y[i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(c.v) + at));
        }
    }
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
        const int row = row0 + i * kRows;
        if (row >= (kTail ? T : len)) continue;
        const long long to = static_cast<long long>(row) * HD + 8 * lane;
        *reinterpret_cast<uint4 *>(k + to) = kInt8 ? values(nx[i], paged_power(ex[i])) : x[i];
        *reinterpret_cast<uint4 *>(v + to) = kInt8 ? values(ny[i], paged_power(ey[i])) : y[i];
    }
}
constexpr int kBlockRows = kRows * kReadRows;
static_assert(kBlockRows == 128, "PagedPlan::blocks");

template <bool kInt8>
__global__ void __launch_bounds__(kThreads) paged_read_kernel(const PagedCache c, __nv_bfloat16 *__restrict__ k,
                                                              __nv_bfloat16 *__restrict__ v, int T, int blocks) {
    const int bh = blockIdx.x / blocks, head = bh % c.Hkv, b = bh / c.Hkv;
    pdl_wait();
    pdl_launch_dependents();
    const long long to = static_cast<long long>(bh) * T * HD;
    copy_rows<kInt8, true>(c, b, head, (blockIdx.x - bh * blocks) * kBlockRows, min(min(max(c.lens[b], 0), c.cap), T), T, k + to,
                           v + to);
}

// The rows of the sequences that have row tiles (see PagedWide), in blocks of 128 rows
// of a head: what attn_paged_bf16.cu would do to an int8 tile for each of the row
// tiles that read it is done once (a chunk of 1,024 x 4 query heads behind 31,744 int8
// rows 268 -> 138 us, this launch 16 of them from cold memory).
template <bool kInt8>
__global__ void __launch_bounds__(kThreads) paged_widen_kernel(const PagedAttnParams p, const PagedWide w) {
    pdl_wait();
    pdl_launch_dependents();
    const PagedPlan at = paged_plan(p.c.B, paged_most_tiles(p.c.N, p.c.B, p.H / p.c.Hkv));
    const int *blocks = p.plan + at.blocks, *slot_b = p.plan + at.slot_b;
    const int slots = min(p.plan[1], w.slots), all = blocks[slots];
    for (long long x = blockIdx.x; x < static_cast<long long>(all) * p.c.Hkv; x += gridDim.x) {
        const int head = static_cast<int>(x / all), i = static_cast<int>(x - static_cast<long long>(head) * all);
        int lo = 0, hi = slots;  // the last place whose first block is at most i
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (blocks[mid] <= i)
                lo = mid;
            else
                hi = mid;
        }
        const int b = slot_b[lo], blk = i - blocks[lo], first = blk * kBlockRows;
        const PagedSeq s = paged_seq(p.c, b);
        const long long to = (static_cast<long long>(lo) * p.c.Hkv + head) * w.cap * HD;
        copy_rows<kInt8, false>(p.c, b, head, first, s.len, s.len, w.k + to, w.v + to);
        if (head == 0 && threadIdx.x < 32) {
            const int key = first + static_cast<int>(threadIdx.x) * 16;
            const bool gone = threadIdx.x < 8 && key < s.len && paged_page(p.c, b, key / p.c.page) < 0;
            const uint32_t bits = __ballot_sync(0xffffffffu, gone);
            if (threadIdx.x == 0) w.gone[static_cast<long long>(lo) * (w.cap / kBlockRows) + blk] = bits;
        }
    }
}

}  // namespace

cudaError_t launch_paged_append(const PagedCache &c, const PagedRows &k, const PagedRows &v, cudaStream_t stream) {
    return launch_kernel(paged_append_kernel, dim3((c.N + kRows - 1) / kRows, c.Hkv), dim3(kThreads), 0, stream, true, 1, c,
                         k, v);
}

cudaError_t launch_paged_read(const PagedCache &c, __nv_bfloat16 *k, __nv_bfloat16 *v, int T, cudaStream_t stream) {
    const int blocks = (T + kBlockRows - 1) / kBlockRows;
    const dim3 grid(static_cast<unsigned>(static_cast<long long>(blocks) * c.B * c.Hkv));
    return c.int8 ? launch_kernel(paged_read_kernel<true>, grid, dim3(kThreads), 0, stream, true, 1, c, k, v, T, blocks)
                  : launch_kernel(paged_read_kernel<false>, grid, dim3(kThreads), 0, stream, true, 1, c, k, v, T, blocks);
}

cudaError_t launch_paged_widen(const PagedAttnParams &p, const PagedWide &w, cudaStream_t stream) {
    const dim3 grid(8 * kSmsPerGpu);
    return p.c.int8 ? launch_kernel(paged_widen_kernel<true>, grid, dim3(kThreads), 0, stream, true, 1, p, w)
                    : launch_kernel(paged_widen_kernel<false>, grid, dim3(kThreads), 0, stream, true, 1, p, w);
}

}  // namespace mha
