// attn_scored_bwd_bf16.cu -- gradients of scored attention for sm_103a
// (scores as defined in scores.cuh).
//
//   P = exp(S - lse),  dV = P^T dO,  dP = dO V^T,  dS = P (.) (dP - D),
//   dZ = dS (.) (1 - t^2)  with t = tanh(z / cap)  (dZ = dS uncapped),
//   dQ = scale dZ K,  dK = scale dZ^T Q,
//   dtable[u, h] = sum over pairs of bucket u of dS,
// dK and dV summed over the query heads that share the K/V head.
//
// Launches: one before (row terms; the expanded bias and document ranges of
// scored_prep.cu), the kernel below, one after (dQ to bf16, sums of partial dK,
// dV and dtable).  The kernel's warp roles, tensor-memory plan and issue order
// are attn_bwd_main's (attn_bwd_bf16.cu).  What differs:
//   * an item is a K/V head's 128 keys and walks (query head of the group, query
//     block) pairs, so dK and dV of the group are summed in tensor memory, in
//     a fixed order.  Where that makes too few items the group's heads are
//     divided among several, which leave fp32 sums for the last launch;
//   * one CTA per SM takes items off a counter and runs their pairs on without
//     a gap: the next item's keys, query blocks and first scores come while the
//     last pair's products run, and dK and dV leave while the next item's
//     first products wait.  A CTA per item instead spent about 8 us of each
//     on its start and end beside 1.6 us a pair; this spends 4 to 5 (B 2, h 16,
//     8,192 in 12 causal documents, capped: 277 -> 238 us; 16 causal heads of
//     8 x 1,024: 113 -> 95; 2 x 16 x 8,192 causal: 815 -> 807);
//   * a key is seen by one interval of queries [lo, hi) (causal, prefix,
//     documents and padding all end in one), which bounds the query blocks
//     walked and masks the ones seen in part;
//   * a bucket bias is read from a window of 256 distances that comes with the
//     query block, for block pairs nearer than the last bucket's first
//     distance; past it, it is one value;
//   * the bias's gradient sums dS over the buckets of its distances.  A block
//     pair past the last bucket's first distance adds up in one register per
//     thread; in a nearer one each warp adds its 32 x 32 pairs along their
//     diagonals (a shuffle and an add per pair), then the diagonals of each
//     bucket (a segmented scan over the lanes), into sums of its own in shared
//     memory.  A CTA adds the warps' sums once per head and leaves one per
//     bucket, and the last launch adds those, all in a fixed order: dtable does
//     not depend on the order in which CTAs finish.  (Adding over the warps in
//     every near pair instead cost 4,300 cycles of its 3,900; a warp set apart
//     for it fell behind.)
//
// Bound: like attn_bwd_main by the score warps, 16 of them on 96 registers,
// issuing in 47 to 56 of 100 cycles and waiting for tensor memory and for one
// another in the others; the tensor cores are 28 to 35 % busy.  Measured, 2 x
// 16 heads x 8,192, causal, all launches: plain 806 us (852 TFLOP/s), slopes
// 843, 32 buckets 991, cap 50 947, both 1,030, 12 documents 208; 16 x 8 heads x 512,
// all keys: plain 53, slopes 56, buckets 71.  Of that the launches before and
// after take what their bytes do (at 8,192: 100 MB read and 67 written, 67
// read and 34 written).
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "scores.cuh"
#include "sm103_ptx.cuh"

namespace mha {
namespace {

constexpr int HD = kAttnHeadDim;
constexpr int BQ = 128;
constexpr int BKB = 128;
constexpr uint32_t kTile = BQ * HD * 2;
constexpr uint32_t kColS = 0, kColDP = 128, kColP = 256, kColDV = 320, kColDK = 384, kColDQ = 448;
constexpr int kSoftmaxWarps = 16;
constexpr int kThreads = 32 * (2 + kSoftmaxWarps);
constexpr int kStages = 3;
constexpr int kItems = 4;

// One item of work: 128 keys of a K/V head and query heads that share it.
struct Item {
    int b, bkv, kb;        // batch entry, b Hkv + K/V head, key block
    int h0, group, split;  // query heads [h0, h0 + group) of the K/V head's
    int kv_len;
    int j_begin, n_j;      // query blocks
    int n_t;               // pairs (query head, query block); -1: no more items
};
// A pair, beside its tiles.
struct __align__(16) Pair {
    int q0;     // first query
    int block;  // query block, of all heads'
    int flags;
    float bias;  // bucket bias of a far pair
};
constexpr int kFirstOfItem = 1, kLastOfItem = 2, kLastOfHead = 4, kNear = 8, kPast = 16;  // kPast: keys before the queries

// What only a bucket bias needs.
struct SmemBuckets {
    alignas(16) float bias[kStages][2 * BQ];   // near block pairs: window of the expanded bias
    alignas(16) uint8_t idx[kStages][2 * BQ];  // and of its buckets
    float sums[kSoftmaxWarps][2 * kMaxBuckets];  // a warp's sums of one head
};
struct SmemNone {};

template <int kBias>
struct __align__(1024) Smem {
    uint8_t k[2][kTile];  // of two items in turn
    uint8_t v[kTile];
    uint8_t q[kStages][kTile];
    uint8_t g[kStages][kTile];
    uint8_t ds[2][2 * kTile];
    float nlse2[kStages][BQ];
    float dvec[kStages][BQ];
    std::conditional_t<kBias == kBiasBuckets, SmemBuckets, SmemNone> bk;
    Pair pair[kStages];
    Item items[kItems];
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t k_full[2], k_empty[2], v_full, v_empty;
    uint64_t stage_full[kStages];
    uint64_t q_empty[kStages];
    uint64_t g_empty[kStages];
    uint64_t sdp_full, sdp_read, pds_full, tmem_free, p_free, dq_full, dq_free, acc_done, acc_free, drain;
    uint64_t buckets_full, buckets_read;  // a head's sums are complete, are read (16 warps)
    uint32_t tmem_base;
    int abort_flag;
};

// Queries [lo, hi) that see key `j` of batch entry `b`.
__device__ __forceinline__ int2 key_queries(const ScoredBwdParams &p, int b, int j, int kv_len) {
    if (j >= kv_len) return make_int2(0, 0);
    int lo = 0, hi = p.Tq;
    if (p.vis.causal && !(p.vis.prefix_lens && j < p.vis.prefix_lens[b])) lo = j;
    if (p.vis.doc_range) {
        const int2 d = p.vis.doc_range[static_cast<long long>(b) * p.Tk + j];
        lo = max(lo, d.x);
        hi = min(hi, d.y);
    }
    return make_int2(lo, hi);
}

// Items go through the key blocks in turn: a causal mask's longest first.
__device__ __forceinline__ Item make_item(const ScoredBwdParams &p, unsigned i) {
    Item it{};
    const unsigned per_block = static_cast<unsigned>(p.B * p.Hkv) * p.splits;
    it.kb = static_cast<int>(i / per_block);
    const unsigned x = i - static_cast<unsigned>(it.kb) * per_block;
    it.bkv = static_cast<int>(x / p.splits);
    it.split = static_cast<int>(x) - it.bkv * p.splits;
    it.b = it.bkv / p.Hkv;
    const int all = p.H / p.Hkv, per = (all + p.splits - 1) / p.splits;
    it.group = max(0, min(per, all - it.split * per));
    it.h0 = (it.bkv - it.b * p.Hkv) * all + it.split * per;
    it.kv_len = p.Tk;
    if (p.vis.key_lens) it.kv_len = min(max(p.vis.key_lens[it.b], 0), p.Tk);
    // lo and hi grow with the key: the block's first and last key bound the
    // query blocks
    const int k0 = it.kb * BKB;
    if (k0 < it.kv_len) {
        const int lo = key_queries(p, it.b, k0, it.kv_len).x;
        const int hi = key_queries(p, it.b, min(k0 + BKB, it.kv_len) - 1, it.kv_len).y;
        it.j_begin = max(lo, 0) / BQ;
        it.n_j = max(0, (min(hi, p.Tq) + BQ - 1) / BQ - it.j_begin);
    }
    it.n_t = it.n_j * it.group;
    return it;
}

// What an item whose keys no query sees leaves: zeros, written by one warp.
template <int kBias>
__device__ __forceinline__ void write_none(const ScoredBwdParams &p, const Item &it, int lane) {
    const int rows = min(BKB, p.Tk - it.kb * BKB), row = it.kb * BKB;
    if (!in_bounds(rows > 0 && it.bkv < p.B * p.Hkv, p.status)) return;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    if (p.splits > 1) {
        const long long at = (((static_cast<long long>(it.split) * p.B * p.Hkv + it.bkv) * p.Tk) + row) * HD;
        for (int x = lane; x < rows * (HD / 4); x += 32) {
            reinterpret_cast<uint4 *>(p.part_dk + at)[x] = zero;
            reinterpret_cast<uint4 *>(p.part_dv + at)[x] = zero;
        }
    } else {
        const long long at = (static_cast<long long>(it.bkv) * p.Tk + row) * HD;
        for (int x = lane; x < rows * (HD / 8); x += 32) {
            reinterpret_cast<uint4 *>(p.dk + at)[x] = zero;
            reinterpret_cast<uint4 *>(p.dv + at)[x] = zero;
        }
    }
    if (kBias == kBiasBuckets && p.bucket_part) {
        const int n_buckets = p.bk.num * (p.bk.both ? 2 : 1), n_kb = (p.Tk + BKB - 1) / BKB;
        for (int h = 0; h < it.group; ++h) {
            float *dst = p.bucket_part + ((static_cast<long long>(it.b) * p.H + it.h0 + h) * n_kb + it.kb) * n_buckets;
            for (int u = lane; u < n_buckets; u += 32) dst[u] = 0.f;
        }
    }
}

// Weights P^T and dZ^T of 16 query columns for the thread's key, as bf16 pairs,
// from S^T and dP^T; leaves dS^T (fp32) in dp.  d0: the key's distance from the
// first query; kNearPair: column e's bucket bias is window[-e], otherwise all
// columns' is `far`.
// kMasked: only the columns of `bits` count.
template <bool kCap, int kBias, bool kMasked, bool kNearPair>
__device__ __forceinline__ void score_terms(uint32_t (&sv)[16], uint32_t (&dp)[16], const float *nlse2,
                                            const float *dvec, const ScoreParams &f, const BiasRow &br, int d0,
                                            const float *window, float far, unsigned bits, uint32_t (&pk)[8],
                                            uint32_t (&dsk)[8]) {
    auto seen = [&](int e) { return !kMasked || (bits >> e & 1u); };
    auto at = [](const uint32_t(&x)[16], int e) { return f32x2_pack(__uint_as_float(x[e]), __uint_as_float(x[e + 1])); };
    if (kCap) {
        // sv := mul tanh(s cap_in); masked scores have no say in how
        if (kMasked) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (!seen(e)) sv[e] = 0u;
        }
        const float big = max_abs(sv);
        if (__all_sync(0xffffffffu, big * big <= f.near_max)) {
            const uint64_t n0 = f32x2_set(f.near[0]), n1 = f32x2_set(f.near[1]), n2 = f32x2_set(f.near[2]);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                const uint64_t s2 = at(sv, e), sq = mul_f32x2(s2, s2);
                float a, b;
                f32x2_unpack(mul_f32x2(s2, fma_f32x2(sq, fma_f32x2(sq, n2, n1), n0)), a, b);
                sv[e] = __float_as_uint(a);
                sv[e + 1] = __float_as_uint(b);
            }
        } else {
            cap_scores(sv, f, __all_sync(0xffffffffu, big * big <= f.wide_max));
        }
    }
    const uint64_t mul2 = f32x2_set(f.mul), one2 = f32x2_set(1.f), far2 = f32x2_set(far);
    const uint64_t inv2 = f32x2_set(kCap ? -1.f / (f.mul * f.mul) : 0.f);
    // Slopes: -slope |d| and -lse, both large where only far keys are seen, meet
    // in one fused multiply-add from the whole distance d, so that their
    // difference loses nothing.  One sign of d for all of the warp's columns
    // but where they straddle the diagonal.
    bool one_sign = false;
    uint64_t dist = 0, slope = 0;
    const uint64_t minus2 = f32x2_set(-2.f);
    if (kBias == kBiasSlopes) {
        const bool past = f.past_only || __all_sync(0xffffffffu, d0 <= 0);
        one_sign = past || __all_sync(0xffffffffu, d0 >= 15);
        const float df = static_cast<float>(d0);
        dist = f32x2_pack(df, df - 1.f);
        slope = f32x2_set(past ? br.slope2 : -br.slope2);
    }
    auto columns = [&](auto one) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float4 l4 = reinterpret_cast<const float4 *>(nlse2)[g];
            const float4 d4 = reinterpret_cast<const float4 *>(dvec)[g];
            const uint64_t nl[2] = {f32x2_pack(l4.x, l4.y), f32x2_pack(l4.z, l4.w)};
            const uint64_t d[2] = {f32x2_pack(d4.x, d4.y), f32x2_pack(d4.z, d4.w)};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int e = 4 * g + 2 * i;
                uint64_t y = at(sv, e);
                if (kBias == kBiasBuckets) {
                    const uint64_t w2 = kNearPair ? f32x2_pack(window[-e], window[-e - 1]) : far2;
                    y = kCap ? add_f32x2(y, w2) : fma_f32x2(y, mul2, w2);
                }
                uint64_t add = nl[i];
                if (kBias == kBiasSlopes) {
                    uint64_t away = dist;
                    if (!decltype(one)::value) {
                        float a0, a1;
                        f32x2_unpack(dist, a0, a1);
                        away = f32x2_pack(fabsf(a0), fabsf(a1));
                    }
                    add = fma_f32x2(away, slope, add);
                    dist = add_f32x2(dist, minus2);
                }
                float x0, x1;
                f32x2_unpack(kCap || kBias == kBiasBuckets ? add_f32x2(y, add) : fma_f32x2(y, mul2, add), x0, x1);
                float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
                if (!seen(e)) p0 = 0.f;
                if (!seen(e + 1)) p1 = 0.f;
                float ds0, ds1;
                f32x2_unpack(mul_f32x2(f32x2_pack(p0, p1), sub_f32x2(at(dp, e), d[i])), ds0, ds1);
                dp[e] = __float_as_uint(ds0);
                dp[e + 1] = __float_as_uint(ds1);
                if (kCap) {
                    // 1 - t^2, t = sv / mul
                    const uint64_t t2 = at(sv, e);
                    f32x2_unpack(mul_f32x2(f32x2_pack(ds0, ds1), fma_f32x2(mul_f32x2(t2, inv2), t2, one2)), ds0, ds1);
                }
                pk[2 * g + i] = pack_bf16x2(p0, p1);
                dsk[2 * g + i] = pack_bf16x2(ds0, ds1);
            }
        }
    };
    if (kBias != kBiasSlopes || one_sign)
        columns(std::true_type{});
    else
        columns(std::false_type{});
}

template <bool kCap, int kBias>
__global__ void __launch_bounds__(kThreads, 1)
    attn_scored_bwd_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                           const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_g,
                           const __grid_constant__ ScoredBwdParams p) {
    extern __shared__ uint8_t smem_raw[];
    Smem<kBias> &sm = *reinterpret_cast<Smem<kBias> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                         ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sm.item_full[i], 1);
            mbar_init(&sm.item_empty[i], 1 + kSoftmaxWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.k_full[i], 1);
            mbar_init(&sm.k_empty[i], 1);
        }
        mbar_init(&sm.v_full, 1);
        mbar_init(&sm.v_empty, 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sm.stage_full[i], 1);
            mbar_init(&sm.q_empty[i], 1);
            mbar_init(&sm.g_empty[i], 1);
        }
        mbar_init(&sm.p_free, 1);
        mbar_init(&sm.sdp_full, 1);
        mbar_init(&sm.sdp_read, kSoftmaxWarps);
        mbar_init(&sm.pds_full, kSoftmaxWarps);
        mbar_init(&sm.tmem_free, 1);
        mbar_init(&sm.dq_full, 1);
        mbar_init(&sm.dq_free, kSoftmaxWarps);
        mbar_init(&sm.acc_done, 1);
        mbar_init(&sm.acc_free, kSoftmaxWarps);
        mbar_init(&sm.drain, 1);
        mbar_init(&sm.buckets_full, kSoftmaxWarps);
        mbar_init(&sm.buckets_read, kSoftmaxWarps);
        sm.abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&sm.tmem_base, 512);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tmap_q);
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
        prefetch_tensormap(&tmap_g);
    }
    if constexpr (kBias == kBiasBuckets) {
        for (int i = threadIdx.x; i < kSoftmaxWarps * 2 * kMaxBuckets; i += kThreads) (&sm.bk.sums[0][0])[i] = 0.f;
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = sm.tmem_base;
    const AbortState ab{&sm.abort_flag, p.status, 0};
    pdl_wait();

    if (warp == 0) {
        // ------------------------------------------------------- items, TMA
        unsigned i = blockIdx.x;
        int n = 0, t = 0;                   // items with pairs, their pairs
        int k_loads = 0, v_loads = 0, stage_loads = 0;
        // Publishes the item (n_t < 0: the end) and loads all that it needs.
        auto issue = [&](const Item &it) -> bool {
            const int slot = n % kItems, kbuf = n & 1;
            if (n >= kItems && !mbar_wait(&sm.item_empty[slot], (n / kItems - 1) & 1, ab)) return false;
            sm.items[slot] = it;
            mbar_arrive(&sm.item_full[slot]);
            if (it.n_t < 0) return true;
            const bool k_ok = in_bounds(it.kb * BKB < p.Tk && it.bkv < p.B * p.Hkv, p.status);
            if (n >= 2 && !mbar_wait(&sm.k_empty[kbuf], ((n >> 1) - 1) & 1, ab)) return false;
            mbar_arrive_expect_tx(&sm.k_full[kbuf], kTile);
            if (k_ok) tma_load_3d(&tmap_k, &sm.k_full[kbuf], sm.k[kbuf], 0, it.kb * BKB, it.bkv);
            ++k_loads;
            int j = it.j_begin, bh = it.b * p.H + it.h0;
            int head = it.h0;
            BiasRow br{};
            if (kBias == kBiasBuckets) br = bias_row<kBias>(p.f, head);
            for (int u = 0; u < it.n_t; ++u, ++t) {
                const int st = t % kStages, use = t / kStages;
                if (t >= kStages && !mbar_wait(&sm.q_empty[st], (use - 1) & 1, ab)) return false;
                const long long vrow = static_cast<long long>(bh) * p.Tq_pad + j * BQ;
                const bool window = kBias == kBiasBuckets && abs(it.kb - j) <= p.near_blocks;
                sm.pair[st] = Pair{j * BQ, bh * (p.Tq_pad / BQ) + j,
                                   (u == 0 ? kFirstOfItem : 0) | (u + 1 == it.n_t ? kLastOfItem : 0) |
                                       (j + 1 == it.j_begin + it.n_j ? kLastOfHead : 0) | (window ? kNear : 0) |
                                       (it.kb < j ? kPast : 0),
                                   kBias == kBiasBuckets ? (it.kb < j ? br.past : br.future) : 0.f};
                mbar_arrive_expect_tx(&sm.stage_full[st], 2 * kTile + 2 * BQ * 4 + (window ? 2 * BQ * 5 : 0));
                const bool j_ok = in_bounds(j * BQ < p.Tq && j * BQ + BQ <= p.Tq_pad && bh < p.B * p.H, p.status);
                if (j_ok) {
                    tma_load_3d(&tmap_q, &sm.stage_full[st], sm.q[st], 0, j * BQ, bh);
                    bulk_load_1d(sm.nlse2[st], p.nlse2 + vrow, BQ * 4, &sm.stage_full[st]);
                    bulk_load_1d(sm.dvec[st], p.dvec + vrow, BQ * 4, &sm.stage_full[st]);
                    if constexpr (kBias == kBiasBuckets) {
                        if (window) {
                            const int d = BKB * (it.kb - j - 1);  // first distance
                            bulk_load_1d(sm.bk.bias[st], br.vec + d, 2 * BQ * 4, &sm.stage_full[st]);
                            bulk_load_1d(sm.bk.idx[st], p.f.idx + p.f.mid + d, 2 * BQ, &sm.stage_full[st]);
                        }
                    }
                }
                ++stage_loads;
                if (t >= kStages && !mbar_wait(&sm.g_empty[st], (use - 1) & 1, ab)) return false;
                if (j_ok) tma_load_3d(&tmap_g, &sm.stage_full[st], sm.g[st], 0, j * BQ, bh);
                if (u == 0) {
                    // V's one buffer is free once the item before has its last
                    // dP, for which nothing of this item is needed
                    if (n >= 1 && !mbar_wait(&sm.v_empty, (n - 1) & 1, ab)) return false;
                    mbar_arrive_expect_tx(&sm.v_full, kTile);
                    if (k_ok) tma_load_3d(&tmap_v, &sm.v_full, sm.v, 0, it.kb * BKB, it.bkv);
                    ++v_loads;
                }
                if (++j == it.j_begin + it.n_j) {
                    j = it.j_begin;
                    ++bh;
                    ++head;
                    if (kBias == kBiasBuckets && u + 1 < it.n_t) br = bias_row<kBias>(p.f, head);
                }
            }
            ++n;
            return true;
        };
        for (;;) {
            Item it{};
            it.n_t = -1;
            if (i < p.total_items) it = make_item(p, i);
            if (lane == 0 && it.n_t >= 0) i = gridDim.x + atomicAdd(p.next_item, 1u);
            i = __shfl_sync(0xffffffffu, i, 0);
            if (it.n_t == 0) {
                write_none<kBias>(p, it, lane);
                continue;
            }
            const bool ok = lane == 0 ? issue(it) : true;
            if (!__all_sync(0xffffffffu, ok) || it.n_t < 0) break;
        }
        // every copy has landed before the CTA goes
        if (lane == 0) {
            for (int x = max(0, k_loads - 2); x < k_loads; ++x) mbar_wait_drain(&sm.k_full[x & 1], (x >> 1) & 1);
            if (v_loads > 0) mbar_wait_drain(&sm.v_full, (v_loads - 1) & 1);
            for (int x = max(0, stage_loads - kStages); x < stage_loads; ++x)
                mbar_wait_drain(&sm.stage_full[x % kStages], (x / kStages) & 1);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------- MMA
        constexpr uint32_t id_s = idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t id_kv = idesc_bf16_f32(128, HD, false, true);
        constexpr uint32_t id_q = idesc_bf16_f32(128, HD, true, true);
        constexpr uint64_t kT = kTile >> 4;
        const uint64_t k_km0 = smem_desc_sw128(smem_u32(sm.k), 16, 1024);
        constexpr uint64_t kMn = static_cast<uint64_t>((1024 >> 4) - 1) << 16;
        constexpr uint64_t kDsMn = static_cast<uint64_t>((kTile >> 4) - 1) << 16;
        const uint64_t v_km = k_km0 + 2 * kT;
        const uint64_t q_km = k_km0 + 3 * kT;
        const uint64_t g_km = k_km0 + (3 + kStages) * kT;
        const uint64_t ds_km0 = k_km0 + (3 + 2 * kStages) * kT;
        const uint64_t q_mn = q_km + kMn;
        const uint64_t g_mn = g_km + kMn;
        const uint64_t ds_mn = ds_km0 + kDsMn;
        bool ok = true;
        int n = 0, n_t = 0, v = 0;  // items taken; pairs of the last; the item of the scores in hand
        // S and dP of pair t, of which `more` pairs follow in its item.
        auto score = [&](int t, bool more) {
            const uint64_t so = static_cast<uint64_t>(t % kStages) * kT, k_km = k_km0 + static_cast<uint64_t>(v & 1) * kT;
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk)
                warp_mma_bf16_ss(tmem + kColS, k_km + 2 * kk, q_km + so + 2 * kk, id_s, kk > 0 ? 1u : 0u);
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk)
                warp_mma_bf16_ss(tmem + kColDP, v_km + 2 * kk, g_km + so + 2 * kk, id_s, kk > 0 ? 1u : 0u);
            warp_commit(&sm.sdp_full);
            if (!more) warp_commit(&sm.v_empty);
        };
        int pad = BKB;  // the item's first padded key
        // To the next item; false at the end, or on failure.
        auto next_item = [&]() -> bool {
            if (!(ok = warp_wait(&sm.item_full[n % kItems], (n / kItems) & 1, ab))) return false;
            const Item &it = sm.items[n % kItems];
            // (shuffled: known to be the same in every lane, so that what
            // follows from them, descriptors too, stays in uniform registers)
            n_t = __shfl_sync(0xffffffffu, it.n_t, 0);
            pad = __shfl_sync(0xffffffffu, it.kv_len < p.Tk ? it.kv_len - it.kb * BKB : BKB, 0);
            if (lane == 0) mbar_arrive(&sm.item_empty[n % kItems]);
            ++n;
            return n_t > 0;
        };
        auto keys_ready = [&]() -> bool {
            if (!warp_wait(&sm.k_full[v & 1], (v >> 1) & 1, ab) || !warp_wait(&sm.v_full, v & 1, ab)) return false;
            // Padded keys: their weight is 0, and 0 times whatever the buffer
            // holds there has to be 0 (rows past Tk the copy zeroed).
            if (pad < BKB) {
                uint4 *dk = reinterpret_cast<uint4 *>(sm.k[v & 1]), *dv = reinterpret_cast<uint4 *>(sm.v);
                for (int x = pad * 8 + lane; x < BKB * 8; x += 32) dk[x] = dv[x] = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
                __syncwarp();
            }
            return true;
        };
        bool live = next_item();
        if (live) {
            ok = keys_ready() && warp_wait(&sm.stage_full[0], 0, ab);
            if (ok) {
                tc_fence_after_sync();
                score(0, n_t > 1);
            }
        }
        for (int t = 0, u = 0; ok && live; ++t) {
            const int st = t % kStages, w = v;
            const uint64_t so = static_cast<uint64_t>(st) * kT;
            const bool last = u + 1 == n_t;
            if (last) {
                live = next_item();
                if (!ok) break;
                if (live) ++v;
            }
            const int nu = last ? 0 : u + 1;
            if (live) {
                if (!(ok = warp_wait(&sm.sdp_read, t & 1, ab))) break;
                if (last && !(ok = keys_ready())) break;
                if (!(ok = warp_wait(&sm.stage_full[(t + 1) % kStages], ((t + 1) / kStages) & 1, ab))) break;
                tc_fence_after_sync();
                score(t + 1, nu + 1 < n_t);
            }
            if (!(ok = warp_wait(&sm.pds_full, t & 1, ab))) break;
            if (u == 0 && w > 0 && !(ok = warp_wait(&sm.acc_free, (w - 1) & 1, ab))) break;
            tc_fence_after_sync();
            const uint64_t dso = static_cast<uint64_t>(t & 1) * (2 * kT);
#pragma unroll
            for (int kk = 0; kk < BQ / 16; ++kk)
                warp_mma_bf16_ss(tmem + kColDK, ds_km0 + dso + (kk >> 2) * kT + 2 * (kk & 3),
                                 q_mn + so + 128 * kk, id_kv, (u > 0 || kk > 0) ? 1u : 0u);
            warp_commit(&sm.q_empty[st]);
            warp_commit(&sm.tmem_free);
#pragma unroll
            for (int kk = 0; kk < BQ / 16; ++kk)
                warp_mma_bf16_ts(tmem + kColDV, tmem + kColP + 8 * kk, g_mn + so + 128 * kk, id_kv,
                                 (u > 0 || kk > 0) ? 1u : 0u);
            warp_commit(&sm.p_free);
            warp_commit(&sm.g_empty[st]);
            if (last) warp_commit(&sm.acc_done);
            if (t >= 1 && !(ok = warp_wait(&sm.dq_free, (t - 1) & 1, ab))) break;
            tc_fence_after_sync();
            const uint64_t k_mn = k_km0 + kMn + static_cast<uint64_t>(w & 1) * kT;
#pragma unroll
            for (int kk = 0; kk < BKB / 16; ++kk)
                warp_mma_bf16_ss(tmem + kColDQ, ds_mn + dso + 128 * kk, k_mn + 128 * kk, id_q,
                                 kk > 0 ? 1u : 0u);
            warp_commit(&sm.dq_full);
            if (last) warp_commit(&sm.k_empty[w & 1]);
            if (!(ok = warp_wait(&sm.tmem_free, t & 1, ab))) break;
            u = nu;
        }
        warp_commit(&sm.drain);
        mbar_wait_drain(&sm.drain, 0);
    } else {
        // ------------------------------------------- per-key score terms
        const int c = (warp - 2) >> 2;  // query chunk [32c, 32c + 32)
        const uint32_t lane_base = static_cast<uint32_t>(warp & 3) * 32;
        const int r = static_cast<int>(lane_base) + lane;
        const uint32_t tl = tmem_addr(tmem, lane_base, 0);
        const int wi = warp - 2;

        const int n_qb = p.Tq_pad / BQ;

        // dQ of the u-th pair, query block `block` of all heads': the quadrant's rows, features
        // [16c, 16c + 16), into the accumulator's layout (attn_bwd_bf16.cu).
        auto add_dq = [&](int u, int block) -> bool {
            if (!__all_sync(0xffffffffu, mbar_wait(&sm.dq_full, u & 1, ab))) return false;
            tc_fence_after_sync();
            uint32_t a[16];
            tmem_ld16(tl + kColDQ + 16u * c, a);
            tmem_ld_wait(a);
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.dq_free);
            float *dst = p.dq_acc + (static_cast<long long>(block) * BQ + lane_base) * HD + 512 * c + 4 * lane;
            if (!in_bounds(block < p.B * p.H * n_qb, p.status)) return true;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                red_add_v4(dst + 128 * x, __uint_as_float(a[4 * x]), __uint_as_float(a[4 * x + 1]),
                           __uint_as_float(a[4 * x + 2]), __uint_as_float(a[4 * x + 3]));
            return true;
        };
        // Bucket bias gradient.  `gen`: heads finished.
        const bool want_bias = kBias == kBiasBuckets && p.bucket_part != nullptr;
        const int n_buckets = p.bk.num * (p.bk.both ? 2 : 1);
        int gen = 0;
        float diag_hi = 0.f, diag_lo = 0.f, far_past = 0.f, far_future = 0.f;
        // x of the lane's distance, which is in bucket u, added over the lanes of
        // the bucket (they are neighbours: distances rise with the lane) to the
        // warp's sums.
        auto put_diagonals = [&](float x, int u) {
            if constexpr (kBias == kBiasBuckets) {
                const int before = __shfl_up_sync(0xffffffffu, u, 1);
                const unsigned heads = __ballot_sync(0xffffffffu, lane == 0 || before != u);
                const int back = lane - (31 - __clz(heads & (0xffffffffu >> (31 - lane))));  // lanes since its first
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float y = __shfl_up_sync(0xffffffffu, x, o);
                    if (back >= o) x += y;
                }
                if (lane == 31 || (heads >> (lane + 1) & 1u)) sm.bk.sums[wi][u] += x;
                __syncwarp();
            }
        };
        // The sums of the head before have been read (and are zero again).
        auto sums_free = [&]() -> bool {
            return gen == 0 || __all_sync(0xffffffffu, mbar_wait(&sm.buckets_read, (gen - 1) & 1, ab));
        };
        auto put_near = [&](int u_hi, int u_lo) -> bool {
            if constexpr (kBias == kBiasBuckets) {
                if (!sums_free()) return false;
                put_diagonals(diag_hi, u_hi);
                put_diagonals(diag_lo, u_lo);
                diag_hi = diag_lo = 0.f;
            }
            return true;
        };
        auto finish_head = [&](const Item &it, int head) -> bool {
            if constexpr (kBias == kBiasBuckets) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    far_past += __shfl_xor_sync(0xffffffffu, far_past, o);
                    far_future += __shfl_xor_sync(0xffffffffu, far_future, o);
                }
                if (!sums_free()) return false;
                float(&mine)[kSoftmaxWarps][2 * kMaxBuckets] = sm.bk.sums;
                if (lane == 0) {
                    // far past: the last bucket; far future: the last of the other
                    // direction, or, with one direction, bucket 0
                    mine[wi][p.bk.num - 1] += far_past;
                    mine[wi][p.bk.both ? 2 * p.bk.num - 1 : 0] += far_future;
                }
                far_past = far_future = 0.f;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.buckets_full);
                if (!__all_sync(0xffffffffu, mbar_wait(&sm.buckets_full, gen & 1, ab))) return false;
                const int u = wi * 32 + lane;
                if (u < n_buckets) {
                    float sum = 0.f;
#pragma unroll
                    for (int w = 0; w < kSoftmaxWarps; ++w) {
                        sum += mine[w][u];
                        mine[w][u] = 0.f;
                    }
                    p.bucket_part[((static_cast<long long>(it.b) * p.H + head) * ((p.Tk + BKB - 1) / BKB) + it.kb) * n_buckets + u] = sum;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.buckets_read);
                ++gen;
            }
            return true;
        };

        // dK and dV of an item: the thread's key, 32 features.
        auto write_kv = [&](const Item &it) {
            const bool is_dv = c >= 2;
            const int f0 = 32 * (c & 1);
            uint32_t a[32];
            tc_fence_after_sync();
            tmem_ld32(tl + (is_dv ? kColDV : kColDK) + f0, a);
            tmem_ld_wait(a);
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.acc_free);
            const int key = it.kb * BKB + r;
            if (key < p.Tk && in_bounds(key >= 0 && it.bkv < p.B * p.Hkv, p.status)) {
                if (p.splits > 1) {
                    uint4 *dst = reinterpret_cast<uint4 *>(
                        (is_dv ? p.part_dv : p.part_dk) +
                        ((static_cast<long long>(it.split) * p.B * p.Hkv + it.bkv) * p.Tk + key) * HD + f0);
#pragma unroll
                    for (int x = 0; x < 8; ++x) dst[x] = make_uint4(a[4 * x], a[4 * x + 1], a[4 * x + 2], a[4 * x + 3]);
                } else {
                    const float f = is_dv ? 1.f : p.scale;
                    uint4 *dst = reinterpret_cast<uint4 *>(
                        (is_dv ? p.dv : p.dk) + (static_cast<long long>(it.bkv) * p.Tk + key) * HD + f0);
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        w[e] = pack_bf16x2(__uint_as_float(a[2 * e]) * f, __uint_as_float(a[2 * e + 1]) * f);
#pragma unroll
                    for (int x = 0; x < 4; ++x) dst[x] = make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
                }
            }
        };

        bool ok = true;
        int t = 0, n = 0;  // pairs, items
        int before = 0;    // query block of pair t - 1, whose dQ is still to be added
        // dK and dV of item n - 1, and its slot given back.
        auto finish_item = [&]() -> bool {
            if (!__all_sync(0xffffffffu, mbar_wait(&sm.acc_done, (n - 1) & 1, ab))) return false;
            const int slot = (n - 1) % kItems;
            write_kv(sm.items[slot]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.item_empty[slot]);
            return true;
        };
        for (;; ++n) {
            const int slot = n % kItems;
            if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sm.item_full[slot], (n / kItems) & 1, ab)))) break;
            const Item &it = sm.items[slot];
            if (it.n_t < 0) break;
            const int key = it.kb * BKB + r;
            const int2 qs = key_queries(p, it.b, key, it.kv_len);
            BiasRow br{};
            if (kBias == kBiasSlopes) br = bias_row<kBias>(p.f, it.h0);
            int flags;
            do {
                const int st = t % kStages;
                ok = __all_sync(0xffffffffu, mbar_wait(&sm.stage_full[st], (t / kStages) & 1, ab)) &&
                     __all_sync(0xffffffffu, mbar_wait(&sm.sdp_full, t & 1, ab));
                if (!ok) break;
                tc_fence_after_sync();
                const Pair pair = sm.pair[st];
                flags = pair.flags;
                const int q0 = pair.q0 + 32 * c;
                const bool near = kBias == kBiasBuckets && (flags & kNear);
                const float *window = nullptr;
                if constexpr (kBias == kBiasBuckets) {
                    if (near) window = sm.bk.bias[st] + (r - 32 * c + BKB);
                }
                uint8_t *blk = sm.ds[t & 1] + (c >> 1) * kTile + r * 128;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const uint32_t col = 32u * c + 16u * h;
                    uint32_t sv[16], dp[16];
                    tmem_ld16(tl + kColS + col, sv);
                    tmem_ld16(tl + kColDP + col, dp);
                    const int lo = qs.x - (q0 + 16 * h), hi = qs.y - (q0 + 16 * h);
                    tmem_ld_wait(sv);
                    tmem_ld_wait(dp);
                    if (h == 1) {
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.sdp_read);
                    }
                    uint32_t pk[8], dsk[8];
                    const float *l2 = sm.nlse2[st] + 32 * c + 16 * h, *dv = sm.dvec[st] + 32 * c + 16 * h;
                    const int d0 = key - (q0 + 16 * h);
                    const float *win = window ? window - 16 * h : nullptr;
                    // columns that see the key
                    const unsigned bits = (hi <= 0 ? 0u : 0xffffu >> (16 - min(hi, 16))) & (0xffffu << min(max(lo, 0), 16));
                    auto terms = [&](auto masked, auto near_pair) {
                        score_terms<kCap, kBias, decltype(masked)::value, decltype(near_pair)::value>(
                            sv, dp, l2, dv, p.f, br, d0, win, pair.bias, bits, pk, dsk);
                    };
                    if (kBias == kBiasBuckets && near)
                        terms(std::true_type{}, std::bool_constant<kBias == kBiasBuckets>{});
                    else if (__all_sync(0xffffffffu, bits == 0xffffu))
                        terms(std::false_type{}, std::false_type{});
                    else if (kBias == kBiasBuckets || __any_sync(0xffffffffu, bits != 0))
                        terms(std::true_type{}, std::false_type{});
                    else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) pk[e] = dsk[e] = 0u;
                    }
                    if (h == 0 && t >= 1 && !(ok = __all_sync(0xffffffffu, mbar_wait(&sm.p_free, (t - 1) & 1, ab))))
                        break;
                    tmem_st8(tl + kColP + 16u * c + 8u * h, pk);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int chunk = 4 * (c & 1) + 2 * h + x;
                        *reinterpret_cast<uint4 *>(blk + ((chunk ^ (r & 7)) << 4)) =
                            make_uint4(dsk[4 * x], dsk[4 * x + 1], dsk[4 * x + 2], dsk[4 * x + 3]);
                    }
                    if (want_bias) {
                        if (near) {
                            // Column e of lane x has distance x - e: moved to
                            // lane x - e modulo 32, where distances L and L - 32
                            // meet.
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const int ee = 16 * h + e;
                                const float y =
                                    __shfl_sync(0xffffffffu, __uint_as_float(dp[e]), (lane + ee) & 31);
                                if (lane + ee < 32)
                                    diag_hi += y;
                                else
                                    diag_lo += y;
                            }
                        } else {
                            uint64_t s2 = f32x2_pack(0.f, 0.f);
#pragma unroll
                            for (int e = 0; e < 16; e += 2)
                                s2 = add_f32x2(s2, f32x2_pack(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1])));
                            float a, z;
                            f32x2_unpack(s2, a, z);
                            if (flags & kPast)
                                far_past += a + z;
                            else
                                far_future += a + z;
                        }
                    }
                }
                if (!ok) break;
                // the buckets of the warp's 32 x 32 pairs, distances -31 .. 31
                // around its own diagonal (read before the stage is given back)
                int u_hi = 0, u_lo = 0;
                if constexpr (kBias == kBiasBuckets)
                    if (want_bias && near) {
                        const uint8_t *u0 = sm.bk.idx[st] + BKB + static_cast<int>(lane_base) - 32 * c + lane;
                        u_hi = u0[0];
                        u_lo = u0[-32];
                    }
                tmem_st_wait();
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.pds_full);
                // what the item and the pair before left, while this pair's
                // products run
                if (n > 0 && (flags & kFirstOfItem) && !(ok = finish_item())) break;
                if (t >= 1 && !(ok = add_dq(t - 1, before))) break;
                if (want_bias && near && !(ok = put_near(u_hi, u_lo))) break;
                before = pair.block;
                ++t;
                if (flags & kLastOfHead) {
                    const int head = before / n_qb - it.b * p.H;
                    if (want_bias && !(ok = finish_head(it, head))) break;
                    if (kBias == kBiasSlopes && !(flags & kLastOfItem)) br = bias_row<kBias>(p.f, head + 1);
                }
            } while (!(flags & kLastOfItem));
            if (!ok) break;
        }
        if (ok && n > 0) ok = add_dq(t - 1, before) && finish_item();
        if (!ok) tmem_st_wait();
    }

    pdl_launch_dependents();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

template <bool kCap, int kBias>
cudaError_t launch(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, const CUtensorMap &tg,
                   const ScoredBwdParams &p, cudaStream_t stream) {
    auto kernel = attn_scored_bwd_kernel<kCap, kBias>;
    constexpr size_t smem = sizeof(Smem<kBias>) + 1024;
    static_assert(smem <= 227 * 1024, "");
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    const unsigned grid = std::min(p.total_items, static_cast<unsigned>(sms));
    return launch_kernel(kernel, dim3(grid), dim3(kThreads), smem, stream, true, 1, tq, tk, tv, tg, p);
}

}  // namespace

cudaError_t launch_attn_scored_bwd(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                                   const CUtensorMap &tg, bool capped, int bias, const ScoredBwdParams &p,
                                   cudaStream_t stream) {
    if (capped) {
        if (bias == kBiasSlopes) return launch<true, kBiasSlopes>(tq, tk, tv, tg, p, stream);
        if (bias == kBiasBuckets) return launch<true, kBiasBuckets>(tq, tk, tv, tg, p, stream);
        return launch<true, kBiasNone>(tq, tk, tv, tg, p, stream);
    }
    if (bias == kBiasSlopes) return launch<false, kBiasSlopes>(tq, tk, tv, tg, p, stream);
    if (bias == kBiasBuckets) return launch<false, kBiasBuckets>(tq, tk, tv, tg, p, stream);
    return launch<false, kBiasNone>(tq, tk, tv, tg, p, stream);
}

}  // namespace mha
