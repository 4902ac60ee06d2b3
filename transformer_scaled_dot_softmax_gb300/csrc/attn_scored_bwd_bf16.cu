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
//   * one CTA per (K/V head, 128 keys) walks (query head of the group, query
//     block) pairs, so dK and dV of the group are summed in tensor memory, in
//     a fixed order.  Where that makes too few CTAs the group's heads are
//     divided among several, which leave fp32 sums for the last launch;
//   * a key is seen by one interval of queries [lo, hi) (causal, prefix,
//     documents and padding all end in one), which bounds the query blocks
//     walked and masks the ones seen in part;
//   * a bucket bias sums dS over the buckets of its distances.  A block pair
//     past the last bucket's first distance adds up in one register per
//     thread; in a nearer one each warp adds its 32 x 32 pairs along their
//     diagonals (a shuffle and an add per pair), then each warp adds the
//     diagonals of the buckets it owns.  A CTA leaves one sum per head and
//     bucket, and the last launch adds those, all in a fixed order: dtable
//     does not depend on the order in which CTAs finish.
#include <cuda_bf16.h>

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
constexpr int kThreads = 576;
constexpr int kSoftmaxWarps = 16;
constexpr int kStages = 3;

struct __align__(1024) Smem {
    uint8_t k[kTile];
    uint8_t v[kTile];
    uint8_t q[kStages][kTile];
    uint8_t g[kStages][kTile];
    uint8_t ds[2][2 * kTile];
    float nlse2[kStages][BQ];
    float dvec[kStages][BQ];
    float diag[2][kSoftmaxWarps][64];  // a warp's 32 x 32 pairs by distance
    float far[2][kSoftmaxWarps][2];    // a warp's far sums of one query head (past, future)
    uint64_t kv_full;
    uint64_t stage_full[kStages];
    uint64_t q_empty[kStages];
    uint64_t g_empty[kStages];
    uint64_t sdp_full, sdp_read, pds_full, tmem_free, p_free, dq_full, dq_free, acc_done, drain;
    uint64_t diag_full;  // a near block's (or a head's far) sums are in shared memory (16 warps)
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

// Weights P^T and dZ^T of 16 query columns for the thread's key, as bf16
// pairs, from S^T and dP^T; returns dS^T (fp32) in dp.  kMasked: columns
// outside [lo, hi) count nothing, whatever S and dP hold there.
template <bool kCap, int kBias, bool kMasked>
__device__ __forceinline__ void score_terms(uint32_t (&sv)[16], uint32_t (&dp)[16], const float *nlse2,
                                            const float *dvec, const ScoreParams &f, const BiasRow &br, int d0,
                                            int lo, int hi, uint32_t (&pk)[8], uint32_t (&dsk)[8]) {
    uint32_t u[kCap ? 16 : 1];
    if (kCap) {
        if (kMasked) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (e < lo || e >= hi) sv[e] = 0u;
        }
        cap_scores(sv, f.cap_in, 1.f, __all_sync(0xffffffffu, max_abs(sv) * fabsf(f.cap_in) <= kTanhWide));
#pragma unroll
        for (int e = 0; e < 16; ++e) u[kCap ? e : 0] = sv[e];
    }
    if (kBias != kBiasNone) add_bias<kBias, -1, false>(sv, f, br, d0, 0.f);
    const uint64_t mul2 = f32x2_set(f.mul), one2 = f32x2_set(1.f);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const float4 l4 = reinterpret_cast<const float4 *>(nlse2)[g];
        const float4 d4 = reinterpret_cast<const float4 *>(dvec)[g];
        const uint64_t nl[2] = {f32x2_pack(l4.x, l4.y), f32x2_pack(l4.z, l4.w)};
        const uint64_t d[2] = {f32x2_pack(d4.x, d4.y), f32x2_pack(d4.z, d4.w)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int e = 4 * g + 2 * h;
            const uint64_t s2 = f32x2_pack(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
            float x0, x1;
            f32x2_unpack(kBias == kBiasNone ? fma_f32x2(s2, mul2, nl[h]) : add_f32x2(s2, nl[h]), x0, x1);
            float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            if (kMasked) {
                if (e < lo || e >= hi) p0 = 0.f;
                if (e + 1 < lo || e + 1 >= hi) p1 = 0.f;
            }
            const uint64_t dd = mul_f32x2(
                f32x2_pack(p0, p1),
                sub_f32x2(f32x2_pack(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1])), d[h]));
            float ds0, ds1;
            f32x2_unpack(dd, ds0, ds1);
            if (kMasked) {
                if (e < lo || e >= hi) ds0 = 0.f;
                if (e + 1 < lo || e + 1 >= hi) ds1 = 0.f;
            }
            dp[e] = __float_as_uint(ds0);
            dp[e + 1] = __float_as_uint(ds1);
            if (kCap) {
                const uint64_t t2 = f32x2_pack(__uint_as_float(u[kCap ? e : 0]), __uint_as_float(u[kCap ? e + 1 : 0]));
                const uint64_t nt = f32x2_pack(-__uint_as_float(u[kCap ? e : 0]), -__uint_as_float(u[kCap ? e + 1 : 0]));
                f32x2_unpack(mul_f32x2(f32x2_pack(ds0, ds1), fma_f32x2(t2, nt, one2)), ds0, ds1);
            }
            pk[2 * g + h] = pack_bf16x2(p0, p1);
            dsk[2 * g + h] = pack_bf16x2(ds0, ds1);
        }
    }
}

template <bool kCap, int kBias>
__global__ void __launch_bounds__(kThreads, 1)
    attn_scored_bwd_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                           const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_g,
                           const __grid_constant__ ScoredBwdParams p) {
    extern __shared__ uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                         ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int bkv = static_cast<int>(blockIdx.x) / p.splits;  // b Hkv + K/V head
    const int kb = static_cast<int>(blockIdx.y);
    const int b = bkv / p.Hkv, kvh = bkv - b * p.Hkv;
    // this CTA's query heads [h0, h0 + group) of the K/V head's
    const int split = static_cast<int>(blockIdx.x) - bkv * p.splits;
    const int all = p.H / p.Hkv, per = (all + p.splits - 1) / p.splits;
    const int group = max(0, min(per, all - split * per));
    const int h0 = kvh * all + split * per;
    const int k0 = kb * BKB;

    if (threadIdx.x == 0) {
        mbar_init(&sm.kv_full, 1);
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
        mbar_init(&sm.drain, 1);
        mbar_init(&sm.diag_full, kSoftmaxWarps);
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
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = sm.tmem_base;
    const AbortState ab{&sm.abort_flag, p.status, 0};
    pdl_launch_dependents();
    pdl_wait();

    int kv_len = p.Tk;
    if (p.vis.key_lens) kv_len = min(max(p.vis.key_lens[b], 0), p.Tk);
    // lo and hi grow with the key: the block's first and last key bound the
    // query blocks [j_begin, j_begin + n_j)
    int j_begin = 0, n_j = 0;
    if (k0 < kv_len) {
        const int lo = key_queries(p, b, k0, kv_len).x;
        const int hi = key_queries(p, b, min(k0 + BKB, kv_len) - 1, kv_len).y;
        j_begin = max(lo, 0) / BQ;
        n_j = max(0, (min(hi, p.Tq) + BQ - 1) / BQ - j_begin);
    }
    const int n_t = n_j * group;

    if (warp == 0) {
        // -------------------------------------------------------------- TMA
        if (lane == 0 && n_t > 0) {
            mbar_arrive_expect_tx(&sm.kv_full, 2 * kTile);
            if (in_bounds(k0 < p.Tk && bkv < p.B * p.Hkv, p.status)) {
                tma_load_3d(&tmap_k, &sm.kv_full, sm.k, 0, k0, bkv);
                tma_load_3d(&tmap_v, &sm.kv_full, sm.v, 0, k0, bkv);
            }
            int issued = 0, j = j_begin, bh = b * p.H + h0;
            for (int t = 0; t < n_t; ++t) {
                const int st = t % kStages, use = t / kStages;
                if (t >= kStages && !mbar_wait(&sm.q_empty[st], (use - 1) & 1, ab)) break;
                const long long vrow = static_cast<long long>(bh) * p.Tq_pad + j * BQ;
                mbar_arrive_expect_tx(&sm.stage_full[st], 2 * kTile + 2 * BQ * 4);
                const bool j_ok =
                    in_bounds(j * BQ < p.Tq && j * BQ + BQ <= p.Tq_pad && bh < p.B * p.H, p.status);
                if (j_ok) {
                    tma_load_3d(&tmap_q, &sm.stage_full[st], sm.q[st], 0, j * BQ, bh);
                    bulk_load_1d(sm.nlse2[st], p.nlse2 + vrow, BQ * 4, &sm.stage_full[st]);
                    bulk_load_1d(sm.dvec[st], p.dvec + vrow, BQ * 4, &sm.stage_full[st]);
                }
                issued = t + 1;
                if (t >= kStages && !mbar_wait(&sm.g_empty[st], (use - 1) & 1, ab)) break;
                if (j_ok) tma_load_3d(&tmap_g, &sm.stage_full[st], sm.g[st], 0, j * BQ, bh);
                if (++j == j_begin + n_j) {
                    j = j_begin;
                    ++bh;
                }
            }
            mbar_wait_drain(&sm.kv_full, 0);
            for (int x = max(0, issued - kStages); x < issued; ++x)
                mbar_wait_drain(&sm.stage_full[x % kStages], (x / kStages) & 1);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------- MMA
        if (n_t > 0) {
            constexpr uint32_t id_s = idesc_bf16_f32(128, 128, false, false);
            constexpr uint32_t id_kv = idesc_bf16_f32(128, HD, false, true);
            constexpr uint32_t id_q = idesc_bf16_f32(128, HD, true, true);
            constexpr uint64_t kT = kTile >> 4;
            const uint64_t k_km = smem_desc_sw128(smem_u32(sm.k), 16, 1024);
            constexpr uint64_t kMn = static_cast<uint64_t>((1024 >> 4) - 1) << 16;
            constexpr uint64_t kDsMn = static_cast<uint64_t>((kTile >> 4) - 1) << 16;
            const uint64_t v_km = k_km + kT;
            const uint64_t q_km = k_km + 2 * kT;
            const uint64_t g_km = k_km + (2 + kStages) * kT;
            const uint64_t ds_km0 = k_km + (2 + 2 * kStages) * kT;
            const uint64_t q_mn = q_km + kMn;
            const uint64_t g_mn = g_km + kMn;
            const uint64_t k_mn = k_km + kMn;
            const uint64_t ds_mn = ds_km0 + kDsMn;
            auto score_s = [&](int s) {
                const uint64_t so = static_cast<uint64_t>(s) * kT;
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk)
                    warp_mma_bf16_ss(tmem + kColS, k_km + 2 * kk, q_km + so + 2 * kk, id_s, kk > 0 ? 1u : 0u);
            };
            auto score_dp = [&](int s) {
                const uint64_t so = static_cast<uint64_t>(s) * kT;
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk)
                    warp_mma_bf16_ss(tmem + kColDP, v_km + 2 * kk, g_km + so + 2 * kk, id_s, kk > 0 ? 1u : 0u);
            };
            bool ok = warp_wait(&sm.kv_full, 0, ab);
            // Padded keys: their dS is 0, and dQ's 0 times whatever the
            // buffer holds has to be 0 (rows past Tk the copy zeroed).
            if (ok && k0 + BKB > kv_len && kv_len < p.Tk) {
                uint4 *dst = reinterpret_cast<uint4 *>(sm.k);
                for (int x = (kv_len - k0) * 8 + lane; x < BKB * 8; x += 32) dst[x] = make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
                __syncwarp();
            }
            ok = ok && warp_wait(&sm.stage_full[0], 0, ab);
            if (ok) {
                tc_fence_after_sync();
                score_s(0);
                score_dp(0);
                warp_commit(&sm.sdp_full);
            }
            for (int t = 0; ok && t < n_t; ++t) {
                const int st = t % kStages, nst = (t + 1) % kStages;
                const uint64_t so = static_cast<uint64_t>(st) * kT;
                if (t + 1 < n_t) {
                    if (!(ok = warp_wait(&sm.sdp_read, t & 1, ab))) break;
                    if (!(ok = warp_wait(&sm.stage_full[nst], ((t + 1) / kStages) & 1, ab))) break;
                    tc_fence_after_sync();
                    score_s(nst);
                    score_dp(nst);
                    warp_commit(&sm.sdp_full);
                }
                if (!(ok = warp_wait(&sm.pds_full, t & 1, ab))) break;
                tc_fence_after_sync();
                const uint64_t dso = static_cast<uint64_t>(t & 1) * (2 * kT);
#pragma unroll
                for (int kk = 0; kk < BQ / 16; ++kk)
                    warp_mma_bf16_ss(tmem + kColDK, ds_km0 + dso + (kk >> 2) * kT + 2 * (kk & 3),
                                     q_mn + so + 128 * kk, id_kv, (t > 0 || kk > 0) ? 1u : 0u);
                warp_commit(&sm.q_empty[st]);
                warp_commit(&sm.tmem_free);
#pragma unroll
                for (int kk = 0; kk < BQ / 16; ++kk)
                    warp_mma_bf16_ts(tmem + kColDV, tmem + kColP + 8 * kk, g_mn + so + 128 * kk, id_kv,
                                     (t > 0 || kk > 0) ? 1u : 0u);
                warp_commit(&sm.p_free);
                warp_commit(&sm.g_empty[st]);
                if (t >= 1 && !(ok = warp_wait(&sm.dq_free, (t - 1) & 1, ab))) break;
                tc_fence_after_sync();
#pragma unroll
                for (int kk = 0; kk < BKB / 16; ++kk)
                    warp_mma_bf16_ss(tmem + kColDQ, ds_mn + dso + 128 * kk, k_mn + 128 * kk, id_q,
                                     kk > 0 ? 1u : 0u);
                warp_commit(&sm.dq_full);
                if (!(ok = warp_wait(&sm.tmem_free, t & 1, ab))) break;
            }
            if (ok) warp_commit(&sm.acc_done);
        }
        warp_commit(&sm.drain);
        mbar_wait_drain(&sm.drain, 0);
    } else {
        // ------------------------------------------- per-key score terms
        const int c = (warp - 2) >> 2;  // query chunk [32c, 32c + 32)
        const uint32_t lane_base = static_cast<uint32_t>(warp & 3) * 32;
        const int r = static_cast<int>(lane_base) + lane;
        const int key = k0 + r;
        const uint32_t tl = tmem_addr(tmem, lane_base, 0);
        const int2 qs = n_t > 0 ? key_queries(p, b, key, kv_len) : make_int2(0, 0);
        const int wi = warp - 2;

        // dQ of the t-th (head, block) pair: the quadrant's rows, features
        // [16c, 16c + 16), into the accumulator's layout (attn_bwd_bf16.cu).
        auto add_dq = [&](int u, int bh, int j) -> bool {
            if (!__all_sync(0xffffffffu, mbar_wait(&sm.dq_full, u & 1, ab))) return false;
            tc_fence_after_sync();
            uint32_t a[16];
            tmem_ld16(tl + kColDQ + 16u * c, a);
            tmem_ld_wait(a);
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.dq_free);
            float *dst = p.dq_acc + (static_cast<long long>(bh) * p.Tq_pad + j * BQ + lane_base) * HD + 512 * c + 4 * lane;
            if (!in_bounds(j * BQ + BQ <= p.Tq_pad && bh < p.B * p.H, p.status)) return true;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                red_add_v4(dst + 128 * x, __uint_as_float(a[4 * x]), __uint_as_float(a[4 * x + 1]),
                           __uint_as_float(a[4 * x + 2]), __uint_as_float(a[4 * x + 3]));
            return true;
        };
        // Bucket bias gradient.  `gen` counts this CTA's exchanges through
        // shared memory (one per near block, one per head for the far sums).
        // Warp wi owns the buckets wi, wi + 16, ...; lane i holds the sum of
        // the i-th of them.
        const bool want_bias = kBias == kBiasBuckets && p.bucket_part != nullptr;
        const int n_buckets = p.bk.num * (p.bk.both ? 2 : 1);
        int gen = 0;
        float diag_hi = 0.f, diag_lo = 0.f, far_past = 0.f, far_future = 0.f, mine = 0.f;
        auto exchange = [&]() -> bool {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.diag_full);
            const bool got = __all_sync(0xffffffffu, mbar_wait(&sm.diag_full, gen & 1, ab));
            ++gen;
            return got;
        };
        auto warp_sum = [](float x) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            return x;
        };
        auto put_near = [&](int j) -> bool {
            const int buf = gen & 1;
            sm.diag[buf][wi][lane + 32] = diag_hi;  // distance `lane` within the warp's 32 x 32
            sm.diag[buf][wi][lane] = diag_lo;       // distance lane - 32
            diag_hi = diag_lo = 0.f;
            if (!exchange()) return false;
            const int mid = BKB * (kb - j);  // distance of the block pair's main diagonal
            for (int i = 0, u = wi; u < n_buckets; ++i, u += kSoftmaxWarps) {
                // the bucket's distances [d0, d1], as bucket_of() has them
                const int x = u < p.bk.num ? u : u - p.bk.num;
                const int near = p.bk.starts[x], far = x + 1 < p.bk.num ? p.bk.starts[x + 1] - 1 : 1 << 30;
                int d0 = u < p.bk.num ? -far : max(near, 1);
                int d1 = u < p.bk.num ? (u == 0 && !p.bk.both ? 1 << 30 : -near) : far;
                d0 = max(d0, mid - (BQ - 1));
                d1 = min(d1, mid + BKB - 1);
                if (d0 > d1) continue;
                float sum = 0.f;
                for (int d = d0 + lane; d <= d1; d += 32) {
                    // the warps' blocks that hold distance d: quadrant q, chunk
                    // q - k or q - k - 1 for k = floor((d - mid) / 32)
                    const int k = (d - mid) >> 5, loc = (d - mid) - 32 * k;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        // warp index of (quadrant q, chunk c): 4 c + (q + 2) % 4
                        const int c0 = q - k, c1 = c0 - 1;
                        if (c0 >= 0 && c0 < 4) sum += sm.diag[buf][4 * c0 + ((q + 2) & 3)][loc + 32];
                        if (c1 >= 0 && c1 < 4) sum += sm.diag[buf][4 * c1 + ((q + 2) & 3)][loc];
                    }
                }
                sum = warp_sum(sum);
                if (lane == i) mine += sum;
            }
            return true;
        };
        auto finish_head = [&](int head) -> bool {
            const int buf = gen & 1;
            far_past = warp_sum(far_past);
            far_future = warp_sum(far_future);
            if (lane == 0) {
                sm.far[buf][wi][0] = far_past;
                sm.far[buf][wi][1] = far_future;
            }
            far_past = far_future = 0.f;
            if (!exchange()) return false;
            const int u = wi + kSoftmaxWarps * lane;
            if (u < n_buckets) {
                // far past: the last bucket; far future: the last of the
                // other direction, or, with one direction, bucket 0
                const bool past = u == p.bk.num - 1, future = u == (p.bk.both ? 2 * p.bk.num - 1 : 0);
                for (int w = 0; past && w < kSoftmaxWarps; ++w) mine += sm.far[buf][w][0];
                for (int w = 0; future && w < kSoftmaxWarps; ++w) mine += sm.far[buf][w][1];
                p.bucket_part[((static_cast<long long>(b) * p.H + head) * gridDim.y + kb) * n_buckets + u] = mine;
            }
            mine = 0.f;
            return true;
        };

        bool ok = true;
        int j = j_begin, head = h0, j_prev = 0, bh_prev = 0;
        BiasRow br = bias_row<kBias>(p.f, head);
        for (int t = 0; t < n_t; ++t) {
            const int st = t % kStages;
            const int q0 = j * BQ + 32 * c;
            ok = __all_sync(0xffffffffu, mbar_wait(&sm.sdp_full, t & 1, ab)) &&
                 __all_sync(0xffffffffu, mbar_wait(&sm.stage_full[st], (t / kStages) & 1, ab));
            if (!ok) break;
            tc_fence_after_sync();
            const bool near = want_bias && abs(kb - j) <= p.near_blocks;
            uint8_t *blk = sm.ds[t & 1] + (c >> 1) * kTile + r * 128;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const uint32_t col = 32u * c + 16u * h;
                uint32_t sv[16], dp[16];
                tmem_ld16(tl + kColS + col, sv);
                tmem_ld16(tl + kColDP + col, dp);
                const int lo = qs.x - (q0 + 16 * h), hi = qs.y - (q0 + 16 * h);  // columns that see the key
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
                if (__all_sync(0xffffffffu, lo <= 0 && hi >= 16))
                    score_terms<kCap, kBias, false>(sv, dp, l2, dv, p.f, br, d0, 0, 16, pk, dsk);
                else
                    score_terms<kCap, kBias, true>(sv, dp, l2, dv, p.f, br, d0, lo, hi, pk, dsk);
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
                        if (kb < j)
                            far_past += a + z;
                        else
                            far_future += a + z;
                    }
                }
            }
            if (!ok) break;
            tmem_st_wait();
            fence_proxy_async_smem();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.pds_full);
            if (t >= 1 && !(ok = add_dq(t - 1, bh_prev, j_prev))) break;
            if (near && !(ok = put_near(j))) break;
            j_prev = j;
            bh_prev = b * p.H + head;
            if (++j == j_begin + n_j) {
                if (want_bias && !(ok = finish_head(head))) break;
                j = j_begin;
                ++head;
                if (t + 1 < n_t) br = bias_row<kBias>(p.f, head);
            }
        }
        if (ok && n_t > 0) ok = add_dq(n_t - 1, bh_prev, j_prev);
        if (n_t == 0 && want_bias)
            for (int x = 0; x < group && ok; ++x) ok = finish_head(h0 + x);
        if (ok && n_t > 0) ok = __all_sync(0xffffffffu, mbar_wait(&sm.acc_done, 0, ab));
        if (ok) {
            const bool is_dv = c >= 2;
            const int f0 = 32 * (c & 1);
            uint32_t a[32];
            if (n_t > 0) {
                tc_fence_after_sync();
                __syncwarp();
                tmem_ld32(tl + (is_dv ? kColDV : kColDK) + f0, a);
                tmem_ld_wait(a);
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) a[e] = 0u;
            }
            if (key < p.Tk && in_bounds(key >= 0 && bkv < p.B * p.Hkv, p.status)) {
                if (p.splits > 1) {
                    uint4 *dst = reinterpret_cast<uint4 *>(
                        (is_dv ? p.part_dv : p.part_dk) +
                        ((static_cast<long long>(split) * p.B * p.Hkv + bkv) * p.Tk + key) * HD + f0);
#pragma unroll
                    for (int x = 0; x < 8; ++x) dst[x] = make_uint4(a[4 * x], a[4 * x + 1], a[4 * x + 2], a[4 * x + 3]);
                } else {
                    const float f = is_dv ? 1.f : p.scale;
                    __nv_bfloat16 *dst = (is_dv ? p.dv : p.dk) + (static_cast<long long>(bkv) * p.Tk + key) * HD + f0;
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        w[e] = pack_bf16x2(__uint_as_float(a[2 * e]) * f, __uint_as_float(a[2 * e + 1]) * f);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        reinterpret_cast<uint4 *>(dst)[x] = make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
                }
            }
        }
        if (!ok) tmem_st_wait();
    }

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
    const size_t smem = sizeof(Smem) + 1024;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    dim3 grid(static_cast<unsigned>(p.B * p.Hkv * p.splits), static_cast<unsigned>((p.Tk + BKB - 1) / BKB));
    return launch_kernel(kernel, grid, dim3(kThreads), smem, stream, true, 1, tq, tk, tv, tg, p);
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
