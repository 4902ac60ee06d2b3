// attn_scored_bf16.cuh -- attention forward whose scores are more than
// scale q.k, for sm_103a: capped by a tanh, biased by distance, masked by
// documents or prefixes (the definition is in scores.cuh), with K/V heads
// shared by groups of query heads; and, as the same kernel over other rows,
// the partial sums of decoding rows against a prefix that a batch shares and
// against the requests' own caches.
//
// Mathematics: the online softmax.  A row keeps a reference m (log2 units)
// and a sum l; P = 2^(y - m), O += P V.  Softmax does not change with m, so the
// first one is simply 0, and only a row whose weights leave the window
// [2^-64, 2^64] moves it, by the exact step: m += the whole part of the
// round's maximum, and what was summed so far (O, l, P not yet multiplied) is
// scaled by that power of two, without rounding.  What a
// row sees is one interval of keys [lo, hi): the causal mask, key padding,
// prefixes and documents all end in one, so a tile is masked by two
// comparisons per key, and only tiles that some row sees in part are.
//
// With the log-sum-exp exported (the training forward) P is multiplied as two
// bf16 parts, P = hi + lo, hi the rounded weight and lo the rounded rest: O and
// with it the backward's row terms D = rowsum(dO O) then carry no rounding of
// the weights.  (With hi alone D is off by sum_j d_j w_j (dP_j - D), d_j the
// weights' relative roundings, and every dS of the row with it: dQ and dtable
// were 1.5 to 1.6 times as far from fp64 as fp32 arithmetic rounded once.)  It
// costs the tensor cores half as much again, which they have to spare, and a
// softmax thread one instruction per score.  The output's own rounding
// remainder can be stored beside it.
//
// The pipeline (persistent CTAs, TMA ring, S issuer, two PV issuers, two
// softmax groups on alternate tiles, output warps, three rotating score
// buffers in tensor memory) is that of attn_bf16.cu, described there.  What
// differs:
//   * an item's key tiles start at the tile that holds its diagonal and go
//     down from there, then up: with a distance bias the largest scores come
//     first, so the reference is set once instead of growing from tile to
//     tile (a rescale of O each);
//   * a softmax thread takes a round of 64 scores in one straight line where
//     it is a common one (every key seen, the bias an arithmetic progression,
//     capped scores in the polynomials' range), any other 32 by 32; in long
//     items, without cap and log-sum-exp, a common tile's two rounds;
//   * V rows past the key length are cleared in shared memory before they are
//     multiplied by their zero weights, so that what a padded buffer holds
//     there (NaN included) never reaches the output.
//
// Bound: like attn_bf16.cu by the softmax warps' instruction stream, not by a
// pipe: a tile takes about 1,200 cycles, of which its weights need 512 of the
// special-function unit (32 a cycle: 45 % busy) and its products 512 of the
// tensor cores; the cap adds 8 issue slots per pair, on the FMA pipe (41 % busy).
// Two warps share a scheduler and issue in 52 to 63 of 100 cycles, waiting for
// tensor memory in most others.
//
// Measured, 2 x 16 heads x 8,192, causal, without / with the log-sum-exp:
// 254 / 343 us (1,082 TFLOP/s without; attn_bf16.cu's plain forward 254), cap 50
// 385 / 504, slopes 304 / 399, both 470 / 605, 32 buckets 288 / 380, cap 20 under
// scores of deviation 4 (some in the wide range) 526 / 663, cap 1,000 under scores
// of deviation 6 (most warps past the polynomials) 709 / 877, 12 documents 100 / 112
// (capped 127 / 149).  Per item of
// 128 rows about 2.5 us (3.5 with the log-sum-exp) and 0.5 to 0.6 (0.7) per key tile;
// a tile seen in part costs two to three whole ones, which is what documents
// and short sequences are bound by.
// Tried and slower: rounds of 32 scores throughout (382 us), key tiles in
// ascending order under slopes (822, a rescale per tile), a straight-line
// variant for masked rounds or for biases from a window in shared memory (the
// common rounds lose 3 to 12 % to its registers and code), both rounds of a tile
// in one line with lo parts (slopes 409 to 448, documents 113 to 119, plain 347
// to 334) or with a cap (cap 50 413 to 392, cap 20 620 to 669, cap 50 with
// slopes 16 x 8 x 512 29 to 37).
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "kernels.h"
#include "scores.cuh"
#include "softmax_sums.cuh"
#include "sm103_ptx.cuh"

namespace mha {
namespace scored {

constexpr int BM = kAttnRowsPerCta;
constexpr int BN = 128;
constexpr int HD = kAttnHeadDim;
constexpr int STAGES = 5;
constexpr int kSBufs = 3;
constexpr int kThreads = 512;
constexpr int kSoftmaxWarps = 8;
constexpr int kLoadWarp = 8;
constexpr int kMmaSWarp = 9;
constexpr int kMmaPvWarp = 10;
constexpr int kOutWarp = 12;
constexpr uint32_t kTileBytes = BM * HD * 2;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 384;
// A row's reference serves while the sums of its rounds' weights lie in
// [2^-64, 2^64]: weights, sums and O are floats, so that their common scale
// costs no precision, and 2^64 times any length stays far from overflow.
constexpr float kSumMin = 5.421010862427522e-20f, kSumMax = 1.8446744073709552e19f;
constexpr int kItemTable = 128;
// Items of so many key tiles take their common tiles in one straight line (see
// kWhole), shorter ones and those with slopes round by round: there more tiles
// move the reference, and the attempt is lost (causal, line / rounds: slopes
// 16 x 8 x 1,024 52 / 44 us, 8 x 8 x 2,048 71 / 62, 2 x 16 x 8,192 310 / 346;
// plain 32 x 8 x 512 28 / 24, 8,192 254 / 285; buckets 8 x 8 x 2,048 60 / 64).
template <int kBias>
constexpr int kFastTiles = kBias == kBiasSlopes ? 16 : 6;
constexpr int kSorted = kThreads;

// What the kernel computes.
enum Mode { kForward, kForwardLse, kDecode };

// One work item: 128 query rows of one head against a range of key tiles.
struct Item {
    int b, hh, q0;         // decoding: (first) batch entry, K/V head, first row of the batch entry's
    int kv_len;            // keys past it are padding
    int j0, n_kv;          // key tiles j0 .. j0 + n_kv - 1
    int jd;                // the first one visited
    int full_lo, full_hi;  // keys [full_lo, full_hi) are seen by every row
    int split;             // decoding: key range, the prefix's before the caches'
};

struct __align__(1024) Smem {
    uint8_t q[2][kTileBytes];
    uint8_t k[STAGES][kTileBytes];
    uint8_t v[STAGES][kTileBytes];
    float red_m[2][BM];
    float red_l[2][BM];
    uint64_t q_full[2];
    uint64_t q_empty[2];
    uint64_t kv_full[STAGES];
    uint64_t kv_empty[STAGES];
    uint64_t s_full[kSBufs];
    uint64_t p_rd[2][2][2];  // [group][round][group tile mod 2]: P of the round written
    uint64_t pv0[2][2];      // [group][group tile mod 2]: round-0 product complete
    uint64_t ml_full, ml_free, o_final, o_free;
    uint64_t drain[3];
    uint16_t len[kSorted], order[kSorted];
    Item item_tab[kItemTable];
    Item item_own[kThreads / 32];
    int n_items;
    uint32_t tmem_base;
    int abort_flag;
};

__device__ __forceinline__ int item_index(int t, int c, int G) {
    return t * G + ((t & 1) ? (G - 1 - c) : c);
}

// Keys [lo, hi) that query row `i` of batch entry `b` sees.
__device__ __forceinline__ int2 row_keys(const VisParams &v, int Tk, int Tq, int b, int i) {
    int lo = 0, hi = Tk;
    if (v.key_lens) hi = min(max(v.key_lens[b], 0), Tk);
    if (v.causal) {
        int seen = i + 1;
        if (v.prefix_lens) seen = max(seen, v.prefix_lens[b]);
        hi = min(hi, seen);
    }
    if (v.doc_range) {
        const int2 d = v.doc_range[static_cast<long long>(b) * Tq + i];
        lo = max(lo, d.x);
        hi = min(hi, d.y);
    }
    return make_int2(lo, hi);
}

// Column, in its score buffer, of the packed weights of keys 64 rd + 16 kk ..
// + 15 (8 columns): over scores already read.  With lo parts, each 32 keys'
// weights lie over their own scores, 16 columns of hi, then 16 of lo.
template <int kMode>
__device__ __forceinline__ constexpr uint32_t weight_col(int rd, int kk) {
    return kMode == kForwardLse ? 64u * rd + 32u * (kk >> 1) + 8u * (kk & 1) : 32u * rd + 8u * kk;
}

// Blocks of query rows are dealt to the CTAs longest first.  Under a causal
// mask alone that is from the last block down; where lengths or documents make
// it another order, up to kSorted blocks (of all batch entries, one head) are
// ranked in the prologue, by every CTA alike.  `order`: null, or the ranking.
template <int kMode>
__device__ __forceinline__ Item make_item(const ScoredFwdParams &p, int k, const uint16_t *order) {
    Item it;
    if (kMode == kDecode) {
        const DecodeRows dr = decode_rows(p.H / p.Hkv * p.Tq);
        const int prefix_items = p.Hkv * p.row_tiles * p.splits;
        it.full_lo = 0;
        if (k < prefix_items) {
            const int tile = k % p.row_tiles;
            const int rest = k / p.row_tiles;
            it.hh = rest % p.Hkv;
            it.split = rest / p.Hkv;
            it.b = dr.chunks > 1 ? tile / dr.chunks : tile * dr.nb;
            it.q0 = dr.chunks > 1 ? (tile - it.b * dr.chunks) * 128 : 0;
            it.kv_len = it.full_hi = p.Tk;
            it.j0 = it.split * p.split_tiles;
            it.n_kv = max(0, min(p.split_tiles, (p.Tk + BN - 1) / BN - it.j0));
        } else {
            const int x = (k - prefix_items) / dr.chunks;
            const int bkv = x % (p.B * p.Hkv), cs = x / (p.B * p.Hkv);
            it.b = bkv / p.Hkv;
            it.hh = bkv - it.b * p.Hkv;
            it.q0 = (k - prefix_items - x * dr.chunks) * 128;
            it.split = p.splits + cs;
            it.kv_len = p.cache_lens ? min(max(p.cache_lens[it.b], 0), p.cache_cap) : p.cache_cap;
            it.full_hi = p.vis.causal ? max(it.kv_len - p.Tq + 1, 0) : it.kv_len;
            it.j0 = cs * p.split_tiles;
            it.n_kv = max(0, min(p.split_tiles, (it.kv_len + BN - 1) / BN - it.j0));
        }
        it.jd = it.j0 + it.n_kv - 1;
        return it;
    }
    // (block, head) pairs, blocks numbered from the last down, all batch
    // entries' last blocks first
    int blk = k / p.H;
    it.hh = k - blk * p.H;
    if (order) blk = order[blk];
    it.b = blk % p.B;
    it.q0 = (p.num_qblocks - 1 - blk / p.B) * BM;
    it.split = 0;
    it.kv_len = p.vis.key_lens ? min(max(p.vis.key_lens[it.b], 0), p.Tk) : p.Tk;
    // lo and hi grow with the row: the first and the last row bound the block
    const int2 first = row_keys(p.vis, p.Tk, p.Tq, it.b, it.q0);
    const int2 last = row_keys(p.vis, p.Tk, p.Tq, it.b, min(it.q0 + BM, p.Tq) - 1);
    it.j0 = max(first.x, 0) / BN;
    it.n_kv = max(0, (last.y + BN - 1) / BN - it.j0);
    it.jd = min(max(it.q0 / BN, it.j0), it.j0 + it.n_kv - 1);
    it.full_lo = last.x;
    it.full_hi = first.y;
    return it;
}

template <int kMode>
__device__ __forceinline__ bool sorted(const ScoredFwdParams &p) {
    return kMode != kDecode && (p.vis.key_lens || p.vis.prefix_lens || p.vis.doc_range) && p.B * p.num_qblocks <= kSorted;
}

// The t-th key tile of an item: down from jd, then up.
__device__ __forceinline__ int tile_of(const Item &it, int t) {
    const int down = it.jd - it.j0;
    return t <= down ? it.jd - t : it.j0 + t;
}

// The CTA's t-th item, in shared memory (read there when needed rather than
// held in registers); past the table each warp computes its own, once all of
// its lanes that take part (`lanes`) are done with the one before: items without
// a key tile pass no other barrier.
template <int kMode>
__device__ __forceinline__ const Item &item_of(Smem &sm, const ScoredFwdParams &p, int t, int cta, int G,
                                               unsigned lanes = 0xffffffffu) {
    if (t < kItemTable) return sm.item_tab[t];
    Item &own = sm.item_own[threadIdx.x >> 5];
    __syncwarp(lanes);
    own = make_item<kMode>(p, item_index(t, cta, G), sorted<kMode>(p) ? sm.order : nullptr);  // every lane writes the same
    __syncwarp(lanes);
    return own;
}

// What a thread's row (r of the item's 128) is.
struct Row {
    bool live;       // an output row
    int head;        // query head
    int pos;         // position, for distances
    long long out;   // row of the output (or of the partial sums of a split)
    int2 keys;       // keys [x, y) seen
};
template <int kMode>
__device__ __forceinline__ Row make_row(const ScoredFwdParams &p, const Item &it, int r) {
    Row w;
    if (kMode == kDecode) {
        const int g = p.H / p.Hkv, rows = g * p.Tq;
        const DecodeRows dr = decode_rows(rows);
        const bool cache = it.split >= p.splits;
        const int bi = r / dr.per;
        const int rem = it.q0 + r - bi * dr.per;
        const int b = it.b + bi;
        w.live = bi < (cache ? 1 : dr.nb) && b < p.B && rem < rows;
        w.head = it.hh * g + (w.live ? rem / p.Tq : 0);
        const int t = w.live ? rem % p.Tq : 0;
        int len = p.cache_cap;
        if (w.live && p.cache_lens) len = min(max(p.cache_lens[b], 0), p.cache_cap);
        w.pos = len - p.Tq + t;  // among the cache's rows
        w.keys = cache ? make_int2(0, p.vis.causal ? min(w.pos + 1, len) : len) : make_int2(0, p.Tk);
        if (!cache) w.pos += p.Tk;
        w.out = w.live ? (static_cast<long long>(b) * p.H + w.head) * p.Tq + t : 0;
    } else {
        const int i = it.q0 + r, ic = min(i, p.Tq - 1);
        w.live = i < p.Tq;
        w.head = it.hh;
        w.pos = i;
        w.out = (static_cast<long long>(it.b) * p.H + it.hh) * p.Tq + ic;
        w.keys = row_keys(p.vis, p.Tk, p.Tq, it.b, ic);
    }
    return w;
}

template <bool kCap, int kBias, int kMode, bool kRuns>
__global__ void __launch_bounds__(kThreads, 1)
    attn_scored_kernel(const __grid_constant__ ScoredMaps maps, const __grid_constant__ ScoredFwdParams p) {
    extern __shared__ uint8_t smem_raw[];
    Smem &sm = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                         ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int G = static_cast<int>(gridDim.x);
    const int cta = static_cast<int>(blockIdx.x);
    const int total = p.total_items;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 1);
            mbar_init(&sm.q_empty[i], 1);
        }
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&sm.kv_full[i], 1);
            mbar_init(&sm.kv_empty[i], 1);
        }
        for (int i = 0; i < kSBufs; ++i) mbar_init(&sm.s_full[i], 1);
        for (int i = 0; i < 8; ++i) mbar_init(&sm.p_rd[i >> 2][(i >> 1) & 1][i & 1], kSoftmaxWarps / 2);
        for (int i = 0; i < 4; ++i) mbar_init(&sm.pv0[i >> 1][i & 1], 1);
        mbar_init(&sm.ml_full, kSoftmaxWarps);
        mbar_init(&sm.ml_free, 4);
        mbar_init(&sm.o_final, 2);
        mbar_init(&sm.o_free, 4);
        for (int i = 0; i < 3; ++i) mbar_init(&sm.drain[i], 1);
        const int F = total / G, rem = total - F * G;
        sm.n_items = F + ((((F & 1) ? (G - 1 - cta) : cta) < rem) ? 1 : 0);
        sm.abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kMmaSWarp) {
        tmem_alloc(&sm.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    if (warp == kLoadWarp && lane == 0) {
        prefetch_tensormap(&maps.q);
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.v);
    }
    // The launch before this one may still run, of a call before it or the
    // one that writes document ranges and the expanded bias (a call after
    // another of these: 1 to 2 us less).  A launch after this one may begin
    // once that one is complete, so it may read its results.
    pdl_wait();
    pdl_launch_dependents();
    if (sorted<kMode>(p)) {
        const int n = p.B * p.num_qblocks, x = threadIdx.x;
        int len = 0;
        if (x < n) {
            len = min(make_item<kMode>(p, x * p.H, nullptr).n_kv, 65535);
            sm.len[x] = static_cast<uint16_t>(len);
        }
        __syncthreads();
        if (x < n) {
            int rank = 0;
            for (int i = 0; i < n; ++i) {
                const int other = sm.len[i];
                rank += other > len || (other == len && i < x) ? 1 : 0;
            }
            sm.order[rank] = static_cast<uint16_t>(x);
        }
        __syncthreads();
    }
    for (int t = threadIdx.x; t < kItemTable; t += kThreads) {
        const int k = item_index(t, cta, G);
        if (k < total) sm.item_tab[t] = make_item<kMode>(p, k, sorted<kMode>(p) ? sm.order : nullptr);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = sm.tmem_base;
    const AbortState ab{&sm.abort_flag, p.status, 0};

    if (warp == kLoadWarp) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0) {
            const int g = p.H / p.Hkv;
            const DecodeRows dr = decode_rows(g * p.Tq);
            int n = 0, v = 0;  // key tiles and items so far
            bool ok = true;
            for (int t = 0; ok && t < sm.n_items; ++t) {
                const Item &it = item_of<kMode>(sm, p, t, cta, G, 1u);
                if (it.n_kv == 0) continue;
                const bool cache = kMode == kDecode && it.split >= p.splits;
                const CUtensorMap *mq = cache ? &maps.q_cache : &maps.q, *mk = cache ? &maps.k_cache : &maps.k,
                                  *mv = cache ? &maps.v_cache : &maps.v;
                const int z = kMode == kDecode ? (cache ? it.b * p.Hkv + it.hh : it.hh) : it.b * p.Hkv + it.hh / g;
                int jt = 0;
                do {
                    const int qbuf = v & 1, run_end = kRuns ? min(jt + kRunTiles, it.n_kv) : it.n_kv;
                    if (v >= 2 && !(ok = mbar_wait(&sm.q_empty[qbuf], ((v - 2) >> 1) & 1, ab))) break;
                    mbar_arrive_expect_tx(&sm.q_full[qbuf], kMode == kDecode
                                                                ? static_cast<uint32_t>(dr.per * (cache ? 1 : dr.nb)) * (HD * 2)
                                                                : kTileBytes);
                    if (in_bounds(it.q0 >= 0 && it.b >= 0 && it.b < p.B && it.hh < (kMode == kDecode ? p.Hkv : p.H), p.status)) {
                        if (kMode == kDecode)
                            tma_load_4d(mq, &sm.q_full[qbuf], sm.q[qbuf], 0, it.q0, it.b, it.hh);
                        else
                            tma_load_3d(mq, &sm.q_full[qbuf], sm.q[qbuf], 0, it.q0, it.b * p.H + it.hh);
                    }
                    ++v;
                    for (; jt < run_end; ++jt, ++n) {
                        const int j = tile_of(it, jt);
                        const int st = n % STAGES;
                        if (n >= STAGES && !(ok = mbar_wait(&sm.kv_empty[st], ((n / STAGES) - 1) & 1, ab))) break;
                        mbar_arrive_expect_tx(&sm.kv_full[st], 2 * kTileBytes);
                        if (in_bounds(j >= 0 && j * BN < (cache ? p.cache_cap : p.Tk) &&
                                          z < (kMode == kDecode && !cache ? 1 : p.B) * p.Hkv,
                                      p.status)) {
                            tma_load_3d(mk, &sm.kv_full[st], sm.k[st], 0, j * BN, z);
                            tma_load_3d(mv, &sm.kv_full[st], sm.v[st], 0, j * BN, z);
                        }
                    }
                } while (kRuns && ok && jt < it.n_kv);
            }
            for (int x = max(0, n - STAGES); x < n; ++x)
                mbar_wait_drain(&sm.kv_full[x % STAGES], (x / STAGES) & 1);
            for (int x = max(0, v - 2); x < v; ++x) mbar_wait_drain(&sm.q_full[x & 1], (x >> 1) & 1);
        }
    } else if (warp == kMmaSWarp) {
        // ----------------------------------------------------- S issuer
        constexpr uint32_t idesc_s = idesc_bf16_f32(BM, BN, false, false);
        constexpr uint64_t kTileDesc = kTileBytes >> 4;
        const uint64_t q_desc0 = smem_desc_sw128(smem_u32(sm.q[0]), 16, 1024);
        const uint64_t k_desc0 = smem_desc_sw128(smem_u32(sm.k[0]), 16, 1024);
        int n = 0, v = 0;
        bool ok = true;
        for (int t = 0; ok && t < sm.n_items; ++t) {
            const int n_kv = item_of<kMode>(sm, p, t, cta, G).n_kv;
            if (n_kv == 0) continue;
            int jt = 0;
            do {
                const int qbuf = v & 1, run_end = kRuns ? min(jt + kRunTiles, n_kv) : n_kv;
                if (!(ok = warp_wait(&sm.q_full[qbuf], (v >> 1) & 1, ab))) break;
                const uint64_t qd = q_desc0 + static_cast<uint64_t>(qbuf) * kTileDesc;
                for (; jt < run_end; ++jt, ++n) {
                    const int st = n % STAGES, sb = n % kSBufs;
                    if (!(ok = warp_wait(&sm.kv_full[st], (n / STAGES) & 1, ab))) break;
                    if (n >= kSBufs) {
                        const int np = n - kSBufs;
                        if (!(ok = warp_wait(&sm.kv_empty[np % STAGES], (np / STAGES) & 1, ab))) break;
                    }
                    tc_fence_after_sync();
                    const uint32_t d = tmem + 128u * static_cast<uint32_t>(sb);
                    const uint64_t kd = k_desc0 + static_cast<uint64_t>(st) * kTileDesc;
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk)
                        warp_mma_bf16_ss(d, qd + 2 * kk, kd + 2 * kk, idesc_s, kk > 0 ? 1u : 0u);
                    warp_commit(&sm.s_full[sb]);
                }
                if (!ok) break;
                warp_commit(&sm.q_empty[qbuf]);
                ++v;
            } while (kRuns && ok && jt < n_kv);
        }
        warp_commit(&sm.drain[0]);
        mbar_wait_drain(&sm.drain[0], 0);
    } else if (warp == kMmaPvWarp || warp == kMmaPvWarp + 1) {
        // ---------------------------------------------------- PV issuers
        const int hf = warp - kMmaPvWarp;
        constexpr uint32_t idesc_o = idesc_bf16_f32(BM, HD, false, true);
        constexpr uint64_t kTileDesc = kTileBytes >> 4;
        const uint64_t v_desc = smem_desc_sw128(smem_u32(sm.v[0]), 1024, 1024);
        const uint32_t d_o = tmem + kOCol + 64u * static_cast<uint32_t>(hf);
        int n = 0, v = 0;
        bool ok = true;
        for (int t = 0; ok && t < sm.n_items; ++t) {
            const Item &it = item_of<kMode>(sm, p, t, cta, G);
            if (it.n_kv == 0) continue;
            int run = 0;
            do {
                const int n_kv = kRuns ? min(it.n_kv - run, kRunTiles) : it.n_kv;
                if (v >= 1 && !(ok = warp_wait(&sm.o_free, (v - 1) & 1, ab))) break;
                for (int jt = 0; jt < n_kv; ++jt, ++n) {
                    if ((n & 1) != hf) continue;
                    const int st = n % STAGES, sb = n % kSBufs;
                    const int slot = (n >> 1) & 1, par = (n >> 2) & 1;
                    if (!(ok = warp_wait(&sm.kv_full[st], (n / STAGES) & 1, ab))) break;
                    // Padding past the key length: weights there are 0, and 0
                    // times whatever the buffer holds has to be 0.  (Rows past Tk
                    // are filled with zeros by the copy.)
                    const int rows = it.kv_len - tile_of(it, run + jt) * BN;
                    if (rows < BN && it.kv_len < (kMode == kDecode && it.split >= p.splits ? p.cache_cap : p.Tk)) {
                        uint4 *dst = reinterpret_cast<uint4 *>(sm.v[st]);
                        for (int x = max(rows, 0) * 8 + lane; x < BN * 8; x += 32) dst[x] = make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    const uint32_t a = tmem + 128u * static_cast<uint32_t>(sb);
                    const uint64_t vd = v_desc + static_cast<uint64_t>(st) * kTileDesc;
#pragma unroll
                    for (int rd = 0; rd < 2; ++rd) {
                        if (!(ok = warp_wait(&sm.p_rd[hf][rd][slot], par, ab))) break;
                        tc_fence_after_sync();
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint32_t acc = jt >= 2 || rd > 0 || kk > 0 ? 1u : 0u;
                            warp_mma_bf16_ts(d_o, a + weight_col<kMode>(rd, kk), vd + 128 * (4 * rd + kk), idesc_o, acc);
                            if (kMode == kForwardLse)
                                warp_mma_bf16_ts(d_o, a + weight_col<kMode>(rd, kk) + 16, vd + 128 * (4 * rd + kk), idesc_o, 1u);
                        }
                        if (rd == 0) warp_commit(&sm.pv0[hf][slot]);
                    }
                    if (!ok) break;
                    warp_commit(&sm.kv_empty[st]);
                }
                if (!ok) break;
                warp_commit(&sm.o_final);
                ++v;
            } while (kRuns && ok && (run += kRunTiles) < it.n_kv);
        }
        warp_commit(&sm.drain[1 + hf]);
        mbar_wait_drain(&sm.drain[1 + hf], 0);
    } else if (warp < kSoftmaxWarps) {
        // --------------------------------------------------------- softmax
        const int half = warp >> 2;
        const uint32_t lane_base = static_cast<uint32_t>(warp & 3) * 32;
        const int r = static_cast<int>(lane_base) + lane;
        const uint32_t tl = tmem_addr(tmem, lane_base, 0);
        const uint32_t to = tl + kOCol + 64u * half;
        // Weights of a pair of keys: packed, with lo parts where they are
        // kept, and added to the row sum -- the rounded weights, which are
        // what P V multiplies, so that normalised weights sum to 1; with lo
        // parts the weights themselves.
        struct Sum {
            uint64_t both = 0;
            float a[4] = {0.f, 0.f, 0.f, 0.f};
            __device__ __forceinline__ float get() const {
                float e0, e1;
                f32x2_unpack(both, e0, e1);
                return kMode == kForwardLse ? e0 + e1 : (a[0] + a[1]) + (a[2] + a[3]);
            }
        };
        auto pack_pair = [](float x0, float x1, int c, uint32_t &hi, uint32_t &lo, Sum &sum) {
            hi = pack_bf16x2(x0, x1);
            if (kMode == kForwardLse) {
                const uint64_t x = f32x2_pack(x0, x1);
                float r0, r1;
                f32x2_unpack(sub_f32x2(x, f32x2_pack(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u))), r0, r1);
                lo = pack_bf16x2(r0, r1);
                sum.both = add_f32x2(sum.both, x);
            } else {
                add_bf16x2_to_f32(sum.a[2 * (c & 1)], sum.a[2 * (c & 1) + 1], hi);
            }
        };
        // The common round, load to packed weights in one straight line:
        // y = u mul + b0 + c step.  a: its first 16 scores, on their way from
        // tensor memory; the others follow 16 by 16 while the ones before them
        // are worked on, and `next` starts the first of the round after it.
        // kind 0: no cap, 1: near, 2: wide range; big: the largest squared
        // argument of the polynomial.  pk: the round's 64 weights; with lo parts
        // 32 keys' hi and lo, of which `half_done` takes the first 32 keys' and
        // says whether to go on.
        // Without cap and lo parts registers are to spare: a round's 64 scores
        // are read at once (decoding 64 x 16 x 2 rows 54.5 -> 53.5 us), and in the
        // forward a common tile's two rounds stand in one line.
        constexpr bool kWhole = kMode != kForwardLse && !kCap;
        auto common_round = [&](auto kind, uint32_t tr, uint32_t(&a)[16], bool next, float b0, float step,
                                uint32_t(&pk)[32], Sum &sum, float &big, auto half_done) -> bool {
            constexpr int kKind = decltype(kind)::value;
            uint32_t b16[16];
            const uint64_t mul2 = f32x2_set(p.f.mul);
            const uint64_t n0 = f32x2_set(p.f.near[0]), n1 = f32x2_set(p.f.near[1]), n2 = f32x2_set(p.f.near[2]);
            const TanhWide poly(p.f);
            constexpr int kChains = kBias == kBiasSlopes ? 4 : 1;
            uint64_t b[kChains];
#pragma unroll
            for (int i = 0; i < kChains; ++i) b[i] = f32x2_pack(fmaf(2.f * i, step, b0), fmaf(2.f * i + 1.f, step, b0));
            const uint64_t step2 = f32x2_set(8.f * step);
            float big0 = 0.f, big1 = 0.f;
            auto take = [&](const auto &sc, int part) {
                constexpr int kPairs = sizeof(sc) / 8;
#pragma unroll
                for (int c = 0; c < kPairs; ++c) {
                    const uint64_t s2 = f32x2_pack(__uint_as_float(sc[2 * c]), __uint_as_float(sc[2 * c + 1]));
                    uint64_t y;
                    if (kKind == 0) {
                        y = fma_f32x2(s2, mul2, b[c % kChains]);
                    } else {
                        const uint64_t sq = mul_f32x2(s2, s2);
                        float w0, w1;
                        f32x2_unpack(sq, w0, w1);
                        if (c & 1)
                            big1 = fmax3(big1, w0, w1);
                        else
                            big0 = fmax3(big0, w0, w1);
                        const uint64_t pol = kKind == 1 ? fma_f32x2(sq, fma_f32x2(sq, n2, n1), n0) : poly(sq);
                        y = fma_f32x2(s2, pol, b[c % kChains]);
                    }
                    if (kBias == kBiasSlopes) b[c % kChains] = add_f32x2(b[c % kChains], step2);
                    float x0, x1;
                    f32x2_unpack(y, x0, x1);
                    x0 = ex2_approx(x0);
                    x1 = ex2_approx(x1);
                    const int at = kMode == kForwardLse ? 8 * (part & 1) + c : 8 * part + c;
                    pack_pair(x0, x1, c, pk[at], pk[(16 + at) & 31], sum);
                }
            };
            if constexpr (kWhole) {
                uint32_t s0[32], s1[32];
                tmem_ld32(tr, s0);
                tmem_ld32(tr + 32, s1);
                tmem_ld_wait(s0);
                reg_fence32(s1);
                take(s0, 0);
                take(s1, 2);
                return true;
            }
            tmem_ld_wait(a);
            tmem_ld16(tr + 16, b16);
            take(a, 0);
            tmem_ld_wait(b16);
            tmem_ld16(tr + 32, a);
            take(b16, 1);
            big = fmaxf(big0, big1);
            if (kMode == kForwardLse && !half_done()) return false;
            tmem_ld_wait(a);
            tmem_ld16(tr + 48, b16);
            take(a, 2);
            tmem_ld_wait(b16);
            if (next) tmem_ld16(tr + 64, a);
            take(b16, 3);
            big = fmaxf(big0, big1);
            return true;
        };

        int n = 0, v = 0;
        bool ok = true;
        for (int t = 0; ok && t < sm.n_items; ++t) {
            const Item &it = item_of<kMode>(sm, p, t, cta, G);
            if (it.n_kv == 0) continue;
            const Row w = make_row<kMode>(p, it, r);
            const BiasRow br = bias_row<kBias>(p.f, w.head);
            // decoding: rows past the stacked ones have nothing to compute
            const bool warp_live = kMode != kDecode || __any_sync(0xffffffffu, w.live);
            const bool long_item = it.n_kv >= kFastTiles<kBias>;
            // the range the warp's capped scores need: near, wide, any
            int tier = !kCap || p.f.near_max != 0.f ? 0 : p.f.wide_max != 0.f ? 1 : 2;
            int run = 0;
            do {
                const int n_kv = kRuns ? min(it.n_kv - run, kRunTiles) : it.n_kv;
                float m_run = -INFINITY;  // log2 units; -inf until this group has seen a visible key
                float l_run = 0.f;

                for (int jt = 0; jt < n_kv; ++jt, ++n) {
                    if ((n & 1) != half) continue;
                    const int j = tile_of(it, run + jt);
                    const int sb = n % kSBufs;
                    ok = __all_sync(0xffffffffu, mbar_wait(&sm.s_full[sb], (n / kSBufs) & 1, ab));
                    if (!ok) break;
                    if (!warp_live) {
                        // P of the warp's rows stays whatever it is: a row of
                        // tensor memory only reaches its own row of O
                        if (lane == 0) {
                            mbar_arrive(&sm.p_rd[half][0][(n >> 1) & 1]);
                            mbar_arrive(&sm.p_rd[half][1][(n >> 1) & 1]);
                        }
                        continue;
                    }
                    tc_fence_after_sync();
                    const uint32_t ts = tl + 128u * static_cast<uint32_t>(sb);
                    const bool edge = j * BN < it.full_lo || j * BN + BN > it.full_hi;
                    float b_tile, step;  // bias of the tile's key c: b_tile + c step, if `linear`
                    const bool linear = linear_bias<kBias>(p.f, br, j * BN - w.pos, BN, 0.f, b_tile, step);
                    uint32_t a[16];
                    int rd_first = 0;
                    if constexpr (kWhole && kMode == kForward) {
                        if (!edge && linear && long_item) {
#pragma unroll
                            for (int rd = 0; rd < 2; ++rd) {
                                uint32_t pk[32];
                                const float ref = m_run == -INFINITY ? 0.f : m_run;
                                const float b0 = kBias == kBiasSlopes ? fmaf(step, static_cast<float>(j * BN + 64 * rd - w.pos), -ref)
                                                                      : b_tile - ref;
                                Sum sum;
                                float big = 0.f;
                                common_round(std::integral_constant<int, 0>{}, ts + 64u * rd, a, false, b0, step, pk, sum, big, [] { return true; });
                                const float lt = sum.get();
                                // a reference has to move: to the rounds below
                                if (__any_sync(0xffffffffu, !(lt <= kSumMax && (m_run != -INFINITY || lt >= kSumMin)))) break;
                                if (m_run == -INFINITY) m_run = 0.f;
                                tmem_st32(ts + 32u * rd, pk);
                                l_run += lt;
                                tmem_st_wait();
                                tc_fence_before_sync();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(&sm.p_rd[half][rd][(n >> 1) & 1]);
                                rd_first = rd + 1;
                            }
                        }
                    }
                    if (!kWhole) tmem_ld16(ts, a);
#pragma unroll 1
                    for (int rd = rd_first; rd < 2; ++rd) {
                        const uint32_t tr = ts + 64u * static_cast<uint32_t>(rd);
                        auto sees_none = [&](int first, int len) {
                            return w.keys.x >= first + len || w.keys.y <= first || (kMode == kDecode && !w.live);
                        };
                        // Does the row need the exact step after a sum against
                        // the reference in hand (0 before there is one)?
                        auto must_move = [&](float sum, bool none) -> bool {
                            if (none) return false;
                            if (m_run != -INFINITY) return !(sum <= kSumMax);
                            if (!(sum >= kSumMin && sum <= kSumMax)) return true;
                            m_run = 0.f;
                            return false;
                        };
                        const int key0 = j * BN + 64 * rd;  // the round's first key
                        int done = 0;  // of the round's two halves
                        if (linear && (!kCap || tier < 2) &&
                            (!edge || __all_sync(0xffffffffu, w.keys.x <= key0 && w.keys.y >= key0 + 64))) {
                            uint32_t pk[32];
                            const float ref = m_run == -INFINITY ? 0.f : m_run;
                            // -ref and the bias's large part meet in one fused
                            // multiply-add: far distances lose nothing
                            const float b0 = kBias == kBiasSlopes ? fmaf(step, static_cast<float>(key0 - w.pos), -ref)
                                                                  : b_tile - ref;
                            Sum sum;
                            float big = 0.f;
                            // The weights in pk, if the round may keep them: col,
                            // their column.
                            auto keep = [&](uint32_t col) -> bool {
                                if (kCap && kMode == kDecode && !w.live) big = 0.f;
                                if (kCap && __any_sync(0xffffffffu, big > (tier == 0 ? p.f.near_max : p.f.wide_max))) {
                                    ++tier;  // out of the polynomial's range: taken again below
                                    return false;
                                }
                                const bool first = m_run == -INFINITY;
                                const float lt = sum.get();
                                if (__any_sync(0xffffffffu, must_move(lt, kMode == kDecode && !w.live))) {
                                    if (first) m_run = -INFINITY;
                                    return false;
                                }
                                tmem_st32(ts + col, pk);
                                l_run += lt;
                                return true;
                            };
                            auto half_done = [&]() {
                                if (!keep(weight_col<kMode>(0, 0) + 64u * static_cast<uint32_t>(rd))) return false;
                                done = 1;
                                sum = Sum();
                                return true;
                            };
                            bool whole;
                            if (!kCap)
                                whole = common_round(std::integral_constant<int, 0>{}, tr, a, rd == 0, b0, step, pk, sum, big, half_done);
                            else if (tier == 0)
                                whole = common_round(std::integral_constant<int, 1>{}, tr, a, rd == 0, b0, step, pk, sum, big, half_done);
                            else
                                whole = common_round(std::integral_constant<int, 2>{}, tr, a, rd == 0, b0, step, pk, sum, big, half_done);
                            if (whole) {
                                if (keep(kMode == kForwardLse ? 64u * static_cast<uint32_t>(rd) + 32u : 32u * static_cast<uint32_t>(rd)))
                                    done = 2;
                            } else {
                                tmem_ld_wait(a);
                                if (rd == 0) tmem_ld16(tr + 64, a);
                            }
                        } else if (!kWhole) {
                            tmem_ld_wait(a);
                            if (rd == 0) tmem_ld16(tr + 64, a);
                        }
                        // Every other round, 32 keys at a time.
#pragma unroll 1
                        for (int h = done; h < 2; ++h) {
                            const int kh = key0 + 32 * h;
                            const bool none = sees_none(kh, 32);
                            const uint32_t tp = ts + weight_col<kMode>(0, 0) + (kMode == kForwardLse ? 64u : 32u) * rd;
                            uint32_t pk[16], pl[16];
                            float lt = 0.f, alpha = 1.f;
                            if (__all_sync(0xffffffffu, none)) {
#pragma unroll
                                for (int c = 0; c < 16; ++c) pk[c] = pl[c] = 0u;
                            } else {
                                const int lo = min(max(w.keys.x - kh, 0), 32), hi = min(w.keys.y - kh, 32);
                                // the keys seen, a bit each
                                const unsigned bits = none ? 0u : (0xffffffffu >> (32 - hi)) & (0xffffffffu << lo);
                                const bool all = __all_sync(0xffffffffu, bits == 0xffffffffu);
                                bool need = false;
                                // attempt 0 against the reference in hand; where a
                                // row needs the exact step, 1 moves its reference
                                // and 2 takes the keys again
#pragma unroll 1
                                for (int attempt = 0;; ++attempt) {
                                    uint32_t y[32];
                                    tmem_ld32(tr + 32u * static_cast<uint32_t>(h), y);
                                    tmem_ld_wait(y);
                                    auto mask_to = [&](float value) {
#pragma unroll
                                        for (int c = 0; c < 32; ++c)
                                            if (!(bits >> c & 1u)) y[c] = __float_as_uint(value);
                                    };
                                    if (kCap) {
                                        const bool dead = kMode == kDecode && !w.live;
                                        float big = max_abs(y);
                                        bool near = __all_sync(0xffffffffu, dead || big * big <= p.f.near_max);
                                        if (!near && !all) {
                                            // masked scores have no say in how tanh is taken
                                            mask_to(0.f);
                                            big = max_abs(y);
                                            near = __all_sync(0xffffffffu, dead || big * big <= p.f.near_max);
                                        }
                                        if (near) {
                                            const uint64_t n0 = f32x2_set(p.f.near[0]), n1 = f32x2_set(p.f.near[1]),
                                                           n2 = f32x2_set(p.f.near[2]);
#pragma unroll
                                            for (int c = 0; c < 32; c += 2) {
                                                const uint64_t s2 = f32x2_pack(__uint_as_float(y[c]), __uint_as_float(y[c + 1]));
                                                const uint64_t sq = mul_f32x2(s2, s2);
                                                float t0, t1;
                                                f32x2_unpack(mul_f32x2(s2, fma_f32x2(sq, fma_f32x2(sq, n2, n1), n0)), t0, t1);
                                                y[c] = __float_as_uint(t0);
                                                y[c + 1] = __float_as_uint(t1);
                                            }
                                        } else {
                                            cap_scores(y, p.f, __all_sync(0xffffffffu, dead || big * big <= p.f.wide_max));
                                        }
                                    }
                                    if (!all) mask_to(p.f.masked);
                                    add_bias<kBias, kCap>(y, p.f, br, kh - w.pos, m_run == -INFINITY ? 0.f : -m_run);
                                    if (attempt == 1) {
                                        if (need) {
                                            float up = -INFINITY;  // above the reference
#pragma unroll
                                            for (int c = 0; c < 32; c += 2)
                                                up = fmax3(up, __uint_as_float(y[c]), __uint_as_float(y[c + 1]));
                                            up = ceilf(up);
                                            if (m_run == -INFINITY) {
                                                m_run = up;
                                            } else if (up > 0.f) {
                                                m_run += up;
                                                alpha = ex2_approx(-up);
                                                l_run *= alpha;
                                            }
                                        }
                                        continue;
                                    }
                                    Sum sum;
#pragma unroll
                                    for (int c = 0; c < 16; ++c)
                                        pack_pair(ex2_approx(__uint_as_float(y[2 * c])), ex2_approx(__uint_as_float(y[2 * c + 1])), c,
                                                  pk[c], pl[c], sum);
                                    lt = sum.get();
                                    if (attempt == 2) break;
                                    need = must_move(lt, none);
                                    if (!__any_sync(0xffffffffu, need)) break;
                                }
                            }
                            const uint32_t th = tp + (kMode == kForwardLse ? 32u : 16u) * static_cast<uint32_t>(h);
                            tmem_st16(th, pk);
                            if (kMode == kForwardLse) tmem_st16(th + 16, pl);
                            l_run += lt;
                            if (!__any_sync(0xffffffffu, alpha != 1.f)) continue;
                            // What was summed before moves with the reference: the
                            // round's first 32 weights, which wait to be multiplied
                            // with these, and O_h, which holds the group's earlier
                            // tiles of the item and, in round 1, this tile's round
                            // 0: wait for the last product it took.
                            if (h == 1) {
                                tmem_st_wait();
#pragma unroll 1
                                for (uint32_t part = 0; part < (kMode == kForwardLse ? 32u : 16u); part += 16u) {
                                    tmem_ld16(tp + part, pk);
                                    tmem_ld_wait(pk);
#pragma unroll
                                    for (int c = 0; c < 16; ++c)
                                        pk[c] = pack_bf16x2(__uint_as_float(pk[c] << 16) * alpha,
                                                            __uint_as_float(pk[c] & 0xffff0000u) * alpha);
                                    tmem_st16(tp + part, pk);
                                }
                            }
                            if (rd == 1) {
                                ok = __all_sync(0xffffffffu, mbar_wait(&sm.pv0[half][(n >> 1) & 1], (n >> 2) & 1, ab));
                            } else if (jt >= 2) {
                                const int np = n - 2;
                                ok = __all_sync(0xffffffffu, mbar_wait(&sm.kv_empty[np % STAGES], (np / STAGES) & 1, ab));
                            } else {
                                continue;  // O_h holds nothing of this item
                            }
                            if (!ok) break;
                            tc_fence_after_sync();
#pragma unroll 1
                            for (int part = 0; part < 2; ++part) {
                                uint32_t o0[32];
                                tmem_ld32(to + 32u * static_cast<uint32_t>(part), o0);
                                tmem_ld_wait(o0);
#pragma unroll
                                for (int c = 0; c < 32; ++c) o0[c] = __float_as_uint(__uint_as_float(o0[c]) * alpha);
                                tmem_st32(to + 32u * static_cast<uint32_t>(part), o0);
                            }
                        }
                        if (!ok) break;
                        tmem_st_wait();
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.p_rd[half][rd][(n >> 1) & 1]);
                    }
                    if (!ok) break;
                }
                if (!ok) break;
                if (v >= 1 && !(ok = __all_sync(0xffffffffu, mbar_wait(&sm.ml_free, (v - 1) & 1, ab)))) break;
                sm.red_m[half][r] = m_run;
                sm.red_l[half][r] = l_run;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.ml_full);
                ++v;
            } while (kRuns && ok && (run += kRunTiles) < it.n_kv);
        }
        if (!ok) tmem_st_wait();
    } else if (warp >= kOutWarp) {
        // ------------------------------------------------------------ output
        const uint32_t lane_base = static_cast<uint32_t>(warp & 3) * 32;
        const int r = static_cast<int>(lane_base) + lane;
        const uint32_t tl = tmem_addr(tmem, lane_base, 0);
        int v = 0;
        bool ok = true;
        for (int t = 0; ok && t < sm.n_items; ++t) {
            const Item &it = item_of<kMode>(sm, p, t, cta, G);
            const Row w = make_row<kMode>(p, it, r);
            const bool row_ok = in_bounds(w.out >= 0 && w.out < static_cast<long long>(p.B) * p.H * p.Tq, p.status) && w.live;
            if (it.n_kv == 0) {
                if (kMode == kDecode) {
                    if (row_ok)
                        p.part_ml[it.split * (static_cast<long long>(p.B) * p.H * p.Tq) + w.out] = make_float2(-INFINITY, 0.f);
                } else if (row_ok) {
                    uint4 *d4 = reinterpret_cast<uint4 *>(p.o + w.out * HD);
#pragma unroll
                    for (int c = 0; c < 8; ++c) d4[c] = make_uint4(0u, 0u, 0u, 0u);
                    if (kMode == kForwardLse) {
                        p.lse[w.out] = -INFINITY;
                        if (p.o_lo) {
                            uint4 *l4 = reinterpret_cast<uint4 *>(p.o_lo + w.out * HD);
#pragma unroll
                            for (int c = 0; c < 8; ++c) l4[c] = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                }
                continue;
            }
            // what an item's runs before have summed (in local memory: few items have any)
            volatile float sum_o[kRuns ? HD : 1];
            float sum_m = -INFINITY, sum_l = 0.f;
            const bool single = !kRuns || it.n_kv <= kRunTiles;
            int run = 0;
            do {
                const bool last = !kRuns || run + kRunTiles >= it.n_kv;
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sm.ml_full, v & 1, ab)))) break;
                const float ma = sm.red_m[0][r], mb = sm.red_m[1][r];
                const float la = sm.red_l[0][r], lb = sm.red_l[1][r];
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.ml_free);
                if (!(ok = __all_sync(0xffffffffu, mbar_wait(&sm.o_final, v & 1, ab)))) break;
                tc_fence_after_sync();
                // A sum of 0: no visible key.  One of NaN (a NaN or +infinity among
                // the visible scores) goes on to o and lse.
                const SumLevel va = sum_level(ma, la), vb = sum_level(mb, lb);
                float M = fmaxf(la != 0.f ? va.m : -INFINITY, lb != 0.f ? vb.m : -INFINITY);
                const float wa = la != 0.f ? ex2_approx(va.m - M) * va.down : 0.f;
                const float wb = lb != 0.f ? ex2_approx(vb.m - M) * vb.down : 0.f;
                float L = la * wa + lb * wb, f = 1.f, keep = 0.f;
                if (!single) {
                    const float m = L > 0.f ? M : L == 0.f ? -INFINITY : 0.f;
                    M = fmaxf(sum_m, m);
                    f = m == -INFINITY ? 0.f : ex2_approx(m - M);
                    keep = sum_m == -INFINITY ? 0.f : ex2_approx(sum_m - M);
                    L = L * f + sum_l * keep;
                    sum_m = M;
                    sum_l = L;
                }
                if (kMode != kDecode && last) {
                    const float inv = L != 0.f ? 1.0f / L : 0.f;
                    f *= inv;
                    keep *= inv;
                }
                const float fa = wa * f, fb = wb * f;
                const long long prow = kMode == kDecode ? it.split * (static_cast<long long>(p.B) * p.H * p.Tq) + w.out : 0;
                if (row_ok && last) {
                    if (kMode == kDecode)
                        // (L in [1, 4): the merge joins by M alone; the reference of a
                        // NaN is as good as any, if the merge takes it)
                        p.part_ml[prow] = make_float2(L > 0.f ? M : L == 0.f ? -INFINITY : 0.f, L);
                    else if (kMode == kForwardLse)
                        p.lse[w.out] = L != 0.f ? fmaf(M, kLn2, logf(L)) : -INFINITY;
                }
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    uint32_t oa[32], ob[32];
                    tmem_ld32(tl + kOCol + 32u * part, oa);
                    tmem_ld32(tl + kOCol + 64u + 32u * part, ob);
                    tmem_ld_wait(oa);
                    reg_fence32(ob);
                    if (part == 1) {
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sm.o_free);
                    }
                    if (!row_ok) continue;
                    // a group without a visible key left its accumulator unwritten
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        oa[c] = __float_as_uint((la != 0.f ? __uint_as_float(oa[c]) * fa : 0.f) +
                                                (lb != 0.f ? __uint_as_float(ob[c]) * fb : 0.f));
                    if constexpr (kRuns) {
                        if (!single) {
#pragma unroll
                            for (int c = 0; c < 32; ++c) {
                                float x = __uint_as_float(oa[c]);
                                if (run > 0) x = fmaf(sum_o[32 * part + c], keep, x);
                                oa[c] = __float_as_uint(x);
                                if (!last) sum_o[32 * part + c] = x;
                            }
                            if (!last) continue;
                        }
                    }
                    if (kMode == kDecode) {
                        uint4 *d4 = reinterpret_cast<uint4 *>(p.part_o + prow * HD) + 8 * part;
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            d4[c] = make_uint4(oa[4 * c], oa[4 * c + 1], oa[4 * c + 2], oa[4 * c + 3]);
                    } else {
                        uint4 *d4 = reinterpret_cast<uint4 *>(p.o + w.out * HD) + 4 * part;
                        uint32_t pk[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            pk[c] = pack_bf16x2(__uint_as_float(oa[2 * c]), __uint_as_float(oa[2 * c + 1]));
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            d4[c] = make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
                        if (kMode == kForwardLse && p.o_lo) {
                            uint4 *l4 = reinterpret_cast<uint4 *>(p.o_lo + w.out * HD) + 4 * part;
#pragma unroll
                            for (int c = 0; c < 16; ++c)
                                pk[c] = pack_bf16x2(__uint_as_float(oa[2 * c]) - __uint_as_float(pk[c] << 16),
                                                    __uint_as_float(oa[2 * c + 1]) - __uint_as_float(pk[c] & 0xffff0000u));
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                l4[c] = make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
                        }
                    }
                }
                ++v;
            } while (kRuns && ok && (run += kRunTiles) < it.n_kv);
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaSWarp) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <bool kCap, int kBias, int kMode, bool kRuns>
cudaError_t launch(const ScoredMaps &maps, const ScoredFwdParams &p, cudaStream_t stream) {
    auto kernel = attn_scored_kernel<kCap, kBias, kMode, kRuns>;
    const size_t smem = sizeof(Smem) + 1024;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    int sms = 0;
    if ((e = sm_count(&sms)) != cudaSuccess) return e;
    const int grid = p.total_items < sms ? p.total_items : sms;
    if (grid <= 0) return cudaSuccess;
    return launch_kernel(kernel, dim3(grid), dim3(kThreads), smem, stream, true, 1, maps, p);
}

template <bool kCap, int kBias, bool kRuns>
cudaError_t launch_form(const ScoredMaps &maps, const ScoredFwdParams &p, cudaStream_t stream) {
    if (p.part_o) return launch<kCap, kBias, kDecode, kRuns>(maps, p, stream);
    if (p.lse) return launch<kCap, kBias, kForwardLse, kRuns>(maps, p, stream);
    return launch<kCap, kBias, kForward, kRuns>(maps, p, stream);
}

template <bool kCap, bool kRuns>
cudaError_t launch_any(const ScoredMaps &maps, int bias, const ScoredFwdParams &p, cudaStream_t stream) {
    if (bias == kBiasSlopes) return launch_form<kCap, kBiasSlopes, kRuns>(maps, p, stream);
    if (bias == kBiasBuckets) return launch_form<kCap, kBiasBuckets, kRuns>(maps, p, stream);
    return launch_form<kCap, kBiasNone, kRuns>(maps, p, stream);
}

}  // namespace scored
}  // namespace mha
