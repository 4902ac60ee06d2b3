// attn_paged_bf16.cu -- attention of chunks of new tokens (prompts, parts of
// them) over a paged K/V cache, for sm_103a.
//
// Row tiles.  A K/V head's query rows are stacked token by token, x = t g + i for
// token t and the i-th of its g query heads, as many whole tokens to a tile of
// 128 rows as fit: a chunk's heads share the K/V tiles they read, and a causal
// tile spans few positions.  The launch before this one lists the row tiles of
// all sequences with their numbers of key tiles (those that some row sees).
// All (K/V head, row tile, key tile) stand in one line, of which every CTA takes
// an equal share: no CTA waits for another's longer one, and a chunk with few rows
// spreads over the GPU along its keys.  A row tile inside a share is written out;
// pieces leave fp32 partial sums that the last launch joins (paged_decode.cu).
//
// Pages come by TMA, boxes of gcd(page, 128) rows out of a tensor of pages; a page
// that is not there, and rows of pages past the length, are boxes past the
// tensor's end, which arrive as zeros, and their keys are not seen.
//
// The pipeline (one CTA an SM, a TMA ring, S issuer, two PV issuers, two softmax
// groups on alternate tiles, output warps, three score buffers in tensor memory)
// and the online softmax with its window of [2^-64, 2^64] around a row's reference
// are attn_scored_bf16.cuh's, without cap and bias.
//
// Bound, like that kernel, by the latency of the chain from a tile's weights over their
// product to the next scores in the same of the three buffers: no pipe is full (issue
// 60 %, tensor 43 %, special functions 43 % of their cycles), and every instruction less
// in the softmax warps' part of it shows.  Measured, causal, 2 x 16 heads x 8,192
// in 64-row pages: the whole call 271 us (1,015 TFLOP/s), listing and joining included;
// 1,024 tokens x 16 heads, 4 to a K/V head, behind 31,744 rows 125 (1,080 TFLOP/s).
//
// int8 pages arrive in a ring of their own, 64 bytes a row, with the rows'
// exponents; the output warps, which are idle while a row tile is worked on, write
// them as bf16 into the K/V ring, in the 128-byte swizzle that TMA leaves
// (n 2^e is exact).  Between two tiles they look for a finished row tile
// first, since the products behind it wait for its accumulators.  A key tile takes 1.25
// us so, 0.53 without, in every row tile that reads it: from kPagedWideRows query rows
// on the rows are laid out as bf16 before instead.
//
// Tried and dropped: stages of their own for K, free earlier, V loaded by an output
// warp, boxes issued by single threads (prompts 318 to 650 us against 291): each
// adds instructions a tile to a warp that gets few to issue beside the softmax, and to
// code that already fills the instruction cache.
#include <cuda_bf16.h>

#include <type_traits>

#include "kernels.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace mha {
namespace {

constexpr int BM = kAttnRowsPerCta;
constexpr int BN = 128;
constexpr int HD = kAttnHeadDim;
constexpr int kSBufs = 3;
constexpr int kThreads = 512;
constexpr int kSoftmaxWarps = 8;
constexpr int kLoadWarp = 8;
constexpr int kMmaSWarp = 9;
constexpr int kMmaPvWarp = 10;
constexpr int kOutWarp = 12;
constexpr uint32_t kTileBytes = BM * HD * 2;
constexpr uint32_t kRawBytes = BN * HD;  // an int8 tile
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 384;
constexpr float kSumMin = 5.421010862427522e-20f, kSumMax = 1.8446744073709552e19f;  // 2^-64, 2^64
// About a second, for a loop of its own between two barriers (the wall clock takes
// microseconds to read).
constexpr long long kSpinClocks = 2000ll * 1000 * 1000;
constexpr int kTable = 48;     // pieces whose geometry is kept on chip

template <bool kInt8>
constexpr int kStages = kInt8 ? 4 : 5;
constexpr int kRaw = 3;  // int8 tiles in flight

// One piece of work: a row tile against key tiles j0 .. j0 + n_kv - 1.
struct Piece {
    int b, head;      // sequence, K/V head
    int tokens, row0; // new tokens, the first one's packed row
    int len, pos0;    // the sequence's length, the position of that token
    int j0, n_kv;
    int full_hi;      // keys below it are seen by every row
    int whole;        // all of the row tile's key tiles
};

template <bool kInt8>
struct RawRing {
    uint8_t k[kRaw][kRawBytes];
    uint8_t v[kRaw][kRawBytes];
    uint8_t ks[kRaw][BN], vs[kRaw][BN];
    uint32_t bad[kRaw];
    uint64_t full[kRaw], empty[kRaw];
};
template <>
struct RawRing<false> {};

template <bool kInt8>
struct __align__(1024) Smem {
    uint8_t q[2][kTileBytes];
    uint8_t k[kStages<kInt8>][kTileBytes];
    uint8_t v[kStages<kInt8>][kTileBytes];
    RawRing<kInt8> raw;
    float red_m[2][BM];
    float red_l[2][BM];
    uint64_t q_full[2];
    uint64_t q_empty[2];
    uint64_t kv_full[kStages<kInt8>];  // by TMA, or (int8) by the output warps
    uint64_t kv_empty[kStages<kInt8>];
    uint64_t s_full[kSBufs];
    uint64_t p_rd[2][2][2];  // [group][round][group tile mod 2]: P of the round written
    uint64_t pv0[2][2];      // [group][group tile mod 2]: round-0 product complete
    uint64_t ml_full, ml_free, o_final, o_free;
    uint64_t drain[3];
    uint32_t bad[kStages<kInt8>];  // a bit for every 16 keys of the tile whose page is not there
    Piece table[kTable];
    Piece own[kThreads / 32];
    int at_x, n_pieces;
    uint32_t tmem_base;
    int abort_flag;
};

// (the ring of one type is not there in the other)
template <bool kInt8>
__device__ __forceinline__ uint64_t *raw_full(Smem<kInt8> &sm, int i) {
    if constexpr (kInt8) return &sm.raw.full[i];
    return nullptr;
}
template <bool kInt8>
__device__ __forceinline__ uint64_t *raw_empty(Smem<kInt8> &sm, int i) {
    if constexpr (kInt8) return &sm.raw.empty[i];
    return nullptr;
}
template <bool kInt8>
__device__ __forceinline__ uint8_t *raw_k(Smem<kInt8> &sm, int i) {
    if constexpr (kInt8) return sm.raw.k[i];
    return nullptr;
}
template <bool kInt8>
__device__ __forceinline__ uint8_t *raw_v(Smem<kInt8> &sm, int i) {
    if constexpr (kInt8) return sm.raw.v[i];
    return nullptr;
}
template <bool kInt8>
__device__ __forceinline__ uint32_t *raw_bad(Smem<kInt8> &sm, int i) {
    if constexpr (kInt8) return &sm.raw.bad[i];
    return nullptr;
}

// Where a CTA's share of the line lies.  A row tile takes kTileCost places on it
// before those of its key tiles: what a piece costs besides them, in key tiles.
// (Causal, 2 x 16 x 8,192: CTAs with the short row tiles of a head have 29 of them,
// others 7.  1 place 285 us, 2 279, 3 271, 4 275, 5 276.)
constexpr int kTileCost = 3;
struct Share {
    int tiles, keys;        // row tiles, places of one K/V head
    int start, end, share;  // of the line
    int head0, x0;          // K/V head and row tile that it starts in
};
__device__ __forceinline__ int place_of(const int *cum, int x) { return cum[x] + kTileCost * x; }

__device__ __forceinline__ Piece make_piece(const PagedAttnParams &p, const Share &sh, int t) {
    const PagedPlan at = paged_plan(p.c.B, paged_most_tiles(p.c.N, p.c.B, p.H / p.c.Hkv));
    const int i = sh.x0 + t, up = i / sh.tiles, x = i - up * sh.tiles;
    const PagedTile tile = reinterpret_cast<const PagedTile *>(p.plan + at.tile)[x];
    Piece w;
    w.head = sh.head0 + up;
    w.b = tile.b;
    w.tokens = tile.tokens;
    w.row0 = tile.row0;
    w.len = tile.len;
    w.pos0 = tile.pos0;
    w.full_hi = p.causal ? min(max(w.pos0 + 1, 0), w.len) : w.len;
    const int n = p.plan[at.cum + x + 1] - p.plan[at.cum + x];
    const int first = w.head * sh.keys + place_of(p.plan + at.cum, x) + kTileCost;  // its first key tile's place
    w.j0 = max(sh.start - first, 0);
    const int end = min(n, sh.end - first);
    w.n_kv = end - w.j0;  // (none or less: the share ends before it)
    w.whole = w.j0 == 0 && end == n;
    return w;
}

// The t-th key tile of a piece: from the last one down.  The tiles that some rows
// see in part are the last ones, and slow; at a piece's end they would hold up the
// accumulators' handing on.
__device__ __forceinline__ int tile_of(const Piece &w, int t) { return w.j0 + w.n_kv - 1 - t; }

template <bool kInt8>
__device__ __forceinline__ const Piece &piece_of(Smem<kInt8> &sm, const PagedAttnParams &p, const Share &sh, int t) {
    if (t < kTable) return sm.table[t];
    Piece &own = sm.own[threadIdx.x >> 5];
    __syncwarp();
    own = make_piece(p, sh, t);  // every lane writes the same
    __syncwarp();
    return own;
}

// The boxes that a warp loads tiles in.  A lane holds where one of the next 32, those
// of 32 / boxes tiles, lies (a look-up a tile would be a trip to L2 for each).
struct Boxes {
    int box, boxes, window;  // rows of a box: gcd(page, 128); boxes of a tile; tiles looked up at once
    int none;                // a page past the tensor: zeros
    int at = 0;              // the tile's first box among the 32
    int page = 0, in_page = 0;
    uint32_t gone = 0;       // 16-key bits of this lane's box in its tile, if it is seen but not there
    bool any_gone = false;
    __device__ __forceinline__ explicit Boxes(const PagedAttnParams &p) {
        box = min(p.c.page & -p.c.page, BN);
        boxes = BN / box;
        window = 32 / boxes;
        none = max(p.c.num_pages, 1);
    }
    // for tile jt of a piece, called for jt = 0, 1, ... by the converged warp
    __device__ __forceinline__ void next(const PagedAttnParams &p, const Piece &w, int jt, int lane) {
        at += boxes;
        if (jt != 0 && at < 32) return;
        at = 0;
        const int j = tile_of(w, jt + lane / boxes), key = j * BN + lane % boxes * box;
        page = none;
        in_page = 0;
        gone = 0;
        if (j >= w.j0 && key < w.len) {
            const int i = key / p.c.page, pg = paged_page(p.c, w.b, i);
            if (pg >= 0) {
                page = pg;
                in_page = key - i * p.c.page;
                if (p.gone) gone = p.gone[static_cast<long long>(pg) * (p.c.page / BN) + j];
            } else {
                gone = ((1u << (box / 16)) - 1u) << (lane % boxes * (box / 16));
            }
        }
        any_gone = __any_sync(0xffffffffu, gone != 0u);
    }
    __device__ __forceinline__ uint32_t bad(int lane) const {
        return any_gone ? __reduce_or_sync(0xffffffffu, lane >= at && lane < at + boxes ? gone : 0u) : 0u;
    }
};

// 16 int8 values of a row as bf16, times 2^e: the two 16-byte pieces.
__device__ __forceinline__ void to_bf16(const uint4 &n, float power, uint4 &a, uint4 &b) {
    const float off = -8388736.f * power;  // 2^23 + 128, the 0x4B000000 and the sign's offset below
    const uint64_t p2 = f32x2_pack(power, power), off2 = f32x2_pack(off, off);
    const uint32_t w[4] = {n.x ^ 0x80808080u, n.y ^ 0x80808080u, n.z ^ 0x80808080u, n.w ^ 0x80808080u};
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = w[i >> 1];
        float y0, y1;
        f32x2_unpack(fma_f32x2(f32x2_pack(__uint_as_float(__byte_perm(u, 0x4B000000u, i & 1 ? 0x7442 : 0x7440)),
                                          __uint_as_float(__byte_perm(u, 0x4B000000u, i & 1 ? 0x7443 : 0x7441))),
                               p2, off2),
                     y0, y1);
        r[i] = pack_bf16x2(y0, y1);
    }
    a = make_uint4(r[0], r[1], r[2], r[3]);
    b = make_uint4(r[4], r[5], r[6], r[7]);
}

template <bool kInt8>
__global__ void __launch_bounds__(kThreads, 1)
    attn_paged_kernel(const __grid_constant__ PagedMaps maps, const __grid_constant__ PagedAttnParams p) {
    constexpr int STAGES = kStages<kInt8>;
    extern __shared__ uint8_t smem_raw[];
    Smem<kInt8> &sm = *reinterpret_cast<Smem<kInt8> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                       ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int cta = static_cast<int>(blockIdx.x), G = static_cast<int>(gridDim.x);
    const int g = p.H / p.c.Hkv, tt = paged_tile_tokens(g);

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 1);
            mbar_init(&sm.q_empty[i], 1);
        }
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&sm.kv_full[i], kInt8 ? 4 : 1);
            mbar_init(&sm.kv_empty[i], 1);
        }
        if constexpr (kInt8)
            for (int i = 0; i < kRaw; ++i) {
                mbar_init(&sm.raw.full[i], 1);
                mbar_init(&sm.raw.empty[i], 4);
            }
        for (int i = 0; i < kSBufs; ++i) mbar_init(&sm.s_full[i], 1);
        for (int i = 0; i < 8; ++i) mbar_init(&sm.p_rd[i >> 2][(i >> 1) & 1][i & 1], kSoftmaxWarps / 2);
        for (int i = 0; i < 4; ++i) mbar_init(&sm.pv0[i >> 1][i & 1], 1);
        mbar_init(&sm.ml_full, kSoftmaxWarps);
        mbar_init(&sm.ml_free, 4);
        mbar_init(&sm.o_final, 2);
        mbar_init(&sm.o_free, 4);
        for (int i = 0; i < 3; ++i) mbar_init(&sm.drain[i], 1);
        sm.abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == kLoadWarp && lane == 0) {
        prefetch_tensormap(&maps.q);
        prefetch_tensormap(&maps.k);
        prefetch_tensormap(&maps.v);
    }
    pdl_wait();
    pdl_launch_dependents();
    Share sh;
    sh.tiles = p.plan[0];
    const PagedPlan at = paged_plan(p.c.B, paged_most_tiles(p.c.N, p.c.B, g));
    const int *cum = p.plan + at.cum;
    sh.keys = p.plan[2] + kTileCost * sh.tiles;
    const int total = p.c.Hkv * sh.keys;
    sh.share = (total + G - 1) / G;
    if (total == 0 || static_cast<long long>(cta) * sh.share >= total) {
        if (threadIdx.x == 0) p.tile_join[cta] = PagedJoin{};
        return;
    }
    if (warp == kMmaSWarp) {
        tmem_alloc(&sm.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    sh.start = cta * sh.share;
    sh.end = min(sh.start + sh.share, total);
    sh.head0 = sh.start / sh.keys;
    const int head1 = (sh.end - 1) / sh.keys;
    {
        const int s0 = sh.start - sh.head0 * sh.keys, s1 = sh.end - 1 - head1 * sh.keys;
        for (int x = threadIdx.x; x < sh.tiles; x += kThreads) {
            const int lo = place_of(cum, x), hi = place_of(cum, x + 1);
            if (lo <= s0 && s0 < hi) sm.at_x = x;
            if (lo <= s1 && s1 < hi) sm.n_pieces = x;
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    sh.x0 = sm.at_x;
    int pieces = (head1 - sh.head0) * sh.tiles + sm.n_pieces - sh.x0 + 1;
    for (int t = threadIdx.x; t < min(pieces, kTable); t += kThreads) sm.table[t] = make_piece(p, sh, t);
    // the last one, if the share ends before its first key tile, is the next CTA's
    if (make_piece(p, sh, pieces - 1).n_kv <= 0) --pieces;
    __syncthreads();
    const uint32_t tmem = sm.tmem_base;
    const AbortState ab{&sm.abort_flag, p.status, 0};

    if (warp == kLoadWarp) {
        // ------------------------------------------------------ TMA producer
        // By the converged warp: an instruction of this warp takes about 10 cycles
        // beside two softmax warps, and 100 of them a tile are more than the tile's
        // weights take.
        Boxes bx(p);
        int n = 0, v = 0, st = 0;
        uint32_t par = 1;
        constexpr int kRing = kInt8 ? kRaw : STAGES;
        const int box_bytes = bx.box * HD * (kInt8 ? 1 : 2);
        bool ok = true, marked = false;  // marked: stages may hold a `bad` other than 0
        if (!kInt8 && lane < STAGES) sm.bad[lane] = 0;
        for (int t = 0; ok && t < pieces; ++t) {
            const Piece &w = piece_of<kInt8>(sm, p, sh, t);
            const int n_kv = w.n_kv, head = w.head;
            for (int jt = 0; ok && jt < n_kv;) {
                const int qbuf = v & 1, run_end = min(jt + kRunTiles, n_kv);
                if (v >= 2 && !(ok = warp_wait(&sm.q_empty[qbuf], ((v - 2) >> 1) & 1, ab))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sm.q_full[qbuf], static_cast<uint32_t>(tt * g) * (HD * 2));
                    if (in_bounds(w.head * g < p.H && w.row0 < p.c.N, p.status))
                        tma_load_3d(&maps.q, &sm.q_full[qbuf], sm.q[qbuf], 0, w.head * g, w.row0);
                }
                __syncwarp();
                ++v;
                for (; jt < run_end; ++jt, ++n) {
                    bx.next(p, w, jt, lane);
                    uint64_t *full = kInt8 ? raw_full(sm, st) : &sm.kv_full[st], *empty = kInt8 ? raw_empty(sm, st) : &sm.kv_empty[st];
                    uint8_t *k = kInt8 ? raw_k(sm, st) : sm.k[st], *vv = kInt8 ? raw_v(sm, st) : sm.v[st];
                    uint32_t bytes = 2 * (kInt8 ? kRawBytes : kTileBytes);
                    if constexpr (kInt8) {
                        const bool there = lane >= bx.at && lane < bx.at + bx.boxes && bx.page < bx.none;
                        bytes += 2u * bx.box * __popc(__ballot_sync(0xffffffffu, there));
                    }
                    if (n >= kRing && !(ok = warp_wait(empty, par, ab))) break;
                    if (bx.any_gone || marked || kInt8) {
                        marked = true;
                        const uint32_t bad = bx.bad(lane);
                        if (lane == 0) *(kInt8 ? raw_bad(sm, st) : &sm.bad[st]) = bad;
                        __syncwarp();
                    }
                    warp_arrive_expect_tx(full, bytes);
#pragma unroll 1
                    for (int i = 0; i < bx.boxes; ++i) {
                        const int pg = __shfl_sync(0xffffffffu, bx.page, bx.at + i), in = __shfl_sync(0xffffffffu, bx.in_page, bx.at + i);
                        warp_tma_load_4d(&maps.k, full, k + i * box_bytes, 0, in, head, pg);
                        warp_tma_load_4d(&maps.v, full, vv + i * box_bytes, 0, in, head, pg);
                        if constexpr (kInt8)
                            if (pg < bx.none) {
                                const long long from = (static_cast<long long>(pg) * p.c.Hkv + head) * p.c.page + in;
                                warp_bulk_load_1d(sm.raw.ks[st] + i * bx.box, p.c.k_scales + from, bx.box, full);
                                warp_bulk_load_1d(sm.raw.vs[st] + i * bx.box, p.c.v_scales + from, bx.box, full);
                            }
                    }
                    if (++st == kRing) {
                        st = 0;
                        par ^= 1u;
                    }
                }
            }
        }
        // Let every copy still in flight land before the CTA exits.
        if (lane == 0) {
            for (int x = max(0, n - kRing); x < n; ++x)
                mbar_wait_drain(kInt8 ? raw_full(sm, x % kRing) : &sm.kv_full[x % kRing], (x / kRing) & 1);
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
        for (int t = 0; ok && t < pieces; ++t) {
            const int n_kv = piece_of<kInt8>(sm, p, sh, t).n_kv;
            for (int jt = 0; ok && jt < n_kv;) {
                const int qbuf = v & 1, run_end = min(jt + kRunTiles, n_kv);
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
            }
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
        for (int t = 0; ok && t < pieces; ++t) {
            const Piece &w = piece_of<kInt8>(sm, p, sh, t);
            for (int run = 0; ok && run < w.n_kv; run += kRunTiles) {
                if (v >= 1 && !(ok = warp_wait(&sm.o_free, (v - 1) & 1, ab))) break;
                const int n_kv = min(w.n_kv - run, kRunTiles);
                for (int jt = 0; jt < n_kv; ++jt, ++n) {
                    if ((n & 1) != hf) continue;
                    const int st = n % STAGES, sb = n % kSBufs;
                    const int slot = (n >> 1) & 1, par = (n >> 2) & 1;
                    if (!(ok = warp_wait(&sm.kv_full[st], (n / STAGES) & 1, ab))) break;
                    // Rows of the last page past the length: their weights are 0, and
                    // 0 times whatever the page holds has to be 0.
                    const int rows = w.len - tile_of(w, run + jt) * BN;
                    if (!kInt8 && rows < BN) {
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
                        for (int kk = 0; kk < 4; ++kk)
                            warp_mma_bf16_ts(d_o, a + 32u * rd + 8u * kk, vd + 128 * (4 * rd + kk), idesc_o,
                                             jt >= 2 || rd > 0 || kk > 0 ? 1u : 0u);
                        if (rd == 0) warp_commit(&sm.pv0[hf][slot]);
                    }
                    if (!ok) break;
                    warp_commit(&sm.kv_empty[st]);
                }
                if (!ok) break;
                warp_commit(&sm.o_final);
                ++v;
            }
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
        const uint64_t mul2 = f32x2_pack(p.mul, p.mul);
        // Weights of N keys against the reference, packed; their sum, of the
        // rounded weights (what the product multiplies, so that they still add up
        // to 1).  bf16, 2^-8 off at most each, is what the matrix instructions take
        // beside bf16 V; a second part for the rest would double their number.
        auto weights = [&](const auto &s, float ref, uint32_t *pk, float (&sum)[4]) {
            constexpr int kPairs = sizeof(s) / 8;
            const uint64_t ref2 = f32x2_pack(-ref, -ref);
#pragma unroll
            for (int c = 0; c < kPairs; ++c) {
                float x0, x1;
                f32x2_unpack(fma_f32x2(f32x2_pack(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), mul2, ref2), x0, x1);
                pk[c] = pack_bf16x2(ex2_approx(x0), ex2_approx(x1));
                add_bf16x2_to_f32(sum[2 * (c & 1)], sum[2 * (c & 1) + 1], pk[c]);
            }
        };
        int n = 0, v = 0;
        int sb = half, s_par = 0, st = half;  // n mod kSBufs and how often that was, n mod STAGES, of this group's next tile
        bool ok = true;
        for (int t = 0; ok && t < pieces; ++t) {
            const Piece &w = piece_of<kInt8>(sm, p, sh, t);
            const int token = r / g;
            const bool live = token < w.tokens;
            const bool warp_live = __any_sync(0xffffffffu, live);
            // keys below it are seen; rows that are none hold nothing up
            const int lim = !live ? 0x7fffffff : p.causal ? min(max(w.pos0 + token + 1, 0), w.len) : w.len;
            const int full_hi = w.full_hi;
            for (int run = 0; ok && run < w.n_kv; run += kRunTiles) {
                float m_run = -INFINITY;  // log2 units; -inf until this group has seen a visible key
                float l_run = 0.f;

                const int n_kv = min(w.n_kv - run, kRunTiles), j_last = w.j0 + w.n_kv - 1 - run;
                const int n0 = n;
                auto step = [&]() {
                    sb += 2;
                    if (sb >= kSBufs) {
                        sb -= kSBufs;
                        s_par ^= 1;
                    }
                    st += 2;
                    if (st >= STAGES) st -= STAGES;
                };
                for (int jt = (n0 ^ half) & 1; jt < n_kv; jt += 2, step()) {
                    n = n0 + jt;
                    const int j = j_last - jt;
                    ok = __all_sync(0xffffffffu, mbar_wait(&sm.s_full[sb], s_par, ab));
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
                    // (written before the tile was handed to the S issuer, which waited
                    // for that before it issued the products whose end s_full tells)
                    const uint32_t bad = *static_cast<volatile uint32_t *>(&sm.bad[st]);
                    const bool edge = j * BN + BN > full_hi || bad != 0;
                    int rd_first = 0;
                    if (!edge) {
#pragma unroll
                        for (int rd = 0; rd < 2; ++rd) {
                            uint32_t s0[32], s1[32], pk[32];
                            tmem_ld32(ts + 64u * rd, s0);
                            tmem_ld32(ts + 64u * rd + 32u, s1);
                            tmem_ld_wait(s0);
                            reg_fence32(s1);
                            const float ref = m_run == -INFINITY ? 0.f : m_run;
                            float sum[4] = {0.f, 0.f, 0.f, 0.f};
                            weights(s0, ref, pk, sum);
                            weights(s1, ref, pk + 16, sum);
                            const float lt = (sum[0] + sum[1]) + (sum[2] + sum[3]);
                            // a reference has to move: to the rounds below
                            if (__any_sync(0xffffffffu, live && !(lt <= kSumMax && (m_run != -INFINITY || lt >= kSumMin)))) break;
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
#pragma unroll 1
                    for (int rd = rd_first; rd < 2; ++rd) {
                        const uint32_t tr = ts + 64u * static_cast<uint32_t>(rd);
                        const int key0 = j * BN + 64 * rd;  // the round's first key
                        const uint32_t gone = bad >> (4 * rd) & 15u;
                        // Does the row need the exact step after a sum against
                        // the reference in hand (0 before there is one)?
                        auto must_move = [&](float sum, bool none) -> bool {
                            if (none || !live) return false;
                            if (m_run != -INFINITY) return !(sum <= kSumMax);
                            if (!(sum >= kSumMin && sum <= kSumMax)) return true;
                            m_run = 0.f;
                            return false;
                        };
                        // 32 keys at a time.
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
                            const int kh = key0 + 32 * h;
                            const uint32_t two = gone >> (2 * h) & 3u;
                            const int hi = min(lim - kh, 32);
                            // the keys seen, a bit each
                            unsigned bits = hi <= 0 ? 0u : 0xffffffffu >> (32 - hi);
                            if (two & 1u) bits &= 0xffff0000u;
                            if (two & 2u) bits &= 0x0000ffffu;
                            const bool none = bits == 0u;
                            const uint32_t tp = ts + 32u * static_cast<uint32_t>(rd);
                            uint32_t pk[16];
                            float lt = 0.f, alpha = 1.f;
                            if (__all_sync(0xffffffffu, none || !live)) {
#pragma unroll
                                for (int c = 0; c < 16; ++c) pk[c] = 0u;
                            } else {
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
                                    const float ref = m_run == -INFINITY ? 0.f : m_run;
#pragma unroll
                                    for (int c = 0; c < 32; ++c) y[c] = __float_as_uint(fmaf(__uint_as_float(y[c]), p.mul, -ref));
                                    if (!all) {
#pragma unroll
                                        for (int c = 0; c < 32; ++c)
                                            if (!(bits >> c & 1u)) y[c] = __float_as_uint(-INFINITY);
                                    }
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
                                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                                    for (int c = 0; c < 16; ++c) {
                                        pk[c] = pack_bf16x2(ex2_approx(__uint_as_float(y[2 * c])), ex2_approx(__uint_as_float(y[2 * c + 1])));
                                        add_bf16x2_to_f32(sum[2 * (c & 1)], sum[2 * (c & 1) + 1], pk[c]);
                                    }
                                    lt = (sum[0] + sum[1]) + (sum[2] + sum[3]);
                                    if (attempt == 2) break;
                                    need = must_move(lt, none);
                                    if (!__any_sync(0xffffffffu, need)) break;
                                }
                            }
                            tmem_st16(tp + 16u * static_cast<uint32_t>(h), pk);
                            l_run += lt;
                            if (!__any_sync(0xffffffffu, alpha != 1.f)) continue;
                            // What was summed before moves with the reference: the
                            // round's first 32 weights, which wait to be multiplied
                            // with these, and O_h, which holds the group's earlier
                            // tiles of the piece and, in round 1, this tile's round
                            // 0: wait for the last product it took.
                            if (h == 1) {
                                tmem_st_wait();
                                tmem_ld16(tp, pk);
                                tmem_ld_wait(pk);
#pragma unroll
                                for (int c = 0; c < 16; ++c)
                                    pk[c] = pack_bf16x2(__uint_as_float(pk[c] << 16) * alpha,
                                                        __uint_as_float(pk[c] & 0xffff0000u) * alpha);
                                tmem_st16(tp, pk);
                            }
                            if (rd == 1) {
                                ok = __all_sync(0xffffffffu, mbar_wait(&sm.pv0[half][(n >> 1) & 1], (n >> 2) & 1, ab));
                            } else if (jt >= 2) {
                                const int np = n - 2;
                                ok = __all_sync(0xffffffffu, mbar_wait(&sm.kv_empty[np % STAGES], (np / STAGES) & 1, ab));
                            } else {
                                continue;  // O_h holds nothing of this piece
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
                n = n0 + n_kv;
                if (v >= 1 && !(ok = __all_sync(0xffffffffu, mbar_wait(&sm.ml_free, (v - 1) & 1, ab)))) break;
                sm.red_m[half][r] = m_run;
                sm.red_l[half][r] = l_run;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.ml_full);
                ++v;
            }
        }
        if (!ok) tmem_st_wait();
    } else {
        // ------------------------------------------------- output, int8 tiles
        const uint32_t lane_base = static_cast<uint32_t>(warp & 3) * 32;
        const int r = static_cast<int>(lane_base) + lane;
        const uint32_t tl = tmem_addr(tmem, lane_base, 0);
        if (warp == kOutWarp && lane == 0) {
            const Piece &w = sm.table[0];
            const int n = cum[sh.x0 + 1] - cum[sh.x0];
            PagedJoin j{};
            const int first = sh.start - w.j0;  // the place of its first key tile
            if (pieces > 0 && w.j0 > 0)
                j = PagedJoin{w.tokens * g, 0, w.head, w.row0, first / sh.share, (first + n - 1) / sh.share};
            p.tile_join[cta] = j;
        }
        // The next run's rows (the v-th of all), once its products are complete: tiles
        // `run` to run + kRunTiles - 1 of piece `t`.  What a piece's runs before have summed
        // waits in its slot.
        int v = 0, t = 0, run = 0;
        auto output = [&]() -> bool {
            const Piece &w = piece_of<kInt8>(sm, p, sh, t);
            const bool first = run == 0, last = run + kRunTiles >= w.n_kv, whole = w.whole && last;
            const int token = r / g, h = w.head * g + r - token * g;
            const bool live = token < w.tokens && in_bounds(h < p.H && w.row0 + token < p.c.N, p.status);
            if (!__all_sync(0xffffffffu, mbar_wait(&sm.ml_full, v & 1, ab))) return false;
            const float ma = sm.red_m[0][r], mb = sm.red_m[1][r];
            const float la = sm.red_l[0][r], lb = sm.red_l[1][r];
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.ml_free);
            if (!__all_sync(0xffffffffu, mbar_wait(&sm.o_final, v & 1, ab))) return false;
            tc_fence_after_sync();
            // A sum of 0: no visible key.  One of NaN goes on to the output.
            const SumLevel va = sum_level(ma, la), vb = sum_level(mb, lb);
            const float M = fmaxf(la != 0.f ? va.m : -INFINITY, lb != 0.f ? vb.m : -INFINITY);
            const float wa = la != 0.f ? ex2_approx(va.m - M) * va.down : 0.f;
            const float wb = lb != 0.f ? ex2_approx(vb.m - M) * vb.down : 0.f;
            float L = la * wa + lb * wb, f = 1.f, keep = 0.f;
            const long long slot = (2ll * cta + (w.j0 > 0 ? 0 : 1)) * BM + r;
            // (the reference of a NaN is as good as any, if the merge takes it)
            float top = L > 0.f ? M : L == 0.f ? -INFINITY : 0.f;
            if (live && !first) {
                const float2 before = p.tile_ml[slot];
                const float m = top;
                top = fmaxf(before.x, m);
                f = m == -INFINITY ? 0.f : ex2_approx(m - top);
                keep = before.x == -INFINITY ? 0.f : ex2_approx(before.x - top);
                L = L * f + before.y * keep;
            }
            if (whole) {
                const float inv = L != 0.f ? 1.0f / L : 0.f;
                f *= inv;
                keep *= inv;
            }
            const float fa = wa * f, fb = wb * f;
            if (live && !whole) p.tile_ml[slot] = make_float2(top, L);
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
                if (!live) continue;
                // a group without a visible key left its accumulator unwritten
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    oa[c] = __float_as_uint((la != 0.f ? __uint_as_float(oa[c]) * fa : 0.f) +
                                            (lb != 0.f ? __uint_as_float(ob[c]) * fb : 0.f));
                uint4 *sum = reinterpret_cast<uint4 *>(p.tile_o + slot * HD) + 8 * part;
                if (!first) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const uint4 x = sum[c];
                        oa[4 * c] = __float_as_uint(fmaf(__uint_as_float(x.x), keep, __uint_as_float(oa[4 * c])));
                        oa[4 * c + 1] = __float_as_uint(fmaf(__uint_as_float(x.y), keep, __uint_as_float(oa[4 * c + 1])));
                        oa[4 * c + 2] = __float_as_uint(fmaf(__uint_as_float(x.z), keep, __uint_as_float(oa[4 * c + 2])));
                        oa[4 * c + 3] = __float_as_uint(fmaf(__uint_as_float(x.w), keep, __uint_as_float(oa[4 * c + 3])));
                    }
                }
                if (!whole) {
#pragma unroll
                    for (int c = 0; c < 8; ++c) sum[c] = make_uint4(oa[4 * c], oa[4 * c + 1], oa[4 * c + 2], oa[4 * c + 3]);
                } else {
                    uint4 *d4 = reinterpret_cast<uint4 *>(p.o + h * p.o_stride_h + (w.row0 + token) * p.o_stride_t) + 4 * part;
                    uint32_t pk[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        pk[c] = pack_bf16x2(__uint_as_float(oa[2 * c]), __uint_as_float(oa[2 * c + 1]));
#pragma unroll
                    for (int c = 0; c < 4; ++c) d4[c] = make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
                }
            }
            ++v;
            run += kRunTiles;
            if (last) {
                run = 0;
                ++t;
            }
            return true;
        };
        // int8: runs are put out as their products are complete, K and V of tile
        // after tile written as stages come free.  Behind a run's last tile it may
        // be a stage that only products after that run's output give back:
        // whichever comes first.  (One place in the code for each: all roles' loops
        // together have to stay in the instruction cache, 32 KB or so; with three
        // copies of output() here a causal prompt took 392 us instead of 290.)
        auto put_first = [&](uint64_t *bar, uint32_t parity, bool &ok) -> bool {
            const long long since = clock64();
            while (true) {
                if (__all_sync(0xffffffffu, mbar_test(&sm.o_final, static_cast<uint32_t>(v & 1)))) return true;
                if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return false;
                bool stop = should_abort(ab);
                if (clock64() - since > kSpinClocks) {
                    raise_abort(ab);
                    stop = true;
                }
                if (__any_sync(0xffffffffu, stop)) {
                    ok = false;
                    return false;
                }
            }
        };
        if constexpr (!kInt8) {
            while (t < pieces && output()) {
            }
        } else {
            const int tid = threadIdx.x - 32 * kOutWarp;
            const int row0 = tid >> 2, quarter = tid & 3;  // rows tid / 4 + 32 i of a tile, a quarter of each
            int runs = 0, piece = 0, jt = 0, st = 0, rs = 0;  // runs: whose tiles are all written
            uint32_t st_par = 1, rs_par = 0;
            int n_kv = 0, keys = 0;
            bool fill = true, ok = true;  // fill: the ring's first round, nothing to wait for
            while (ok && (piece < pieces || v < runs)) {
                bool put = piece == pieces;
                if (!put && jt == 0) {
                    const Piece &w = piece_of<true>(sm, p, sh, piece);
                    n_kv = w.n_kv;
                    keys = w.len - (w.j0 + n_kv - 1) * BN;  // of the tile; rows past them are cleared
                }
                if (!put && !fill) {
                    if (v < runs) put = put_first(&sm.kv_empty[st], st_par, ok);
                    if (ok && !put) ok = warp_wait(&sm.kv_empty[st], st_par, ab);
                    if (!ok) break;
                }
                if (put) {
                    ok = output();
                    continue;
                }
                // (raw tiles wait for nothing but these warps)
                if (!(ok = warp_wait(&sm.raw.full[rs], rs_par, ab))) break;
                const uint32_t bad = sm.raw.bad[rs];
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv) {
                    const uint4 *from = reinterpret_cast<const uint4 *>(kv ? sm.raw.v[rs] : sm.raw.k[rs]) + tid;
                    const uint8_t *es = (kv ? sm.raw.vs[rs] : sm.raw.ks[rs]) + row0;
                    uint4 *to = reinterpret_cast<uint4 *>(kv ? sm.v[st] : sm.k[st]) + row0 * 8 + ((2 * quarter) ^ (row0 & 7));
                    const int other = (row0 & 1) ? -1 : 1;
                    uint4 u[4];
                    uint32_t e[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {  // (all loads before the first store: they may not pass it)
                        u[i] = from[i * 128];
                        e[i] = es[32 * i];
                    }
                    if (keys < BN || bad != 0u) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (row0 + 32 * i >= keys || (bad >> ((row0 + 32 * i) >> 4) & 1u)) e[i] = 0u;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint4 a, b;
                        to_bf16(u[i], paged_power(e[i]), a, b);
                        to[256 * i] = a;
                        to[256 * i + other] = b;
                    }
                }
                if (tid == 0) sm.bad[st] = bad;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sm.kv_full[st]);
                    mbar_arrive(&sm.raw.empty[rs]);
                }
                if (++st == STAGES) {
                    st = 0;
                    st_par ^= 1u;
                    fill = false;
                }
                if (++rs == kRaw) {
                    rs = 0;
                    rs_par ^= 1u;
                }
                keys += BN;
                ++jt;
                if (jt == n_kv || jt % kRunTiles == 0) ++runs;
                if (jt == n_kv) {
                    jt = 0;
                    ++piece;
                }
            }
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaSWarp) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <bool kInt8>
cudaError_t launch(const PagedMaps &maps, const PagedAttnParams &p, cudaStream_t stream) {
    auto kernel = attn_paged_kernel<kInt8>;
    const size_t smem = sizeof(Smem<kInt8>) + 1024;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_kernel(kernel, dim3(kPagedTileCtas), dim3(kThreads), smem, stream, true, 1, maps, p);
}
static_assert(sizeof(Smem<true>) + 1024 <= 227 * 1024 && sizeof(Smem<false>) + 1024 <= 227 * 1024, "shared memory");

}  // namespace

cudaError_t launch_attn_paged(const PagedMaps &maps, const PagedAttnParams &p, cudaStream_t stream) {
    return p.c.int8 ? launch<true>(maps, p, stream) : launch<false>(maps, p, stream);
}

}  // namespace mha
