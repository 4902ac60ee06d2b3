// paged_decode.cu -- attention of few query rows (single tokens, drafted
// tokens, short chunks) over a paged K/V cache, and the joining of partial sums.
//
// A K/V head's query rows are stacked: x = t g + i for token t and the i-th of
// its g query heads.  An item is up to kRows of them against all cached rows of
// the sequence, in units of 16 keys (bf16) or 32 (int8): 4 KB of K and V.  All
// units of the batch stand in one line; every worker takes an equal share of it,
// whatever the lengths, keeps the online softmax of the item it is in (reference
// m in log2 units, sum l, unnormalised O) and leaves it behind where the item ends
// inside the share: whole items are written out, pieces as partial sums that
// paged_merge_kernel joins, in a fixed order.  A worker is a warp, or, where items
// would be divided among more than two of those, the four warps of a CTA, which take
// every fourth unit and meet in shared memory (8 to 16 rows of 4 K/V heads behind
// 32,768 keys: about 600 pieces an item to join, 59 to 104 us, against 15 to 18).  Short
// sequences' items are taken whole, without anything to join (kPagedWholeRows).
//
// The products run on mma.sync with the keys as rows: S^T = K Q^T and
// O^T = V^T P^T, m16n8k16, because the work is bound by memory and a tile of 8
// query rows wastes the least (a tcgen05 tile has 128).  K and V go from global
// memory straight into the fragments: the order of the 64 features in a dot product
// is free, so that a lane's fragments of a K row are 16 consecutive bytes, four lanes a
// row; for V^T a lane holds 8 consecutive features of the four keys its fragments
// need, and pairs of keys are merged by byte permutes.  A unit's K is on its way while
// the weights of the one before it are taken, its V while its scores are.
//
// int8: K n and q are multiplied as fp16, K's whole numbers exactly, a query row
// scaled by a power of two so that its largest element lies in [2^14, 2^15)
// (elements below 2^-31 of it lose bits, 2^-39 of it at most); the keys' powers of
// two and the row's meet the fp32 score.  V's whole numbers are bf16 numbers, and its
// rows' powers of two, times 2^kPowerUp, meet the weights, without rounding but for weights
// below 2^-kPowerUp beside rows as small as there are.  The numbers come out of
// their bytes by permutes: 0x6400 | u is 1024 + u in fp16, u = n + 128, and u alone
// u 2^-133 in bf16.
//
// Measured, single tokens, whole calls: 16 sequences of up to 8,192 bf16 rows x 16
// heads 68 us back to back, 65 between a layer's projections (403 MB, 6.2 TB/s; of up to
// 32,768 rows 238, 6.7 TB/s); 64 sequences of up to 8,192 int8 rows x 2 heads, 8 query
// heads each, 29 us (102 MB, 3.5 TB/s; of up to 32,768 rows 83, 4.9 TB/s).  bf16 is bound
// by DRAM, but for 7 us of launches and joining.  int8 fills no pipe (issue 40 %, ALU 35 %,
// DRAM 46 %; of up to 32,768 rows 45, 41, 61 %): a warp runs 430 instructions a unit, most
// of which wait for one another, at 16 warps an SM, and with 10 units a warp another
// quarter outside that loop.  32 less a unit on the ALU pipe (V's numbers by 2 and a
// multiply-add instead of 3 and a subtraction) took 33.2 to 30.9 us; 40 less on other
// pipes (first products without cleared accumulators, powers before their shuffles, pairs
// of scores at a time) and K or V asked for earlier gained nothing.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kernels.h"
#include "paged.cuh"
#include "sm103_ptx.cuh"

namespace mha {
namespace {

constexpr int HD = kAttnHeadDim;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMergeThreads = 128;
// A row's reference serves until a unit's weights sum to more than this.
constexpr float kSumMax = 65536.0f;
// A worker's least share of the line, in units: what a piece costs to write and
// join is worth a few units of reading.  (Alone, and of the four warps of a CTA.)
constexpr int kLeastShare = 4, kLeastTeamShare = 8;

// CTAs of an SM, by the rows of an item in eights.
constexpr int ctas_of_sm(int n) { return n == 4 ? 2 : n == 2 ? 3 : 4; }

template <bool kInt8>
constexpr int kUnitKeys = kInt8 ? 32 : 16;
// Places on the line that an item takes before those of its units, for what beginning
// one costs a worker: a CTA's four warps together, or a warp.  Without / with them, us:
// 64 sequences of up to 8,192 int8 rows x 2 heads 30.8 / 29.4, 32 of up to 4,096 bf16
// rows x 8 heads 31.2 / 27.5; of warps, 128 of up to 2,048 x 16 heads 134.8 / 131.5.
template <bool kInt8>
constexpr int kTeamCost = kInt8 ? 12 : 8;
constexpr int kAloneCost = 1;
static_assert(kTeamCost<true> <= kPagedItemPlaces && kTeamCost<false> <= kPagedItemPlaces);

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transposes an 8 x 8 matrix of 16-bit elements held as an accumulator's halves are.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint4 load16(const void *p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
__device__ __forceinline__ uint2 load8(const void *p) {
    uint2 r;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}

// The two fp16 pairs n0 n1, n2 n3 of four whole numbers.
__device__ __forceinline__ void to_f16(uint32_t n, uint32_t &lo, uint32_t &hi) {
    const uint32_t u = n ^ 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1024 + 128
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), off), y = __hsub2(*reinterpret_cast<__half2 *>(&b), off);
    lo = *reinterpret_cast<uint32_t *>(&x);
    hi = *reinterpret_cast<uint32_t *>(&y);
}

// Whole number e of a and of b times 2^-6, as a bf16 pair: the half word n + 128 is the
// bf16 number (n + 128) 2^-133 (of its numbers below 2^-125 the bits count multiples of
// 2^-133), and times 2^127, less 128 2^-6, that is exact.
constexpr float kIntUnit = 0.015625f;
__device__ __forceinline__ uint32_t to_bf16(uint32_t a, uint32_t b, int e) {
    const uint32_t u = (__byte_perm(a, b, 0x4400 + 0x1111 * e) & 0x00ff00ffu) ^ 0x00800080u;
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(u), "r"(0x7f007f00u), "r"(0xc000c000u));
    return d;
}

// Weights times V's powers of two are bf16 numbers of their own, whole down to 2^-126 only:
// a weight of 2^-10 beside a row of 2^-120 would keep no bit.  They are taken 2^40 times
// as large, which keeps weights down to 2^-40 of a row whole beside any power.  Up to
// the 2^46 that V may hold there is room: powers of 2^40, weights of 2^16 and sums of 2^26
// units of them come to 2^122.
constexpr int kPowerUp = 40;
constexpr float kPowerDown = 1.f / static_cast<float>(1ull << kPowerUp);
// The exponent that it makes of a stored one; 255 (NaN) stays.
__device__ __forceinline__ uint32_t raised(uint32_t stored) { return min(stored + kPowerUp, 255u); }

// Units of an item that a warp sums in its accumulators without a break, 65,536 keys: then
// they are added to what lies in shared memory.  (The matrix instructions drop, towards
// zero, what lies below a sum's last places: 64 x 16 heads over 2^22 rows each, 1.7 million
// of them a warp, averaged values of one sign to 0.5 % too little.)
template <bool kInt8>
constexpr int kRunUnits = (1 << 16) / kUnitKeys<kInt8>;

// One lane's part of a unit's K, or of its V.
struct Part {
    // K, bf16: keys l/4 and l/4 + 8, two pieces of 8 features; int8: keys l/4 + 8 i,
    // 16 features.  V, bf16: keys 2c, 2c+1, 2c+8, 2c+9 (c = l % 4), features 8 (l/4)
    // on; int8: two such keys in each.
    uint4 x[4];
    uint32_t s;  // int8: the stored exponent of the unit's key `lane`
};

struct Shape {
    int units, places;  // of an item: units, and places on the line (1 where items are not divided)
    int tiles, total;   // row tiles, places of the sequence
};
template <bool kInt8, int kRows>
__device__ __forceinline__ Shape shape_of(const PagedAttnParams &p, const PagedSeq &s, int g, int cost) {
    Shape r;
    const int rows = min(s.n, p.max_new) * g;
    r.units = max((s.len + kUnitKeys<kInt8> - 1) / kUnitKeys<kInt8>, 1);
    r.places = p.undivided ? 1 : r.units + cost;
    r.tiles = rows > p.small_rows ? 0 : (rows + kRows - 1) / kRows;
    r.total = p.c.Hkv * r.tiles * r.places;
    return r;
}

// Sum over the block of one value a thread; `excl`: of the threads before it.
__device__ __forceinline__ int block_sum(int x, int *warp_sums, int &excl) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += warp_sums[w];
        total += warp_sums[w];
    }
    excl = before + incl - x;
    return total;
}

// The row tiles of the sequences that attn_paged_bf16.cu goes through, with
// their key tiles, in plan.
__device__ void list_tiles(const PagedAttnParams &p, int *warp_sums) {
    const int g = p.H / p.c.Hkv, tt = paged_tile_tokens(g);
    const PagedPlan at = paged_plan(p.c.B, paged_most_tiles(p.c.N, p.c.B, g));
    int *first = p.plan + at.first, *cum = p.plan + at.cum;
    PagedTile *tile = reinterpret_cast<PagedTile *>(p.plan + at.tile);
    const int most = paged_most_tiles(p.c.N, p.c.B, g);
    int *slot = p.plan + at.slot, *slot_b = p.plan + at.slot_b, *blocks = p.plan + at.blocks;
    int tiles = 0, slots = 0, rows = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        int n = 0, len = 0, excl;
        if (b < p.c.B) {
            const PagedSeq s = paged_seq(p.c, b);
            const int tokens = min(s.n, p.max_new);
            if (tokens * g > p.small_rows) n = (tokens + tt - 1) / tt;
            len = s.len;
        }
        const int total = block_sum(n, warp_sums, excl);
        if (b < p.c.B) first[b] = min(tiles + excl, most);
        tiles = min(tiles + total, most);  // (more than that only where sequences overlap)
        const int taken = block_sum(n > 0 ? 1 : 0, warp_sums, excl);
        const int mine = slots + excl;
        if (b < p.c.B) {
            slot[b] = n > 0 ? mine : -1;
            if (n > 0) slot_b[mine] = b;
        }
        const int all = block_sum(n > 0 ? (len + 127) / 128 : 0, warp_sums, excl);
        if (b < p.c.B && n > 0) blocks[mine] = rows + excl;
        slots += taken;
        rows += all;
    }
    if (threadIdx.x == 0) {
        first[p.c.B] = tiles;
        blocks[slots] = rows;
        p.plan[1] = slots;
    }
    __syncthreads();
    int keys = 0;
    for (int x0 = 0; x0 < tiles; x0 += kThreads) {
        const int x = x0 + threadIdx.x;
        int n = 0, excl;
        if (x < tiles) {
            int lo = 0, hi = p.c.B;  // the last sequence whose first tile is at most x
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (first[mid] <= x)
                    lo = mid;
                else
                    hi = mid;
            }
            const PagedSeq s = paged_seq(p.c, lo);
            const int t0 = (x - first[lo]) * tt, tokens = min(tt, min(s.n, p.max_new) - t0), pos0 = s.len - s.n + t0;
            const int end = p.causal ? min(max(pos0 + tokens, 0), s.len) : s.len;
            n = max((end + 127) / 128, 1);
            tile[x] = PagedTile{lo, s.len, s.row0 + t0, pos0, tokens, {}};
        }
        const int total = block_sum(n, warp_sums, excl);
        if (x < tiles) cum[x] = keys + excl;
        keys += total;
    }
    if (threadIdx.x == 0) {
        cum[tiles] = keys;
        p.plan[0] = tiles;
        p.plan[2] = keys;
    }
}

template <bool kInt8, int kN>
__global__ void __launch_bounds__(kThreads, ctas_of_sm(kN)) paged_decode_kernel(const PagedAttnParams p, int list) {
    constexpr int kRows = 8 * kN, kKeys = kUnitKeys<kInt8>, kBlocks = kKeys / 16;
    __shared__ int warp_sums[kWarps];
    // Where every warp is on the line: sequence, place in it, places left to it.  Read
    // anew around an item's keys, and not kept over them: registers.
    __shared__ volatile int at_b[kWarps], at_rel[kWarps], at_left[kWarps];
    __shared__ float4 sh_o[kWarps][kRows][HD / 4];
    __shared__ float2 sh_ml[kWarps][kRows];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l4 = lane >> 2, c = lane & 3;
    pdl_wait();
    pdl_launch_dependents();
    if (list && blockIdx.x == gridDim.x - 1) {
        list_tiles(p, warp_sums);
        return;
    }
    const int ctas = gridDim.x - (list ? 1 : 0);
    const int g = p.H / p.c.Hkv;
    const int per_page = p.c.page / 16;

    // The line's length, the shares, and where this worker's begins.
    if (lane == 0) at_b[warp] = -1;
    int total = 0, items = 0, mine = 0, excl = 0, my_items = 0, items_excl = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        Shape sh{};
        if (b < p.c.B) sh = shape_of<kInt8, kRows>(p, paged_seq(p.c, b), g, 0);
        mine = sh.total;
        my_items = p.c.Hkv * sh.tiles;
        items += block_sum(my_items, warp_sums, items_excl);
        total += block_sum(mine, warp_sums, excl);
    }
    // A CTA's warps are workers of their own, or, where items would be divided among
    // more than two of those, one together.
    const int alone = (total + ctas * kWarps - 1) / (ctas * kWarps);
    const bool team = p.undivided || total >= 2ll * alone * items;
    const int cost = p.undivided ? 0 : team ? kTeamCost<kInt8> : kAloneCost;
    total += cost * items;
    mine += cost * my_items;
    excl += cost * items_excl;
    const int share = p.undivided ? (total + ctas - 1) / ctas
                      : team      ? max((total + ctas - 1) / ctas, kLeastTeamShare)
                                  : max((total + ctas * kWarps - 1) / (ctas * kWarps), kLeastShare);
    const int me = team ? blockIdx.x : blockIdx.x * kWarps + warp;
    int base = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        if (p.c.B > kThreads) mine = b < p.c.B ? shape_of<kInt8, kRows>(p, paged_seq(p.c, b), g, cost).total : 0;
        const int sum = p.c.B > kThreads ? block_sum(mine, warp_sums, excl) : 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            // (a share past the line's end may start past 2^31)
            const long long s = static_cast<long long>(team ? blockIdx.x : blockIdx.x * kWarps + w) * share;
            if (s >= base + excl && s < base + excl + mine) {
                at_b[w] = b;
                at_rel[w] = static_cast<int>(s - (base + excl));
                at_left[w] = min(share, static_cast<int>(total - s));
            }
        }
        base += sum;
    }
    // (a record for every warp, whether it is a worker or not)
    if (!p.undivided && team && warp > 0 && lane == 0) p.join[ctas + blockIdx.x * (kWarps - 1) + warp - 1] = PagedJoin{};
    const int sub = team ? warp : 0, step = team ? kWarps : 1;
    __syncthreads();
    if (at_b[warp] < 0) {
        if (!p.undivided && lane == 0 && sub == 0) p.join[me] = PagedJoin{};
        return;
    }
    struct Item {
        PagedSeq s;
        int b, places, total, at0, at1;  // places of the item, of the sequence; of these, this worker's
        int u0, u1;                      // its units
        int units, head, tile, rows;     // of the item
    };
    auto item_now = [&]() {
        Item w;
        w.b = at_b[warp];
        w.s = paged_seq(p.c, w.b);
        const Shape sh = shape_of<kInt8, kRows>(p, w.s, g, cost);
        const int rel = at_rel[warp], item = rel / sh.places;
        w.places = sh.places;
        w.total = sh.total;
        w.units = sh.units;
        w.at0 = rel - item * sh.places;
        w.at1 = min(sh.places, w.at0 + at_left[warp]);
        w.u0 = max(w.at0 - cost, 0);
        w.u1 = p.undivided ? sh.units : w.at1 - cost;
        w.head = item / sh.tiles;
        w.tile = item - w.head * sh.tiles;
        w.rows = min(min(w.s.n, p.max_new) * g - w.tile * kRows, kRows);
        return w;
    };
    if (!p.undivided && lane == 0 && sub == 0) {
        const Item w = item_now();
        PagedJoin j{};
        if (w.u0 > 0) {
            const int first = me * share - w.at0;  // the item's place on the line
            j = PagedJoin{w.rows, w.tile * kRows, w.head, w.s.row0, (first + cost) / share, (first + w.places - 1) / share};
        }
        p.join[me] = j;
    }

    while (true) {
        const Item it = item_now();
        const PagedSeq s = it.s;
        const int b = it.b, u0 = it.u0, u1 = it.u1, head = it.head, tile = it.tile, rows = it.rows;
        if (u1 <= u0) break;  // the share ends before its first key

        // Where the warp's next 32 blocks of 16 keys lie, those of units window0,
        // window0 + step, ..., a lane each: offsets of the rows and of their exponents,
        // how many of the 16 are there; and a bit for each block with all of them.
        int window0 = 0, my_valid = 0;
        unsigned all_there = 0;
        long long my_at = 0, my_scales = 0;
        auto look_up = [&](int u) {
            window0 = u;
            const int block = (u + lane / kBlocks * step) * kBlocks + lane % kBlocks, i = block / per_page;
            const int row = head * p.c.page + (block - i * per_page) * 16;
            const int pg = block * 16 < s.len ? paged_page(p.c, b, i) : -1;
            my_valid = pg >= 0 ? min(s.len - block * 16, 16) : 0;
            my_at = pg * p.c.stride + row * HD;
            if (kInt8) my_scales = static_cast<long long>(pg) * (p.c.Hkv * p.c.page) + row;
            all_there = __ballot_sync(0xffffffffu, my_valid == 16);
        };
        look_up(u0 + sub);
        // The same for a unit's blocks; the exponent of its key `lane`.
        long long at[kBlocks], s_at = 0;
        int valid[kBlocks], s_valid = 16;
        bool full = false;  // all its keys are there
        auto place = [&](int u) {
            if (u - window0 >= 32 / kBlocks * step) look_up(u);
            const int from = (team ? (u - window0) / kWarps : u - window0) * kBlocks;
            constexpr unsigned kAll = (1u << kBlocks) - 1u;
            full = (all_there >> from & kAll) == kAll;
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
                at[i] = __shfl_sync(0xffffffffu, my_at, from + i);
                valid[i] = 16;
            }
            if (kInt8) s_at = __shfl_sync(0xffffffffu, my_scales, from + (lane >> 4)) + (lane & 15);
            if (!full) {
#pragma unroll
                for (int i = 0; i < kBlocks; ++i) valid[i] = __shfl_sync(0xffffffffu, my_valid, from + i);
                if (kInt8) s_valid = __shfl_sync(0xffffffffu, my_valid, from + (lane >> 4));
            }
        };
        // K or V of the unit that place() has found
        auto load = [&](auto is_v, Part &to) {
            constexpr bool kV = decltype(is_v)::value;
            auto rows = [&](auto all) {
                constexpr bool kAll = decltype(all)::value;
                to.s = 0u;
                if (kInt8 && (kAll || (lane & 15) < s_valid)) to.s = __ldg((kV ? p.c.v_scales : p.c.k_scales) + s_at);
#pragma unroll
                for (int i = 0; i < kBlocks; ++i) {
                    const void *base = kV ? p.c.v : p.c.k;
                    if constexpr (kInt8) {
                        const int8_t *from = static_cast<const int8_t *>(base) + at[i];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            uint4 &x = to.x[2 * i + j];
                            if constexpr (kV) {
                                const int key = 2 * c + 8 * j;
                                uint2 v0 = make_uint2(0u, 0u), v1 = v0;
                                if (kAll || key < valid[i]) v0 = load8(from + key * HD + 8 * l4);
                                if (kAll || key + 1 < valid[i]) v1 = load8(from + (key + 1) * HD + 8 * l4);
                                x = make_uint4(v0.x, v0.y, v1.x, v1.y);
                            } else {
                                x = make_uint4(0u, 0u, 0u, 0u);
                                if (kAll || l4 + 8 * j < valid[i]) x = load16(from + (l4 + 8 * j) * HD + 16 * c);
                            }
                        }
                    } else {
                        const __nv_bfloat16 *from = static_cast<const __nv_bfloat16 *>(base) + at[i];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int key = kV ? 2 * c + (j & 1) + 8 * (j >> 1) : l4 + 8 * (j >> 1);
                            to.x[j] = make_uint4(0u, 0u, 0u, 0u);
                            if (kAll || key < valid[i]) to.x[j] = load16(from + key * HD + (kV ? 8 * l4 : 8 * c + 32 * (j & 1)));
                        }
                    }
                }
            };
            if (full)
                rows(std::true_type{});
            else
                rows(std::false_type{});
        };

        float o[kN][4][4], m[kN][2], l[kN][2];
        bool set = false;  // every row has a reference
#pragma unroll
        for (int n = 0; n < kN; ++n) {
#pragma unroll
            for (int i = 0; i < 16; ++i) o[n][i / 4][i % 4] = 0.f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
        }

        // K of the next unit is on its way while this one's weights are taken, its V
        // while the next one's scores are: 32 registers instead of 64, and four
        // CTAs an SM.
        Part kp, vp;
        if (u0 + sub < u1) {
            place(u0 + sub);
            load(std::false_type{}, kp);
            load(std::true_type{}, vp);
        }
        // Queries: a lane's features of row l/4, in every 8 rows.
        uint32_t q[kN][8];
        float mul[kN][2];  // of the scores of rows 2c, 2c + 1
        int lim[kN][2];    // keys below it are seen
        int least = s.len;
#pragma unroll
        for (int n = 0; n < kN; ++n) {
            const int x = tile * kRows + 8 * n + l4;
            uint4 a = make_uint4(0u, 0u, 0u, 0u), d = a;
            if (8 * n + l4 < rows) {
                const int t = x / g;
                const __nv_bfloat16 *src = p.q.x + (head * g + x - t * g) * p.q.stride_h + (s.row0 + t) * p.q.stride_t;
                a = *reinterpret_cast<const uint4 *>(src + (kInt8 ? 16 * c : 8 * c));
                d = *reinterpret_cast<const uint4 *>(src + (kInt8 ? 16 * c + 8 : 8 * c + 32));
            }
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, d.x, d.y, d.z, d.w};
            float f = p.mul;
            if (kInt8) {
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // 2^k, the largest element's (at least the least normal number's)
                const int k = max(static_cast<int>(top >> 7), 1) - 127;
                const float up0 = __uint_as_float((127 - k / 2) << 23), up1 = __uint_as_float((127 + 14 - (k - k / 2)) << 23);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const __half2 h = __floats2half2_rn(__uint_as_float(w[i] << 16) * up0 * up1,
                                                        __uint_as_float(w[i] & 0xffff0000u) * up0 * up1);
                    q[n][i] = *reinterpret_cast<const uint32_t *>(&h);
                }
                f *= __uint_as_float((127 + k / 2) << 23) * __uint_as_float((127 - 14 + (k - k / 2)) << 23);
                if (top >= 0x7f80u) f = __uint_as_float(0x7fc00000u);  // an infinity or NaN in the row: NaN
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) q[n][i] = w[i];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 8 * n + 2 * c + i;
                mul[n][i] = __shfl_sync(0xffffffffu, f, (2 * c + i) * 4);
                lim[n][i] = 0x7fffffff;
                if (r < rows) {
                    lim[n][i] = p.causal ? min(s.len, max(s.len - s.n + (tile * kRows + r) / g + 1, 0)) : s.len;
                    least = min(least, lim[n][i]);
                }
            }
        }
        least = __reduce_min_sync(0xffffffffu, least);

        int u = u0 + sub;
#pragma unroll 1
        for (bool carried = false;; carried = true) {
            const int run_end = min(u1, u + kRunUnits<kInt8> * step);
#pragma unroll 1
            for (; u < run_end; u += step) {
                // scores: key l/4 + 8 j (+ 16 i) of row 2c + r in st[n][i][2 j + r]
                float st[kN][kBlocks][4];
#pragma unroll
                for (int i = 0; i < kBlocks; ++i) {
                    uint32_t ka[2][8];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if constexpr (kInt8) {
                            const uint4 &w = kp.x[2 * i + j];
                            to_f16(w.x, ka[j][0], ka[j][1]);
                            to_f16(w.y, ka[j][2], ka[j][3]);
                            to_f16(w.z, ka[j][4], ka[j][5]);
                            to_f16(w.w, ka[j][6], ka[j][7]);
                        } else {
                            const uint4 &w = kp.x[2 * j], &z = kp.x[2 * j + 1];
                            ka[j][0] = w.x, ka[j][1] = w.y, ka[j][2] = w.z, ka[j][3] = w.w;
                            ka[j][4] = z.x, ka[j][5] = z.y, ka[j][6] = z.z, ka[j][7] = z.w;
                        }
                    }
#pragma unroll
                    for (int n = 0; n < kN; ++n) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) st[n][i][e] = 0.f;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t a[4] = {ka[0][2 * k], ka[1][2 * k], ka[0][2 * k + 1], ka[1][2 * k + 1]};
                            if constexpr (kInt8)
                                mma_f16(st[n][i], a, q[n][2 * k], q[n][2 * k + 1]);
                            else
                                mma_bf16(st[n][i], a, q[n][2 * k], q[n][2 * k + 1]);
                        }
                    }
                }
                int here[kBlocks];  // keys of a block that are there
#pragma unroll
                for (int i = 0; i < kBlocks; ++i) here[i] = valid[i];
                const bool whole = full && (u + 1) * kKeys <= least;  // every row sees every key
                if constexpr (kInt8) {
#pragma unroll
                    for (int i = 0; i < kBlocks; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float power = paged_power(__shfl_sync(0xffffffffu, kp.s, 16 * i + 8 * j + l4));
#pragma unroll
                            for (int n = 0; n < kN; ++n) {
                                st[n][i][2 * j] *= power;
                                st[n][i][2 * j + 1] *= power;
                            }
                        }
                }
                if (u + step < u1) {
                    place(u + step);
                    load(std::false_type{}, kp);
                }
                // Weights against the reference in hand, 0 before there is one.  Masked:
                // of scores in log2 units.  They are rounded to bf16, 2^-8 off at most
                // each, for the matrix instructions; the sums are of the rounded ones, so
                // that they still add up to 1.
                uint32_t pk[kN][kBlocks][2];
                float sum[kN][2];
                auto weights = [&](auto is_masked, bool has_ref) -> bool {
                    constexpr bool masked = decltype(is_masked)::value;
                    bool need = !has_ref;
#pragma unroll
                    for (int n = 0; n < kN; ++n) {
                        const float r0 = masked && m[n][0] == -INFINITY ? 0.f : m[n][0];
                        const float r1 = masked && m[n][1] == -INFINITY ? 0.f : m[n][1];
                        sum[n][0] = sum[n][1] = 0.f;
#pragma unroll
                        for (int i = 0; i < kBlocks; ++i)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                float y0 = masked ? st[n][i][2 * j] - r0 : fmaf(st[n][i][2 * j], mul[n][0], -r0);
                                float y1 = masked ? st[n][i][2 * j + 1] - r1 : fmaf(st[n][i][2 * j + 1], mul[n][1], -r1);
                                pk[n][i][j] = pack_bf16x2(ex2_approx(y0), ex2_approx(y1));
                                add_bf16x2_to_f32(sum[n][0], sum[n][1], pk[n][i][j]);
                            }
                        need |= !(sum[n][0] <= kSumMax) || !(sum[n][1] <= kSumMax);
                    }
                    return __any_sync(0xffffffffu, need);
                };
                if (!whole || !set || weights(std::false_type{}, true)) {
                    // Scores in log2 units, a key that is not seen at minus infinity;
                    // where a row has no reference yet, or its sum leaves the
                    // range, against the unit's maximum.
#pragma unroll
                    for (int n = 0; n < kN; ++n)
#pragma unroll
                        for (int i = 0; i < kBlocks; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int in = l4 + 8 * (e >> 1), key = u * kKeys + 16 * i + in;
                                st[n][i][e] = in < here[i] && key < lim[n][e & 1] ? st[n][i][e] * mul[n][e & 1] : -INFINITY;
                            }
                    if (weights(std::true_type{}, set)) {
#pragma unroll
                        for (int n = 0; n < kN; ++n)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                float top = m[n][r];
#pragma unroll
                                for (int i = 0; i < kBlocks; ++i) top = fmax3(top, st[n][i][r], st[n][i][2 + r]);
                                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                                if (m[n][r] != -INFINITY) {
                                    const float alpha = ex2_approx(m[n][r] - top);
                                    l[n][r] *= alpha;
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        o[n][i][r] *= alpha;
                                        o[n][i][2 + r] *= alpha;
                                    }
                                }
                                m[n][r] = top;
                            }
                        weights(std::true_type{}, true);
                        bool all = true;
#pragma unroll
                        for (int n = 0; n < kN; ++n) all = all && m[n][0] != -INFINITY && m[n][1] != -INFINITY;
                        set = __all_sync(0xffffffffu, all);
                    }
                }
#pragma unroll
                for (int n = 0; n < kN; ++n) {
                    l[n][0] += sum[n][0];
                    l[n][1] += sum[n][1];
                }
                const uint32_t v_power = kInt8 ? raised(vp.s) * 0x00800080u : 0u;  // of the unit's key `lane`
#pragma unroll
                for (int i = 0; i < kBlocks; ++i) {
                    // V^T: features 8 (l/4) + 2 f, + 1 in rows l/4, l/4 + 8 of tile f
                    uint32_t va[4][4];
                    if constexpr (kInt8) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint4 &w = vp.x[2 * i + j];
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                va[e >> 1][2 * j + (e & 1)] = to_bf16(e < 4 ? w.x : w.y, e < 4 ? w.z : w.w, e & 3);
                        }
                    } else {
                        const uint32_t w[4][4] = {{vp.x[0].x, vp.x[0].y, vp.x[0].z, vp.x[0].w},
                                                  {vp.x[1].x, vp.x[1].y, vp.x[1].z, vp.x[1].w},
                                                  {vp.x[2].x, vp.x[2].y, vp.x[2].z, vp.x[2].w},
                                                  {vp.x[3].x, vp.x[3].y, vp.x[3].z, vp.x[3].w}};
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            va[f][0] = __byte_perm(w[0][f], w[1][f], 0x5410);
                            va[f][1] = __byte_perm(w[0][f], w[1][f], 0x7632);
                            va[f][2] = __byte_perm(w[2][f], w[3][f], 0x5410);
                            va[f][3] = __byte_perm(w[2][f], w[3][f], 0x7632);
                        }
                    }
                    // (as bf16 a power's bits are its stored exponent, 7 bits up)
                    uint32_t power[2] = {0u, 0u};
                    if constexpr (kInt8) {
                        power[0] = __shfl_sync(0xffffffffu, v_power, 16 * i + l4);
                        power[1] = __shfl_sync(0xffffffffu, v_power, 16 * i + 8 + l4);
                    }
#pragma unroll
                    for (int n = 0; n < kN; ++n) {
                        if constexpr (kInt8) {
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const __nv_bfloat162 w = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&pk[n][i][j]),
                                                                 *reinterpret_cast<const __nv_bfloat162 *>(&power[j]));
                                pk[n][i][j] = *reinterpret_cast<const uint32_t *>(&w);
                            }
                        }
                        const uint32_t b0 = transpose8(pk[n][i][0]), b1 = transpose8(pk[n][i][1]);
#pragma unroll
                        for (int f = 0; f < 4; ++f) mma_bf16(o[n][f], va[f], b0, b1);
                    }
                }
                if (u + step < u1) load(std::true_type{}, vp);
            }
            // what the runs before have left in shared memory, against the references of then
            if (carried) {
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int row = 8 * n + 2 * c + r;
                        const float was = sh_ml[warp][row].x, f = was == -INFINITY ? 0.f : ex2_approx(was - m[n][r]);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float4 x = sh_o[warp][row][2 * l4 + i];
                            o[n][2 * i][r] = fmaf(x.x, f, o[n][2 * i][r]);
                            o[n][2 * i][2 + r] = fmaf(x.y, f, o[n][2 * i][2 + r]);
                            o[n][2 * i + 1][r] = fmaf(x.z, f, o[n][2 * i + 1][r]);
                            o[n][2 * i + 1][2 + r] = fmaf(x.w, f, o[n][2 * i + 1][2 + r]);
                        }
                    }
                __syncwarp();
            }
            if (u >= u1) break;
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int row = 8 * n + 2 * c + r;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        sh_o[warp][row][2 * l4 + i] =
                            make_float4(o[n][2 * i][r], o[n][2 * i][2 + r], o[n][2 * i + 1][r], o[n][2 * i + 1][2 + r]);
                        o[n][2 * i][r] = o[n][2 * i][2 + r] = o[n][2 * i + 1][r] = o[n][2 * i + 1][2 + r] = 0.f;
                    }
                    if (l4 == 0) sh_ml[warp][row].x = m[n][r];
                }
            __syncwarp();
        }

        // The sums of the worker's warps meet in shared memory.
        auto meet = [team]() {
            if (team)
                __syncthreads();
            else
                __syncwarp();
        };
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float sum = l[n][r];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const int row = 8 * n + 2 * c + r;
                constexpr float f = kInt8 ? 1.f / kIntUnit * kPowerDown : 1.f;
                sh_o[warp][row][2 * l4] = make_float4(o[n][0][r] * f, o[n][0][2 + r] * f, o[n][1][r] * f, o[n][1][2 + r] * f);
                sh_o[warp][row][2 * l4 + 1] = make_float4(o[n][2][r] * f, o[n][2][2 + r] * f, o[n][3][r] * f, o[n][3][2 + r] * f);
                if (l4 == 0) sh_ml[warp][row] = make_float2(m[n][r], sum);
            }
        meet();
        // The item, or the piece: slot 2 me of one that began before this worker,
        // 2 me + 1 of one that goes on behind it.  16 lanes take a row.
        {
            const Item w = item_now();
            const bool whole = w.u0 == 0 && w.u1 == w.units;
            const long long slot = (2ll * me + (w.u0 > 0 ? 0 : 1)) * kRows;
            const int w0 = team ? 0 : warp, wn = team ? kWarps : 1, part = lane & 15;
            for (int row = (team ? threadIdx.x : lane) / 16; row < w.rows; row += 2 * wn) {
                float top = -INFINITY, sum = 0.f;
                for (int i = w0; i < w0 + wn; ++i) top = fmaxf(top, sh_ml[i][row].x);
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int i = w0; i < w0 + wn; ++i) {
                    const float2 ml = sh_ml[i][row];
                    if (ml.y == 0.f) continue;  // no visible key
                    const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - top);
                    const float4 x = sh_o[i][row][part];
                    sum += ml.y * f;
                    y = make_float4(y.x + x.x * f, y.y + x.y * f, y.z + x.z * f, y.w + x.w * f);
                }
                if (whole) {
                    const float inv = sum != 0.f ? 1.f / sum : 0.f;
                    const int at = w.tile * kRows + row, t = at / g, h = w.head * g + at - t * g;
                    if (in_bounds(h < p.H && w.s.row0 + t < p.c.N, p.status))
                        reinterpret_cast<uint2 *>(p.o + h * p.o_stride_h + (w.s.row0 + t) * p.o_stride_t)[part] =
                            make_uint2(pack_bf16x2(y.x * inv, y.y * inv), pack_bf16x2(y.z * inv, y.w * inv));
                } else if (in_bounds(me < ctas * kWarps, p.status)) {
                    reinterpret_cast<float4 *>(p.part_o + (slot + row) * HD)[part] = y;
                    if (part == 0) p.part_ml[slot + row] = make_float2(top, sum);
                }
            }
            const int left = at_left[warp] - (w.at1 - w.at0);
            int next = w.b, rel = at_rel[warp] + w.at1 - w.at0;
            if (rel == w.total) {
                rel = 0;
                do ++next;
                while (left > 0 && next < p.c.B && shape_of<kInt8, kRows>(p, paged_seq(p.c, next), g, cost).total == 0);
            }
            meet();
            if (left <= 0 || next >= p.c.B) break;
            if (lane == 0) {
                at_b[warp] = next;
                at_rel[warp] = rel;
                at_left[warp] = left;
            }
            __syncwarp();
        }
    }
}

// ------------------------------------------------------------ joining partial sums
//   o = (sum_s w_s O_s) / (sum_s w_s l_s),  w_s = 2^(m_s - M),  M = max_s m_s
// over the pieces of an item: the tail slot of its first worker, then the head slots
// up to its last one, in that order whatever the timing.
// 16 lanes take one row (4 features each), up to kBatch pieces at a time; groups that
// would be idle share a row's pieces.  A piece without a visible key has m = -inf,
// l = 0; one with a NaN or infinity among its scores l = NaN.  m_s is taken as
// sum_level gives it.
//
// Bound by latency: small blocks, most of which find nothing to join.  Behind row
// tiles, whose blocks come on top, one looks at four workers' records, and takes fewer
// pieces at a time to be resident with the others (10 us -> 7).
constexpr int kTileBlocks = 8;  // for a worker of attn_paged_bf16.cu
constexpr int kGroups = kMergeThreads / 16;

__device__ __forceinline__ float piece_weight(float m, float top) { return m == -INFINITY ? 0.f : ex2_approx(m - top); }

// A partial sum, and others joined to it.
template <int kBatch>
struct Sum {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    // pieces with l = 0 are left out
    __device__ __forceinline__ void add(const float2 (&ml)[kBatch], const float4 (&x)[kBatch]) {
        float top = m;
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (ml[i].y != 0.f) top = fmaxf(top, sum_level(ml[i].x, ml[i].y).m);
        const float a = piece_weight(m, top);
        m = top;
        l *= a;
        o = make_float4(o.x * a, o.y * a, o.z * a, o.w * a);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (ml[i].y != 0.f) {
                const SumLevel v = sum_level(ml[i].x, ml[i].y);
                const float w = piece_weight(v.m, top) * v.down;
                l += ml[i].y * w;
                o = make_float4(o.x + x[i].x * w, o.y + x[i].y * w, o.z + x[i].z * w, o.w + x[i].w * w);
            }
    }
};

template <int kBatch>
__device__ __forceinline__ void join_rows(const PagedAttnParams &p, const PagedJoin &j, bool small, int slot_rows, int from, int rows,
                                          float4 (&sh_o)[kGroups][16], float2 (&sh_ml)[kGroups]) {
    const int g = p.H / p.c.Hkv;
    const int grp = threadIdx.x / 16, lane = threadIdx.x & 15;
    const float *part_o = small ? p.part_o : p.tile_o;
    const float2 *part_ml = small ? p.part_ml : p.tile_ml;
    const int pieces = j.last - j.first + 1;
    int per = 1;  // groups of a row
    while (per < kGroups && per * 2 * rows <= kGroups) per *= 2;
    for (int r0 = 0; r0 < rows; r0 += kGroups / per) {
        const int row = r0 + grp / per, part = grp % per;
        float2 ml[kBatch];
        float4 o[kBatch];
        Sum<kBatch> sum;
        if (row < rows) {
            for (int i0 = part; i0 < pieces; i0 += kBatch * per) {
#pragma unroll
                for (int e = 0; e < kBatch; ++e) {
                    const int i = i0 + e * per;
                    ml[e] = make_float2(-INFINITY, 0.f);
                    o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i < pieces) {
                        const long long slot = (2ll * (j.first + i) + (i == 0 ? 1 : 0)) * slot_rows + from + row;
                        ml[e] = part_ml[slot];
                        o[e] = reinterpret_cast<const float4 *>(part_o + slot * HD)[lane];
                    }
                }
                sum.add(ml, o);
            }
        }
        if (per > 1) {
            __syncthreads();
            sh_o[grp][lane] = sum.o;
            if (lane == 0) sh_ml[grp] = make_float2(sum.m, sum.l);
            __syncthreads();
            if (part == 0) {
                sum = Sum<kBatch>();
                for (int i0 = 0; i0 < per; i0 += kBatch) {
#pragma unroll
                    for (int e = 0; e < kBatch; ++e) {
                        ml[e] = i0 + e < per ? sh_ml[grp + i0 + e] : make_float2(-INFINITY, 0.f);
                        o[e] = i0 + e < per ? sh_o[grp + i0 + e][lane] : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
                    sum.add(ml, o);
                }
            }
        }
        if (part == 0 && row < rows) {
            const float inv = sum.l != 0.f ? 1.f / sum.l : 0.f;
            const int at = j.x0 + from + row, t = at / g, h = j.head * g + at - t * g;
            if (in_bounds(h < p.H && j.row0 + t < p.c.N, p.status))
                reinterpret_cast<uint2 *>(p.o + h * p.o_stride_h + (j.row0 + t) * p.o_stride_t)[lane] =
                    make_uint2(pack_bf16x2(sum.o.x * inv, sum.o.y * inv), pack_bf16x2(sum.o.z * inv, sum.o.w * inv));
        }
    }
}

// Blocks 0 .. workers / kRecords - 1 look at kRecords of the warps' records each, far
// apart; the others, kTileBlocks for each of attn_paged_bf16.cu's CTAs, at that CTA's.
// The rows of an item are divided among the blocks of all workers that began inside.
template <int kBatch, int kRecords>
__global__ void __launch_bounds__(kMergeThreads, kBatch == 8 ? 5 : 8) paged_merge_kernel(const PagedAttnParams p, int workers,
                                                                                         int tile_rows) {
    __shared__ float4 sh_o[kGroups][16];
    __shared__ float2 sh_ml[kGroups];
    pdl_wait();
    pdl_launch_dependents();
    const int own = workers / kRecords, x = blockIdx.x;
    auto join = [&](const PagedJoin &j, bool small, int w, int per, int block) {
        if (j.rows == 0) return;
        const int blocks = (j.last - j.first) * per, at = (w - 1 - j.first) * per + block;
        const int from = j.rows * at / blocks, rows = j.rows * (at + 1) / blocks - from;
        if (rows > 0) join_rows<kBatch>(p, j, small, small ? tile_rows : 128, from, rows, sh_o, sh_ml);
    };
    if (x >= own) {
        const int w = (x - own) / kTileBlocks;
        join(p.tile_join[w], false, w, kTileBlocks, (x - own) % kTileBlocks);
    } else if (kRecords == 1) {
        join(p.join[x], true, x, 1, 0);
    } else {
        __shared__ PagedJoin sh_j[kRecords];
        if (threadIdx.x < kRecords) sh_j[threadIdx.x] = p.join[x + threadIdx.x * own];
        __syncthreads();
        for (int i = 0; i < kRecords; ++i) join(sh_j[i], true, x + i * own, 1, 0);
    }
}

template <bool kInt8>
cudaError_t launch_rows(const PagedAttnParams &p, int list, int tile_rows, cudaStream_t stream) {
    const dim3 grid(paged_decode_ctas(tile_rows) + list), block(kThreads);
    if (tile_rows == 8) return launch_kernel(paged_decode_kernel<kInt8, 1>, grid, block, 0, stream, true, 1, p, list);
    if constexpr (kInt8)  // (paged_small_rows())
        if (tile_rows == 32) return launch_kernel(paged_decode_kernel<true, 4>, grid, block, 0, stream, true, 1, p, list);
    return launch_kernel(paged_decode_kernel<kInt8, 2>, grid, block, 0, stream, true, 1, p, list);
}

}  // namespace

int paged_decode_rows(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }

int paged_decode_ctas(int tile_rows) { return kSmsPerGpu * ctas_of_sm(tile_rows / 8); }
int paged_decode_workers(int tile_rows) { return paged_decode_ctas(tile_rows) * kWarps; }

cudaError_t launch_paged_decode(const PagedAttnParams &p, bool tiles, int tile_rows, cudaStream_t stream) {
    return p.c.int8 ? launch_rows<true>(p, tiles ? 1 : 0, tile_rows, stream) : launch_rows<false>(p, tiles ? 1 : 0, tile_rows, stream);
}

cudaError_t launch_paged_merge(const PagedAttnParams &p, bool tiles, int tile_rows, cudaStream_t stream) {
    const int workers = paged_decode_workers(tile_rows);
    if (!tiles)
        return launch_kernel(paged_merge_kernel<8, 1>, dim3(workers), dim3(kMergeThreads), 0, stream, true, 1, p, workers, tile_rows);
    const dim3 grid(workers / 4 + kPagedTileCtas * kTileBlocks);
    return launch_kernel(paged_merge_kernel<4, 4>, grid, dim3(kMergeThreads), 0, stream, true, 1, p, workers, tile_rows);
}

}  // namespace mha
