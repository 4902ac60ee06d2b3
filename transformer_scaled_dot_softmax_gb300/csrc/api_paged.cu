// api_paged.cu -- the paged K/V cache entry points of include/mha.h: argument
// checks, workspace layout and launches.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/mha.h"
#include "kernels.h"

#define MHA_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

using namespace mha;

constexpr int kMostPageRows = 1 << 16;
constexpr long long kMostRows = 1ll << 30;  // of a sequence, or packed
// Units of the kernels' work lines: 32 bits, with room to round up to equal shares.
constexpr long long kMostLine = (1ll << 31) - (1 << 14);

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
mha_status launched(cudaError_t e, const char *what) {
    return e == cudaSuccess ? MHA_OK : record_cuda_failure(what, cudaGetErrorName(e));
}

// Everything but the pointers.
mha_status check_sizes(const mha_paged_cache *x, int d, int N, PagedCache &c) {
    if (x->dtype != MHA_BF16 && x->dtype != MHA_INT8)
        return x->dtype == MHA_F32 ? MHA_ERR_UNSUPPORTED : MHA_ERR_INVALID_ARG;
    if (x->B < 0 || x->h_kv < 0 || x->num_pages < 0 || x->max_pages < 0 || x->page_rows <= 0 || N < 0 || d <= 0)
        return MHA_ERR_INVALID_ARG;
    if (d != kAttnHeadDim || x->page_rows % 16 != 0 || x->page_rows > kMostPageRows || x->h_kv > 65535 || x->B > 65535)
        return MHA_ERR_UNSUPPORTED;
    if (static_cast<long long>(x->max_pages) * x->page_rows >= kMostRows) return MHA_ERR_UNSUPPORTED;
    const long long rows_of_page = static_cast<long long>(x->h_kv) * x->page_rows;
    if (rows_of_page > (1 << 24)) return MHA_ERR_UNSUPPORTED;
    c.int8 = x->dtype == MHA_INT8;
    c.k = x->k_pages;
    c.v = x->v_pages;
    c.k_scales = x->k_scales;
    c.v_scales = x->v_scales;
    c.stride = x->page_stride;
    c.table = x->page_table;
    c.starts = x->row_starts;
    c.lens = x->seq_lens;
    c.B = x->B;
    c.Hkv = x->h_kv;
    c.page = x->page_rows;
    c.num_pages = x->num_pages;
    c.max_pages = x->max_pages;
    c.cap = x->max_pages * x->page_rows;
    c.N = N;
    if (x->num_pages > 1 && (x->page_stride < rows_of_page * kAttnHeadDim || x->page_stride % 16 != 0)) return MHA_ERR_INVALID_ARG;
    if (x->num_pages <= 1) c.stride = rows_of_page * kAttnHeadDim;
    return c.stride < (1ll << 38) ? MHA_OK : MHA_ERR_UNSUPPORTED;
}

// `rows`: the call takes packed rows (row_starts).
mha_status check_cache(const mha_paged_cache *x, int d, bool rows, int N, PagedCache &c) {
    if (!x) return MHA_ERR_INVALID_ARG;
    const mha_status s = check_sizes(x, d, N, c);
    if (s != MHA_OK) return s;
    if (x->B == 0 || x->h_kv == 0) return MHA_OK;
    if (!x->seq_lens || (rows && !x->row_starts) || (x->max_pages > 0 && !x->page_table)) return MHA_ERR_INVALID_ARG;
    if (x->num_pages > 0) {
        if (!c.k || !c.v || (c.int8 && (!c.k_scales || !c.v_scales))) return MHA_ERR_INVALID_ARG;
        if (!aligned16(c.k) || !aligned16(c.v) || (c.int8 && (!aligned16(c.k_scales) || !aligned16(c.v_scales))))
            return MHA_ERR_MISALIGNED;
    }
    return MHA_OK;
}

// Rows (heads, N, 64) at strides of their own.
mha_status check_rows(const void *x, long long stride_h, long long stride_t, int heads, int N, PagedRows &r) {
    if (!x) return MHA_ERR_INVALID_ARG;
    if (!aligned16(x)) return MHA_ERR_MISALIGNED;
    if ((heads > 1 && stride_h < kAttnHeadDim) || (N > 1 && stride_t < kAttnHeadDim)) return MHA_ERR_INVALID_ARG;
    if ((heads > 1 && stride_h % 8 != 0) || (N > 1 && stride_t % 8 != 0)) return MHA_ERR_MISALIGNED;
    if (stride_h >= (1ll << 38) || stride_t >= (1ll << 38)) return MHA_ERR_UNSUPPORTED;
    r.x = static_cast<const __nv_bfloat16 *>(x);
    // the stride of a single head or row is never used but in a tensor map
    r.stride_h = heads > 1 ? stride_h : kAttnHeadDim;
    r.stride_t = N > 1 ? stride_t : kAttnHeadDim;
    return MHA_OK;
}

// What a call's workspace holds.
struct Layout {
    bool tiles;      // sequences may have more than paged_small_rows() stacked rows
    bool undivided;  // no key range is divided
    int tile_rows;   // of paged_decode.cu
    int slots, wide_cap;  // places for rows laid out as bf16 (0: none), their rows
    size_t part_o, part_ml, join, plan, tile_o, tile_ml, tile_join, wide_k, wide_v, gone, bytes;
};
Layout layout(const PagedCache &c, int g, int max_new) {
    Layout l{};
    const long long most = static_cast<long long>(std::min(max_new, c.N)) * g;
    const int small = paged_small_rows(c.int8 != 0);
    l.tiles = most > small;
    // among longer chunks the short ones are taken for single tokens
    l.tile_rows = paged_decode_rows(l.tiles ? std::min(g, small) : static_cast<int>(most));
    const long long items = static_cast<long long>(c.B) * c.Hkv * ((most + l.tile_rows - 1) / l.tile_rows);
    l.undivided = !l.tiles && c.cap <= kPagedWholeRows && items <= paged_decode_ctas(l.tile_rows);
    if (l.undivided) return l;
    const size_t workers = static_cast<size_t>(paged_decode_workers(l.tile_rows));
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t was = at;
        at += round256(bytes);
        return was;
    };
    l.part_o = take(2 * workers * l.tile_rows * kAttnHeadDim * sizeof(float));
    l.part_ml = take(2 * workers * l.tile_rows * sizeof(float2));
    l.join = take(workers * sizeof(PagedJoin));
    if (l.tiles) {
        l.plan = take(sizeof(int) * static_cast<size_t>(paged_plan(c.B, paged_most_tiles(c.N, c.B, g)).ints));
        l.tile_o = take(static_cast<size_t>(2) * kPagedTileCtas * 128 * kAttnHeadDim * sizeof(float));
        l.tile_ml = take(static_cast<size_t>(2) * kPagedTileCtas * 128 * sizeof(float2));
        l.tile_join = take(kPagedTileCtas * sizeof(PagedJoin));
        // sequences with more than `small` rows are no more than these
        const int slots = static_cast<int>(std::min<long long>(c.B, static_cast<long long>(c.N) * g / (small + 1)));
        const int cap = (c.cap + 127) / 128 * 128;
        const size_t rows = static_cast<size_t>(slots) * c.Hkv * cap;
        const bool wide = c.int8 || c.page % 32 != 0
                              ? most >= kPagedWideRows
                              : c.page % 64 != 0 && most >= kPagedWideRows32 && c.cap >= kPagedWideKeys32;
        if (wide && rows > 0 &&
            rows <= kPagedWideBytes / (2 * kAttnHeadDim * sizeof(__nv_bfloat16))) {
            l.slots = slots;
            l.wide_cap = cap;
            l.wide_k = take(rows * kAttnHeadDim * sizeof(__nv_bfloat16));
            l.wide_v = take(rows * kAttnHeadDim * sizeof(__nv_bfloat16));
            l.gone = take(static_cast<size_t>(slots) * (cap / 128) * sizeof(uint32_t));
        }
    }
    l.bytes = at;
    return l;
}

// Do 32 bits number the kernels' work lines, for whatever lengths and starts the device
// holds?  (Units of 16 bf16 or 32 int8 keys of what is taken as few rows; key tiles.)
bool lines_fit(const PagedCache &c, const Layout &l, int g, int max_new) {
    const long long cap = c.cap, unit = c.int8 ? 32 : 16;
    const long long rows = std::min<long long>(static_cast<long long>(std::min(max_new, c.N)) * g, paged_small_rows(c.int8 != 0));
    const long long row_tiles = (rows + l.tile_rows - 1) / l.tile_rows;
    if (static_cast<long long>(c.B) * c.Hkv * row_tiles * (cap / unit + 1 + kPagedItemPlaces) >= kMostLine) return false;
    return !l.tiles || static_cast<long long>(paged_most_tiles(c.N, c.B, g)) * c.Hkv * (cap / 128 + 8) < kMostLine;
}

mha_status check_heads(int B, int h, int h_kv, int N, int max_new) {
    if (B < 0 || h < 0 || h_kv < 0 || N < 0 || max_new < 0) return MHA_ERR_INVALID_ARG;
    if (h > 0 && (h_kv == 0 || h % h_kv != 0)) return MHA_ERR_INVALID_ARG;
    if (h > 0 && h / h_kv > 128) return MHA_ERR_UNSUPPORTED;
    if (B > 65535 || h > 65535 || static_cast<long long>(N) * h >= (1ll << 30)) return MHA_ERR_UNSUPPORTED;
    return MHA_OK;
}

}  // namespace

MHA_EXPORT mha_status paged_cache_append(const mha_paged_cache *cache, const void *k, long long k_stride_h,
                                         long long k_stride_t, const void *v, long long v_stride_h, long long v_stride_t,
                                         int N, int d, cudaStream_t stream) {
    PagedCache c{};
    PagedRows kr, vr;
    mha_status s = check_cache(cache, d, true, N, c);
    if (s != MHA_OK) return s;
    if (N >= kMostRows) return MHA_ERR_UNSUPPORTED;
    if (N == 0 || c.B == 0 || c.Hkv == 0 || c.max_pages == 0 || c.num_pages == 0) return MHA_OK;
    if ((s = check_rows(k, k_stride_h, k_stride_t, c.Hkv, N, kr)) != MHA_OK) return s;
    if ((s = check_rows(v, v_stride_h, v_stride_t, c.Hkv, N, vr)) != MHA_OK) return s;
    return launched(launch_paged_append(c, kr, vr, stream), "paged cache append launch");
}

MHA_EXPORT mha_status paged_cache_read(const mha_paged_cache *cache, void *k, void *v, int T, int d, cudaStream_t stream) {
    PagedCache c{};
    mha_status s = check_cache(cache, d, false, 0, c);
    if (s != MHA_OK) return s;
    if (T < 0) return MHA_ERR_INVALID_ARG;
    if (T == 0 || c.B == 0 || c.Hkv == 0) return MHA_OK;
    if (!k || !v) return MHA_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v)) return MHA_ERR_MISALIGNED;
    if (T >= kMostRows || static_cast<long long>(c.B) * c.Hkv * ((T + 127) / 128) >= (1ll << 31)) return MHA_ERR_UNSUPPORTED;
    return launched(launch_paged_read(c, static_cast<__nv_bfloat16 *>(k), static_cast<__nv_bfloat16 *>(v), T, stream),
                    "paged cache read launch");
}

MHA_EXPORT size_t sdpa_paged_workspace_bytes(const mha_paged_cache *cache, int h, int N, int max_new) {
    PagedCache c{};
    // (sizes alone: the pointers may be missing)
    if (!cache || check_sizes(cache, kAttnHeadDim, N, c) != MHA_OK || check_heads(c.B, h, c.Hkv, N, max_new) != MHA_OK) return 0;
    if (c.B == 0 || h == 0 || N == 0 || max_new == 0) return 0;
    const Layout l = layout(c, h / c.Hkv, max_new);
    return lines_fit(c, l, h / c.Hkv, max_new) ? l.bytes : 0;
}

MHA_EXPORT mha_status sdpa_paged_forward(const mha_paged_cache *cache, const void *q, long long q_stride_h,
                                         long long q_stride_t, void *o, long long o_stride_h, long long o_stride_t,
                                         void *workspace, size_t workspace_bytes, int h, int N, int max_new, int d,
                                         float scale, mha_mask mask, int *status_dev, cudaStream_t stream) {
    PagedAttnParams p{};
    mha_status s = check_cache(cache, d, true, N, p.c);
    if (s != MHA_OK) return s;
    if ((s = check_heads(p.c.B, h, p.c.Hkv, N, max_new)) != MHA_OK) return s;
    if (!isfinite(scale) || !isfinite(scale * 1.4426950408889634f)) return MHA_ERR_INVALID_ARG;
    if (mask < MHA_MASK_NONE || mask > MHA_MASK_CAUSAL_KEY_PADDING) return MHA_ERR_INVALID_ARG;
    if (p.c.B == 0 || h == 0 || N == 0 || max_new == 0) return MHA_OK;
    PagedRows out;
    if ((s = check_rows(q, q_stride_h, q_stride_t, h, N, p.q)) != MHA_OK) return s;
    if ((s = check_rows(o, o_stride_h, o_stride_t, h, N, out)) != MHA_OK) return s;
    const int g = h / p.c.Hkv;
    const Layout l = layout(p.c, g, max_new);
    if (!lines_fit(p.c, l, g, max_new)) return MHA_ERR_UNSUPPORTED;
    if (l.bytes > 0 && (!workspace || workspace_bytes < l.bytes)) return MHA_ERR_WORKSPACE;
    if (l.bytes > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return MHA_ERR_MISALIGNED;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.o_stride_h = out.stride_h;
    p.o_stride_t = out.stride_t;
    p.H = h;
    p.max_new = std::min(max_new, N);
    p.causal = (mask & MHA_MASK_CAUSAL) ? 1 : 0;
    p.mul = scale * 1.4426950408889634f;
    p.small_rows = l.tiles ? paged_small_rows(p.c.int8 != 0) : 1 << 30;
    p.undivided = l.undivided ? 1 : 0;
    if (!l.undivided) {
        p.part_o = reinterpret_cast<float *>(ws + l.part_o);
        p.part_ml = reinterpret_cast<float2 *>(ws + l.part_ml);
        p.join = reinterpret_cast<PagedJoin *>(ws + l.join);
    }
    p.status = status_dev;
    PagedMaps maps;
    if (l.tiles) {
        p.plan = reinterpret_cast<int *>(ws + l.plan);
        p.tile_o = reinterpret_cast<float *>(ws + l.tile_o);
        p.tile_ml = reinterpret_cast<float2 *>(ws + l.tile_ml);
        p.tile_join = reinterpret_cast<PagedJoin *>(ws + l.tile_join);
    }
    PagedAttnParams t = p;  // of the row tiles
    PagedWide w{};
    if (l.slots > 0) {
        w.k = reinterpret_cast<__nv_bfloat16 *>(ws + l.wide_k);
        w.v = reinterpret_cast<__nv_bfloat16 *>(ws + l.wide_v);
        w.gone = reinterpret_cast<uint32_t *>(ws + l.gone);
        w.cap = l.wide_cap;
        w.slots = l.slots;
        // a bf16 cache with a page for every such sequence
        t.gone = w.gone;
        t.c.int8 = 0;
        t.c.k = w.k;
        t.c.v = w.v;
        t.c.stride = static_cast<long long>(p.c.Hkv) * w.cap * kAttnHeadDim;
        t.c.table = p.plan + paged_plan(p.c.B, paged_most_tiles(N, p.c.B, g)).slot;
        t.c.max_pages = 1;
        t.c.num_pages = w.slots;
        t.c.page = w.cap;
    }
    if (l.tiles && (s = encode_paged_maps(&maps, t)) != MHA_OK) return s;
    if ((s = launched(launch_paged_decode(p, l.tiles, l.tile_rows, stream), "paged attention, few rows")) != MHA_OK) return s;
    if (l.slots > 0 && (s = launched(launch_paged_widen(p, w, stream), "paged attention, rows to bf16")) != MHA_OK) return s;
    if (l.tiles && (s = launched(launch_attn_paged(maps, t, stream), "paged attention, row tiles")) != MHA_OK) return s;
    if (l.undivided) return MHA_OK;
    return launched(launch_paged_merge(p, l.tiles, l.tile_rows, stream), "paged attention, joining");
}
