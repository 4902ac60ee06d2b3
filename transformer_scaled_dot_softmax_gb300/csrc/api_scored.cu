// api_scored.cu -- the scored attention entry points of include/mha.h:
// argument checks, workspace layout, tensor maps and launches.
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

constexpr int kMaxFar = 1 << 16;      // last bucket's first distance
constexpr int kMaxLength = 1 << 24;   // distances are exact in fp32
// Caps between which the score, its derivative and their factors stay well
// inside fp32's range.
constexpr float kLeastCap = 1e-18f, kMostCap = 1e18f;
// What the capping polynomials may take from a score, in natural units: a
// seventh of a weight's bf16 half step (2^-8 relative).
constexpr double kCapError = 6e-4;

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
mha_status launched(cudaError_t e, const char *what) {
    return e == cudaSuccess ? MHA_OK : record_cuda_failure(what, cudaGetErrorName(e));
}

// A checked form.
struct Form {
    bool capped = false;
    int bias = kBiasNone;
    ScoreParams f{};
    BucketParams bk{};
    const int32_t *prefix_lens = nullptr, *doc_ids = nullptr;
    size_t vec_bytes(int h) const {
        return bias == kBiasBuckets ? round256(static_cast<size_t>(h) * vec_stride(f.mid) * 4) : 0;
    }
};

// Sizes only (no pointer of the form is needed): what a workspace depends on.
bool form_sizes(const mha_score_form *form, Form &out) {
    if (!form) return true;
    if (form->num_buckets < 0 || form->num_buckets > kMaxBuckets) return false;
    if (form->num_buckets > 0) {
        if (!form->bucket_starts) return false;
        out.bias = kBiasBuckets;
        out.bk.num = form->num_buckets;
        out.bk.both = form->bidirectional ? 1 : 0;
        for (int i = 0; i < form->num_buckets; ++i) {
            const int32_t s = form->bucket_starts[i];
            if (i == 0 ? s != 0 : s <= form->bucket_starts[i - 1]) return false;
            out.bk.starts[i] = s;
        }
        out.f.far = std::max(out.bk.starts[form->num_buckets - 1], 1);
        if (out.f.far > kMaxFar) return false;
        out.f.mid = vec_mid(out.f.far);
    }
    return true;
}

mha_status check_form(const mha_score_form *form, float scale, int mask, bool decode, int T_q, int T_k, Form &out) {
    if (!isfinite(scale)) return MHA_ERR_INVALID_ARG;
    if (mask < MHA_MASK_NONE || mask > MHA_MASK_CAUSAL_KEY_PADDING) return MHA_ERR_INVALID_ARG;
    const mha_score_form none{};
    if (!form) form = &none;
    if (!(form->cap >= 0.f && form->cap <= kMostCap) || (form->cap > 0.f && form->cap < kLeastCap)) return MHA_ERR_INVALID_ARG;
    if (form->num_buckets < 0 || (form->table != nullptr) != (form->num_buckets > 0)) return MHA_ERR_INVALID_ARG;
    if (form->slopes && form->table) return MHA_ERR_INVALID_ARG;
    if (form->num_buckets > kMaxBuckets) return MHA_ERR_UNSUPPORTED;
    if (form->num_buckets > 0) {
        if (!form->bucket_starts || form->bucket_starts[0] != 0) return MHA_ERR_INVALID_ARG;
        for (int i = 1; i < form->num_buckets; ++i)
            if (form->bucket_starts[i] <= form->bucket_starts[i - 1]) return MHA_ERR_INVALID_ARG;
        if (form->bucket_starts[form->num_buckets - 1] > kMaxFar) return MHA_ERR_UNSUPPORTED;
    }
    if (decode ? (form->prefix_lens || form->doc_ids)
               : ((form->prefix_lens && !(mask & MHA_MASK_CAUSAL)) || (form->doc_ids && T_q != T_k)))
        return MHA_ERR_INVALID_ARG;
    if (!form_sizes(form, out)) return MHA_ERR_INVALID_ARG;
    out.capped = form->cap > 0.f;
    if (form->slopes) out.bias = kBiasSlopes;
    constexpr float kLog2e = 1.4426950408889634f;
    out.f.cap_in = out.capped ? scale / form->cap : 0.f;
    out.f.mul = out.capped ? form->cap * kLog2e : scale * kLog2e;
    out.f.lin = scale * kLog2e;
    if (!isfinite(out.f.cap_in) || !isfinite(out.f.mul) || !isfinite(out.f.lin)) return MHA_ERR_INVALID_ARG;
    if (out.capped) {
        // fits of tanh(x) / x in x^2 over [0, 0.5^2] and [0, 1.7^2] (scores.cuh)
        constexpr double kNear[3] = {0.999978295, -0.331718863, 0.115318969};
        constexpr double kWide[7] = {0.999964321,  -0.332565284,   0.129537331,   -0.0458991416,
                                     0.0125609041, -0.00216785714, 0.000168549304};
        // ... and their errors, those of x p(x^2) against tanh(x): near's in
        // parts of x, wide's absolute; times the cap they are a score's.
        constexpr double kNearError = 2.2e-5, kWideError = 9.1e-6;
        const double near_x = std::min(0.5, kCapError / (kNearError * form->cap));
        const double wide_x = kWideError * form->cap <= kCapError ? 1.7 : 0.0;
        // In s = x / cap_in, with the factor mul; usable where every coefficient
        // and the squares stay within fp32's normal range.
        const double a = out.f.cap_in;
        auto in_scores = [&](const double *k, int n, double most_x, float *to) -> float {
            bool fine = a != 0.0;
            double pow = out.f.mul * a;
            for (int i = 0; i < n; ++i, pow *= a * a) {
                to[i] = static_cast<float>(k[i] * pow);
                fine = fine && fabs(k[i] * pow) > 1e-36 && fabs(k[i] * pow) < 1e36;
            }
            const double most = most_x * most_x / (a * a);
            if (fine && most > 1e-18 && most < 1e18) return static_cast<float>(most);
            std::fill(to, to + n, 0.f);  // scores of 0 alone
            return 0.f;
        };
        out.f.near_max = in_scores(kNear, 3, near_x, out.f.near);
        out.f.wide_max = in_scores(kWide, 7, wide_x, out.f.wide);
    }
    // A masked score is u = -inf before the multiplication by mul: with scale
    // 0 a factor that makes every other product vanish beside 1 keeps it so.
    if (out.f.mul == 0.f) out.f.mul = 1e-37f;
    // The capped forward masks after its scores are multiplied: mul > 0 there.
    out.f.masked = out.f.mul < 0.f ? INFINITY : -INFINITY;
    out.f.slopes = form->slopes;
    out.bk.table = static_cast<const __nv_bfloat16 *>(form->table);
    out.f.past_only = (mask & MHA_MASK_CAUSAL) && !form->prefix_lens && !decode;
    out.prefix_lens = form->prefix_lens;
    out.doc_ids = form->doc_ids;
    return MHA_OK;
}

mha_status check_sizes(mha_dtype dt, int B, int h, int h_kv, int T_q, int T_k, int d_k, int d_v) {
    if (B < 0 || h < 0 || h_kv < 0 || T_q < 0 || T_k < 0 || d_k <= 0 || d_v <= 0) return MHA_ERR_INVALID_ARG;
    if (dt != MHA_BF16) return dt == MHA_F32 ? MHA_ERR_UNSUPPORTED : MHA_ERR_INVALID_ARG;
    if (h > 0 && (h_kv == 0 || h % h_kv != 0)) return MHA_ERR_INVALID_ARG;
    if (d_k != 64 || d_v != 64) return MHA_ERR_UNSUPPORTED;
    if (h > 65535 || static_cast<long long>(B) * h >= (1ll << 31)) return MHA_ERR_UNSUPPORTED;
    if (T_q >= kMaxLength || T_k >= kMaxLength || (T_k + 127) / 128 > 65535) return MHA_ERR_UNSUPPORTED;
    if (static_cast<long long>(B) * h * ((T_q + 127) / 128) >= (1ll << 30)) return MHA_ERR_UNSUPPORTED;
    return MHA_OK;
}

// Scratch of the preparing launch, at the start of every workspace.
struct Prep {
    size_t vec, docs, end;
};
Prep prep_layout(const Form &f, bool docs, int B, int h, int T) {
    Prep p;
    p.vec = 0;
    p.docs = f.vec_bytes(h);
    p.end = p.docs + (docs ? round256(static_cast<size_t>(B) * T * 8) : 0);
    return p;
}

// Runs the preparing launch if the form needs one and fills in what it writes.
mha_status prepare(const Form &f, const Prep &lay, void *workspace, int B, int h, int T, ScoreParams &sp, VisParams &vis,
                   cudaStream_t stream) {
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    float *vec = f.bias == kBiasBuckets ? reinterpret_cast<float *>(ws + lay.vec) : nullptr;
    int2 *docs = f.doc_ids ? reinterpret_cast<int2 *>(ws + lay.docs) : nullptr;
    sp = f.f;
    sp.vec = vec;
    vis.doc_range = docs;
    vis.prefix_lens = f.prefix_lens;
    return launched(launch_scored_prep(vec, f.f.far, h, f.bk, docs, f.doc_ids, B, T, stream), "scored attention preparation");
}

struct BwdLayout {
    Prep prep;
    size_t next, dq, nlse2, dvec, idx, buckets, part_dk, part_dv, end;
    int splits, near_blocks;
};
BwdLayout bwd_layout(const Form &f, bool docs, int B, int h, int h_kv, int T_q, int T_k) {
    BwdLayout l{};
    l.prep = prep_layout(f, docs, B, h, T_k);
    const size_t BH = static_cast<size_t>(B) * h;
    const int n_qb = (T_q + 127) / 128, n_kb = (T_k + 127) / 128;
    const size_t rows = BH * n_qb * 128;
    l.next = l.prep.end;
    l.dq = l.next + 256;
    l.nlse2 = l.dq + round256(rows * 256);
    l.dvec = l.nlse2 + round256(rows * 4);
    l.idx = l.dvec + round256(rows * 4);
    l.buckets = l.idx + (f.bias == kBiasBuckets ? round256(vec_stride(f.f.mid)) : 0);
    l.part_dk = l.buckets;
    l.splits = 1;
    if (f.bias == kBiasBuckets) {
        // block pairs with |key - query| < far for some pair
        l.near_blocks = std::min((f.f.far + 126) / 128, std::max(n_qb, n_kb));
        l.part_dk += round256(BH * n_kb * f.bk.num * (f.bk.both ? 2 : 1) * 4);
    }
    if (h_kv > 0 && T_q > 0) {
        // CTAs share a K/V head's query heads until there are about three for
        // every SM (blocks of a causal mask differ in length), or one per head
        const long long ctas = static_cast<long long>(B) * h_kv * n_kb;
        const int group = h / h_kv;
        while (l.splits < group && ctas * l.splits < 3 * kSmsPerGpu) ++l.splits;
        const int per = (group + l.splits - 1) / l.splits;
        l.splits = (group + per - 1) / per;
    }
    const size_t part = l.splits > 1 ? round256(static_cast<size_t>(l.splits) * B * h_kv * T_k * 256) : 0;
    l.part_dv = l.part_dk + part;
    l.end = l.part_dv + part;
    return l;
}

// Division of a decoding step's keys into ranges of `tiles` 128-key tiles each:
// an item (a range of the prefix for 128 stacked rows, or of one cache) costs
// its tiles and about three more (query rows, pipeline start, partial sums).
// Few items go in whole rounds over the SMs, many even out.
struct Splits {
    int row_tiles, prefix, cache, tiles;
    size_t parts() const { return static_cast<size_t>(prefix) + cache; }
};
Splits decode_splits(int B, int h, int h_kv, int T_q, int T_p, int T_k) {
    Splits s{};
    if (h <= 0 || B <= 0 || T_q <= 0) return s;
    const DecodeRows dr = decode_rows(h / h_kv * T_q);
    s.row_tiles = dr.chunks > 1 ? B * dr.chunks : (B + dr.nb - 1) / dr.nb;
    const long long np = static_cast<long long>(h_kv) * s.row_tiles, nc = static_cast<long long>(h_kv) * B * dr.chunks;
    const bool single = h / h_kv * T_q == 1;  // the caches are launch_decode_row's
    const int tp = (T_p + 127) / 128, tc = single ? 0 : (T_k + 127) / 128;
    long long best = -1;
    for (int n = 2; n <= 32; ++n) {
        const int prefix = (tp + n - 1) / n, cache = (tc + n - 1) / n;
        const long long items = np * prefix + nc * cache;
        long long cost = np * (tp + 3 * prefix) + nc * (tc + 3 * cache);  // all items', in tiles
        if (items <= 4 * kSmsPerGpu)
            cost = (items + kSmsPerGpu - 1) / kSmsPerGpu * (n + 3) * kSmsPerGpu;
        else
            cost += static_cast<long long>(n) * kSmsPerGpu / 2;
        if (best < 0 || cost < best) {
            best = cost;
            s.prefix = prefix;
            s.cache = cache;
            s.tiles = n;
        }
    }
    return s;
}

}  // namespace

MHA_EXPORT size_t sdpa_scored_workspace_bytes(int B, int h, int T_q, int T_k, const mha_score_form *form) {
    Form f;
    if (B < 0 || h < 0 || T_q < 0 || T_k < 0 || !form_sizes(form, f)) return 0;
    return prep_layout(f, form && form->doc_ids, B, h, T_k).end;
}

MHA_EXPORT mha_status sdpa_scored_forward(mha_dtype dt, const void *q, const void *k, const void *v, void *o, float *lse,
                                          void *o_lo, void *workspace, size_t workspace_bytes, int B, int h, int h_kv, int T_q,
                                          int T_k, int d_k, int d_v, float scale, mha_mask mask,
                                          const int32_t *key_lens, const mha_score_form *form, int *status_dev,
                                          cudaStream_t stream) {
    Form f;
    mha_status s = check_sizes(dt, B, h, h_kv, T_q, T_k, d_k, d_v);
    if (s != MHA_OK) return s;
    if ((s = check_form(form, scale, mask, false, T_q, T_k, f)) != MHA_OK) return s;
    if ((mask & MHA_MASK_KEY_PADDING) && !key_lens) return MHA_ERR_INVALID_ARG;
    if (o_lo && !lse && B > 0 && h > 0 && T_q > 0) return MHA_ERR_INVALID_ARG;
    if (B == 0 || h == 0 || T_q == 0) return MHA_OK;
    if (!q || !o || (T_k > 0 && (!k || !v))) return MHA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(o) || !aligned16(o_lo) || (T_k > 0 && (!aligned16(k) || !aligned16(v)))) return MHA_ERR_MISALIGNED;
    const Prep lay = prep_layout(f, f.doc_ids != nullptr, B, h, T_k);
    if (lay.end > 0 && (!workspace || workspace_bytes < lay.end)) return MHA_ERR_WORKSPACE;
    if (lay.end > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return MHA_ERR_MISALIGNED;

    // T_k == 0: a one-row tensor that the kernel never loads
    const int Tk_map = T_k > 0 ? T_k : 1;
    ScoredMaps maps;
    if ((s = encode_heads_map(&maps.q, q, static_cast<long long>(B) * h, T_q)) != MHA_OK) return s;
    if ((s = encode_heads_map(&maps.k, T_k > 0 ? k : q, static_cast<long long>(B) * h_kv, Tk_map)) != MHA_OK) return s;
    if ((s = encode_heads_map(&maps.v, T_k > 0 ? v : q, static_cast<long long>(B) * h_kv, Tk_map)) != MHA_OK) return s;
    maps.q_cache = maps.k_cache = maps.v_cache = maps.q;
    ScoredFwdParams p{};
    if ((s = prepare(f, lay, workspace, B, h, T_k, p.f, p.vis, stream)) != MHA_OK) return s;
    p.B = B;
    p.H = h;
    p.Hkv = h_kv;
    p.Tq = T_q;
    p.Tk = T_k;
    p.vis.causal = (mask & MHA_MASK_CAUSAL) ? 1 : 0;
    p.vis.key_lens = (mask & MHA_MASK_KEY_PADDING) ? key_lens : nullptr;
    p.o = static_cast<__nv_bfloat16 *>(o);
    p.lse = lse;
    p.o_lo = static_cast<__nv_bfloat16 *>(o_lo);
    p.num_qblocks = (T_q + 127) / 128;
    p.total_items = B * h * p.num_qblocks;
    p.status = status_dev;
    return launched(launch_attn_scored(maps, f.capped, f.bias, p, stream), "scored attention launch");
}

MHA_EXPORT size_t sdpa_scored_backward_workspace_bytes(int B, int h, int h_kv, int T_q, int T_k,
                                                       const mha_score_form *form) {
    Form f;
    if (B < 0 || h < 0 || h_kv < 0 || T_q < 0 || T_k < 0 || !form_sizes(form, f)) return 0;
    if (h > 0 && (h_kv == 0 || h % h_kv != 0)) return 0;
    return bwd_layout(f, form && form->doc_ids, B, h, h_kv, T_q, T_k).end;
}

MHA_EXPORT mha_status sdpa_scored_backward(mha_dtype dt, const void *q, const void *k, const void *v, const void *o,
                                           const void *o_lo, const void *dout, const float *lse, void *dq, void *dk, void *dv, void *dtable,
                                           void *workspace, size_t workspace_bytes, int B, int h, int h_kv, int T_q,
                                           int T_k, int d_k, int d_v, float scale, mha_mask mask,
                                           const int32_t *key_lens, const mha_score_form *form, int *status_dev,
                                           cudaStream_t stream) {
    Form f;
    mha_status s = check_sizes(dt, B, h, h_kv, T_q, T_k, d_k, d_v);
    if (s != MHA_OK) return s;
    if ((s = check_form(form, scale, mask, false, T_q, T_k, f)) != MHA_OK) return s;
    if ((mask & MHA_MASK_KEY_PADDING) && !key_lens) return MHA_ERR_INVALID_ARG;
    if (dtable && f.bias != kBiasBuckets) return MHA_ERR_INVALID_ARG;
    const long long BH = static_cast<long long>(B) * h;
    if (h == 0 || (BH == 0 && !dtable) || (T_q == 0 && T_k == 0 && !dtable)) return MHA_OK;
    if (BH > 0 && ((T_q > 0 && (!q || !o || !dout || !lse || !dq)) || (T_k > 0 && (!k || !v || !dk || !dv))))
        return MHA_ERR_INVALID_ARG;
    const BwdLayout lay = bwd_layout(f, f.doc_ids != nullptr, B, h, h_kv, T_q, T_k);
    if (lay.end > 0 && (!workspace || workspace_bytes < lay.end)) return MHA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return MHA_ERR_MISALIGNED;
    if (BH > 0 && ((T_q > 0 && (!aligned16(q) || !aligned16(o) || !aligned16(o_lo) || !aligned16(dout) || !aligned16(dq))) ||
                   (T_k > 0 && (!aligned16(k) || !aligned16(v) || !aligned16(dk) || !aligned16(dv)))))
        return MHA_ERR_MISALIGNED;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    ScoredBwdParams p{};
    p.B = B;
    p.H = h;
    p.Hkv = h_kv;
    p.Tq = T_q;
    p.Tk = T_k;
    p.Tq_pad = (T_q + 127) / 128 * 128;
    p.scale = scale;
    p.f = f.f;
    p.bk = f.bk;
    p.vis.causal = (mask & MHA_MASK_CAUSAL) ? 1 : 0;
    p.vis.key_lens = (mask & MHA_MASK_KEY_PADDING) ? key_lens : nullptr;
    p.vis.prefix_lens = f.prefix_lens;
    p.dq_acc = reinterpret_cast<float *>(ws + lay.dq);
    p.dk = static_cast<__nv_bfloat16 *>(dk);
    p.dv = static_cast<__nv_bfloat16 *>(dv);
    p.splits = lay.splits;
    p.part_dk = reinterpret_cast<float *>(ws + lay.part_dk);
    p.part_dv = reinterpret_cast<float *>(ws + lay.part_dv);
    p.next_item = reinterpret_cast<unsigned *>(ws + lay.next);
    const long long items = static_cast<long long>(B) * h_kv * lay.splits * ((T_k + 127) / 128);
    if (items >= (1ll << 31)) return MHA_ERR_UNSUPPORTED;
    p.total_items = static_cast<unsigned>(items);
    p.near_blocks = lay.near_blocks;
    if (dtable) p.bucket_part = reinterpret_cast<float *>(ws + lay.buckets);
    p.status = status_dev;
    if (BH > 0 && (T_q > 0 || T_k > 0)) {
        // an empty side is described by a one-row tensor that is never loaded
        const void *q_src = T_q > 0 ? q : k, *g_src = T_q > 0 ? dout : k;
        const void *k_src = T_k > 0 ? k : q, *v_src = T_k > 0 ? v : q;
        const long long BHk = static_cast<long long>(B) * h_kv;
        CUtensorMap tq, tk, tv, tg;
        if ((s = encode_heads_map(&tq, q_src, T_q > 0 ? BH : BHk, T_q > 0 ? T_q : 1)) != MHA_OK) return s;
        if ((s = encode_heads_map(&tg, g_src, T_q > 0 ? BH : BHk, T_q > 0 ? T_q : 1)) != MHA_OK) return s;
        if ((s = encode_heads_map(&tk, k_src, BHk, T_k > 0 ? T_k : 1)) != MHA_OK) return s;
        if ((s = encode_heads_map(&tv, v_src, BHk, T_k > 0 ? T_k : 1)) != MHA_OK) return s;
        float *vec = f.bias == kBiasBuckets ? reinterpret_cast<float *>(ws + lay.prep.vec) : nullptr;
        uint8_t *idx = vec ? ws + lay.idx : nullptr;
        int2 *docs = f.doc_ids ? reinterpret_cast<int2 *>(ws + lay.prep.docs) : nullptr;
        float *nlse2 = reinterpret_cast<float *>(ws + lay.nlse2), *dvec = reinterpret_cast<float *>(ws + lay.dvec);
        p.f.vec = vec;
        p.f.idx = idx;
        p.vis.doc_range = docs;
        p.nlse2 = nlse2;
        p.dvec = dvec;
        if ((s = launched(launch_scored_bwd_pre(static_cast<const __nv_bfloat16 *>(o), static_cast<const __nv_bfloat16 *>(o_lo),
                                                static_cast<const __nv_bfloat16 *>(dout), lse, nlse2, dvec, p, vec, idx, docs,
                                                f.doc_ids, stream),
                          "scored attention backward, row terms")) != MHA_OK)
            return s;
        if (T_k > 0 && (s = launched(launch_attn_scored_bwd(tq, tk, tv, tg, f.capped, f.bias, p, stream),
                                     "scored attention backward launch")) != MHA_OK)
            return s;
    }
    return launched(launch_scored_bwd_post(p, static_cast<__nv_bfloat16 *>(dq), static_cast<__nv_bfloat16 *>(dtable), stream),
                    "scored attention backward, conversion");
}

MHA_EXPORT size_t sdpa_decode_shared_workspace_bytes(int B, int h, int h_kv, int T_q, int T_p, int T_k,
                                                     const mha_score_form *form) {
    Form f;
    if (B < 0 || h < 0 || h_kv < 0 || T_q < 0 || T_p < 0 || T_k < 0 || !form_sizes(form, f)) return 0;
    if (h > 0 && (h_kv == 0 || h % h_kv != 0)) return 0;
    const size_t rows = static_cast<size_t>(B) * h * T_q;
    const size_t parts = decode_splits(B, h, h_kv, T_q, T_p, T_k).parts();
    return f.vec_bytes(h) + round256(parts * rows * 256) + round256(parts * rows * 8);
}

MHA_EXPORT mha_status sdpa_decode_shared_forward(const void *q, const void *k_prefix, const void *v_prefix,
                                                 const void *k_cache, const void *v_cache, void *o, void *workspace,
                                                 size_t workspace_bytes, int B, int h, int h_kv, int T_q, int T_p, int T_k,
                                                 int d_k, int d_v, float scale, mha_mask mask, const int32_t *cache_lens,
                                                 const mha_score_form *form, int *status_dev, cudaStream_t stream) {
    Form f;
    mha_status s = check_sizes(MHA_BF16, B, h, h_kv, T_q, T_k, d_k, d_v);
    if (s != MHA_OK) return s;
    if (T_p < 0) return MHA_ERR_INVALID_ARG;
    if (T_q > kDecodeMaxRows) return MHA_ERR_UNSUPPORTED;
    if (static_cast<long long>(T_p) + T_k >= kMaxLength) return MHA_ERR_UNSUPPORTED;
    if ((s = check_form(form, scale, mask, true, T_q, T_k, f)) != MHA_OK) return s;
    if ((mask & MHA_MASK_KEY_PADDING) && !cache_lens) return MHA_ERR_INVALID_ARG;
    if (B == 0 || h == 0 || T_q == 0) return MHA_OK;
    if (!q || !o || (T_k > 0 && (!k_cache || !v_cache)) || (T_p > 0 && (!k_prefix || !v_prefix))) return MHA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(o) || (T_k > 0 && (!aligned16(k_cache) || !aligned16(v_cache))) ||
        (T_p > 0 && (!aligned16(k_prefix) || !aligned16(v_prefix))))
        return MHA_ERR_MISALIGNED;
    const int rows = h / h_kv * T_q;
    const size_t n_rows = static_cast<size_t>(B) * h * T_q;
    const DecodeRows dr = decode_rows(rows);
    const Splits sp = decode_splits(B, h, h_kv, T_q, T_p, T_k);
    const long long items = static_cast<long long>(h_kv) * sp.row_tiles * sp.prefix +
                            static_cast<long long>(h_kv) * B * dr.chunks * sp.cache;
    if (items >= (1ll << 30) || n_rows >= (1ull << 28)) return MHA_ERR_UNSUPPORTED;
    const size_t at_o = f.vec_bytes(h), at_ml = at_o + round256(sp.parts() * n_rows * 256);
    const size_t need = at_ml + round256(sp.parts() * n_rows * 8);
    if (need > 0 && (!workspace || workspace_bytes < need)) return MHA_ERR_WORKSPACE;
    if (need > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return MHA_ERR_MISALIGNED;
    uint8_t *ws = static_cast<uint8_t *>(workspace);

    // an empty side is described by a one-row tensor that is never loaded
    ScoredMaps maps;
    DecodeRows one = dr;
    one.nb = 1;
    if ((s = encode_stacked_rows_map(&maps.q, q, B, h_kv, rows, dr)) != MHA_OK) return s;
    if ((s = encode_stacked_rows_map(&maps.q_cache, q, B, h_kv, rows, one)) != MHA_OK) return s;
    if ((s = encode_heads_map(&maps.k, T_p > 0 ? k_prefix : q, T_p > 0 ? h_kv : 1, std::max(T_p, 1))) != MHA_OK) return s;
    if ((s = encode_heads_map(&maps.v, T_p > 0 ? v_prefix : q, T_p > 0 ? h_kv : 1, std::max(T_p, 1))) != MHA_OK) return s;
    const long long BHk = T_k > 0 ? static_cast<long long>(B) * h_kv : 1;
    if ((s = encode_heads_map(&maps.k_cache, T_k > 0 ? k_cache : q, BHk, std::max(T_k, 1))) != MHA_OK) return s;
    if ((s = encode_heads_map(&maps.v_cache, T_k > 0 ? v_cache : q, BHk, std::max(T_k, 1))) != MHA_OK) return s;
    ScoredFwdParams p{};
    if ((s = prepare(f, prep_layout(f, false, B, h, 0), workspace, B, h, 0, p.f, p.vis, stream)) != MHA_OK)
        return s;
    p.B = B;
    p.H = h;
    p.Hkv = h_kv;
    p.Tq = T_q;
    p.Tk = T_p;
    p.vis.causal = (mask & MHA_MASK_CAUSAL) ? 1 : 0;
    p.total_items = static_cast<int>(items);
    p.status = status_dev;
    p.cache_lens = cache_lens;
    p.cache_cap = T_k;
    p.splits = sp.prefix;
    p.cache_splits = sp.cache;
    p.split_tiles = sp.tiles;
    p.row_tiles = sp.row_tiles;
    p.part_o = reinterpret_cast<float *>(ws + at_o);
    p.part_ml = reinterpret_cast<float2 *>(ws + at_ml);
    if ((s = launched(launch_attn_scored(maps, f.capped, f.bias, p, stream), "shared prefix decoding launch")) !=
        MHA_OK)
        return s;
    if (rows == 1) {
        DecodeRowParams d{};
        d.B = B;
        d.H = h;
        d.Tk = T_k;
        d.capped = f.capped ? 1 : 0;
        d.f = p.f;
        d.cache_lens = cache_lens;
        d.q = static_cast<const __nv_bfloat16 *>(q);
        d.k = static_cast<const __nv_bfloat16 *>(k_cache);
        d.v = static_cast<const __nv_bfloat16 *>(v_cache);
        d.o = static_cast<__nv_bfloat16 *>(o);
        d.prefix_splits = sp.prefix;
        d.part_o = p.part_o;
        d.part_ml = p.part_ml;
        return launched(launch_decode_row(d, f.bias, stream), "shared prefix decoding, caches and merge");
    }
    return launched(launch_decode_merge(p.part_o, p.part_ml, static_cast<__nv_bfloat16 *>(o), static_cast<int>(sp.parts()),
                                        static_cast<long long>(n_rows), stream),
                    "shared prefix decoding, merge");
}
