// kernels.h -- launch interfaces between the C ABI (api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mha.h"

namespace mha {

constexpr int kMaskCausalBit = 1;
constexpr int kMaskPaddingBit = 2;

// ------------------------------------------------ launch helper
// Launches `kernel` on `stream`.  With pdl the launch may begin while the
// kernel before it on the stream finishes (programmatic dependent launch);
// every kernel launched that way waits for its predecessor (pdl_wait) after
// its prologue and before it touches global memory.  Optional cluster size.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_kernel(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                 cudaStream_t stream, bool pdl, unsigned cluster, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ------------------------------------------------ fused bf16 attention
struct AttnParams {
    int B, H, Tq, Tk;
    float scale_log2;  // scale * log2(e): scores are exponentiated with ex2
    float scale;
    float *lse;        // optional (B, H, Tq) fp32: log sum_j exp(scale q.k_j); null: not written
    int mask;          // kMaskCausalBit | kMaskPaddingBit
    const int32_t *key_lens;
    __nv_bfloat16 *o;  // output; element (b, h, t, c) at o + b*sb + h*sh + t*st + c
    long long o_stride_b, o_stride_h, o_stride_t;
    int num_qblocks;   // ceil(Tq / rows per item)
    int total_items;   // B * H * num_qblocks work items (query tiles)
    int *status;
    // Failure-detection drill only (both 0 on every product path): the wait
    // limit in ns (0: the default 1 s), and n > 0 makes every CTA's loader
    // issue no copy for its (n-1)-th key tile, so the waits on it run out.
    unsigned long long wait_limit_ns;
    int drill_skip_tile;
};
constexpr int kAttnRowsPerCta = 128;  // one work item = one 128-row query tile
constexpr int kAttnHeadDim = 64;

// The kernel's two softmax groups split a row's keys either into the two
// 64-key halves of every tile or into alternate tiles; alternate tiles keep
// the groups out of lockstep and pay once a query tile has, on average,
// kAttnTilesSplitMin key tiles or more (measured on GB300: +3 % at causal
// T = 8192), while short items finish sooner by halves.
constexpr int kAttnTilesSplitMin = 8;
bool attn_bf16_splits_by_tiles(int Tq, int Tk, int mask);

// q, k, v: head-split (B, H, T, 64) bf16 tensors described by 3-D TMA maps
// over (64, T, B*H) with 128-byte swizzling and 128-row boxes.
cudaError_t launch_attn_bf16(const CUtensorMap &tq, const CUtensorMap &tk,
                             const CUtensorMap &tv, const AttnParams &p, cudaStream_t stream,
                             bool pdl = false);

// ------------------------------------------------ bf16 decode attention
constexpr int kDecodeMaxRows = 8;  // query rows per (b, h) in one decode call
struct DecodeParams {
    int B, H, Tq, Tk;
    float scale_log2;          // scale * log2(e)
    const int32_t *key_lens;   // cached keys per batch entry; null: all Tk
};
// q (B, H, Tq, 64), k and v (B, H, Tk, 64), o (B, H, Tq, 64), all bf16 and
// contiguous; Tq <= kDecodeMaxRows.
cudaError_t launch_decode_bf16(const __nv_bfloat16 *q, const __nv_bfloat16 *k,
                               const __nv_bfloat16 *v, __nv_bfloat16 *o, const DecodeParams &p,
                               cudaStream_t stream);

// ------------------------------------------------ bf16 attention backward
struct BwdParams {
    int B, H, Tq, Tk, Tq_pad;   // Tq_pad: Tq rounded up to whole 128-row blocks
    float scale, scale_log2;
    int mask;
    const int32_t *key_lens;
    const float *nlse2;         // (B, H, Tq_pad) -lse * log2(e), -inf for padded / empty rows
    const float *dvec;          // (B, H, Tq_pad) rowsum(dO * O)
    float *dq_acc;              // (B, H, Tq_pad, 64) fp32
    __nv_bfloat16 *dk, *dv;     // (B, H, Tk, 64)
    int *status;
};
// Bytes of workspace the backward needs (fp32 dQ accumulator, lse, D).
size_t bwd_workspace_bytes(long long BH, int Tq);
// q, k, v, dout: 3-D TMA maps like the forward's; o, dout, lse as device
// arrays; fills dq (bf16), p.dk, p.dv.  `workspace`: bwd_workspace_bytes(),
// 256-byte aligned.
cudaError_t launch_attn_bwd_bf16(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                                 const CUtensorMap &tg, const __nv_bfloat16 *o,
                                 const __nv_bfloat16 *dout, const float *lse, __nv_bfloat16 *dq,
                                 BwdParams p, void *workspace, cudaStream_t stream);

// ------------------------------------------------ scored attention
// Scores beyond scale q.k (see scores.cuh): what the kernels need of them.
enum BiasKind { kBiasNone = 0, kBiasSlopes = 1, kBiasBuckets = 2 };
struct ScoreParams {
    float cap_in;         // scale / cap (capped scores), else unused
    float mul;            // y = u mul + bias, u = q.k or tanh(q.k cap_in), y in log2 units; never 0
    // Capped scores with |q.k cap_in| <= 0.5: y = s (near[0] + near[1] s^2 +
    // near[2] s^4), s = q.k; s^2 <= near_max (less than that of 0.5 where the
    // fit's error would show; 0: unused, all coefficients 0).  With
    // |q.k cap_in| <= 1.7: the same of wide, s^2 <= wide_max.
    float near[3], near_max;
    float wide[7], wide_max;
    float masked;         // the u of a masked score: minus infinity times the sign of mul
    // scale in log2 units: a capped score's y far below the cap is s lin, s = q.k.
    // (Behind the others: ahead of them it moved the coefficients off their
    // 8-byte pairs, and capped slopes took 484 us instead of 470.)
    float lin;
    const float *slopes;  // (H) fp32, kBiasSlopes
    // kBiasBuckets, written by the preparing launch for distances -mid .. mid:
    const float *vec;     // (H, vec_stride(mid)) the bias, in log2 units
    const uint8_t *idx;   // (vec_stride(mid)) the bucket (backward only)
    int far, mid;         // distances from `far` on share the last bucket; mid = vec_mid(far)
    int past_only;        // no visible key lies past its query (causal mask without prefixes)
};
// Which keys a query sees.
struct VisParams {
    int causal;
    const int32_t *key_lens;     // (B) or null
    const int32_t *prefix_lens;  // (B) or null: keys every query sees in spite of the causal mask
    const int2 *doc_range;       // (B, T) or null: first position of a position's document, and past its last
};

// The expanded bias of a head: distances -mid .. mid and padding, so that the
// 256 distances of a 128 x 128 block pair with one below `far`, from a multiple
// of 128 on, are inside and 16-byte aligned.
inline __host__ __device__ int vec_mid(int far) { return (far + 256 + 15) / 16 * 16; }
inline __host__ __device__ int vec_stride(int mid) { return 2 * mid + 16; }

constexpr int kMaxBuckets = 64;  // per direction
struct BucketParams {
    const __nv_bfloat16 *table;  // (num [* 2], H)
    int num, both;
    int32_t starts[kMaxBuckets];
};
// Writes vec and doc_range (each if not null) for one call.
cudaError_t launch_scored_prep(float *vec, int far, int H, const BucketParams &bk, int2 *doc_range,
                               const int32_t *doc_ids, int B, int T, cudaStream_t stream);

struct ScoredFwdParams {
    int B, H, Hkv, Tq, Tk;
    ScoreParams f;
    VisParams vis;
    __nv_bfloat16 *o;  // (B, H, Tq, 64)
    float *lse;        // optional (B, H, Tq)
    __nv_bfloat16 *o_lo;  // optional with lse, (B, H, Tq, 64): what rounding took from o
    int num_qblocks, total_items;
    int *status;
    // Decoding over a shared prefix (part_o not null): Tk keys of the prefix,
    // seen by a K/V head's query rows of all batch entries stacked, then each
    // batch entry's cache, seen by its own; every key range of split_tiles
    // 128-key tiles leaves unnormalised partial sums instead of an output.
    const int32_t *cache_lens;  // (B) or null: cache_cap rows everywhere
    int cache_cap;
    int splits, cache_splits;   // key ranges of the prefix and of a cache
    int split_tiles;
    int row_tiles;              // 128-row tiles per K/V head, all batch entries stacked
    float *part_o;              // (splits + cache_splits, B, H, Tq, 64)
    float2 *part_ml;            // (splits + cache_splits, B, H, Tq): reference in log2 units, sum
};
// q: (64, Tq, B H); k, v: (64, Tk, B Hkv); 128-row boxes, 128-byte swizzling.
// Decoding: q (64, g Tq, B, Hkv) in boxes of decode_rows(), k, v of the prefix
// (64, Tk, Hkv), q_cache in boxes of one batch entry, the caches (64, cap, B Hkv).
struct ScoredMaps {
    CUtensorMap q, k, v, q_cache, k_cache, v_cache;
};
cudaError_t launch_attn_scored(const ScoredMaps &maps, bool capped, int bias, const ScoredFwdParams &p,
                               cudaStream_t stream);

// How the g Tq query rows of a K/V head and batch entry are stacked into
// 128-row tiles: `per` rows of each of `nb` batch entries, `chunks` tiles per
// batch entry when they are more than 128.
struct DecodeRows {
    int per, nb, chunks;
};
inline __host__ __device__ DecodeRows decode_rows(int rows) {
    DecodeRows d;
    d.per = rows < 128 ? rows : 128;
    d.nb = 128 / d.per;
    d.chunks = (rows + 127) / 128;
    return d;
}

struct ScoredBwdParams {
    int B, H, Hkv, Tq, Tk, Tq_pad;
    float scale;
    ScoreParams f;
    VisParams vis;
    const float *nlse2, *dvec;  // as BwdParams
    float *dq_acc;
    __nv_bfloat16 *dk, *dv;     // (B, Hkv, Tk, 64)
    // CTAs that share a K/V head's query heads; more than one leave fp32 sums,
    // part_dk, part_dv (splits, B, Hkv, Tk, 64), instead of dk and dv
    int splits;
    float *part_dk, *part_dv;
    unsigned total_items;  // (key block, batch entry, K/V head, split)
    unsigned *next_item;   // the counter that items past the grid's come from, zeroed before
    // bucket bias gradient (bucket_part null: none): (B, H, key blocks, buckets);
    // block pairs up to near_blocks apart hold distances below the last bucket's
    float *bucket_part;
    int near_blocks;
    BucketParams bk;
    int *status;
};
// Before it: row terms of o (+ o_lo, may be null) and dout, a zeroed dq_acc,
// and what launch_scored_prep writes.  After it: dq, and dk, dv (splits > 1)
// and dtable (not null) from the partial sums.
cudaError_t launch_scored_bwd_pre(const __nv_bfloat16 *o, const __nv_bfloat16 *o_lo, const __nv_bfloat16 *dout,
                                  const float *lse, float *nlse2, float *dvec, const ScoredBwdParams &p, float *vec,
                                  uint8_t *idx, int2 *doc_range, const int32_t *doc_ids, cudaStream_t stream);
cudaError_t launch_scored_bwd_post(const ScoredBwdParams &p, __nv_bfloat16 *dq, __nv_bfloat16 *dtable,
                                   cudaStream_t stream);
cudaError_t launch_attn_scored_bwd(const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                                   const CUtensorMap &tg, bool capped, int bias, const ScoredBwdParams &p,
                                   cudaStream_t stream);

// ------------------------------------------------ decoding: partial sums to outputs
constexpr int kSmsPerGpu = 152;  // for the choice of key ranges, which fixes the workspace
// o[row] = sum_s w_s O_s / sum_s w_s l_s, w_s = 2^(m_s - max m), over `parts` key ranges.
cudaError_t launch_decode_merge(const float *part_o, const float2 *part_ml, __nv_bfloat16 *o, int parts, long long rows,
                                cudaStream_t stream);

// With one query row per K/V head and batch entry (H K/V heads, Tq = 1) the
// caches are gone through by this launch, which also merges the prefix's
// partial sums.
struct DecodeRowParams {
    int B, H, Tk;
    int capped;
    ScoreParams f;
    const int32_t *cache_lens;
    const __nv_bfloat16 *q, *k, *v;  // (B, H, 1, 64), (B, H, Tk, 64) twice
    __nv_bfloat16 *o;
    int prefix_splits;               // partial sums of the prefix
    const float *part_o;
    const float2 *part_ml;
};
cudaError_t launch_decode_row(const DecodeRowParams &p, int bias, cudaStream_t stream);

// ------------------------------------------------ positional encoding
// out (rows, D) = x + PE(pos0 + row % T); D % 8 == 0; x and out may alias.
cudaError_t launch_posenc_add_bf16(const __nv_bfloat16 *x, __nv_bfloat16 *out, long long rows, int T,
                                   int D, int pos0, cudaStream_t stream);

// ------------------------------------------------ fp32 SIMT attention
constexpr int kF32RowsPerCta = 8;  // query rows per CTA (one warp each)
cudaError_t launch_sdpa_f32(const float *q, const float *k, const float *v, float *o, int B,
                            int H, int Tq, int Tk, int dk, int dv, float scale, int mask,
                            const int32_t *key_lens, cudaStream_t stream);

// ------------------------------------------------ bf16 projection GEMM
constexpr int kGemmMaxProblems = 3;
enum GemmOutMode { kOutRowMajor = 0, kOutHeadSplit = 1 };
struct GemmProblem {
    int M, N, K;
    int tiles_n, tile_start, tile_count;
    __nv_bfloat16 *out;
    int out_mode;  // kOutRowMajor: out (M, N); kOutHeadSplit: row m = b*T + t,
                   // column n = head*64 + c -> out ((b*H + head)*T + t)*64 + c
    int T, H;
    const __nv_bfloat16 *bias;  // optional (N): added to every row
    int relu;                   // nonzero: max(0, .) after the bias
    int tma_store;              // nonzero: the output goes out through its TMA map (y below)
};
struct GemmParams {
    int num_problems;
    int total_tiles;
    int bn;  // output tile width: 128 or 256
    GemmProblem prob[kGemmMaxProblems];
    int *status;
};
constexpr int kGemmBM = 128, kGemmBK = 64;

// a[i]: 2-D TMA map over the activation (K inner, M rows), box (64, 128).
// b[i]: 3-D TMA map over the weight viewed as (64, K, N/64), box (64, 64, bn/64).
// y[i] (problems with tma_store): the output, 2-D (N inner, M rows) box (64, 128)
// for row-major, 3-D (64, T, B*H) box (64, 128, 1) for head-split with T a
// multiple of 128.
cudaError_t launch_gemm_bf16(const CUtensorMap (&a)[kGemmMaxProblems],
                             const CUtensorMap (&b)[kGemmMaxProblems],
                             const CUtensorMap (&y)[kGemmMaxProblems], const GemmParams &p,
                             cudaStream_t stream, bool pdl = false);

// Number of SMs of the current device.
cudaError_t sm_count(int *sms);

// Records "what: detail" as the calling thread's mha_last_error() text and
// returns MHA_ERR_CUDA.
mha_status record_cuda_failure(const char *what, const char *detail);

// Tensor maps: (BH, T, 64) heads in 128-row boxes; the query rows of decoding,
// (B, Hkv, rows, 64) in boxes of dr.per rows of dr.nb batch entries.
mha_status encode_heads_map(CUtensorMap *m, const void *base, long long BH, int T);
mha_status encode_stacked_rows_map(CUtensorMap *m, const void *base, int B, int Hkv, int rows, const DecodeRows &dr);

// ------------------------------------ output projection + residual + LayerNorm
constexpr int kLnMaxCluster = 8;  // CTAs per 128-row block (portable cluster size)
struct LnParams {
    int M, D, K;                  // out (M, D) = LN(resid + A (M, K) W (K, D) [+ bias])
    int bn;                       // columns per CTA: ln_tile_width(D)
    const __nv_bfloat16 *resid;   // (M, D)
    const __nv_bfloat16 *bias;    // optional (D): added to the product before the residual
    const __nv_bfloat16 *gamma;   // (D)
    const __nv_bfloat16 *beta;    // (D)
    float eps;
    __nv_bfloat16 *out;           // (M, D)
    int *status;
};
// 256 or 128 columns per CTA for rows of D features (D / width CTAs <= 8) over
// M rows on `sms` SMs, or 0 if D is not supported.
int ln_tile_width(int D, long long M, int sms);
// a: 2-D TMA map over A (K inner, M rows), box (64, 128); b: 3-D map over W
// viewed as (64, K, D/64), box (64, 64, bn/64); x, y: 2-D maps over the
// residual and the output (D inner, M rows), box (64, 128).
cudaError_t launch_gemm_ln_bf16(const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &x,
                                const CUtensorMap &y, const LnParams &p, cudaStream_t stream,
                                bool pdl = false);

}  // namespace mha
