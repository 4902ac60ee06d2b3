// scores.cuh -- the score definition shared by the scored attention kernels
// (forward, backward, decoding over a shared prefix):
//
//   z = scale q.k,   s = cap tanh(z / cap)  (or z),   s += bias_h(d),
//   d = key position - query position,
//   bias_h(d) = -slope_h |d|   or   table[bucket(d), h].
//
// Scores are kept in log2 units (y = s log2 e) because the weights are taken
// with 2^x.  The bucket bias is read from an expanded per-head row
// vec[d], d in [-mid, mid], mid >= far + 256, that a preparing launch writes
// once per call (already times log2 e): from |d| >= far on all distances
// share one bucket, so a run of keys that lies wholly past `far` needs one
// value, and any other run is read at d clamped per run, not per key.
#pragma once

#include "kernels.h"
#include "sm103_ptx.cuh"

namespace mha {

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint64_t f32x2_set(float v) { return f32x2_pack(v, v); }

// tanh(x) as x p(x^2), on the FMA pipe, two scores per operation, and nothing
// on the special-function unit, which the weights' 2^x need.  Three ranges, each
// a warp's choice by the largest score it holds; near and wide only as far as
// they take less than 6e-4 from a score (one step of a weight's bf16 is 3.9e-3
// to 7.8e-3 of it), which is near whole up to a cap of 54 and to scores of 27
// above, and wide up to a cap of 65:
//   near  |x| <= 0.5, p of degree 2, off by 2.2e-5 x at most (2.4e-5 of tanh x,
//         1.1e-5 of the cap).  The coefficients (ScoreParams.near) hold mul and
//         the powers of cap_in, so that y = s p(s^2) + bias is four packed
//         operations per pair of scores, three more than uncapped;
//   wide  |x| <= 1.7, degree 6, coefficients likewise (ScoreParams.wide), off by
//         8.8e-6 of the cap at most and by 3.6e-5 of a small score: eight
//         operations (degree 7, 2.2e-6 of the cap, with x made first took ten,
//         2 x 16 x 8,192 causal, cap 20: 730 us against 620);
//   any   cap_any, to fp32's own precision, two special-function operations per
//         score.
// (1 - tanh^2 of the backward is off by 1.0e-5 in near's range, 1.7e-5 in wide's.)

// p(s^2) of the wide range: s times it is mul tanh(s cap_in).
struct TanhWide {
    uint64_t c[7];
    __device__ __forceinline__ explicit TanhWide(const ScoreParams &f) {
#pragma unroll
        for (int i = 0; i < 7; ++i) c[i] = f32x2_set(f.wide[i]);
    }
    __device__ __forceinline__ uint64_t operator()(uint64_t w) const {
        uint64_t p = fma_f32x2(w, c[6], c[5]);
#pragma unroll
        for (int i = 4; i >= 0; --i) p = fma_f32x2(w, p, c[i]);
        return p;
    }
};

// mul tanh(x), x = s cap_in, for any s, to 2^-20 of itself: below |x| = 1/4 the
// Taylor series (its next term is 9e-9 there), taken from s so that large caps
// lose nothing; above, tanh(x) = 1 - 2 / (1 + e^(2x)), absolute error ~2^-22
// (e^(2x) overflowing to infinity gives 1, underflowing to 0 gives -1).
__device__ __forceinline__ float cap_any(float s, const ScoreParams &f) {
    const float x = s * f.cap_in, w = x * x;
    const float p = fmaf(w, fmaf(w, fmaf(w, fmaf(w, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f), 1.f);
    const float far = f.mul * (1.f - __fdividef(2.f, 1.f + ex2_approx(x * (2.f * kLog2E))));
    return w <= 0.0625f ? s * f.lin * p : far;
}

// s := mul tanh(s cap_in) of N scores in place.  wide (warp-uniform): no s^2 of
// the warp is past f.wide_max.
template <int N>
__device__ __forceinline__ void cap_scores(uint32_t (&s)[N], const ScoreParams &f, bool wide) {
    if (wide) {
        const TanhWide poly(f);
#pragma unroll
        for (int c = 0; c < N; c += 2) {
            const uint64_t x = f32x2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
            float t0, t1;
            f32x2_unpack(mul_f32x2(x, poly(mul_f32x2(x, x))), t0, t1);
            s[c] = __float_as_uint(t0);
            s[c + 1] = __float_as_uint(t1);
        }
    } else {
#pragma unroll
        for (int c = 0; c < N; ++c) s[c] = __float_as_uint(cap_any(__uint_as_float(s[c]), f));
    }
}

// Largest |s| of N values (NaN ignored).
template <int N>
__device__ __forceinline__ float max_abs(const uint32_t (&s)[N]) {
    float t0 = 0.f, t1 = 0.f;
#pragma unroll
    for (int c = 0; c < N; c += 4) {
        t0 = fmax3(t0, fabsf(__uint_as_float(s[c])), fabsf(__uint_as_float(s[c + 1])));
        t1 = fmax3(t1, fabsf(__uint_as_float(s[c + 2])), fabsf(__uint_as_float(s[c + 3])));
    }
    return fmaxf(t0, t1);
}

// One thread's bias: of head `h`.
struct BiasRow {
    float slope2;        // slope log2 e
    const float *vec;    // vec[d]
    float past, future;  // vec of the distances past `far`
};

__device__ __forceinline__ const float *bias_vec(const ScoreParams &f, int h) {
    return f.vec + static_cast<long long>(h) * vec_stride(f.mid) + f.mid;
}

template <int kBias>
__device__ __forceinline__ BiasRow bias_row(const ScoreParams &f, int h) {
    BiasRow r{0.f, nullptr, 0.f, 0.f};
    if (kBias == kBiasSlopes) r.slope2 = f.slopes[h] * kLog2E;
    if (kBias == kBiasBuckets) {
        r.vec = bias_vec(f, h);
        r.past = r.vec[-f.mid];
        r.future = r.vec[f.mid];
    }
    return r;
}

// The bias of a run of keys as an arithmetic progression b0 + c step, c = 0 ..
// n-1, where it is one for every lane of the warp; returns whether it is.
template <int kBias>
__device__ __forceinline__ bool linear_bias(const ScoreParams &f, const BiasRow &r, int d0, int n, float add, float &b0,
                                            float &step) {
    step = 0.f;
    b0 = add;
    if (kBias == kBiasNone) return true;
    const int lim = kBias == kBiasSlopes ? 0 : f.far;
    const bool past = __all_sync(0xffffffffu, d0 + n - 1 <= -lim || (kBias == kBiasSlopes && f.past_only));
    if (!past && !__all_sync(0xffffffffu, d0 >= lim)) return false;
    if (kBias == kBiasSlopes) {
        step = past ? r.slope2 : -r.slope2;
        b0 = fmaf(step, static_cast<float>(d0), add);
    } else {
        b0 = (past ? r.past : r.future) + add;
    }
    return true;
}

// y = u mul + bias(d0 + c) + add of N values in place, c = 0 .. N-1 (kScaled: u
// holds u mul already): keys run along the registers, the lanes of a warp hold
// one query each with its own d0.  add: minus the reference the weights are
// taken against; the bias's large part and `add` meet in one fused
// multiply-add, so that far distances lose nothing to cancellation.
template <int kBias, bool kScaled, int N>
__device__ __forceinline__ void add_bias(uint32_t (&u)[N], const ScoreParams &f, const BiasRow &r, int d0,
                                         float add) {
    const uint64_t mul2 = f32x2_set(f.mul);
    auto fma2 = [&](uint64_t u2, uint64_t b2) { return kScaled ? add_f32x2(u2, b2) : fma_f32x2(u2, mul2, b2); };
    auto fma1 = [&](uint32_t x, float b) {
        return __float_as_uint(kScaled ? __uint_as_float(x) + b : fmaf(__uint_as_float(x), f.mul, b));
    };
    auto at = [&](int c) { return f32x2_pack(__uint_as_float(u[c]), __uint_as_float(u[c + 1])); };
    auto put = [&](int c, uint64_t v) {
        float a, b;
        f32x2_unpack(v, a, b);
        u[c] = __float_as_uint(a);
        u[c + 1] = __float_as_uint(b);
    };
    if (kBias == kBiasNone) {
        const uint64_t add2 = f32x2_set(add);
#pragma unroll
        for (int c = 0; c < N; c += 2) put(c, fma2(at(c), add2));
    } else if (kBias == kBiasSlopes) {
        const bool past = __all_sync(0xffffffffu, d0 + N - 1 <= 0 || f.past_only);
        if (past || __all_sync(0xffffffffu, d0 >= 0)) {
            // one sign for all: the bias is an arithmetic progression
            const float sl = past ? r.slope2 : -r.slope2;
            const float b0 = fmaf(sl, static_cast<float>(d0), add);
            uint64_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = f32x2_pack(fmaf(2.f * i, sl, b0), fmaf(2.f * i + 1.f, sl, b0));
            const uint64_t step = f32x2_set(8.f * sl);
#pragma unroll
            for (int c = 0; c < N; c += 2) {
                put(c, fma2(at(c), b[(c >> 1) & 3]));
                if (c + 8 < N) b[(c >> 1) & 3] = add_f32x2(b[(c >> 1) & 3], step);
            }
        } else {
            const float df = static_cast<float>(d0);
#pragma unroll
            for (int c = 0; c < N; ++c)
                u[c] = fma1(u[c], fmaf(-r.slope2, fabsf(df + static_cast<float>(c)), add));
        }
    } else {
        const bool past = __all_sync(0xffffffffu, d0 + N - 1 <= -f.far);
        if (past || __all_sync(0xffffffffu, d0 >= f.far)) {
            const uint64_t add2 = f32x2_set((past ? r.past : r.future) + add);
#pragma unroll
            for (int c = 0; c < N; c += 2) put(c, fma2(at(c), add2));
        } else {
            const int dc = min(max(d0, -f.mid), f.far);
            const float *src = r.vec + dc;
#pragma unroll
            for (int c = 0; c < N; ++c)
                u[c] = fma1(u[c], src[c] + add);
        }
    }
}

}  // namespace mha
