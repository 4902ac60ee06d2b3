// scores.cuh -- the score definition shared by the scored attention kernels
// (forward, backward, decoding over a shared prefix):
//
//   z = scale q.k,   s = cap tanh(z / cap)  (or z),   s += bias_h(d),
//   d = key position - query position,
//   bias_h(d) = -slope_h |d|   or   table[bucket(d), h].
//
// Scores are kept in log2 units (y = s log2 e) because the weights are taken
// with 2^x.  The bucket bias is read from an expanded per-head row
// vec[d], d in [-mid, mid], mid = far + 64, that a preparing launch writes
// once per call (already times log2 e): from |d| >= far on all distances
// share one bucket, so a run of 64 keys that lies wholly past `far` needs one
// value, and any other run is read at d clamped per run, not per key.
#pragma once

#include "kernels.h"
#include "sm103_ptx.cuh"

namespace mha {

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// tanh(x) for |x| <= 1 as x p(x^2), p of degree 4: least maximum error
// fitted over [-1, 1], 2.8e-6 absolute, i.e. 1.4e-4 in a score capped at 50
// (a weight's bf16 rounding is 3.9e-3 of it).  Seven packed operations per
// pair and none on the special-function unit, which the weights' 2^x already
// fill; scores past the cap itself (|x| > 1) are rare and take tanh_any.
constexpr float kTanhRange = 1.0f;
constexpr float kTanhP0 = 0.999968469f, kTanhP1 = -0.332658231f, kTanhP2 = 0.129220663f,
                kTanhP3 = -0.0432998549f, kTanhP4 = 0.00836588231f;

__device__ __forceinline__ uint64_t f32x2_set(float v) { return f32x2_pack(v, v); }

__device__ __forceinline__ uint64_t tanh_small_x2(uint64_t x) {
    const uint64_t w = mul_f32x2(x, x);
    uint64_t p = fma_f32x2(w, f32x2_set(kTanhP4), f32x2_set(kTanhP3));
    p = fma_f32x2(w, p, f32x2_set(kTanhP2));
    p = fma_f32x2(w, p, f32x2_set(kTanhP1));
    p = fma_f32x2(w, p, f32x2_set(kTanhP0));
    return mul_f32x2(x, p);
}

// tanh(x) = 1 - 2 / (1 + e^(2x)) for any x (absolute error ~2^-22; e^(2x)
// overflowing to infinity gives 1, underflowing to 0 gives -1).
__device__ __forceinline__ float tanh_any(float x) {
    return 1.f - __fdividef(2.f, 1.f + ex2_approx(x * (2.f * kLog2E)));
}

// u = tanh(s cap_in) of N scores in place; `any_large` (warp-uniform): some
// |s cap_in| of the warp is past kTanhRange.
template <int N>
__device__ __forceinline__ void cap_scores(uint32_t (&s)[N], float cap_in, bool any_large) {
    if (any_large) {
#pragma unroll
        for (int c = 0; c < N; ++c) s[c] = __float_as_uint(tanh_any(__uint_as_float(s[c]) * cap_in));
    } else {
        const uint64_t a2 = f32x2_set(cap_in);
#pragma unroll
        for (int c = 0; c < N; c += 2) {
            float t0, t1;
            f32x2_unpack(tanh_small_x2(mul_f32x2(f32x2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), a2)), t0,
                         t1);
            s[c] = __float_as_uint(t0);
            s[c + 1] = __float_as_uint(t1);
        }
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
    float slope2;      // slope log2 e
    const float *vec;  // vec[d]
};

template <int kBias>
__device__ __forceinline__ BiasRow bias_row(const ScoreParams &f, int h) {
    BiasRow r{0.f, nullptr};
    if (kBias == kBiasSlopes) r.slope2 = f.slopes[h] * kLog2E;
    if (kBias == kBiasBuckets) r.vec = f.vec + static_cast<long long>(h) * (2 * f.mid + 1) + f.mid;
    return r;
}

// y = u mul + bias(d0 + kStep c) + add of N values in place, c = 0 .. N-1,
// kStep = +1 (keys run along the registers) or -1 (queries do).  The lanes of
// a warp hold one query (key) each with its own d0.  add: minus the reference
// the weights are taken against; the bias's large part and `add` meet in one
// fused multiply-add, so that far distances lose nothing to cancellation.
template <int kBias, int kStep, int N>
__device__ __forceinline__ void add_bias(uint32_t (&u)[N], const ScoreParams &f, const BiasRow &r, int d0,
                                         float add) {
    const uint64_t mul2 = f32x2_set(f.mul);
    auto at = [&](int c) { return f32x2_pack(__uint_as_float(u[c]), __uint_as_float(u[c + 1])); };
    auto put = [&](int c, uint64_t v) {
        float a, b;
        f32x2_unpack(v, a, b);
        u[c] = __float_as_uint(a);
        u[c + 1] = __float_as_uint(b);
    };
    constexpr int kEnd = kStep * (N - 1);
    if (kBias == kBiasNone) {
        const uint64_t add2 = f32x2_set(add);
#pragma unroll
        for (int c = 0; c < N; c += 2) put(c, fma_f32x2(at(c), mul2, add2));
    } else if (kBias == kBiasSlopes) {
        const int dmin = kStep > 0 ? d0 : d0 + kEnd, dmax = kStep > 0 ? d0 + kEnd : d0;
        const bool past = __all_sync(0xffffffffu, dmax <= 0 || f.past_only);
        if (past || __all_sync(0xffffffffu, dmin >= 0)) {
            // one sign for all: the bias is an arithmetic progression
            const float sl = past ? r.slope2 : -r.slope2;
            const float b0 = fmaf(sl, static_cast<float>(d0), add), st = kStep * sl;
            uint64_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = f32x2_pack(fmaf(2.f * i, st, b0), fmaf(2.f * i + 1.f, st, b0));
            const uint64_t step = f32x2_set(8.f * st);
#pragma unroll
            for (int c = 0; c < N; c += 2) {
                put(c, fma_f32x2(at(c), mul2, b[(c >> 1) & 3]));
                if (c + 8 < N) b[(c >> 1) & 3] = add_f32x2(b[(c >> 1) & 3], step);
            }
        } else {
            const float df = static_cast<float>(d0);
#pragma unroll
            for (int c = 0; c < N; ++c)
                u[c] = __float_as_uint(
                    fmaf(__uint_as_float(u[c]), f.mul, fmaf(-r.slope2, fabsf(df + static_cast<float>(kStep * c)), add)));
        }
    } else {
        const int dmin = kStep > 0 ? d0 : d0 + kEnd, dmax = kStep > 0 ? d0 + kEnd : d0;
        const bool past = __all_sync(0xffffffffu, dmax <= -f.far);
        if (past || __all_sync(0xffffffffu, dmin >= f.far)) {
            const uint64_t add2 = f32x2_set(r.vec[past ? -f.mid : f.mid] + add);
#pragma unroll
            for (int c = 0; c < N; c += 2) put(c, fma_f32x2(at(c), mul2, add2));
        } else {
            const int dc = kStep > 0 ? min(max(d0, -f.mid), f.far) : min(max(d0, -f.far), f.mid);
            const float *src = r.vec + dc;
#pragma unroll
            for (int c = 0; c < N; ++c)
                u[c] = __float_as_uint(fmaf(__uint_as_float(u[c]), f.mul, src[kStep * c] + add));
        }
    }
}

}  // namespace mha
