// softmax_sums.cuh -- joining a row's partial sums (reference m, sum l of the weights
// against it, unnormalised O) of different keys.
#pragma once

namespace mha {

// A partial sum (m in log2 units, l > 0) is 2^m l, and where a reference serves
// as long as sums fit (m = 0 for scores of -70 as well) l may be as far from 1 as
// 2^+-64 and more: two of them are compared and joined by m + e, e the whole part of
// log2 l, with O and l taken times 2^-e.  By m alone 64 keys at -130 and 64 at -72.5
// against -130, a sum of 2^63.5, would vanish beside 64 at -68 against 0, one of 2^-62:
// 2^-130 is flushed to 0, although they weigh a 23rd of those.
struct SumLevel {
    float m, down;  // m + e, 2^-e
};
__device__ __forceinline__ SumLevel sum_level(float m, float l) {
    const int e = min(max(static_cast<int>(__float_as_uint(l) >> 23 & 255u) - 127, -100), 100);  // (any, for a NaN)
    SumLevel r;
    r.m = m + static_cast<float>(e);
    r.down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    return r;
}

// Key tiles (of 128) of a query block that are summed in tensor memory without a break: a
// longer range goes through the pipeline in runs of so many, whose sums are joined
// outside it.  The tensor cores' accumulators drop, towards zero, what lies below a sum's
// last places when it is added: values of one sign averaged over 2^20 rows came out 0.4 %
// too small in one run, over 2^26 18 %; in runs of 2,048 / 1,024 / 512 tiles 2.5e-4 / 8e-5 /
// 2e-5, whatever the length (a head's prompt of 131,072 takes 1 % longer than without).
constexpr int kRunTiles = 1024;
// Whether the contiguous forwards go about it so, in instances of their own: the loop and
// the joining cost their softmax warps 9 % (1 head of 270,000 x 270,000: 17.5 ms against
// 16.1; as part of the common instances 2 x 16 x 8,192 causal took 277 us against 251), and
// up to this many keys the bias is below 2.5e-4, a 16th of a rounding to bf16.
inline bool needs_runs(int keys) { return keys > 2 * kRunTiles * 128; }

}  // namespace mha
