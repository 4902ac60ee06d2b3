// paged.cuh -- what the kernels over a paged K/V cache share: where a
// sequence's rows are.
//
// Sequence b holds len rows; row j is row j % page of the page
// table[b][j / page].  Its n new tokens are packed rows row0 .. row0 + n - 1 and
// the last n of its len rows.  Nothing on the device is trusted: packed rows
// are cut to [0, N), lengths to [0, cap] (max_pages page), and a table entry
// outside [0, num_pages) is a page that is not there.
#pragma once

#include "kernels.h"

namespace mha {

struct PagedSeq {
    int row0, n, len;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedCache &c, int b) {
    PagedSeq s;
    s.row0 = min(max(c.starts[b], 0), c.N);
    s.n = max(min(c.starts[b + 1], c.N) - s.row0, 0);
    s.len = min(max(c.lens[b], 0), c.cap);
    return s;
}

// Entry i < max_pages of sequence b, or -1.
__device__ __forceinline__ int paged_page(const PagedCache &c, int b, int i) {
    const int pg = c.table[static_cast<long long>(b) * c.max_pages + i];
    return pg >= 0 && pg < c.num_pages ? pg : -1;
}

// 2^(stored - 127) of a row's stored exponent, 1 to 254; infinity for 255, under
// which the row's zeros read as NaN.
__device__ __forceinline__ float paged_power(uint32_t stored) { return __uint_as_float(stored << 23); }

// A partial sum (reference m in log2 units, sum l > 0) is 2^m l, and l may be as
// far from 1 as 2^+-64 and more: two of them are compared and joined by m + e, e the
// whole part of log2 l, with O and l taken times 2^-e.  (By m alone a sum of 2^64
// against m = -130 would vanish beside one of 2^-60 against 0, a 64th of it.)
struct PagedLevel {
    float m, down;  // m + e, 2^-e
};
__device__ __forceinline__ PagedLevel paged_level(float m, float l) {
    const int e = min(max(static_cast<int>(__float_as_uint(l) >> 23 & 255u) - 127, -100), 100);  // (any, for a NaN)
    PagedLevel r;
    r.m = m + static_cast<float>(e);
    r.down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    return r;
}

}  // namespace mha
