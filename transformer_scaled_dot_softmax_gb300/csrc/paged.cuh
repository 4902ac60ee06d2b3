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
#include "softmax_sums.cuh"

namespace mha {

struct PagedSeq {
    int row0, n, len;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedCache &c, int b) {
    PagedSeq s;
    s.row0 = min(max(c.starts[b], 0), c.N);
    s.n = max(min(max(c.starts[b + 1], 0), c.N) - s.row0, 0);  // (the least int less row0 would wrap)
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

}  // namespace mha
