// How a split sum's ranges lie (shared by the kernels, and without HIP, so that a
// plain C++ program can look at it).
#pragma once

#include <stdint.h>

namespace dg {

// Length of the first of `splits` ranges over n summed indices (the last ones may be
// shorter or empty): whole slabs of 64.  Counted in slabs, so that no n below 2^31
// and no number of ranges overflows.
constexpr int32_t range_length(int32_t n, int32_t splits)
{
    const int32_t slabs = n / 64 + (n % 64 != 0);
    return (slabs + splits - 1) / splits * 64;
}

// First index and length of range `i`.
constexpr void range_of(int32_t n, int32_t splits, int32_t i, int32_t &first, int32_t &length)
{
    const int32_t chunk = range_length(n, splits);
    const int64_t b = (int64_t)i * chunk;
    first = b < n ? (int32_t)b : n;
    length = n - first < chunk ? n - first : chunk;
}

}  // namespace dg
