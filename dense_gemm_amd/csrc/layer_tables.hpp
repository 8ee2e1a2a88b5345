// Kernels of a layer's products for one operand type T.  Each .hip file
// instantiates one type, so that they compile in parallel.
#pragma once

#include "layer_tile.hpp"

namespace dg {

// [forward and gradient with B stored K x N, with B stored N x K, weights]
#define DG_LAYER_STAGED(BM, BN, BK, WM, WN, MINW)                                              \
    {(const void *)&layer_staged_kernel<T, BM, BN, BK, WM, WN, false, false, MINW>,            \
     (const void *)&layer_staged_kernel<T, BM, BN, BK, WM, WN, false, true, MINW>,             \
     (const void *)&layer_staged_kernel<T, BM, BN, BK, WM, WN, true, false, MINW>}

template <typename T>
const void *layer_kernel_of(int config, int variant)
{
    constexpr int BK = sizeof(T) == 4 ? 16 : 64;
    static const void *const table[][3] = {
        DG_LAYER_STAGED(64, 64, BK, 32, 32, 2),
        DG_LAYER_STAGED(128, 128, BK, 64, 64, 2),
    };
    return table[config][variant];
}
#undef DG_LAYER_STAGED

}  // namespace dg
