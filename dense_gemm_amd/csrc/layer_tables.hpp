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

#define DG_LAYER_PIPE(BM, BN, WM, WN, STAGES, BKS)                                             \
    {(const void *)&layer_pipe_kernel<T, BM, BN, WM, WN, false, false, STAGES, BKS>,           \
     (const void *)&layer_pipe_kernel<T, BM, BN, WM, WN, false, true, STAGES, BKS>,            \
     (const void *)&layer_pipe_kernel<T, BM, BN, WM, WN, true, false, STAGES, BKS>}

template <typename T>
const void *layer_kernel_of(int config, int variant)
{
    if constexpr (sizeof(T) == 4) {
        static const void *const table[][3] = {
            DG_LAYER_STAGED(64, 64, 16, 32, 32, 2),
            DG_LAYER_STAGED(128, 128, 16, 64, 64, 2),
            DG_LAYER_PIPE(64, 64, 32, 32, 3, 32),
            DG_LAYER_PIPE(128, 128, 64, 64, 4, 16),
            {nullptr, nullptr, nullptr},
        };
        return table[config][variant];
    } else {
        static const void *const table[][3] = {
            DG_LAYER_STAGED(64, 64, 64, 32, 32, 2),
            DG_LAYER_STAGED(128, 128, 64, 64, 64, 2),
            DG_LAYER_PIPE(64, 64, 32, 32, 4, 16),
            DG_LAYER_PIPE(128, 128, 64, 64, 2, 16),
            DG_LAYER_PIPE(256, 256, 128, 64, 2, 16),
        };
        return table[config][variant];
    }
}
#undef DG_LAYER_STAGED
#undef DG_LAYER_PIPE

}  // namespace dg
