// Kernels of a layer's products for one operand type T.  Each .hip file
// instantiates one type, so that they compile in parallel.
#pragma once

#include "layer_rows.hpp"
#include "layer_tile.hpp"

namespace dg {

// [forward and gradient with B stored K x N, with B stored N x K, weights]
#define DG_LAYER_PIPE(BM, BN, WM, WN, KG, STAGES, BK, RA, RB)                                \
    {(const void *)&layer_pipe_kernel<T, BM, BN, WM, WN, KG, false, false, STAGES, BK, RA, RB>,    \
     (const void *)&layer_pipe_kernel<T, BM, BN, WM, WN, KG, false, true, STAGES, BK, RA, RB>,     \
     (const void *)&layer_pipe_kernel<T, BM, BN, WM, WN, KG, true, false, STAGES, BK, RA, RB>}
// an operand that the direct loads do not take: A, B, both
#define DG_LAYER_ANY(BM, BN, WM, WN, BK)                                                       \
    DG_LAYER_PIPE(BM, BN, WM, WN, 1, 2, BK, true, false), DG_LAYER_PIPE(BM, BN, WM, WN, 1, 2, BK, false, true), \
        DG_LAYER_PIPE(BM, BN, WM, WN, 1, 2, BK, true, true)
#define DG_LAYER_ROWS(NWV)                                                                 \
    {(const void *)&layer_rows_kernel<T, false, NWV, false>,                               \
     (const void *)&layer_rows_kernel<T, true, NWV, false>, nullptr}
#define DG_LAYER_STREAM(NWV) {nullptr, (const void *)&layer_rows_kernel<T, true, NWV, true>, nullptr}
#define DG_LAYER_NONE {nullptr, nullptr, nullptr}

template <typename T>
const void *layer_kernel_of(int config, int variant)
{
    if constexpr (sizeof(T) == 4) {
        static const void *const table[][3] = {
            DG_LAYER_ANY(64, 64, 32, 32, 32),
            DG_LAYER_ANY(128, 128, 64, 64, 16),
            DG_LAYER_PIPE(64, 64, 32, 32, 1, 4, 32, false, false),
            DG_LAYER_PIPE(64, 64, 32, 32, 1, 3, 32, false, false),
            DG_LAYER_NONE,
            DG_LAYER_PIPE(128, 128, 64, 64, 1, 4, 16, false, false),
            DG_LAYER_NONE,
            DG_LAYER_ROWS(8),
            DG_LAYER_STREAM(8),
        };
        return table[config][variant];
    } else {
        static const void *const table[][3] = {
            DG_LAYER_ANY(64, 64, 32, 32, 64),
            DG_LAYER_ANY(128, 128, 64, 64, 64),
            DG_LAYER_PIPE(64, 64, 64, 32, 2, 4, 64, false, false),
            DG_LAYER_PIPE(64, 64, 32, 32, 1, 2, 64, false, false),
            DG_LAYER_PIPE(128, 128, 64, 64, 2, 4, 64, false, false),
            DG_LAYER_PIPE(128, 128, 64, 64, 1, 2, 64, false, false),
            DG_LAYER_PIPE(256, 256, 128, 64, 1, 2, 64, false, false),
            DG_LAYER_ROWS(8),
            DG_LAYER_STREAM(8),
        };
        return table[config][variant];
    }
}
#undef DG_LAYER_PIPE
#undef DG_LAYER_ANY
#undef DG_LAYER_ROWS
#undef DG_LAYER_STREAM
#undef DG_LAYER_NONE

}  // namespace dg
