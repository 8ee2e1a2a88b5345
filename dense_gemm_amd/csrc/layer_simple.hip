// Passes beside a layer's products: the join of a split sum, and the column sums
// of a weight gradient's bias.
#include "layer_common.hpp"

namespace dg {

namespace {

// Joins the splits' raw sums (ws[split][group][M][N], fp32), added in their order, and
// applies the epilogue: 4 columns of a row a thread, n of which exist, so that small
// outputs too have many threads; 8 splits' loads in flight.  Behind the rows, a thread
// for every column sum of the bias's gradient.  Latency bounds it: 2048 x 32 of 12 ranges
// with a bias 3.9 us (7.6 with 8 columns a thread, 4 splits' loads and the column sums
// in the rows' first threads).
template <typename TC>
__global__ __launch_bounds__(256) void layer_join_kernel(LayerParams p)
{
    constexpr int W = 4, FLY = 8;
    const int per_row = (p.N + W - 1) / W;
    const int64_t gm = (int64_t)p.groups * p.M, total = gm * per_row, mn = gm * p.N;
    const int64_t all = total + (p.dbias ? gm : 0);
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < all; at += (int64_t)gridDim.x * 256) {
        const bool column = at >= total;                     // a column sum
        const int64_t grow = column ? at - total : at / per_row;
        const int col = column ? 0 : (int)(at - grow * per_row) * W, n = column ? 1 : p.N - col;
        const float *w = column ? p.ws + p.splits * mn + grow : p.ws + grow * p.N + col;
        const int64_t step = column ? gm : mn;
        LayerTile t;
        t.group = (int)(grow / p.M);
        t.row0 = t.out0 = 0;
        const int row = (int)(grow - (int64_t)t.group * p.M);
        LayerAux<TC, W> aux;
        float v[W], bias[W];
        if (!column) {
            aux.fetch(p, t, row, col, n);
            layer_bias<TC, W>(p, t.group, col, bias, n);
        }
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = 0.f;
        for (int s = 0; s < p.splits; s += FLY) {
            float x[FLY][W];
#pragma unroll
            for (int u = 0; u < FLY; ++u)
                if (s + u < p.splits) load_row<float, W>(w + (s + u) * step, x[u], n);
#pragma unroll
            for (int u = 0; u < FLY; ++u)
                if (s + u < p.splits)
#pragma unroll
                    for (int e = 0; e < W; ++e) v[e] += x[u][e];
        }
        if (column) p.dbias[grow] = p.beta != 0.f ? __builtin_fmaf(p.beta, p.dbias[grow], v[0]) : v[0];
        else layer_finish<TC, W>(p, t, row, col, v, aux, bias, n);
    }
}

// dbias where there is no product to compute it with (no column in B, or alpha = 0):
// dbias[g][m] = sum over group g's rows of A[r][m] (+ beta * dbias).  A workgroup
// takes 64 columns of a group, 64 rows at a time, 8 columns of a row a lane; the
// 64 partial sums of a column are added in a fixed order.
template <typename T>
__global__ __launch_bounds__(512) void layer_colsum_kernel(LayerParams p)
{
    __shared__ float red[64][65];
    const int g = blockIdx.y, lc = (threadIdx.x & 7) * 8, lr = threadIdx.x >> 3;
    const int col = blockIdx.x * 64 + lc, n = p.M - col;
    int begin = 0, rows = p.K;
    if (p.offsets) group_rows(p, g, p.K, begin, rows);
    const T *a = (const T *)p.A + (int64_t)begin * p.lda + col;
    float s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = 0.f;
    if (n >= 8) {
        for (int r = lr; r < rows; r += 256) {
            float v[4][8];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (r + 64 * u < rows) load_row<T, 8>(a + (int64_t)(r + 64 * u) * p.lda, v[u], 8);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (r + 64 * u < rows)
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[e] += v[u][e];
        }
    } else if (n > 0) {
        for (int r = lr; r < rows; r += 64)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) s[e] += (float)a[(int64_t)r * p.lda + e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) red[lr][lc + e] = s[e];
    __syncthreads();
    if (threadIdx.x < 64 && blockIdx.x * 64 + (int)threadIdx.x < p.M) {
        float v = 0.f;
#pragma unroll 8
        for (int r = 0; r < 64; ++r) v += red[r][threadIdx.x];
        float *d = p.dbias + (int64_t)g * p.M + blockIdx.x * 64 + threadIdx.x;
        *d = p.beta != 0.f ? __builtin_fmaf(p.beta, *d, v) : v;
    }
}

}  // namespace

hipError_t launch_layer_join(const LayerParams &p, hipStream_t s)
{
    const int64_t gm = (int64_t)p.groups * p.M, total = gm * ((p.N + 3) / 4) + (p.dbias ? gm : 0), blocks = (total + 255) / 256;
    LayerParams arg = p;
    void *args[] = {&arg};
    const void *f = p.ctype == 0 ? (const void *)&layer_join_kernel<float>
                                 : p.ctype == 1 ? (const void *)&layer_join_kernel<_Float16>
                                                : (const void *)&layer_join_kernel<__bf16>;
    return hipLaunchKernel(f, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), args, 0, s);
}

// type: of the operands (0 fp32, 1 fp16, 2 bf16)
hipError_t launch_layer_colsum(const LayerParams &p, int type, hipStream_t s)
{
    LayerParams arg = p;
    void *args[] = {&arg};
    const void *f = type == 0 ? (const void *)&layer_colsum_kernel<float>
                              : type == 1 ? (const void *)&layer_colsum_kernel<_Float16>
                                          : (const void *)&layer_colsum_kernel<__bf16>;
    return hipLaunchKernel(f, dim3((unsigned)((p.M + 63) / 64), (unsigned)p.groups), dim3(512), args, 0, s);
}

}  // namespace dg
