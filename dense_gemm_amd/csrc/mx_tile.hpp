// Parts shared by the product kernels with MX operands: the parameters and
// the epilogue of one 32 x 32 accumulator block.
#pragma once

#include "gemm_pipe.hpp"
#include "mx_common.hpp"

namespace dg {

// A product with MX operands.  `g` holds the sizes, C and the epilogue as in
// the dense kernels; the row stride of an MX operand is in bytes, that of its
// scales in rows of 8 bytes (one group of 256 k, or of 256 columns).
struct MxGemmParams {
    GemmParams g;
    const uint8_t *SA;
    const uint8_t *SB;
    int64_t ldsa, ldsb;
    int32_t ctype;        // ELEM_* of C and the bias
};

typedef hipError_t (*mx_launch_fn)(const MxGemmParams &p, hipStream_t s);

#ifdef __HIPCC__

// Epilogue of a wave's 32 x W strip of blocks (W = 32 * TN): the sums go to
// this wave's staging slot as fp32 [32][W + 8], then a lane forms 8 columns of
// a row per pass, so that W / 8 lanes write a row's W columns in one piece.
template <int W> constexpr int kEpiBytes = 32 * (W + 8) * 4;

template <typename TC, int W>
__device__ __forceinline__ void store_staged(const GemmParams &p, const lds_char_t *stg, int row0, int col0, int lane)
{
    typedef __attribute__((address_space(3))) f32x4 lds_f32x4_t;
    // 16-byte accesses of C; its rows need only be aligned to their element
    typedef TC VC __attribute__((ext_vector_type(16 / sizeof(TC))));
    typedef VC __attribute__((aligned(sizeof(TC)))) VCu;
    constexpr int PER = 16 / sizeof(TC);                 // elements of a 16-byte access
    constexpr int LPR = W / 8, RPP = 64 / LPR;           // lanes per row, rows per pass
    const int lc = (lane % LPR) * 8, gcol = col0 + lc;
    const bool vec = gcol + 8 <= p.N;
    // the lane's 8 columns are the same in every pass: their bias is read once
    float bias[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[e] = p.bias && gcol + e < p.N ? (float)((const TC *)p.bias)[gcol + e] : 0.f;
#pragma unroll 1
    for (int lr = lane / LPR; lr < 32; lr += RPP) {
        const int64_t grow = (int64_t)row0 + lr;
        if (grow >= p.M) break;
        TC *c = (TC *)p.C + grow * p.ldc + gcol;
        float v[8];
#pragma unroll
        for (int c4 = 0; c4 < 2; ++c4) {
            const f32x4 x = *(const lds_f32x4_t *)(stg + (lr * (W + 8) + lc + 4 * c4) * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * c4 + e] = x[e] * p.alpha;
        }
        if (p.beta != 0.f) {
            if (vec) {
#pragma unroll
                for (int q = 0; q < 8 / PER; ++q) {
                    const VC x = *(const VCu *)(c + q * PER);
#pragma unroll
                    for (int e = 0; e < PER; ++e) v[q * PER + e] = __builtin_fmaf(p.beta, (float)x[e], v[q * PER + e]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (gcol + e < p.N) v[e] = __builtin_fmaf(p.beta, (float)c[e], v[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += bias[e];
        if (p.act == ACT_GELU) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = gelu(v[e]);
        } else if (p.act == ACT_RELU) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = activate(ACT_RELU, v[e]);
        }
        if (vec) {
#pragma unroll
            for (int q = 0; q < 8 / PER; ++q) {
                VC x;
#pragma unroll
                for (int e = 0; e < PER; ++e) x[e] = (TC)v[q * PER + e];
                *(VCu *)(c + q * PER) = x;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (gcol + e < p.N) c[e] = (TC)v[e];
        }
    }
}

// The raw sums into a split's partials (row stride N).
template <int W>
__device__ __forceinline__ void store_partial(const GemmParams &p, const lds_char_t *stg, int row0, int col0, int lane,
                                              int split)
{
    typedef __attribute__((address_space(3))) f32x4 lds_f32x4_t;
    constexpr int LPR = W / 4, RPP = 64 / LPR;
    const int lc = (lane % LPR) * 4, gcol = col0 + lc;
#pragma unroll 1
    for (int lr = lane / LPR; lr < 32; lr += RPP) {
        const f32x4 x = *(const lds_f32x4_t *)(stg + (lr * (W + 8) + lc) * 4);
        const int64_t grow = (int64_t)row0 + lr;
        if (grow >= p.M) break;
        float *w = p.ws + ((int64_t)split * p.M + grow) * p.N + gcol;
        if (gcol + 4 <= p.N && (p.N & 3) == 0) {
            *(f32x4 *)w = x;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (gcol + e < p.N) w[e] = x[e];
        }
    }
}

// The wave's TM strips, one after the other (a loop, so that the code is
// there once; the strip's registers are picked by a uniform branch).
template <int TM, int TN>
__device__ __forceinline__ void store_tile(const MxGemmParams &q, lds_char_t *stg, const f32x16 (&acc)[TM][TN], int row0,
                                           int col0, int lane, int split)
{
    typedef __attribute__((address_space(3))) float lds_float_t;
    constexpr int W = 32 * TN;
#pragma unroll 1
    for (int i = 0; i < TM; ++i) {
        // register r of lane l holds row 8*(r/4) + 4*(l/32) + r%4, column l%32
#pragma unroll
        for (int s = 0; s < TM; ++s)
            if (s == i) {
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int row = 8 * (r >> 2) + (lane >> 5) * 4 + (r & 3);
                        *(lds_float_t *)(stg + (row * (W + 8) + 32 * j + (lane & 31)) * 4) = acc[s][j][r];
                    }
            }
        __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the strip is staged
        __builtin_amdgcn_wave_barrier();
        if (q.g.splits > 1) store_partial<W>(q.g, stg, row0 + 32 * i, col0, lane, split);
        else if (q.ctype == ELEM_F32) store_staged<float, W>(q.g, stg, row0 + 32 * i, col0, lane);
        else if (q.ctype == ELEM_F16) store_staged<_Float16, W>(q.g, stg, row0 + 32 * i, col0, lane);
        else store_staged<__bf16, W>(q.g, stg, row0 + 32 * i, col0, lane);
        __builtin_amdgcn_s_waitcnt(0xc07f);  // reads done before the slot is rewritten
        __builtin_amdgcn_wave_barrier();
    }
}

#endif

}  // namespace dg
