// Tile kernels of a layer's products (see layer_common.hpp for what they compute):
//
//   forward, gradient   C[row][n] = epilogue(sum_k A[row][k] op(B_g)[k][n]), row in group g
//   weights             C_g[m][n] = epilogue(sum_r A[r][m] B[r][n]),         r over group g's rows
//
// One workgroup takes one BM x BN tile of one group and walks its sum in slabs.
// A group's last tile row and last slab end inside a tile: rows and columns past
// the end are fetched from valid places and never stored, summed indices past the
// end are zero.
//
// layer_staged_kernel  any strides and alignment: operands through registers.
#pragma once

#include <type_traits>

#include "gemm_mfma.hpp"
#include "gemm_pipe.hpp"
#include "layer_common.hpp"

namespace dg {

// ---- epilogue of a wave's blocks -----------------------------------------------
// Strips of 32 rows x W columns (W = 32 * TN): the sums go to this wave's slot as
// fp32 [32][W + 8], then a lane takes 8 columns of a row per pass, so that W / 8
// lanes read and write a row's W columns in one piece.  What the epilogue reads
// beside the sums is fetched before the strip is staged.
template <int W> constexpr int kStripBytes = 32 * (W + 8) * 4;

template <typename TC, int TM, int TN>
__device__ __forceinline__ void layer_store_as(const LayerParams &p, const LayerTile &t, lds_char_t *stg,
                                               const f32x16 (&acc)[TM][TN], int row0, int col0, int lane, bool partial)
{
    typedef __attribute__((address_space(3))) float lds_float_t;
    typedef __attribute__((address_space(3))) f32x4 lds_f32x4_t;
    constexpr int W = 32 * TN, LPR = W / 8, RPP = 64 / LPR, PASSES = 32 / RPP;
    const int lc = (lane % LPR) * 8, lr0 = lane / LPR, col = col0 + lc, n = p.N - col;
    float bias[8];
    if (!partial) layer_bias<TC, 8>(p, t.group, col, n, bias);
#pragma unroll 1
    for (int i = 0; i < TM; ++i) {
        LayerAux<TC, 8> aux[PASSES];
        if (!partial) {
#pragma unroll
            for (int ps = 0; ps < PASSES; ++ps) {
                const int row = row0 + 32 * i + lr0 + ps * RPP;
                aux[ps].fetch(p, t, row < t.rows ? row : t.rows - 1, n > 0 ? col : 0, row < t.rows ? n : 0);
            }
        }
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
#pragma unroll
        for (int ps = 0; ps < PASSES; ++ps) {
            const int lr = lr0 + ps * RPP, row = row0 + 32 * i + lr;
            float v[8];
#pragma unroll
            for (int c4 = 0; c4 < 2; ++c4) {
                const f32x4 x = *(const lds_f32x4_t *)(stg + (lr * (W + 8) + lc + 4 * c4) * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[4 * c4 + e] = x[e];
            }
            if (row < t.rows && n > 0) {
                if (partial) layer_partial<8>(p, t, row, col, n, v);
                else layer_finish<TC, 8>(p, t, row, col, n, v, aux[ps], bias);
            }
        }
        __builtin_amdgcn_s_waitcnt(0xc07f);  // reads done before the slot is rewritten
        __builtin_amdgcn_wave_barrier();
    }
}

template <typename T, int TM, int TN>
__device__ __forceinline__ void layer_store(const LayerParams &p, const LayerTile &t, lds_char_t *stg,
                                            const f32x16 (&acc)[TM][TN], int row0, int col0, int lane)
{
    if (p.splits > 1) layer_store_as<float>(p, t, stg, acc, row0, col0, lane, true);
    else if (sizeof(T) == 2 && p.ctype != 0) layer_store_as<T>(p, t, stg, acc, row0, col0, lane, false);
    else layer_store_as<float>(p, t, stg, acc, row0, col0, lane, false);
}

// ---- any strides and alignment ----------------------------------------------------
// Operands go through registers into a double-buffered LDS slab, in 16-byte loads
// that need only the element's alignment (the GPU takes misaligned vectors).
template <typename T, int BMN, int BK, bool KCONT>
struct StagedOperand : Operand<T, BMN, BK, KCONT, true> {
    typedef Operand<T, BMN, BK, KCONT, true> Base;
    typedef typename Base::vec vec;
    typedef vec __attribute__((aligned(sizeof(T)))) vecu;
    static constexpr int V = Base::V;

    __device__ __forceinline__ static vec load_piece(const T *p, int valid)
    {
        vec v;
        if (valid >= V) {
            v = *(const vecu *)p;
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                T x = (T)0.f;
                if (e < valid) x = p[e];
                v[e] = x;
            }
        }
        return v;
    }

    // the slab at (mn0, k0) of a matrix of ext rows (or columns) and K summed indices
    __device__ __forceinline__ void load(const T *g, int64_t ld, int mn0, int k0, int ext, int K, int tid)
    {
        if constexpr (KCONT) {
            const int rr = tid / Base::LPR, c = (tid % Base::LPR) * V;
#pragma unroll
            for (int q = 0; q < Base::NV; ++q) {
                const int mn = mn0 + q * Base::RPP + rr, k = k0 + c;
                this->r[q] = load_piece(g + (int64_t)mn * ld + k, mn < ext ? K - k : 0);
            }
        } else {
            // consecutive k rows per thread where the store transposes them (16 bits)
            const int kg = tid / Base::LPK, c = (tid % Base::LPK) * V;
#pragma unroll
            for (int q = 0; q < Base::NV; ++q) {
                const int k = k0 + (Base::F16 ? kg * Base::KV + q : q * Base::KG + kg), mn = mn0 + c;
                this->r[q] = load_piece(g + (int64_t)k * ld + mn, k < K ? ext - mn : 0);
            }
        }
    }
};

template <typename T, int BM, int BN, int BK, int WM, int WN, bool DW, bool TB, int MINW>
__global__ __launch_bounds__(256, MINW) void layer_staged_kernel(LayerParams p)
{
    constexpr int WAVES_N = BN / WN, TM = WM / 32, TN = WN / 32;
    static_assert((BM / WM) * WAVES_N == 4, "4 waves per workgroup");
    typedef StagedOperand<T, BM, BK, !DW> OpA;
    typedef StagedOperand<T, BN, BK, TB && !DW> OpB;
    constexpr int STAGE = OpA::ELEMS + OpB::ELEMS;
    constexpr int RING = 2 * STAGE * (int)sizeof(T), STRIPS = 4 * kStripBytes<WN>;
    __shared__ __attribute__((aligned(16))) char smem_raw[RING > STRIPS ? RING : STRIPS];
    T *smem = (T *)smem_raw;

    LayerTile t;
    if (!layer_tile(p, BM, BN, t)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm0 = (wave / WAVES_N) * WM, wn0 = (wave % WAVES_N) * WN;
    const T *A = (const T *)p.A + (DW ? (t.row0 + t.k0) * p.lda : t.row0 * p.lda + t.k0);
    const T *B = (const T *)p.B + (DW ? (t.row0 + t.k0) * p.ldb
                                      : t.group * p.strideB + (TB ? (int64_t)t.k0 : t.k0 * p.ldb));
    const int K = t.k_len, nk = (K + BK - 1) / BK;

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    OpA ga;
    OpB gb;
    if (nk > 0) {
        ga.load(A, p.lda, t.m0, 0, t.rows, K, tid);
        gb.load(B, p.ldb, t.n0, 0, p.N, K, tid);
        ga.store(smem, tid);
        gb.store(smem + OpA::ELEMS, tid);
    }
    __syncthreads();
    const int lrow = lane & 31, khalf = (lane >> 5) * (BK / 2);
    for (int kt = 0; kt < nk; ++kt) {
        const T *sA = smem + (kt & 1) * STAGE;
        const T *sB = sA + OpA::ELEMS;
        const bool more = kt + 1 < nk;
        if (more) {
            ga.load(A, p.lda, t.m0, (kt + 1) * BK, t.rows, K, tid);
            gb.load(B, p.ldb, t.n0, (kt + 1) * BK, p.N, K, tid);
        }
        if constexpr (sizeof(T) == 4) {
            // 32x32x2 steps, four at a time; lane half h takes k of the slab's half h
#pragma unroll
            for (int c = 0; c < BK / 8; ++c) {
                float a[TM][4], b[TN][4];
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        a[i][e] = OpA::LDS_KMAJOR ? sA[(wm0 + 32 * i + lrow) * OpA::LD + khalf + 4 * c + e]
                                                  : sA[(khalf + 4 * c + e) * OpA::LD + wm0 + 32 * i + lrow];
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        b[j][e] = OpB::LDS_KMAJOR ? sB[(wn0 + 32 * j + lrow) * OpB::LD + khalf + 4 * c + e]
                                                  : sB[(khalf + 4 * c + e) * OpB::LD + wn0 + 32 * j + lrow];
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int j = 0; j < TN; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i][e], b[j][e], acc[i][j], 0, 0, 0);
            }
        } else {
            // 32x32x16 steps, 8 k a lane
            typedef typename ElemTraits<T>::vec v8;
#pragma unroll
            for (int c = 0; c < BK / 16; ++c) {
                v8 a[TM], b[TN];
#pragma unroll
                for (int i = 0; i < TM; ++i) a[i] = *(const v8 *)(sA + (wm0 + 32 * i + lrow) * OpA::LD + khalf + 8 * c);
#pragma unroll
                for (int j = 0; j < TN; ++j) b[j] = *(const v8 *)(sB + (wn0 + 32 * j + lrow) * OpB::LD + khalf + 8 * c);
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j) acc[i][j] = mfma_32x32x16(a[i], b[j], acc[i][j]);
            }
        }
        if (more) {
            T *s = smem + ((kt + 1) & 1) * STAGE;
            ga.store(s, tid);
            gb.store(s + OpA::ELEMS, tid);
        }
        __syncthreads();
    }
    lds_char_t *stg = (lds_char_t *)smem_raw + wave * kStripBytes<WN>;
    layer_store<T>(p, t, stg, acc, t.m0 + wm0, t.n0 + wn0, lane);
}

}  // namespace dg
