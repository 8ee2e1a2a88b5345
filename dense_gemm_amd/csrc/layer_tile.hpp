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
// layer_staged_kernel  any strides and alignment: operands through registers;
// layer_pipe_kernel    4-byte aligned rows: a ring of slabs in LDS filled by direct loads.
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
    // passes fetched together: half of an fp32 strip's, for the registers
    constexpr int TOGETHER = sizeof(TC) == 4 && PASSES > 1 ? PASSES / 2 : PASSES;
    const int lc = (lane % LPR) * 8, col = col0 + lc;
    const bool whole = col0 + W <= p.N;
    float bias[8];
    if (whole && !partial) layer_bias<TC, 8>(p, t.group, col, bias);
#pragma unroll 1
    for (int i = 0; i < TM; ++i) {
        const int rows = t.rows - row0 - 32 * i;         // of this strip on
        // (opaque to the compiler, which would otherwise keep every pass's addresses
        // in registers from strip to strip)
        int lr0 = lane / LPR, lane1 = lane;
        asm volatile("" : "+v"(lr0), "+v"(lane1));
        LayerAux<TC, 8> aux[TOGETHER];
        auto fetch = [&](int from) {
            if (whole && !partial) {
#pragma unroll
                for (int ps = 0; ps < TOGETHER; ++ps)
                    if (lr0 + (from + ps) * RPP < rows) aux[ps].fetch(p, t, row0 + 32 * i + lr0 + (from + ps) * RPP, col);
            }
        };
        fetch(0);
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
        if (whole) {
#pragma unroll
            for (int ps = 0; ps < PASSES; ++ps) {
                const int lr = lr0 + ps * RPP;
                if (ps > 0 && ps % TOGETHER == 0) fetch(ps);
                float v[8];
#pragma unroll
                for (int c4 = 0; c4 < 2; ++c4) {
                    const f32x4 x = *(const lds_f32x4_t *)(stg + (lr * (W + 8) + lc + 4 * c4) * 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[4 * c4 + e] = x[e];
                }
                if (lr < rows) {
                    if (partial) layer_partial<8>(p, t, row0 + 32 * i + lr, col, v);
                    else layer_finish<TC, 8>(p, t, row0 + 32 * i + lr, col, v, aux[ps % TOGETHER], bias);
                }
                __builtin_amdgcn_sched_barrier(0);    // a pass's registers at a time
            }
        } else {
            // the last columns: one element a lane
#pragma unroll 1
            for (int at = lane1; at < 32 * W; at += 64) {
                const int lr = at / W, c = at % W;
                if (lr >= rows || col0 + c >= p.N) continue;
                float v[1] = {*(const lds_float_t *)(stg + (lr * (W + 8) + c) * 4)};
                if (partial) {
                    layer_partial<1>(p, t, row0 + 32 * i + lr, col0 + c, v);
                } else {
                    float b[1];
                    LayerAux<TC, 1> x;
                    layer_bias<TC, 1>(p, t.group, col0 + c, b);
                    x.fetch(p, t, row0 + 32 * i + lr, col0 + c);
                    layer_finish<TC, 1>(p, t, row0 + 32 * i + lr, col0 + c, v, x, b);
                }
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


// ---- 4-byte aligned rows -------------------------------------------------------------
// The operands of the direct loads (gemm_pipe.hpp), for any extents: a piece of a
// row that is no whole number of pieces long reaches past the row's end, into the
// next row (rows are at least a piece long), and the last slab, which has no next
// row, goes through registers element by element (`tail`), as does a last slab of
// fewer summed indices than a slab has.  What lies past a row's end only feeds
// outputs that are never stored.
template <typename T, int BMN, bool KCONT, int NW, int BKS>
struct LayerOperand : std::conditional<sizeof(T) == 2, PipeOperandH<T, BMN, KCONT, NW, 16>,
                                       PipeOperandS<BMN, KCONT, NW, 16, BKS>>::type {
    typedef typename std::conditional<sizeof(T) == 2, PipeOperandH<T, BMN, KCONT, NW, 16>,
                                      PipeOperandS<BMN, KCONT, NW, 16, BKS>>::type Base;
    static constexpr bool H = sizeof(T) == 2;
    static constexpr int PER = 16 / (int)sizeof(T);       // elements of a piece, which a lane loads

    // Row (KCONT) or summed index, and first column, of the piece at byte b of a stage.
    __device__ static __forceinline__ void place(int b, int &r, int &c)
    {
        r = b / Base::ROW_BYTES;
        const int p = (b % Base::ROW_BYTES) >> 4;
        if constexpr (H) {
            c = KCONT ? (p ^ ((r >> 1) & 7)) * 8 : (((p >> 2) ^ Base::swz(r)) << 5) + (p & 3) * 8;
        } else if constexpr (KCONT) {
            c = (p ^ Base::swz(r)) * 4;
        } else {
            r = Base::krow(r);
            c = (((p >> 3) ^ Base::hsw(r)) << 5) + (p & 7) * 4;
        }
    }

    __device__ __forceinline__ void init(const T *g, int64_t ld, int mn0, int ext, int wave, int lane)
    {
        this->base = (const char *)(KCONT ? g + (int64_t)mn0 * ld : g + mn0);
#pragma unroll
        for (int i = 0; i < Base::LOADS; ++i) {
            int r, c;
            place((i * NW + wave) * Base::SPAN + lane * 16, r, c);
            if constexpr (KCONT) {
                if (mn0 + r >= ext) r = ext - 1 - mn0;
            } else {
                if (mn0 + c >= ext) c = ((ext - 1) / PER) * PER - mn0;
            }
            this->off[i] = (uint32_t)(((int64_t)r * ld + c) * (int)sizeof(T));
        }
        this->step = (KCONT ? Base::BK : Base::BK * ld) * (int)sizeof(T);
    }

    // the last slab, with krem summed indices left
    __device__ __forceinline__ void tail(lds_char_t *lds, int wave, int lane, int krem, int mn0, int ext)
    {
        typedef T V __attribute__((ext_vector_type(PER)));
        typedef V __attribute__((aligned(sizeof(T)))) Vu;
        typedef __attribute__((address_space(3))) V lds_v_t;
#pragma unroll 1
        for (int i = 0; i < Base::LOADS; ++i) {
            const int b = (i * NW + wave) * Base::SPAN + lane * 16;
            int r, c;
            place(b, r, c);
            int valid;
            if constexpr (KCONT) {
                valid = mn0 + r < ext ? krem - c : 0;
            } else {
                valid = r < krem ? ext - mn0 - c : 0;
            }
            const T *x = (const T *)(this->base + ((int64_t)r * row_step + (int64_t)c * (int)sizeof(T)));
            V v;
            if (valid >= PER) {
                v = *(const Vu *)x;
            } else {
#pragma unroll
                for (int e = 0; e < PER; ++e) v[e] = e < valid ? x[e] : (T)0.f;
            }
            *(lds_v_t *)(lds + b) = v;
        }
        this->advance();
    }

    int64_t row_step;                                     // bytes from a stored row to the next
};

// BM x BN tile, waves of WM x WN, a ring of STAGES slabs of BK summed indices.
//
// 16 bits (slabs of 64): fragments are double-buffered per step of 16 k.  The
// barrier of a slab sits before its last step, which runs from registers while the
// next slab's first fragments are read and the slab STAGES ahead is loaded into the
// stage just finished (A's loads there, B's during the following step), so that
// no fragment read waits at a barrier and loads and reads lie between MFMAs.
// fp32 (slabs of BKS): one barrier at a slab's start, the loads of slab kt + STAGES -
// 1 spread over its MFMAs.
template <typename T, int BM, int BN, int WM, int WN, bool DW, bool TB, int STAGES, int BKS>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN), 2) void layer_pipe_kernel(LayerParams p)
{
    constexpr bool H = sizeof(T) == 2;
    constexpr int WAVES_N = BN / WN, NW = (BM / WM) * WAVES_N, TM = WM / 32, TN = WN / 32, NM = TM * TN;
    typedef LayerOperand<T, BM, !DW, NW, BKS> OpA;
    typedef LayerOperand<T, BN, TB && !DW, NW, BKS> OpB;
    constexpr int BK = OpA::BK, LOADS = OpA::LOADS + OpB::LOADS, STAGE = OpA::BYTES + OpB::BYTES;
    constexpr int RING = STAGES * STAGE, STRIPS = NW * kStripBytes<WN>;
    static_assert((RING > STRIPS ? RING : STRIPS) <= 160 * 1024, "the ring and the strips fit the LDS");
    static_assert((STAGES - 2) * LOADS + OpA::LOADS < 64, "the loads in flight can be counted");
    __shared__ __attribute__((aligned(1024))) char smem_raw[RING > STRIPS ? RING : STRIPS];
    lds_char_t *smem = (lds_char_t *)smem_raw;

    LayerTile t;
    if (!layer_tile(p, BM, BN, t)) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm0 = (wave / WAVES_N) * WM, wn0 = (wave % WAVES_N) * WN;
    const T *A = (const T *)p.A + (DW ? (t.row0 + t.k0) * p.lda : t.row0 * p.lda + t.k0);
    const T *B = (const T *)p.B + (DW ? (t.row0 + t.k0) * p.ldb
                                      : t.group * p.strideB + (TB ? (int64_t)t.k0 : t.k0 * p.ldb));
    const int nk = (t.k_len + BK - 1) / BK, krem = t.k_len - (nk - 1) * BK;
    // the last slab through registers: it ends early, or its rows in part of a piece
    const bool tail = krem < BK || (DW && t.rows % OpA::PER != 0) || (!(TB && !DW) && p.N % OpB::PER != 0);
    const int nfull = tail ? nk - 1 : nk;

    OpA ga;
    OpB gb;
    ga.init(A, p.lda, t.m0, t.rows, wave, lane);
    gb.init(B, p.ldb, t.n0, p.N, wave, lane);
    ga.row_step = p.lda * (int)sizeof(T);
    gb.row_step = p.ldb * (int)sizeof(T);
    auto slab_tail = [&](lds_char_t *st) {
        ga.tail(st, wave, lane, krem, t.m0, t.rows);
        gb.tail(st + OpA::BYTES, wave, lane, krem, t.n0, p.N);
    };

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    if constexpr (H) {
        typedef T V8 __attribute__((ext_vector_type(8)));
        constexpr int KPW = BK / 16;
        V8 fa[2][TM], fb[2][TN];
        auto read_a = [&](const lds_char_t *st, int i, int s) { return ga.frag(st, wm0 + 32 * i, s, lane); };
        auto read_b = [&](const lds_char_t *st, int j, int s) { return gb.frag(st + OpA::BYTES, wn0 + 32 * j, s, lane); };
        // the ring, but for B of its last stage, which the first step loads
#pragma unroll
        for (int s = 0; s < STAGES; ++s) {
            lds_char_t *st = smem + s * STAGE;
            if (s < nfull) {
                ga.issue(st, wave);
                if (s < STAGES - 1) gb.issue(st + OpA::BYTES, wave);
            } else if (s < nk) {
                slab_tail(st);
            }
        }
        if (nfull >= STAGES) wait_vmcnt<(STAGES - 2) * LOADS + OpA::LOADS>();
        else wait_vmcnt<0>();
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[0][i] = read_a(smem, i, 0);
#pragma unroll
        for (int j = 0; j < TN; ++j) fb[0][j] = read_b(smem, j, 0);

        int stage = 0;
        // FAST: slab kt + STAGES is whole (and so is kt + STAGES - 1)
        auto slab = [&](auto fast_tag, int kt) {
            constexpr bool FAST = decltype(fast_tag)::value;
            lds_char_t *st = smem + stage * STAGE;
            lds_char_t *prev = smem + (stage == 0 ? STAGES - 1 : stage - 1) * STAGE;
            const bool pend = FAST || kt + STAGES - 1 < nfull;
#pragma unroll
            for (int s = 0; s + 1 < KPW; ++s) {
                const int cur = s & 1, nxt = cur ^ 1;
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        const int m = i * TN + j;
                        if (s == 0) {
#pragma unroll
                            for (int l = 0; l < OpB::LOADS; ++l)
                                if (l * NM / OpB::LOADS == m && pend) gb.issue_one(prev + OpA::BYTES, wave, l);
                        }
#pragma unroll
                        for (int f = 0; f < TM + TN; ++f)
                            if (f * NM / (TM + TN) == m) {
                                if (f < TM) fa[nxt][f] = read_a(st, f, s + 1);
                                else fb[nxt][f - TM] = read_b(st, f - TM, s + 1);
                            }
                        acc[i][j] = mfma_32x32x16(fa[cur][i], fb[cur][j], acc[i][j]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                if (s == 0 && pend) gb.advance();
            }
            // slab kt + 1 has landed in every wave's part, and every wave holds
            // its last fragments of slab kt
            if constexpr (FAST) wait_vmcnt<(STAGES - 2) * LOADS>();
            else wait_vmcnt<0>();
            __syncthreads();
            stage = stage + 1 == STAGES ? 0 : stage + 1;
            const lds_char_t *nst = smem + stage * STAGE;
            const bool more = FAST || kt + STAGES < nfull;
            if constexpr (!FAST) {
                if (!more && kt + STAGES < nk) slab_tail(st);
            }
            constexpr int cur = (KPW - 1) & 1, nxt = cur ^ 1;
            // (after the last slab these reads fetch a stale stage, never used)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const int m = i * TN + j;
#pragma unroll
                    for (int l = 0; l < OpA::LOADS; ++l)
                        if (l * NM / OpA::LOADS == m && more) ga.issue_one(st, wave, l);
#pragma unroll
                    for (int f = 0; f < TM + TN; ++f)
                        if (f * NM / (TM + TN) == m) {
                            if (f < TM) fa[nxt][f] = read_a(nst, f, 0);
                            else fb[nxt][f - TM] = read_b(nst, f - TM, 0);
                        }
                    acc[i][j] = mfma_32x32x16(fa[cur][i], fb[cur][j], acc[i][j]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            if (more) ga.advance();
        };
        int kt = 0;
        for (; kt + STAGES < nfull; ++kt) slab(std::true_type(), kt);
        for (; kt < nk; ++kt) slab(std::false_type(), kt);
    } else {
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) {
            lds_char_t *st = smem + s * STAGE;
            if (s < nfull) {
                ga.issue(st, wave);
                gb.issue(st + OpA::BYTES, wave);
            } else if (s < nk) {
                slab_tail(st);
            }
        }
        int stage = 0;
        // FAST: slab kt + STAGES - 1 is whole
        auto slab = [&](auto fast_tag, int kt) {
            constexpr bool FAST = decltype(fast_tag)::value;
            if constexpr (FAST) wait_vmcnt<(STAGES - 2) * LOADS>();
            else wait_vmcnt<0>();
            __syncthreads();           // slab kt is there, and every wave is done with slab kt - 1
            const int ns = kt + STAGES - 1;
            lds_char_t *dst = smem + ((stage == 0 ? STAGES : stage) - 1) * STAGE;
            const bool more = FAST || ns < nfull;
            if constexpr (!FAST) {
                if (!more && ns < nk) slab_tail(dst);
            }
            const lds_char_t *sA = smem + stage * STAGE;
            const lds_char_t *sB = sA + OpA::BYTES;
            constexpr int C2 = BK / 8, TOTAL = C2 * 4 * NM;
#pragma unroll
            for (int c2 = 0; c2 < C2; ++c2) {
                f32x4 a[TM], b[TN];
#pragma unroll
                for (int i = 0; i < TM; ++i) a[i] = ga.frag4(sA, wm0 + 32 * i, c2, lane);
#pragma unroll
                for (int j = 0; j < TN; ++j) b[j] = gb.frag4(sB, wn0 + 32 * j, c2, lane);
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int j = 0; j < TN; ++j) {
                            const int m = ((c2 * 4 + e) * TM + i) * TN + j;
#pragma unroll
                            for (int l = 0; l < LOADS; ++l)
                                if (l * TOTAL / LOADS == m && more) {
                                    if (l < OpA::LOADS) ga.issue_one(dst, wave, l);
                                    else gb.issue_one(dst + OpA::BYTES, wave, l - OpA::LOADS);
                                }
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i][e], b[j][e], acc[i][j], 0, 0, 0);
                        }
            }
            if (more) {
                ga.advance();
                gb.advance();
            }
            stage = stage + 1 == STAGES ? 0 : stage + 1;
        };
        int kt = 0;
        for (; kt + STAGES - 1 < nfull; ++kt) slab(std::true_type(), kt);
        for (; kt < nk; ++kt) slab(std::false_type(), kt);
    }
    wait_vmcnt<0>();
    __syncthreads();                   // every wave is done with the ring
    layer_store<T>(p, t, smem + wave * kStripBytes<WN>, acc, t.m0 + wm0, t.n0 + wn0, lane);
}

}  // namespace dg
