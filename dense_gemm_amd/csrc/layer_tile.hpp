// Tile kernels of a layer's products (see layer_common.hpp for what they compute):
//
//   forward, gradient   C[row][n] = epilogue(sum_k A[row][k] op(B_g)[k][n]), row in group g
//   weights             C_g[m][n] = epilogue(sum_r A[r][m] B[r][n]),         r over group g's rows
//
// One workgroup takes one BM x BN tile of one group and walks its sum in slabs.
// A group's last tile row and last slab end inside a tile: rows and columns past
// the end are fetched from valid places and never stored, summed indices past the
// end are zero.
#pragma once

#include <type_traits>

#include "gemm_pipe.hpp"
#include "layer_common.hpp"

namespace dg {

// ---- epilogue of a wave's blocks -----------------------------------------------
// Strips of SR rows x W columns (W = 32 * TN): the sums go to this wave's slot as fp32
// [SR][W], then a lane takes 8 columns of a row per pass, so that W / 8 lanes read
// and write a row's W columns in one piece.  The 16-byte chunk c of row r sits at c ^
// strip_swz(r): the chunks that 16 lanes read together lie on all banks.  What the epilogue
// reads beside the sums is fetched before the strip is staged.
template <int W, int SR> constexpr int kStripBytes = SR * W * 4;
template <int W> __device__ __forceinline__ int strip_swz(int r) { return W == 64 ? r & 1 : (r >> 1) & 1; }

template <typename TC, int SR, bool NT, int TM, int TN>
__device__ __forceinline__ void layer_store_as(const LayerParams &p, const LayerTile &t, lds_char_t *stg,
                                               const f32x16 (&acc)[TM][TN], int row0, int col0, int lane, bool partial)
{
    typedef __attribute__((address_space(3))) float lds_float_t;
    typedef __attribute__((address_space(3))) f32x4 lds_f32x4_t;
    constexpr int W = 32 * TN, LPR = W / 8, RPP = 64 / LPR, PASSES = SR / RPP, PER32 = 32 / SR;
    // passes fetched together: half of an fp32 strip's, for the registers
    constexpr int TOGETHER = sizeof(TC) == 4 && PASSES > 2 ? PASSES / 2 : PASSES;
    const int lc = (lane % LPR) * 8, col = col0 + lc;
    const bool whole = col0 + W <= p.N;
    float bias[8];
    if (!partial) layer_bias<TC, 8>(p, t.group, col < p.N ? col : 0, bias, col < p.N ? p.N - col : 0);
#pragma unroll 1
    for (int i = 0; i < TM * PER32; ++i) {
        const int top = row0 + SR * i, rows = t.rows - top;      // of this strip on
        // (opaque to the compiler, which would otherwise keep every pass's addresses
        // in registers from strip to strip)
        int lr0 = lane / LPR;
        asm volatile("" : "+v"(lr0));
        LayerAux<TC, 8> aux[TOGETHER];
        auto fetch = [&](int from) {
            if (whole && !partial) {
#pragma unroll
                for (int ps = 0; ps < TOGETHER; ++ps)
                    if (lr0 + (from + ps) * RPP < rows) aux[ps].fetch(p, t, top + lr0 + (from + ps) * RPP, col);
            }
        };
        fetch(0);
        // register r of lane l holds row 8*(r/4) + 4*(l/32) + r%4, column l%32
#pragma unroll
        for (int s = 0; s < TM * PER32; ++s)
            if (s == i) {
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int r = 0; r < SR / 2; ++r) {
                        const int row = 8 * (r >> 2) + (lane >> 5) * 4 + (r & 3);
                        *(lds_float_t *)(stg + (row * W + ((32 * j + (lane & 31)) ^ (strip_swz<W>(row) << 2))) * 4) =
                            acc[s / PER32][j][s % PER32 * (SR / 2) + r];
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
                    const f32x4 x = *(const lds_f32x4_t *)(stg + (lr * W + ((lc + 4 * c4) ^ (strip_swz<W>(lr) << 2))) * 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[4 * c4 + e] = x[e];
                }
                if (lr < rows) {
                    if (partial) layer_partial<8>(p, t, top + lr, col, v);
                    else layer_finish<TC, 8, NT>(p, t, top + lr, col, v, aux[ps % TOGETHER], bias);
                }
                __builtin_amdgcn_sched_barrier(0);    // a pass's registers at a time
            }
        } else {
            // the last columns: a pass at a time, the piece across the end one by one
#pragma unroll 1
            for (int lr = lr0; lr < SR; lr += RPP) {
                const int n = p.N - col;
                float v[8];
#pragma unroll
                for (int c4 = 0; c4 < 2; ++c4) {
                    const f32x4 x = *(const lds_f32x4_t *)(stg + (lr * W + ((lc + 4 * c4) ^ (strip_swz<W>(lr) << 2))) * 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[4 * c4 + e] = x[e];
                }
                if (lr >= rows || n <= 0) continue;
                if (partial) {
                    layer_partial<8>(p, t, top + lr, col, v, n);
                } else {
                    LayerAux<TC, 8> x;
                    x.fetch(p, t, top + lr, col, n);
                    layer_finish<TC, 8>(p, t, top + lr, col, v, x, bias, n);
                }
            }
        }
        __builtin_amdgcn_s_waitcnt(0xc07f);  // reads done before the slot is rewritten
        __builtin_amdgcn_wave_barrier();
    }
}

template <typename T, int SR, bool NT, int TM, int TN>
__device__ __forceinline__ void layer_store(const LayerParams &p, const LayerTile &t, lds_char_t *stg,
                                            const f32x16 (&acc)[TM][TN], int row0, int col0, int lane)
{
    if (p.splits > 1) layer_store_as<float, SR, false>(p, t, stg, acc, row0, col0, lane, true);
    else if (sizeof(T) == 4 || p.ctype == 0) layer_store_as<float, SR, false>(p, t, stg, acc, row0, col0, lane, false);
    else if (NT && p.past_caches) layer_store_as<T, SR, true>(p, t, stg, acc, row0, col0, lane, false);
    else layer_store_as<T, SR, false>(p, t, stg, acc, row0, col0, lane, false);
}

// ---- operands -------------------------------------------------------------------------
// A 16-bit operand's slab of 64 summed indices in LDS, as PipeOperandH lays out its own.
// KCONT (rows of 64): the 16-byte chunk c of row r sits at chunk c ^ swz(r), so that the
// 16 rows which a quarter wave reads together hit 16 distinct bank groups.  Else (64 rows
// of BMN): the 64-byte quad q of row k sits at q ^ swz(k), and fragments come from the
// transposing read.
template <typename T, int BMN, bool KCONT, int NW>
struct SlabOperandH {
    typedef T V8 __attribute__((ext_vector_type(8)));
    typedef __attribute__((address_space(3))) V8 lds_v8_t;
    static constexpr int BK = 64, BYTES = BMN * BK * 2, SPAN = 1024, LOADS = BYTES / (NW * SPAN);
    static constexpr int ROW_BYTES = KCONT ? BK * 2 : BMN * 2;
    static_assert(LOADS * NW * SPAN == BYTES, "whole loads");
    static_assert(KCONT || BMN == 64 || BMN % 128 == 0, "two quads, or four and more");

    const char *base;            // the current slab's tile origin (wave-uniform)
    uint32_t off[LOADS];         // a lane's byte offsets from it
    int64_t step;                // bytes from a slab to the next

    __device__ static __forceinline__ int swz(int r)
    {
        if constexpr (KCONT) return (r >> 1) & 7;
        else return BMN == 64 ? (r >> 1) & 1 : r & 3;
    }
    // row and first column of the piece at byte b of a stage
    __device__ static __forceinline__ void place(int b, int &r, int &c)
    {
        r = b / ROW_BYTES;
        const int p = (b % ROW_BYTES) >> 4;
        c = KCONT ? (p ^ swz(r)) * 8 : (((p >> 2) ^ swz(r)) << 5) + (p & 3) * 8;
    }
    __device__ __forceinline__ void issue_one(lds_char_t *lds, int wave, int i)
    {
        load_lds16(off[i], buffer_rsrc(base), (unsigned)(uintptr_t)(lds + (i * NW + wave) * SPAN));
    }
    // the operand of 32 rows from b0 on, for step kk of 16 summed indices
    __device__ __forceinline__ V8 frag(const lds_char_t *lds, int b0, int kk, int lane) const
    {
        if constexpr (KCONT) {
            const int r = b0 + (lane & 31);
            return *(const lds_v8_t *)(lds + r * ROW_BYTES + (((2 * kk + (lane >> 5)) ^ swz(r)) << 4));
        } else {
            const int g = lane >> 4, t = (lane & 15) >> 2, s = lane & 3;
            const int colb = (16 * (g & 1) + 4 * s) * 2, k0 = 16 * kk + 8 * (g >> 1) + t;
            const lds_char_t *p0 = lds + k0 * ROW_BYTES + (((b0 >> 5) ^ swz(k0)) << 6) + colb;
            const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)p0);
            const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)(p0 + 4 * ROW_BYTES));
            typedef short i16x8 __attribute__((ext_vector_type(8)));
            const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            return __builtin_bit_cast(V8, v);
        }
    }
};

// An fp32 operand's (PipeOperandS).
template <int BMN, bool KCONT, int NW, int BK_>
struct SlabOperandS : PipeOperandS<BMN, KCONT, NW, 16, BK_> {
    typedef PipeOperandS<BMN, KCONT, NW, 16, BK_> Base;
    __device__ static __forceinline__ void place(int b, int &r, int &c)
    {
        r = b / Base::ROW_BYTES;
        const int p = (b % Base::ROW_BYTES) >> 4;
        if constexpr (KCONT) {
            c = (p ^ Base::swz(r)) * 4;
        } else {
            r = Base::krow(r);
            c = (((p >> 3) ^ Base::hsw(r)) << 5) + (p & 7) * 4;
        }
    }
};

// An operand of any extents.  A piece of a row that is no whole number of pieces long
// reaches past the row's end, into the next row; the last slab, which has no next row,
// goes element by element (`tail`), as does a last slab of fewer summed indices than a
// slab has, and every slab of rows shorter than a piece.  What lies past a row's end
// only feeds outputs that are never stored.
//   REG = false: direct loads into LDS, of rows that are 4-byte aligned, 256 of which
//     lie within 32-bit byte offsets.
//   REG = true: any strides and alignment, through registers: fetch() loads a slab
//     (the GPU takes misaligned vectors), commit() writes it to its stage.
template <typename T, int BMN, bool KCONT, int NW, int BK_, bool REG>
struct LayerOperand : std::conditional<sizeof(T) == 2, SlabOperandH<T, BMN, KCONT, NW>,
                                       SlabOperandS<BMN, KCONT, NW, BK_>>::type {
    typedef typename std::conditional<sizeof(T) == 2, SlabOperandH<T, BMN, KCONT, NW>,
                                      SlabOperandS<BMN, KCONT, NW, BK_>>::type Base;
    static_assert(Base::BK == BK_, "16 bits: slabs of 64");
    static constexpr int PER = 16 / (int)sizeof(T);       // elements of a piece, which a lane loads
    typedef T V __attribute__((ext_vector_type(PER)));
    typedef V __attribute__((aligned(sizeof(T)))) Vu;
    typedef __attribute__((address_space(3))) V lds_v_t;
    int64_t row_step;                                     // bytes from a stored row to the next
    int64_t far[REG ? Base::LOADS : 1];
    V held[REG ? Base::LOADS : 1];

    __device__ __forceinline__ void init(const T *g, int64_t ld, int mn0, int ext, int wave, int lane)
    {
        this->base = (const char *)(KCONT ? g + (int64_t)mn0 * ld : g + mn0);
        row_step = ld * (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < Base::LOADS; ++i) {
            int r, c;
            Base::place((i * NW + wave) * Base::SPAN + lane * 16, r, c);
            if constexpr (KCONT) {
                if (mn0 + r >= ext) r = ext - 1 - mn0;
            } else {
                if (mn0 + c >= ext) c = ((ext - 1) / PER) * PER - mn0;
            }
            const int64_t at = ((int64_t)r * ld + c) * (int)sizeof(T);
            if constexpr (REG) far[i] = at;
            else this->off[i] = (uint32_t)at;
        }
        this->step = (KCONT ? Base::BK : Base::BK * ld) * (int)sizeof(T);
    }

    // the last slab is not whole, or not made of whole pieces
    __device__ static __forceinline__ bool ragged(int krem, int ext) { return krem < Base::BK || (!KCONT && ext % PER != 0); }
    __device__ static __forceinline__ bool narrow(int ext) { return !KCONT && ext < PER; }

    __device__ __forceinline__ void issue(lds_char_t *lds, int wave)
    {
        static_assert(!REG, "direct loads");
#pragma unroll
        for (int i = 0; i < Base::LOADS; ++i) this->issue_one(lds, wave, i);
    }
    __device__ __forceinline__ void fetch()
    {
        static_assert(REG, "loads into registers");
#pragma unroll
        for (int i = 0; i < Base::LOADS; ++i) held[i] = *(const Vu *)(this->base + far[i]);
    }
    __device__ __forceinline__ void commit(lds_char_t *lds, int wave, int lane) const
    {
#pragma unroll
        for (int i = 0; i < Base::LOADS; ++i) *(lds_v_t *)(lds + (i * NW + wave) * Base::SPAN + lane * 16) = held[i];
    }

    // a slab with krem summed indices left, straight to its stage: whole pieces first,
    // then those across an end
    __device__ __forceinline__ void tail(lds_char_t *lds, int wave, int lane, int krem, int mn0, int ext)
    {
        auto place_of = [&](int i, int &valid) {
            int r, c;
            Base::place((i * NW + wave) * Base::SPAN + lane * 16, r, c);
            if constexpr (KCONT) {
                valid = mn0 + r < ext ? krem - c : 0;
            } else {
                valid = r < krem ? ext - mn0 - c : 0;
            }
            return (const T *)(this->base + ((int64_t)r * row_step + (int64_t)c * (int)sizeof(T)));
        };
        V v[Base::LOADS];
        int valid;
#pragma unroll
        for (int i = 0; i < Base::LOADS; ++i) {
            const T *x = place_of(i, valid);
            v[i] = (V)(T)0.f;
            if (valid >= PER) v[i] = *(const Vu *)x;
        }
#pragma unroll
        for (int i = 0; i < Base::LOADS; ++i) {
            const T *x = place_of(i, valid);
            if (valid > 0 && valid < PER) {
#pragma unroll
                for (int e = 0; e < PER - 1; ++e)
                    if (e < valid) v[i][e] = x[e];
            }
            *(lds_v_t *)(lds + (i * NW + wave) * Base::SPAN + lane * 16) = v[i];
        }
    }

    // on to the next slab (without a branch, in which the compiler would merge the
    // two operands' and keep their addresses in memory)
    __device__ __forceinline__ void skip(bool on) { this->base += on ? this->step : 0; }
};

template <typename V8>
__device__ __forceinline__ float sum8(V8 x)
{
    return (((float)x[0] + (float)x[1]) + ((float)x[2] + (float)x[3])) +
           (((float)x[4] + (float)x[5]) + ((float)x[6] + (float)x[7]));
}

// BM x BN tile, waves of WM x WN, a ring of STAGES slabs of BK summed indices.
//
// 16 bits: fragments are double-buffered per step of 16 k.  The barrier of a slab sits
// before its last step, which runs from registers while the next slab's first
// fragments are read and the slab STAGES ahead is loaded into the stage just finished
// (A's loads there, B's during the following step), so that no fragment read waits at
// a barrier and loads and reads lie between MFMAs.  An operand through registers
// (RA, RB; two stages) is fetched in a slab's last step and written to its stage before
// the next slab's barrier.
// Two K groups (KG): each runs half of a slab's steps, so that a tile has twice the
// waves; their sums meet in LDS at the end.
// fp32: one barrier at a slab's start, the loads of slab kt + STAGES - 1 spread over its
// MFMAs (or fetched before them and written after them).
//
// Measured, and what bounds it (M x N x K, weights N x K, in a graph):
//   256 tile, bf16 16384 x 5632 x 2048 with gelu and Z: 368 us, 1.03 PFLOP/s, the matrix
//     cores busy 55% of the units' cycles, no bank conflicts.  Its 1408 tiles are 5.5 rounds,
//     each 44 us of products at the clock that the chip holds under them and 17 us of the first
//     slabs, gelu and 64 MB of outputs.  Grouped (8 uneven experts) 412, the gradient through
//     gelu 421, weight gradients 376; 8192^3 857 us, 1.28 PFLOP/s.
//   128 tile with two K groups, fp16 512 x 5632 x 2048 through gelu's gradient: 21.6 us; 176
//     tiles on 256 units, 11.7 us of them products.
//   64 tile, fp16 over 64 experts of 64 rows, A's odd rows through registers, weights 2040 x 1032
//     direct: 102 us for 287 MB, two slabs in flight (an operand through registers has two stages).
//   64 tile, fp32 511 x 1031 x 2047 in 3 ranges: 30 us (the matrix cores of units that hold two
//     of the 408 workgroups 20 us) and 5 of join.
template <typename T, int BM, int BN, int WM, int WN, int KG, bool DW, bool TB, int STAGES, int BK, bool RA, bool RB>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN) * KG, 2) void layer_pipe_kernel(LayerParams p)
{
    constexpr bool H = sizeof(T) == 2;
    constexpr int WAVES_N = BN / WN, NWG = (BM / WM) * WAVES_N, NW = NWG * KG, TM = WM / 32, TN = WN / 32, NM = TM * TN;
    static_assert(KG == 1 || (H && KG == 2 && TM % 2 == 0), "two K groups: 16 bits, an even number of strips");
    typedef LayerOperand<T, BM, !DW, NW, BK, RA> OpA;
    typedef LayerOperand<T, BN, TB && !DW, NW, BK, RB> OpB;
    static_assert(!(RA || RB) || STAGES == 2, "an operand through registers: two stages");
    // direct loads of a slab, by operand
    constexpr int LA = RA ? 0 : OpA::LOADS, LBN = RB ? 0 : OpB::LOADS, LOADS = LA + LBN, STAGE = OpA::BYTES + OpB::BYTES;
    constexpr int PA = LA ? LA : 1, PB = LBN ? LBN : 1, PL = LOADS ? LOADS : 1;     // divisors
    // The 256 tile's 16-bit outputs bypass the caches from 64 MB on (the host's rule): its
    // rounds of tiles end in 32 to 64 MB of them at once.  16384 x 5632 with gelu and Z,
    // K = 2048: 414 us, 387 so; a whole layer forward of 16384 rows 722 and 681, of 8192 353
    // and 344, of 4096 211 and 214; fp32 outputs 390 and 387, smaller tiles no difference.
    constexpr bool NT = BM == 256;
    constexpr int SR = 32, RING = STAGES * STAGE, STRIPS = NW * kStripBytes<WN, SR>, SMEM = RING > STRIPS ? RING : STRIPS;
    static_assert(SMEM <= 160 * 1024, "the ring and the strips fit the LDS");
    static_assert((STAGES - 2) * LOADS + LA < 64, "the loads in flight can be counted");
    __shared__ __attribute__((aligned(1024))) char smem_raw[SMEM];
    lds_char_t *smem = (lds_char_t *)smem_raw;

    LayerTile t;
    if (!layer_tile(p, BM, BN, blockIdx.x, t)) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kgroup = wave / NWG, wm0 = (wave % NWG / WAVES_N) * WM, wn0 = (wave % WAVES_N) * WN;
    OpA ga;
    OpB gb;
    const T *A = (const T *)p.A + (DW ? (t.row0 + t.k0) * p.lda : t.row0 * p.lda + t.k0);
    const T *B = (const T *)p.B + (DW ? (t.row0 + t.k0) * p.ldb
                                      : t.group * p.strideB + (TB ? (int64_t)t.k0 : t.k0 * p.ldb));
    const int nk = (t.k_len + BK - 1) / BK, krem = t.k_len - (nk - 1) * BK;
    int nfull = OpA::ragged(krem, t.rows) || OpB::ragged(krem, p.N) ? nk - 1 : nk;
    if (OpA::narrow(t.rows) || OpB::narrow(p.N)) nfull = 0;
    ga.init(A, p.lda, t.m0, t.rows, wave, lane);
    gb.init(B, p.ldb, t.n0, p.N, wave, lane);
    auto slab_tail = [&](lds_char_t *st, int slab) {
        const int left = slab == nk - 1 ? krem : BK;
        ga.tail(st, wave, lane, left, t.m0, t.rows);
        gb.tail(st + OpA::BYTES, wave, lane, left, t.n0, p.N);
    };

    f32x16 acc[TM][TN];
    float sums[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        sums[i] = 0.f;
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    }
    // weights: the first tile column adds up A's columns for the bias's gradient from
    // the fragments that it multiplies, each step in one of the waves that share them
    const bool summing = DW && p.dbias && t.n0 == 0;
    const int wcol = wave % WAVES_N;
    auto add_up = [&]() {
        // [wave][32 * strip + row]: added over the waves that share the rows, in order
        typedef __attribute__((address_space(3))) float lds_float_t;
        lds_float_t *red = (lds_float_t *)smem;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const float both = sums[i] + __shfl_xor(sums[i], 32);     // the lane halves' parts of the sum
            if (lane < 32) red[wave * WM + 32 * i + lane] = both;
        }
        __syncthreads();
        for (int m = threadIdx.x; m < BM; m += 64 * NW) {
            if (t.m0 + m >= p.M) break;
            float v = 0.f;
#pragma unroll
            for (int g = 0; g < KG; ++g)
#pragma unroll
                for (int c = 0; c < WAVES_N; ++c) v += red[(g * NWG + m / WM * WAVES_N + c) * WM + m % WM];
            layer_dbias(p, t.group, t.m0 + m, v);
        }
        __syncthreads();
    };

    if constexpr (H) {
        typedef T V8 __attribute__((ext_vector_type(8)));
        constexpr int KPW = BK / 16 / KG;
        const int kk0 = kgroup * KPW;
        static_assert(KPW % 2 == 0, "steps alternate between the two fragment sets");
        V8 fa[2][TM], fb[2][TN];
        auto read_a = [&](const lds_char_t *st, int i, int s) { return ga.frag(st, wm0 + 32 * i, kk0 + s, lane); };
        auto read_b = [&](const lds_char_t *st, int j, int s) { return gb.frag(st + OpA::BYTES, wn0 + 32 * j, kk0 + s, lane); };
        // the ring, but for B of its last stage, which the first step loads (and
        // for an operand through registers, which holds its second slab)
#pragma unroll
        for (int s = 0; s < STAGES; ++s) {
            lds_char_t *st = smem + s * STAGE;
            if (s < nfull) {
                if constexpr (RA) {
                    ga.fetch();
                    if (s == 0) ga.commit(st, wave, lane);
                } else {
                    ga.issue(st, wave);
                }
                if constexpr (RB) {
                    gb.fetch();
                    if (s == 0) gb.commit(st + OpA::BYTES, wave, lane);
                } else {
                    if (s < STAGES - 1) gb.issue(st + OpA::BYTES, wave);
                }
            } else if (s < nk) {
                slab_tail(st, s);
            }
            ga.skip(s < nk);
            if (RB || s < STAGES - 1) gb.skip(s < nk);
        }
        if (!(RA || RB) && nfull >= STAGES) wait_vmcnt<(STAGES - 2) * LOADS + LA>();
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
                if (DW && summing && s % WAVES_N == wcol) {
#pragma unroll
                    for (int i = 0; i < TM; ++i) sums[i] += sum8(fa[cur][i]);
                }
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        const int m = i * TN + j;
                        if (s == 0) {
#pragma unroll
                            for (int l = 0; l < LBN; ++l)
                                if (l * NM / PB == m && pend) gb.issue_one(prev + OpA::BYTES, wave, l);
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
                if (s == 0 && !RB) gb.skip(FAST || kt + STAGES - 1 < nk);
            }
            if constexpr (RA) {
                if (pend) ga.commit(prev, wave, lane);
            }
            if constexpr (RB) {
                if (pend) gb.commit(prev + OpA::BYTES, wave, lane);
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
                if (!more && kt + STAGES < nk) slab_tail(st, kt + STAGES);
            }
            if constexpr (RA) {
                if (more) ga.fetch();
            }
            if constexpr (RB) {
                if (more) gb.fetch();
            }
            constexpr int cur = (KPW - 1) & 1, nxt = cur ^ 1;
            if (DW && summing && (KPW - 1) % WAVES_N == wcol) {
#pragma unroll
                for (int i = 0; i < TM; ++i) sums[i] += sum8(fa[cur][i]);
            }
            // (after the last slab these reads fetch a stale stage, never used)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const int m = i * TN + j;
#pragma unroll
                    for (int l = 0; l < LA; ++l)
                        if (l * NM / PA == m && more) ga.issue_one(st, wave, l);
#pragma unroll
                    for (int f = 0; f < TM + TN; ++f)
                        if (f * NM / (TM + TN) == m) {
                            if (f < TM) fa[nxt][f] = read_a(nst, f, 0);
                            else fb[nxt][f - TM] = read_b(nst, f - TM, 0);
                        }
                    acc[i][j] = mfma_32x32x16(fa[cur][i], fb[cur][j], acc[i][j]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            ga.skip(FAST || kt + STAGES < nk);
            if (RB) gb.skip(FAST || kt + STAGES < nk);
        };
        int kt = 0;
        for (; kt + STAGES < nfull; ++kt) slab(std::true_type(), kt);
        for (; kt < nk; ++kt) slab(std::false_type(), kt);
    } else {
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) {
            lds_char_t *st = smem + s * STAGE;
            if (s < nfull) {
                if constexpr (RA) {
                    ga.fetch();
                    ga.commit(st, wave, lane);
                } else {
                    ga.issue(st, wave);
                }
                if constexpr (RB) {
                    gb.fetch();
                    gb.commit(st + OpA::BYTES, wave, lane);
                } else {
                    gb.issue(st + OpA::BYTES, wave);
                }
            } else if (s < nk) {
                slab_tail(st, s);
            }
            ga.skip(s < nk);
            gb.skip(s < nk);
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
                if (!more && ns < nk) slab_tail(dst, ns);
            }
            if constexpr (RA) {
                if (more) ga.fetch();
            }
            if constexpr (RB) {
                if (more) gb.fetch();
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
                if (DW && summing && c2 % WAVES_N == wcol) {
#pragma unroll
                    for (int i = 0; i < TM; ++i) sums[i] += (a[i][0] + a[i][1]) + (a[i][2] + a[i][3]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int j = 0; j < TN; ++j) {
                            const int m = ((c2 * 4 + e) * TM + i) * TN + j;
#pragma unroll
                            for (int l = 0; l < LOADS; ++l)
                                if (l * TOTAL / PL == m && more) {
                                    if (l < LA) ga.issue_one(dst, wave, l);
                                    else gb.issue_one(dst + OpA::BYTES, wave, l - LA);
                                }
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i][e], b[j][e], acc[i][j], 0, 0, 0);
                        }
            }
            if (more) {
                if constexpr (RA) ga.commit(dst, wave, lane);
                if constexpr (RB) gb.commit(dst + OpA::BYTES, wave, lane);
            }
            ga.skip(FAST || ns < nk);
            gb.skip(FAST || ns < nk);
            stage = stage + 1 == STAGES ? 0 : stage + 1;
        };
        // Every 1024 products the sums go to a second set.  A chain of K roundings of random terms is
        // off by about sqrt(K / 2) rounding errors (1.0e-6 by norm at K = 4000, 1.6e-6 at 8192), chains
        // of 1024 and their sums by 6e-7.  The 64 tile is 0 to 3% slower by it, the 128 tile no slower.
        constexpr int FOLD = 1024 / BK;
        f32x16 folded[TM][TN];
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) folded[i][j] = (f32x16)0.f;
        auto fold = [&]() {
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    folded[i][j] += acc[i][j];
                    acc[i][j] = (f32x16)0.f;
                }
        };
        // (a loop of its own for a chain: a test in every slab costs the 64 tile 15%)
        int kt = 0, end = FOLD;
        for (const int whole = nfull - STAGES + 1; kt < whole;) {
            for (const int stop = end < whole ? end : whole; kt < stop; ++kt) slab(std::true_type(), kt);
            if (kt == end) {
                fold();
                end += FOLD;
            }
        }
        for (; kt < nk; ++kt) {
            if (kt == end) {
                fold();
                end += FOLD;
            }
            slab(std::false_type(), kt);
        }
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] += folded[i][j];
    }
    wait_vmcnt<0>();
    __syncthreads();                   // every wave is done with the ring
    if (summing) add_up();
    if constexpr (KG == 1) {
        layer_store<T, SR, NT>(p, t, smem + wave * kStripBytes<WN, SR>, acc, t.m0 + wm0, t.n0 + wn0, lane);
    } else {
        // the two K groups' sums: each wave keeps half of the strips and hands the
        // other half to its partner, the same part of the tile in the other group
        constexpr int HS = TM / 2, SLOT = HS * TN * 4096;
        static_assert(NW * SLOT <= sizeof(smem_raw), "the exchange fits");
        f32x16 mine[HS][TN];
        lds_char_t *out = smem + wave * SLOT;
        const lds_char_t *in = smem + (wave + NWG) % NW * SLOT;
        typedef __attribute__((address_space(3))) f32x4 lds_f32x4_t;
#pragma unroll
        for (int i = 0; i < HS; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const f32x16 give = kgroup ? acc[i][j] : acc[HS + i][j];
                mine[i][j] = kgroup ? acc[HS + i][j] : acc[i][j];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *(lds_f32x4_t *)(out + ((i * TN + j) * 4 + c) * 1024 + lane * 16) =
                        (f32x4){give[4 * c], give[4 * c + 1], give[4 * c + 2], give[4 * c + 3]};
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < HS; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const f32x4 x = *(const lds_f32x4_t *)(in + ((i * TN + j) * 4 + c) * 1024 + lane * 16);
#pragma unroll
                    for (int e = 0; e < 4; ++e) mine[i][j][4 * c + e] += x[e];
                }
        __syncthreads();               // read before the strips are staged
        layer_store<T, SR, NT>(p, t, smem + wave * kStripBytes<WN, SR>, mine, t.m0 + wm0 + 32 * HS * kgroup, t.n0 + wn0, lane);
    }
}

}  // namespace dg
