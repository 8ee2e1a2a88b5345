// Products of a 16-bit matrix and an MX matrix whose blocks run along the
// output columns (the products of a backward pass):
//
//   C[m][n] = alpha * sum_k op(A)[m][k] * 2^(e[k][n / 32]) * b[k][n] + beta * C[m][n]
//
// A is fp16 or bf16, stored M x K or K x M; B is K x N in mxfp4, mxfp8 or
// mxint8.  The scale changes with k, the summed index, so the scaled matrix
// instruction (one scale per block of 32 k) does not apply; B is instead
// brought to A's type, where every value of the three formats is exact, and
// multiplied by v_mfma_f32_32x32x16 with fp32 sums.
//
// Per slab of 64 k: A goes to LDS by direct loads, in the layout of the dense
// kernels; B's codes are converted in registers, 16 bytes per thread and piece
// with one scale, and written to LDS as 16-bit elements once per workgroup (not
// once per wave that uses them).
//
// B's 16-bit buffer is [64 k][BN], rows of BN * 2 bytes: the 64-byte quad q
// (32 n) of row k sits at quad q ^ swz(k), and its 16-byte chunk c at chunk
// c ^ (k & 3).  The fragment reads (ds_read_b64_tr_b16, four rows of a quad per
// 16 lanes) see four distinct quads and have no bank conflicts.  The 16-byte
// writes have: they are served 8 lanes at a time over 128 bytes of banks, and
// those lanes' quads meet on each 16 bytes twice (8 conflict cycles a write; four
// times and 24 for mxfp4 on the 256-wide tile, whose 8 lanes hold one chunk number of
// 8 quads).  The counters agree to the cycle: 4096^3 on the 256 x 256 tile, 131072
// slabs of a wave with 4 writes each, 1.26e7 cycles with mxfp4 and 4.2e6 with mxfp8,
// and 5.2e5 of the epilogue's, of 3.1e7 and 2.2e7 that the LDS is at work.
//
// Measured: 4096^3 (mxfp4) 108 us, 1.26 PFLOP/s, the rate of a large bf16
// product of the library that ships with torch (1.24); 5632 x 2048 x 16384 (tn,
// mxint8) 354-362 us, 1.05 PFLOP/s on the 176 compute units that have a tile, mxfp8
// 335.  The matrix cores are busy at the clock they hold under load there.
// Smaller outputs are bound by LDS bytes: a 128 x 128 tile moves 106 KB a slab
// for a quarter of the work of the 256 x 256 tile's 256 KB, and converted
// elements go in at about 48 bytes a clock (conflicts and all).  Tried and left: B's codes through
// an LDS ring, more slabs deep (no faster at 512 x 2048 x 5632, slower at
// 2048^3); the 128 x 128 tile in two K groups of four waves (62 us against 68 in
// one range there, 185 against 134 at 4096^3); a 192 x 256 tile (335 us at the tn
// product's mxfp8, as the 256 x 256 one); four 128 x 128 waves (380 against 360).
#include "mx_tile.hpp"

namespace dg {

namespace {

constexpr int DQ_BK = 64;

// Values of T from codes and their block's scale.
template <typename T, int FB>
struct Decode {
    typedef T V8 __attribute__((ext_vector_type(8)));
    typedef T V2 __attribute__((ext_vector_type(2)));
    // eight elements: 4 bytes of codes (mxfp4) or 8
    static __device__ __forceinline__ V8 eight(uint32_t lo, uint32_t hi, float sc)
    {
        V2 r[4];
        if constexpr (FB == MX_FP4) {
            if constexpr (std::is_same<T, __bf16>::value) {
                r[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(lo, sc, 0);
                r[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(lo, sc, 1);
                r[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(lo, sc, 2);
                r[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(lo, sc, 3);
            } else {
                r[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(lo, sc, 0);
                r[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(lo, sc, 1);
                r[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(lo, sc, 2);
                r[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(lo, sc, 3);
            }
        } else if constexpr (FB == MX_FP8) {
            if constexpr (std::is_same<T, __bf16>::value) {
                r[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, sc, false);
                r[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, sc, true);
                r[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, sc, false);
                r[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, sc, true);
            } else {
                r[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, sc, false);
                r[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, sc, true);
                r[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, sc, false);
                r[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, sc, true);
            }
        } else {
            // the scale of one 64th; 2^-133 at the least, a subnormal
            const float s64 = sc * 0.015625f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int32_t c = (int32_t)((i < 4 ? lo : hi) << (24 - 8 * (i & 3))) >> 24;
                r[i >> 1][i & 1] = (T)((float)c * s64);
            }
        }
        return (V8){r[0][0], r[0][1], r[1][0], r[1][1], r[2][0], r[2][1], r[3][0], r[3][1]};
    }
};

// B: codes in registers, 16-bit elements in LDS.
template <typename T, int FB, int BN, int NW>
struct DqOperand {
    typedef T V8 __attribute__((ext_vector_type(8)));
    typedef __attribute__((address_space(3))) V8 lds_v8_t;
    static constexpr int ROW = BN * 2;                                  // LDS bytes per k
    static constexpr int BYTES = DQ_BK * ROW;
    static constexpr int EPP = FB == MX_FP4 ? 32 : 16;                  // elements of a 16-byte piece
    static constexpr int PIECES = BN / EPP;                             // pieces per k
    static constexpr int THREADS = NW * 64;
    static constexpr int PER = DQ_BK * PIECES / THREADS;                // pieces per thread
    static constexpr int CH = EPP / 8;                                  // 16-byte output chunks per piece
    static_assert(PER >= 1 && PER * THREADS == DQ_BK * PIECES, "whole pieces per thread");

    __device__ static __forceinline__ int swz(int k) { return BN >= 128 ? k & 3 : (k >> 1) & 1; }

    const uint8_t *q0, *s0;      // this thread's first piece and its scale, of the current slab
    int64_t ldq;
    int tid, lane;
    u32x4 raw[PER];
    uint32_t byte[PER];

    __device__ __forceinline__ void init(const MxGemmParams &p, int k_begin, int n0, int t)
    {
        tid = t;
        lane = t & 63;
        ldq = p.g.ldb;
        const int n = n0 + (t % PIECES) * EPP;
        const int64_t k = k_begin + t / PIECES;
        q0 = (const uint8_t *)p.g.B + k * ldq + (FB == MX_FP4 ? n / 2 : n);
        s0 = p.SB + ((int64_t)(n / MX_GROUP) * p.ldsb + k) * 8 + (n % MX_GROUP) / 32;
    }
    // piece i of the current slab; WHOLE: every k of the slab lies before K,
    // else rows at or past krem are zeros
    template <bool WHOLE>
    __device__ __forceinline__ void load(int i, int krem)
    {
        const int dk = i * (THREADS / PIECES);
        if (WHOLE || tid / PIECES + dk < krem) {
            raw[i] = *(const u32x4 *)(q0 + dk * ldq);
            byte[i] = s0[dk * 8];
        } else {
            raw[i] = (u32x4){0u, 0u, 0u, 0u};
            byte[i] = 127;
        }
    }
    __device__ __forceinline__ void advance()
    {
        q0 += DQ_BK * ldq;
        s0 += DQ_BK * 8;
    }
    // output chunk c of piece i into the buffer
    __device__ __forceinline__ void convert(lds_char_t *buf, int i, int c) const
    {
        const int k = tid / PIECES + i * (THREADS / PIECES), pc = tid % PIECES;
        const int quad = pc * EPP / 32, ch = FB == MX_FP4 ? c : 2 * (pc & 1) + c;
        const float sc = mx_scale(byte[i]);
        V8 v;
        if constexpr (FB == MX_FP4) v = Decode<T, FB>::eight(raw[i][c], 0, sc);
        else v = Decode<T, FB>::eight(raw[i][2 * c], raw[i][2 * c + 1], sc);
        *(lds_v8_t *)(buf + k * ROW + ((quad ^ swz(k)) << 6) + ((ch ^ (k & 3)) << 4)) = v;
    }
    // columns b0 .. b0+31, step kk of 16 k (the transposing read: in each
    // 16-lane group, lanes 4t .. 4t+3 name row t of a 4 x 16 block)
    __device__ __forceinline__ V8 frag(const lds_char_t *buf, int b0, int kk) const
    {
        const int g = lane >> 4, t = (lane & 15) >> 2, s = lane & 3;
        const int k0 = 16 * kk + 8 * (g >> 1) + t;
        const int ch = 2 * (g & 1) + (s >> 1);
        const lds_char_t *p0 = buf + k0 * ROW + (((b0 >> 5) ^ swz(t)) << 6) + ((ch ^ t) << 4) + (s & 1) * 8;
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)p0);
        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)(p0 + 4 * ROW));
        typedef short i16x8 __attribute__((ext_vector_type(8)));
        const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        return __builtin_bit_cast(V8, v);
    }
};

// A's slab in LDS, 16-byte pieces in the order of the direct loads: piece
// (i * NW + wave) * 64 + lane holds 8 elements that begin at (mn, k) = at(i).
//   k-contiguous (A stored M x K): the layout of the dense kernels, [BM][64]
//     with chunk c of row r at c ^ ((r >> 1) & 7);
//   m-contiguous (K x M): [64][BM], quad q of row k at q ^ swz(k) as in B's
//     buffer, any BM that is a multiple of 32.
template <typename T, int BM, bool KCONT, int NW>
struct DqA {
    typedef T V8 __attribute__((ext_vector_type(8)));
    typedef V8 __attribute__((aligned(2))) V8u;
    typedef __attribute__((address_space(3))) V8 lds_v8_t;
    static constexpr int BYTES = BM * DQ_BK * 2;
    static constexpr int LOADS = BYTES / (NW * 1024);
    static_assert(LOADS * NW * 1024 == BYTES, "whole loads");
    static constexpr int ROW = KCONT ? DQ_BK * 2 : BM * 2;
    const T *base;               // the current slab's tile origin
    int64_t ld;
    uint32_t off[LOADS];         // direct loads: byte offsets from base
    V8 r[LOADS];                 // through registers
    int mn0, ext, wave, lane;

    __device__ static __forceinline__ int swz(int k) { return BM % 128 == 0 ? k & 3 : BM % 64 == 0 ? (k >> 1) & 1 : 0; }

    __device__ __forceinline__ void at(int i, int &mn, int &k) const
    {
        const int id = (i * NW + wave) * 64 + lane;
        if constexpr (KCONT) {
            mn = id >> 3;
            k = ((id & 7) ^ ((mn >> 1) & 7)) * 8;
        } else {
            const int p = id % (ROW / 16);
            k = id / (ROW / 16);
            mn = ((p >> 2) ^ swz(k)) * 32 + (p & 3) * 8;
        }
    }
    // direct: a row (or piece) past the matrix is fetched from the last one; it
    // only feeds outputs that are never stored
    __device__ __forceinline__ void init(const T *g, int64_t l, int m0, int e, int w, int ln, bool direct)
    {
        ld = l;
        mn0 = m0;
        ext = e;
        wave = w;
        lane = ln;
        base = KCONT ? g + (int64_t)m0 * l : g + m0;
        if (!direct) return;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            int mn, k;
            at(i, mn, k);
            if constexpr (KCONT) {
                const int row = m0 + mn < e ? mn : e - 1 - m0;
                off[i] = (uint32_t)(((int64_t)row * l + k) * 2);
            } else {
                const int col = m0 + mn < e ? mn : e - 8 - m0;
                off[i] = (uint32_t)(((int64_t)k * l + col) * 2);
            }
        }
    }
    __device__ __forceinline__ void advance() { base += KCONT ? DQ_BK : DQ_BK * ld; }
    __device__ __forceinline__ void issue_one(lds_char_t *st, int i)
    {
        load_lds16(off[i], buffer_rsrc((const char *)base), (unsigned)(uintptr_t)(st + (i * NW + wave) * 1024));
    }
    // through registers, k at or past krem and rows past the matrix as zeros;
    // rows need be aligned to their elements only
    __device__ __forceinline__ void load(int krem)
    {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            int mn, k;
            at(i, mn, k);
            const T *src = base + (KCONT ? (int64_t)mn * ld + k : (int64_t)k * ld + mn);
            const int valid = KCONT ? (mn0 + mn < ext ? krem - k : 0) : (k < krem ? ext - mn0 - mn : 0);
            if (valid >= 8) {
                r[i] = *(const V8u *)src;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    T x = (T)0.f;
                    if (e < valid) x = src[e];
                    r[i][e] = x;
                }
            }
        }
    }
    __device__ __forceinline__ void store(lds_char_t *st) const
    {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) *(lds_v8_t *)(st + (i * NW + wave) * 1024 + lane * 16) = r[i];
    }
    // the same for a whole slab of a matrix of at least 8 m, without a branch
    // (which would wait for the loads): rows past the matrix come from its
    // last one; an m-contiguous piece that crosses the end is read from the
    // last 8 elements and moved to its place when it is stored
    __device__ __forceinline__ void load_whole()
    {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            int mn, k;
            at(i, mn, k);
            const int last = ext - mn0 - (KCONT ? 1 : 8);
            const int64_t m = mn < last ? mn : last;
            r[i] = *(const V8u *)(base + (KCONT ? m * ld + k : (int64_t)k * ld + m));
        }
    }
    __device__ __forceinline__ void store_whole(lds_char_t *st) const
    {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            V8 x = r[i];
            if constexpr (!KCONT) {
                int mn, k;
                at(i, mn, k);
                const int n = mn - (ext - mn0 - 8);      // elements to drop, when above 0
                u32x4 w = __builtin_bit_cast(u32x4, x);
                w = n > 0 && (n & 4) ? (u32x4){w[2], w[3], 0u, 0u} : w;
                w = n > 0 && (n & 2) ? (u32x4){w[1], w[2], w[3], 0u} : w;
                w = n > 0 && (n & 1) ? (u32x4){w[0] >> 16 | w[1] << 16, w[1] >> 16 | w[2] << 16, w[2] >> 16 | w[3] << 16, w[3] >> 16}
                                     : w;
                x = __builtin_bit_cast(V8, w);
            }
            *(lds_v8_t *)(st + (i * NW + wave) * 1024 + lane * 16) = x;
        }
    }
    // rows b0 .. b0+31, step kk of 16 k
    __device__ __forceinline__ V8 frag(const lds_char_t *st, int b0, int kk) const
    {
        if constexpr (KCONT) {
            const int row = b0 + (lane & 31), c = 2 * kk + (lane >> 5);
            return *(const lds_v8_t *)(st + row * ROW + ((c ^ ((row >> 1) & 7)) << 4));
        } else {
            const int g = lane >> 4, t = (lane & 15) >> 2, s = lane & 3;
            const int k0 = 16 * kk + 8 * (g >> 1) + t;
            const lds_char_t *p0 = st + k0 * ROW + (((b0 >> 5) ^ swz(t)) << 6) + (16 * (g & 1) + 4 * s) * 2;
            const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)p0);
            const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)(p0 + 4 * ROW));
            typedef short i16x8 __attribute__((ext_vector_type(8)));
            const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            return __builtin_bit_cast(V8, v);
        }
    }
};

// DIRECT: A by direct loads (4-byte aligned rows, an m-contiguous extent of
// whole 16-byte pieces), else through registers.
template <typename T, int FB, bool TA, bool DIRECT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN), 2) void dq_gemm_kernel(MxGemmParams p)
{
    constexpr int WAVES_N = BN / WN, NW = (BM / WM) * WAVES_N;
    constexpr int TM = WM / 32, TN = WN / 32, NM = TM * TN, KPW = DQ_BK / 16;
    typedef DqA<T, BM, !TA, NW> OpA;
    typedef DqOperand<T, FB, BN, NW> OpB;
    typedef T V8 __attribute__((ext_vector_type(8)));
    constexpr int B_AT = 2 * OpA::BYTES, RING = B_AT + 2 * OpB::BYTES, EPI = NW * kEpiBytes<WN>;
    constexpr int SMEM = RING > EPI ? RING : EPI;
    static_assert(SMEM <= 160 * 1024, "LDS");
    __shared__ __attribute__((aligned(1024))) char smem_raw[SMEM];
    lds_char_t *smem = (lds_char_t *)smem_raw;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm0 = (wave / WAVES_N) * WM, wn0 = (wave % WAVES_N) * WN;
    int bid, split, k_begin, Kl, tm, tn;
    split_of(p.g, bid, split, k_begin, Kl);
    tile_coords(bid, p.g, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int nk = (Kl + DQ_BK - 1) / DQ_BK, krem = Kl - (nk - 1) * DQ_BK;

    OpA ga;
    OpB gb;
    ga.init((const T *)p.g.A + (TA ? (int64_t)k_begin * p.g.lda : (int64_t)k_begin), p.g.lda, m0, p.g.M, wave, lane,
            DIRECT);
    gb.init(p, k_begin, n0, wave * 64 + lane);

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    auto a_at = [&](int s) { return smem + (s & 1) * OpA::BYTES; };
    auto b_at = [&](int s) { return smem + B_AT + (s & 1) * OpB::BYTES; };
    V8 fa[2][TM], fb[2][TN];
    auto frag = [&](int set, int s, int step, int f) {
        if (f < TM) fa[set][f] = ga.frag(a_at(s), wm0 + 32 * f, step);
        else fb[set][f - TM] = gb.frag(b_at(s), wn0 + 32 * (f - TM), step);
    };
    // A through registers without a branch: a whole slab, and 8 m at least
    auto whole = [&](int s) { return p.g.M >= 8 && (s < nk - 1 || krem == DQ_BK); };
    // a slab at once (the prologue and the end): A by direct loads into
    // its stage (a short last slab through registers), or into registers until
    // the slab is converted
    auto load = [&](int s) {
        const int rem = s == nk - 1 ? krem : DQ_BK;
        if (!DIRECT && whole(s)) {
            ga.load_whole();
        } else if (!DIRECT) {
            ga.load(rem);
        } else if (rem < DQ_BK) {
            ga.load(rem);
            ga.store(a_at(s));
        } else {
#pragma unroll
            for (int i = 0; i < OpA::LOADS; ++i) ga.issue_one(a_at(s), i);
        }
        ga.advance();
#pragma unroll
        for (int i = 0; i < OpB::PER; ++i) gb.template load<false>(i, rem);
        gb.advance();
    };
    auto convert = [&](int s) {
        if (!DIRECT && whole(s)) ga.store_whole(a_at(s));
        else if (!DIRECT) ga.store(a_at(s));
#pragma unroll
        for (int i = 0; i < OpB::PER; ++i)
#pragma unroll
            for (int c = 0; c < OpB::CH; ++c) gb.convert(b_at(s), i, c);
    };

    load(0);
    convert(0);
    if (nk > 1) load(1);
    wait_vmcnt<0>();
    __syncthreads();
#pragma unroll
    for (int f = 0; f < TM + TN; ++f) frag(0, 0, 0, f);

    // Slab kt.  Fragments are double-buffered per step of 16 k.  The barrier
    // sits before the last step: by then slab kt+1's A has landed and its B is
    // converted (during step 2, so that the loads have three steps to arrive);
    // the last step runs from registers while the first fragments of slab kt+1
    // are read and slab kt+2 is loaded.  FAST: slabs kt+1 and kt+2 exist and
    // are whole, so the conversion and the loads are spread between the matrix
    // instructions.
    auto slab = [&](auto fast_tag, int kt) {
        constexpr bool FAST = decltype(fast_tag)::value;
        constexpr int NC = OpB::PER * OpB::CH, cur = (KPW - 1) & 1;
#pragma unroll
        for (int s = 0; s + 1 < KPW; ++s)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const int m = i * TN + j;
#pragma unroll
                    for (int f = 0; f < TM + TN; ++f)
                        if (f * NM / (TM + TN) == m) frag((s & 1) ^ 1, kt, s + 1, f);
                    if (FAST && s == KPW - 2) {
                        if (!DIRECT && m == 0) ga.store_whole(a_at(kt + 1));
#pragma unroll
                        for (int c = 0; c < NC; ++c)
                            if (c * NM / NC == m) gb.convert(b_at(kt + 1), c / OpB::CH, c % OpB::CH);
                    }
                    acc[i][j] = mfma_32x32x16(fa[s & 1][i], fb[s & 1][j], acc[i][j]);
                    __builtin_amdgcn_sched_barrier(0);
                }
        if (!FAST && kt + 1 < nk) convert(kt + 1);
        wait_vmcnt<0>();
        __syncthreads();
        if (!FAST && kt + 2 < nk) load(kt + 2);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int m = i * TN + j;
                if constexpr (FAST) {
#pragma unroll
                    for (int l = 0; l < OpB::PER; ++l)
                        if (l * NM / OpB::PER == m) gb.template load<true>(l, DQ_BK);
                    if constexpr (DIRECT) {
#pragma unroll
                        for (int l = 0; l < OpA::LOADS; ++l)
                            if (l * NM / OpA::LOADS == m) ga.issue_one(a_at(kt), l);
                    } else {
                        if (m == 0) ga.load_whole();
                    }
                }
                // (after the last slab these reads fetch a stale stage, never used)
#pragma unroll
                for (int f = 0; f < TM + TN; ++f)
                    if (f * NM / (TM + TN) == m) frag(cur ^ 1, kt + 1, 0, f);
                acc[i][j] = mfma_32x32x16(fa[cur][i], fb[cur][j], acc[i][j]);
                __builtin_amdgcn_sched_barrier(0);
            }
        if constexpr (FAST) {
            ga.advance();
            gb.advance();
        }
    };
    int kt = 0;
    int nfast = (krem == DQ_BK ? nk : nk - 1) - 2;
    if (!DIRECT && !whole(0)) nfast = 0;
    for (; kt < nfast; ++kt) slab(std::true_type(), kt);
    for (; kt < nk; ++kt) slab(std::false_type(), kt);

    __syncthreads();  // every wave is done with the ring
    store_tile<TM, TN>(p, smem + wave * kEpiBytes<WN>, acc, m0 + wm0, n0 + wn0, lane, split);
}

template <typename T, int FB, bool TA, bool DIRECT, int BM, int BN, int WM, int WN>
hipError_t launch_dq(const MxGemmParams &p, hipStream_t s)
{
    const unsigned nwg = (unsigned)p.g.tiles_m * (unsigned)p.g.tiles_n * (unsigned)p.g.splits;
    MxGemmParams arg = p;
    void *args[] = {&arg};
    return hipLaunchKernel((const void *)&dq_gemm_kernel<T, FB, TA, DIRECT, BM, BN, WM, WN>, dim3(nwg),
                           dim3(64 * (BM / WM) * (BN / WN)), args, 0, s);
}

}  // namespace

// [config][format][transA][direct]
#define DG_DQ4(T, FB, ...)                                                                          \
    {{launch_dq<T, FB, false, false, __VA_ARGS__>, launch_dq<T, FB, false, true, __VA_ARGS__>},     \
     {launch_dq<T, FB, true, false, __VA_ARGS__>, launch_dq<T, FB, true, true, __VA_ARGS__>}}
// A through registers: not on the 256 x 256 tile, where it would spill
#define DG_DQ4D(T, FB, ...)                                                                         \
    {{nullptr, launch_dq<T, FB, false, true, __VA_ARGS__>}, {nullptr, launch_dq<T, FB, true, true, __VA_ARGS__>}}
#define DG_DQ12D(T, ...)                                                                            \
    {DG_DQ4D(T, MX_FP4, __VA_ARGS__), DG_DQ4D(T, MX_FP8, __VA_ARGS__), DG_DQ4D(T, MX_INT8, __VA_ARGS__)}
#define DG_DQ12(T, ...)                                                                             \
    {DG_DQ4(T, MX_FP4, __VA_ARGS__), DG_DQ4(T, MX_FP8, __VA_ARGS__), DG_DQ4(T, MX_INT8, __VA_ARGS__)}
template <typename T>
mx_launch_fn dq_launcher_of(int config, int format, int ta, int direct)
{
    static const mx_launch_fn table[][3][2][2] = {
        DG_DQ12(T, 32, 128, 32, 32),
        DG_DQ12(T, 64, 128, 32, 64),
        DG_DQ12(T, 128, 128, 64, 64),
        DG_DQ12D(T, 256, 256, 128, 64),
    };
    return table[config][format][ta][direct];
}

mx_launch_fn dq_gemm_launcher(int type, int config, int format, int ta, int direct)
{
    return type == ELEM_F16 ? dq_launcher_of<_Float16>(config, format, ta, direct)
                            : dq_launcher_of<__bf16>(config, format, ta, direct);
}

}  // namespace dg
