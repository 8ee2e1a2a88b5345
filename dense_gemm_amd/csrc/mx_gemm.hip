// Products of two MX matrices on the scaled matrix cores of gfx950:
//
//   C = act(alpha * A B^T + beta * C + bias),
//   A[m][k] (mxfp4 or mxfp8) and B[n][k] (mxfp4), k contiguous and in blocks
//   of 32 with a power-of-two scale each:
//   C[m][n] = sum over blocks b of 2^(ea[m][b] + eb[n][b]) * sum_{k in b} a[m][k] b[n][k].
//
// v_mfma_scale_f32_32x32x64_f8f6f4 does a 32 x 32 block over 64 k, the two
// blocks' scales included: lane l holds row l%32, and the scale byte that a
// lane half h passes belongs to the h-th block of 32 k.  The elements:
//   mxfp4: lane half h holds the 32 k of block h (16 bytes, contiguous);
//   mxfp8: lane half h holds k 16h .. 16h+15 of block 0 and of block 1.
// The sum runs in fp32, except that the instruction adds 8 neighbouring k in
// fixed point first: with E the largest sum of exponents ea + eb among their 8
// products, every product is cut, towards zero, to a multiple of 2^(E - 13)
// (measured on gfx950, the same in both shapes).  A product of two mxfp4
// elements is always such a multiple, so nothing is lost.  mxfp8 times mxfp4
// loses up to 2^-13 of the 8 products' largest per product: 2.5e-6 of the
// result by norm on normal data, 1.4e-5 where a few columns of A are eight
// times the others.  Two instructions lose nothing: one on A's elements of 2 or
// more (exponents 1 .. 8, so products are multiples of 2^-3 with E <= 10) and one
// on the others (multiples of 2^-10 with E <= 2).  The row kernels, which wait for
// memory, always take both, and so do the tiled ones for an fp32 C (EXACT): 3e-8 by
// norm.  With a 16-bit C the tiled kernels take one, whose loss lies 15 times
// below an fp16 C's own rounding (120 times below a bf16 C's), for half the matrix
// cores' time: 4096^3 55 us against 100, 8192^3 389 against 735.
//
// Which k an instruction takes is free as long as A and B agree: with two
// mxfp4 operands a slab is 256 k and step kk takes blocks kk and 4 + kk, so
// that a lane half's four scale bytes are one word of the row's 8 (step kk
// selects byte kk), and its elements are 64 contiguous bytes of the row.
#include "mx_tile.hpp"

namespace dg {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) i32x4 lds_i32x4_t;
typedef __attribute__((address_space(3))) uint32_t lds_u32_t;

// A fragment: 4 registers of mxfp4, or 8 of mxfp8.
template <int F> struct Frag;
template <> struct Frag<MX_FP4> {
    i32x4 v;
    __device__ __forceinline__ i32x8 wide() const { return (i32x8){v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }
};
template <> struct Frag<MX_FP8> {
    i32x8 v;
    __device__ __forceinline__ i32x8 wide() const { return v; }
    // one part, zeros in place of the other's elements: those below 2, whose
    // code has its highest exponent bit clear (flip = 0), or the others and NaN
    // (flip = -1).  v_perm_b32's selectors 8 to 11 repeat the top bits of the
    // odd bytes, which the two shifts fill with that exponent bit.
    __device__ __forceinline__ i32x8 part(uint32_t flip) const
    {
        i32x8 o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t x = (uint32_t)v[i];
            const uint32_t large = __builtin_amdgcn_perm(x << 1, x << 9, 0x0b090a08u);
            o[i] = (int)(x & ~(large ^ flip));
        }
        return o;
    }
};

// the instruction's format field (a constant: the builtin takes no call)
template <int F> constexpr int kCode = F == MX_FP4 ? 4 : 0;

// One operand of the tiled kernel: BMN rows, ROWB bytes of k per slab (128,
// or 64), fetched by direct loads into [BMN][ROWB] bytes of LDS.  The 16-byte
// chunk c of row r sits at chunk c ^ swz(r), so that the 16 rows which a
// quarter wave reads together hit 16 distinct bank groups.
template <int BMN, int ROWB, int NW>
struct MxOperand {
    static constexpr int BYTES = BMN * ROWB;
    static constexpr int LOADS = BYTES / (NW * 1024);    // wave-wide 16-byte loads per wave and slab
    static constexpr int CH = ROWB / 16;
    static_assert(LOADS * NW * 1024 == BYTES, "whole loads");
    const char *base;
    uint32_t off[LOADS];

    __device__ static __forceinline__ int swz(int r) { return ROWB == 128 ? (r >> 1) & 7 : (r >> 2) & 3; }

    // rows past ext are fetched from the last row: they only feed outputs
    // that are never stored
    __device__ __forceinline__ void init(const uint8_t *q, int64_t ld, int mn0, int ext, int wave, int lane)
    {
        base = (const char *)(q + (int64_t)mn0 * ld);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int r = (i * NW + wave) * (1024 / ROWB) + lane / CH;
            const int c = (lane % CH) ^ swz(r);
            const int row = mn0 + r < ext ? r : ext - 1 - mn0;
            off[i] = (uint32_t)((int64_t)row * ld + c * 16);
        }
    }
    __device__ __forceinline__ void issue_one(lds_char_t *st, int wave, int i)
    {
        load_lds16(off[i], buffer_rsrc(base), (unsigned)(uintptr_t)(st + (i * NW + wave) * 1024));
    }
    __device__ __forceinline__ void advance() { base += ROWB; }
    __device__ static __forceinline__ i32x4 chunk(const lds_char_t *st, int r, int c)
    {
        return *(const lds_i32x4_t *)(st + r * ROWB + ((c ^ swz(r)) << 4));
    }
};

// The scales of both operands' rows for one slab: DW words per row (2 for a
// slab of 256 k, 1 for 128), [BM][DW] then [BN][DW] words of LDS, by 4-byte
// direct loads (a row's 8 bytes of a group lie 8-byte aligned only).
template <int BM, int BN, int DW, int NW>
struct MxScales {
    static constexpr int BYTES = (BM + BN) * DW * 4;
    static constexpr int TOTAL = BYTES / 256;                       // wave-wide loads per slab
    static constexpr int LOADS = TOTAL < NW ? 1 : TOTAL / NW;       // per wave (fewer loads than waves: some twice)
    static_assert(TOTAL >= NW ? LOADS * NW == TOTAL : NW % TOTAL == 0, "whole loads");
    static_assert((BM * DW) % 64 == 0 && (BN * DW) % 64 == 0, "a load serves one operand");
    const char *base[LOADS];
    int64_t step[LOADS];       // bytes per group
    uint32_t off[LOADS];
    int odd;                   // DW = 1: the slab is the group's second half

    __device__ __forceinline__ void init(const MxGemmParams &p, int m0, int n0, int wave, int lane)
    {
        odd = 0;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int t = (i * NW + wave) % TOTAL;
            const bool isb = t >= BM * DW / 64;
            const int d = (isb ? t - BM * DW / 64 : t) * 64 + lane;
            const int mn0 = isb ? n0 : m0, ext = isb ? p.g.N : p.g.M;
            const int r = d / DW;
            const int row = mn0 + r < ext ? r : ext - 1 - mn0;
            base[i] = (const char *)((isb ? p.SB : p.SA) + (int64_t)mn0 * 8);
            step[i] = (isb ? p.ldsb : p.ldsa) * 8;
            off[i] = (uint32_t)(row * 8 + (d % DW) * 4);
        }
    }
    __device__ __forceinline__ void issue_one(lds_char_t *st, int wave, int i)
    {
        const int t = (i * NW + wave) % TOTAL;
        load_lds4(off[i], buffer_rsrc(base[i]), (unsigned)(uintptr_t)(st + t * 256));
    }
    __device__ __forceinline__ void advance()
    {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            if constexpr (DW == 2) base[i] += step[i];
            else base[i] += odd ? step[i] - 4 : 4;
        }
        if constexpr (DW == 1) odd ^= 1;
    }
};

// The tiled kernel.  BM x BN tile, waves of WM x WN, a ring of STAGES slabs
// in LDS filled by direct loads.  Fragments are double-buffered per step of 64
// k; the barrier of a slab sits before its last step, which runs from
// registers while the next slab's first fragments and scales are read and the
// slab STAGES ahead is loaded into the stage just finished (A's loads there,
// B's and the scales' during the following step).
//
// Two mxfp4 operands move as many LDS bytes per matrix instruction as the
// dense 16-bit kernels (an instruction takes 16 bytes a lane and lasts as
// long), so the tiles are theirs, for four times the work: 8192^3 mxfp4 in 252
// us (4.4 PFLOP/s, 88% of four times the 1.24 PFLOP/s that a large bf16 product
// reaches), mxfp8 times mxfp4 in 385 us (2.9 PFLOP/s: the instruction takes
// twice as long).  256 x 256: eight 128 x 64 waves; four 128 x 128 ones, a
// quarter fewer LDS reads, took 268 us.  What bounds it is the matrix cores at
// the clock that they hold under this load.  128 x 128 (two workgroups a
// unit) and 64 x 64 (two, three with mxfp8) serve outputs with fewer tiles than units, where a
// slab's latency counts: 0.23 us a slab of the 64 x 64 tile, 0.36 of the
// 128 x 128 one.
template <int FA, bool EXACT, int BM, int BN, int WM, int WN, int STAGES>
__global__ __launch_bounds__(64 * (BM / WM) * (BN / WN), 2) void mx_gemm_kernel(MxGemmParams p)
{
    constexpr int WAVES_N = BN / WN, NW = (BM / WM) * WAVES_N;
    constexpr int TM = WM / 32, TN = WN / 32, NM = TM * TN;
    constexpr bool BOTH4 = FA == MX_FP4;
    constexpr int BK = BOTH4 ? 256 : 128, KPW = BK / 64, DW = BK / 128;
    typedef MxOperand<BM, 128, NW> OpA;
    typedef MxOperand<BN, BOTH4 ? 128 : 64, NW> OpB;
    typedef MxScales<BM, BN, DW, NW> Sc;
    constexpr int LOADS = OpA::LOADS + OpB::LOADS + Sc::LOADS;
    constexpr int STAGE = OpA::BYTES + OpB::BYTES + Sc::BYTES;
    constexpr int SMEM = STAGES * STAGE;
    static_assert(NW * kEpiBytes<WN> <= SMEM, "the staged strips fit the ring");
    static_assert(SMEM <= 160 * 1024, "the ring fits the LDS");
    __shared__ __attribute__((aligned(1024))) char smem_raw[SMEM];
    lds_char_t *smem = (lds_char_t *)smem_raw;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, l32 = lane & 31;
    const int wm0 = (wave / WAVES_N) * WM, wn0 = (wave % WAVES_N) * WN;
    int tm, tn;
    tile_coords(blockIdx.x, p.g, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int nk = p.g.K / BK;               // K is a whole number of groups

    OpA ga;
    OpB gb;
    Sc gs;
    ga.init((const uint8_t *)p.g.A, p.g.lda, m0, p.g.M, wave, lane);
    gb.init((const uint8_t *)p.g.B, p.g.ldb, n0, p.g.N, wave, lane);
    gs.init(p, m0, n0, wave, lane);

    typedef Frag<FA> FragA;
    typedef Frag<MX_FP4> FragB;
    FragA fa[2][TM];
    FragB fb[2][TN];
    uint32_t sa[TM], sb[TN];
    auto read_a = [&](const lds_char_t *st, int i, int s) {
        FragA f;
        const int r = wm0 + 32 * i + l32;
        if constexpr (BOTH4) {
            f.v = OpA::chunk(st, r, half * 4 + s);
        } else {
            const i32x4 lo = OpA::chunk(st, r, 4 * s + half), hi = OpA::chunk(st, r, 4 * s + 2 + half);
            f.v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
        return f;
    };
    auto read_b = [&](const lds_char_t *st, int j, int s) {
        FragB f;
        f.v = OpB::chunk(st + OpA::BYTES, wn0 + 32 * j + l32, BOTH4 ? half * 4 + s : 2 * s + half);
        return f;
    };
    // this lane half's scale bytes of a row: byte s (BOTH4) or 2s serves step s
    auto read_s = [&](const lds_char_t *st, int row) -> uint32_t {
        const lds_char_t *q = st + OpA::BYTES + OpB::BYTES;
        if constexpr (BOTH4) return *(const lds_u32_t *)(q + (row * 2 + half) * 4);
        else return *(const lds_u32_t *)(q + row * 4) >> (8 * half);
    };
    auto issue_a = [&](lds_char_t *st, int i) { ga.issue_one(st, wave, i); };
    auto issue_bs = [&](lds_char_t *st, int i) {
        if (i < OpB::LOADS) gb.issue_one(st + OpA::BYTES, wave, i);
        else gs.issue_one(st + OpA::BYTES + OpB::BYTES, wave, i - OpB::LOADS);
    };
    constexpr int BSL = OpB::LOADS + Sc::LOADS;

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    // prologue: the ring, except B and the scales of its last stage, which the
    // first step issues (as every step does for the slab STAGES - 1 ahead)
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
        if (s < nk) {
            lds_char_t *st = smem + s * STAGE;
#pragma unroll
            for (int i = 0; i < OpA::LOADS; ++i) issue_a(st, i);
            ga.advance();
            if (s < STAGES - 1) {
#pragma unroll
                for (int i = 0; i < BSL; ++i) issue_bs(st, i);
                gb.advance();
                gs.advance();
            }
        }
    }
    if (nk >= STAGES) wait_vmcnt<(STAGES - 2) * LOADS + OpA::LOADS>();
    else wait_vmcnt<0>();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        fa[0][i] = read_a(smem, i, 0);
        sa[i] = read_s(smem, wm0 + 32 * i + l32);
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        fb[0][j] = read_b(smem, j, 0);
        sb[j] = read_s(smem, BM + wn0 + 32 * j + l32);
    }

    // one step of 64 k from fragment set s & 1: MFMA m after what `before(m)`
    // does (the order pinned, so that reads and loads sit between the MFMAs)
    auto mfmas = [&](auto step_tag, auto before) {
        constexpr int s = decltype(step_tag)::value, SEL = BOTH4 ? s : 2 * s;
        auto one = [&](i32x8 a, int i, int j) {
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, fb[s & 1][j].wide(), acc[i][j], kCode<FA>,
                                                                        kCode<MX_FP4>, SEL, (int)sa[i], SEL, (int)sb[j]);
            __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            if constexpr (EXACT) {
                const i32x8 small = fa[s & 1][i].part(0);
#pragma unroll
                for (int j = 0; j < TN; ++j) one(small, i, j);
                fa[s & 1][i].v ^= small;
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                before(i * TN + j);
                one(fa[s & 1][i].wide(), i, j);
            }
        }
    };

    int stage = 0;
    // slab kt.  PEND: B and the scales of slab kt + STAGES - 1 are to be
    // loaded (A's loads went out in the step before); MORE: slab kt + STAGES
    // exists
    auto slab = [&](auto pend_tag, auto more_tag) {
        constexpr bool PEND = decltype(pend_tag)::value, MORE = decltype(more_tag)::value;
        lds_char_t *st = smem + stage * STAGE;
        lds_char_t *prev = smem + (stage == 0 ? STAGES - 1 : stage - 1) * STAGE;
        auto inner = [&](auto s_tag) {
            constexpr int s = decltype(s_tag)::value, nxt = (s & 1) ^ 1;
            mfmas(s_tag, [&](int m) {
                if constexpr (s == 0 && PEND) {
#pragma unroll
                    for (int l = 0; l < BSL; ++l)
                        if (l * NM / BSL == m) issue_bs(prev, l);
                }
#pragma unroll
                for (int f = 0; f < TM + TN; ++f)
                    if (f * NM / (TM + TN) == m) {
                        if (f < TM) fa[nxt][f] = read_a(st, f, s + 1);
                        else fb[nxt][f - TM] = read_b(st, f - TM, s + 1);
                    }
            });
            if constexpr (s == 0 && PEND) {
                gb.advance();
                gs.advance();
            }
        };
        inner(std::integral_constant<int, 0>());
        if constexpr (KPW == 4) {
            inner(std::integral_constant<int, 1>());
            inner(std::integral_constant<int, 2>());
        }
        // slab kt + 1 has landed in every wave's part, and every wave holds its
        // last fragments of slab kt
        if constexpr (PEND) wait_vmcnt<(STAGES - 2) * LOADS>();
        else wait_vmcnt<0>();
        __syncthreads();
        stage = stage + 1 == STAGES ? 0 : stage + 1;
        const lds_char_t *nst = smem + stage * STAGE;
        constexpr int nxt = KPW & 1;
        uint32_t na[TM], nb[TN];
        // (after the last slab these reads fetch a stale stage, never used)
        mfmas(std::integral_constant<int, KPW - 1>(), [&](int m) {
            if constexpr (MORE) {
#pragma unroll
                for (int l = 0; l < OpA::LOADS; ++l)
                    if (l * NM / OpA::LOADS == m) issue_a(st, l);
            }
#pragma unroll
            for (int f = 0; f < TM + TN; ++f)
                if (f * NM / (TM + TN) == m) {
                    if (f < TM) {
                        fa[nxt][f] = read_a(nst, f, 0);
                        na[f] = read_s(nst, wm0 + 32 * f + l32);
                    } else {
                        fb[nxt][f - TM] = read_b(nst, f - TM, 0);
                        nb[f - TM] = read_s(nst, BM + wn0 + 32 * (f - TM) + l32);
                    }
                }
        });
        if constexpr (MORE) ga.advance();
#pragma unroll
        for (int i = 0; i < TM; ++i) sa[i] = na[i];
#pragma unroll
        for (int j = 0; j < TN; ++j) sb[j] = nb[j];
    };
    int kt = 0;
    for (; kt + STAGES < nk; ++kt) slab(std::true_type(), std::true_type());
    if (kt + STAGES == nk) {
        slab(std::true_type(), std::false_type());
        ++kt;
    }
    for (; kt < nk; ++kt) slab(std::false_type(), std::false_type());

    __syncthreads();  // every wave is done with the ring
    lds_char_t *stg = smem + wave * kEpiBytes<WN>;
    store_tile<TM, TN>(p, stg, acc, m0 + wm0, n0 + wn0, lane, 0);
}

// Few rows of A (single tokens): bound by reading B once.  A workgroup takes
// 16 rows of B and 16 * MT rows of A; its 8 waves split K by groups of 256 and
// their sums meet in LDS in wave order.  B is the instruction's row operand,
// so a lane ends with 4 consecutive columns of C.  Everything comes straight
// from global memory in fragment order (16 bytes a lane; 64 contiguous bytes
// of a row per instruction, both halves of a line in one group), with 64-bit
// addresses, so any row stride will do.  One token: 5632 x 2048 in 3.9 us (6.3
// MB; the launch and one round trip to memory), 8192 x 8192 in 9.1 us (3.9
// TB/s); 16 rows 5.1 and 14.6 us, where A's rows, read again by every
// workgroup, add to it.
//
// mxfp8: both parts of A (see the top) go through the instruction.  PAIR, for 8
// rows at most: they share one, the elements of 2 or more in the odd operand
// rows and the others in the even ones, side by side so that the two lanes'
// loads are one (8 x 8192 x 8192 10.8 us; two instructions 12.4).
template <int FA, int MT, bool PAIR>
__global__ __launch_bounds__(512) void mx_skinny_kernel(MxGemmParams p)
{
    static_assert(!PAIR || (FA == MX_FP8 && MT == 1), "PAIR: the parts of 8 rows of mxfp8");
    constexpr int NWV = 8;
    __shared__ float red[NWV][MT][256];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
    const int groups = p.g.K / MX_GROUP;
    const int64_t brow = n0 + r < p.g.N ? n0 + r : p.g.N - 1;
    const uint8_t *B = (const uint8_t *)p.g.B + brow * p.g.ldb + q * 16;
    const uint8_t *SB = p.SB + brow * 8;
    const uint8_t *A[MT], *SA[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int64_t ar = m0 + 16 * t + (PAIR ? r >> 1 : r), arow = ar < p.g.M ? ar : p.g.M - 1;
        A[t] = (const uint8_t *)p.g.A + arow * p.g.lda + q * 16;
        SA[t] = p.SA + arow * 8;
    }
    f32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    // U of the wave's groups at a time, all loads first (twice as many take more
    // than 128 registers, and fewer workgroups fit a unit: 5632 x 2048 4.7 us
    // against 3.9, 8192 x 8192 10.8 against 9.1)
    constexpr int U = MT == 1 ? 2 : 1;
    for (int g0 = wave; g0 < groups; g0 += NWV * U) {
        Frag<MX_FP4> b[U][2];
        Frag<FA> a[U][MT][2];
        uint64_t ub[U], ua[U][MT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t g = g0 + u * NWV;
            if (g >= groups) break;
            ub[u] = *(const uint64_t *)(SB + g * p.ldsb * 8);
#pragma unroll
            for (int s = 0; s < 2; ++s) b[u][s].v = *(const i32x4 *)(B + g * 128 + s * 64);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                ua[u][t] = *(const uint64_t *)(SA[t] + g * p.ldsa * 8);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if constexpr (FA == MX_FP4) {
                        a[u][t][s].v = *(const i32x4 *)(A[t] + g * 128 + s * 64);
                    } else {
                        const i32x4 lo = *(const i32x4 *)(A[t] + g * 256 + s * 128);
                        const i32x4 hi = *(const i32x4 *)(A[t] + g * 256 + s * 128 + 64);
                        a[u][t][s].v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                    }
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);    // the loads stay ahead of the sums
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (g0 + u * NWV >= groups) break;
            // byte q of each word to the front: steps 0 and 1 take blocks q and 4 + q
            const uint64_t sb = ub[u] >> (8 * q);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const uint64_t sa = ua[u][t] >> (8 * q);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    i32x8 x = a[u][t][s].wide();
                    if constexpr (PAIR) {
                        x = a[u][t][s].part(0u - (uint32_t)(r & 1));
                    } else if constexpr (FA == MX_FP8) {
                        const i32x8 small = a[u][t][s].part(0);
                        acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            b[u][s].wide(), small, acc[t], kCode<MX_FP4>, kCode<FA>, 0, (int)(uint32_t)(sb >> (32 * s)),
                            0, (int)(uint32_t)(sa >> (32 * s)));
                        x ^= small;
                    }
                    acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        b[u][s].wide(), x, acc[t], kCode<MX_FP4>, kCode<FA>, 0, (int)(uint32_t)(sb >> (32 * s)), 0,
                        (int)(uint32_t)(sa >> (32 * s)));
                }
            }
        }
    }
    // register e of lane l: row (of B) 4 * (l / 16) + e, column (of A) l % 16
#pragma unroll
    for (int t = 0; t < MT; ++t) *(f32x4 *)&red[wave][t][lane * 4] = acc[t];
    __syncthreads();
    for (int o = threadIdx.x; o < (PAIR ? 128 : MT * 256); o += 512) {
        const int n = o & 15, m = o >> 4;
        const int at = ((n >> 2) * 16 + (PAIR ? 2 * m : m & 15)) * 4 + (n & 3);
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < NWV; ++w) v += red[w][m >> 4][at];
        if constexpr (PAIR) {
#pragma unroll
            for (int w = 0; w < NWV; ++w) v += red[w][0][at + 4];    // the other part
        }
        const int64_t gm = m0 + m;
        const int gn = (int)(n0 + n);
        if (gm >= p.g.M || n0 + n >= p.g.N) continue;
        const int64_t c = gm * p.g.ldc + gn;
        if (p.ctype == ELEM_F32) {
            float *C = (float *)p.g.C;
            C[c] = epilogue_value<float>(p.g, v, p.g.beta != 0.f ? C[c] : 0.f, gn);
        } else if (p.ctype == ELEM_F16) {
            _Float16 *C = (_Float16 *)p.g.C;
            C[c] = (_Float16)epilogue_value<_Float16>(p.g, v, p.g.beta != 0.f ? (float)C[c] : 0.f, gn);
        } else {
            __bf16 *C = (__bf16 *)p.g.C;
            C[c] = (__bf16)epilogue_value<__bf16>(p.g, v, p.g.beta != 0.f ? (float)C[c] : 0.f, gn);
        }
    }
}

template <int FA, bool EXACT, int BM, int BN, int WM, int WN, int STAGES>
hipError_t launch_tile(const MxGemmParams &p, hipStream_t s)
{
    MxGemmParams arg = p;
    void *args[] = {&arg};
    return hipLaunchKernel((const void *)&mx_gemm_kernel<FA, EXACT, BM, BN, WM, WN, STAGES>,
                           dim3((unsigned)p.g.tiles_m * (unsigned)p.g.tiles_n), dim3(64 * (BM / WM) * (BN / WN)), args, 0,
                           s);
}

template <int FA, int MT>
hipError_t launch_skinny(const MxGemmParams &p, hipStream_t s)
{
    MxGemmParams arg = p;
    void *args[] = {&arg};
    const void *f = (const void *)&mx_skinny_kernel<FA, MT, false>;
    if constexpr (FA == MX_FP8 && MT == 1)
        if (p.g.M <= 8) f = (const void *)&mx_skinny_kernel<FA, MT, true>;
    return hipLaunchKernel(f, dim3((unsigned)p.g.tiles_n, (unsigned)p.g.tiles_m),
                           dim3(512), args, 0, s);
}

}  // namespace

// [config][mxfp4, mxfp8, mxfp8 without loss]
#define DG_MX_TILE(BM, BN, WM, WN, S4, S8)                                                       \
    {launch_tile<MX_FP4, false, BM, BN, WM, WN, S4>, launch_tile<MX_FP8, false, BM, BN, WM, WN, S8>, \
     launch_tile<MX_FP8, true, BM, BN, WM, WN, S8>}
mx_launch_fn mx_gemm_launcher(int config, int format_a, bool exact)
{
    static const mx_launch_fn table[][3] = {
        {launch_skinny<MX_FP4, 1>, launch_skinny<MX_FP8, 1>, launch_skinny<MX_FP8, 1>},
        {launch_skinny<MX_FP4, 2>, launch_skinny<MX_FP8, 2>, launch_skinny<MX_FP8, 2>},
        DG_MX_TILE(64, 64, 32, 32, 4, 4),
        DG_MX_TILE(128, 128, 64, 64, 2, 3),
        DG_MX_TILE(256, 256, 128, 64, 2, 2),
    };
    return table[config][format_a == MX_FP8 ? 1 + exact : 0];
}

}  // namespace dg
