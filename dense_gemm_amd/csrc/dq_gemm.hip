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
// Per slab of 64 k, with everything fetched by direct global->LDS loads two
// slabs ahead: A in the layout of the dense kernels, B and its scales as
// stored (8 bytes of scales per k).  Each thread then takes 16 bytes of B
// from LDS, converts them (one scale for all of them) and writes 16-bit
// elements into a second buffer, once per workgroup and slab rather than
// once per wave, while the previous slab's matrix instructions run.
//
// B's 16-bit buffer is [64 k][128 n], rows of 256 bytes: the 64-byte quad q
// (32 n) of row k sits at quad q ^ (k & 3), and its 16-byte chunk c at chunk
// c ^ (k & 3).  The fragment reads (ds_read_b64_tr_b16, four rows of a quad per
// 16 lanes) see four distinct quads, and the 16 lanes of a write, which hold
// the same chunk number of two or four rows, 16 distinct chunks.
#include "mx_tile.hpp"

namespace dg {

namespace {

constexpr int DQ_BK = 64, DQ_BN = 128;

// Two 16-bit values of T from the low or high half of codes q.
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

// B's raw ring slot and 16-bit buffer.
template <typename T, int FB, int NW>
struct DqOperand {
    typedef T V8 __attribute__((ext_vector_type(8)));
    typedef __attribute__((address_space(3))) V8 lds_v8_t;
    typedef __attribute__((address_space(3))) u32x4 lds_u32x4_t;
    typedef __attribute__((address_space(3))) uint8_t lds_u8_t;
    static constexpr int RROW = FB == MX_FP4 ? DQ_BN / 2 : DQ_BN;      // raw bytes per k
    static constexpr int PIECES = RROW / 16;                            // 16-byte pieces per k
    static constexpr int RAW = DQ_BK * RROW;
    static constexpr int RAW_BYTES = RAW + DQ_BK * 8;                   // and the scales
    static constexpr int BYTES = DQ_BK * DQ_BN * 2;
    static constexpr int RTOT = RAW / 1024;                             // wave-wide loads
    static constexpr int RLOADS = RTOT < NW ? 1 : RTOT / NW;            // per wave (some twice)
    static constexpr int LOADS = RLOADS + 1;
    static constexpr int THREADS = NW * 64;
    static constexpr int PER = (DQ_BK * PIECES + THREADS - 1) / THREADS;   // pieces per thread
    const char *base, *sbase;
    int64_t ldq;
    uint32_t off[RLOADS], soff;
    int wave, lane;

    __device__ __forceinline__ void init(const MxGemmParams &p, int k_begin, int n0, int w, int l)
    {
        wave = w;
        lane = l;
        ldq = p.g.ldb;
        base = (const char *)p.g.B + (int64_t)k_begin * ldq + (FB == MX_FP4 ? n0 / 2 : n0);
        sbase = (const char *)p.SB + ((int64_t)(n0 / MX_GROUP) * p.ldsb + k_begin) * 8;
        offsets(DQ_BK);
    }
    // byte offsets of this lane's loads; rows at or past krem come from the
    // slab's last valid row (their elements are zeroed on conversion)
    __device__ __forceinline__ void offsets(int krem)
    {
#pragma unroll
        for (int i = 0; i < RLOADS; ++i) {
            const int b = ((i * NW + wave) % RTOT) * 1024 + lane * 16;
            const int k = b / RROW;
            off[i] = (uint32_t)((int64_t)(k < krem ? k : krem - 1) * ldq + b % RROW);
        }
        const int d = (wave & 1) * 64 + lane;
        soff = (uint32_t)((d / 2 < krem ? d / 2 : krem - 1) * 8 + (d & 1) * 4);
    }
    __device__ __forceinline__ void issue(lds_char_t *raw)
    {
#pragma unroll
        for (int i = 0; i < RLOADS; ++i)
            load_lds16(off[i], buffer_rsrc(base), (unsigned)(uintptr_t)(raw + ((i * NW + wave) % RTOT) * 1024));
        load_lds4(soff, buffer_rsrc(sbase), (unsigned)(uintptr_t)(raw + RAW + (wave & 1) * 256));
        base += DQ_BK * ldq;
        sbase += DQ_BK * 8;
    }
    // this thread's pieces of a raw slot into the 16-bit buffer; blk0: the
    // tile's first block within its group
    __device__ __forceinline__ void convert(const lds_char_t *raw, lds_char_t *dst, int blk0, int krem) const
    {
        const int tid = wave * 64 + lane;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = i * THREADS + tid;
            if (DQ_BK * PIECES % THREADS != 0 && t >= DQ_BK * PIECES) break;
            const int k = t / PIECES, pc = t % PIECES;
            const u32x4 q = *(const lds_u32x4_t *)(raw + t * 16);
            const int blk = FB == MX_FP4 ? pc : pc >> 1;               // 32 n: the quad, too
            const float sc = mx_scale(*(const lds_u8_t *)(raw + RAW + k * 8 + blk0 + blk));
            lds_char_t *row = dst + k * (DQ_BN * 2) + ((blk ^ (k & 3)) << 6);
            constexpr int CH = FB == MX_FP4 ? 4 : 2;                   // 16-byte chunks of the output
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                V8 v;
                if constexpr (FB == MX_FP4) v = Decode<T, FB>::eight(q[c], 0, sc);
                else v = Decode<T, FB>::eight(q[2 * c], q[2 * c + 1], sc);
                if (k >= krem)
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = (T)0.f;
                const int ch = FB == MX_FP4 ? c : 2 * (pc & 1) + c;
                *(lds_v8_t *)(row + ((ch ^ (k & 3)) << 4)) = v;
            }
        }
    }
    // columns b0 .. b0+31, step kk of 16 k (the transposing read: in each
    // 16-lane group, lanes 4t .. 4t+3 name row t of a 4 x 16 block)
    __device__ __forceinline__ V8 frag(const lds_char_t *buf, int b0, int kk) const
    {
        const int g = lane >> 4, t = (lane & 15) >> 2, s = lane & 3;
        const int k0 = 16 * kk + 8 * (g >> 1) + t;
        const int ch = 2 * (g & 1) + (s >> 1);
        const lds_char_t *p0 = buf + k0 * (DQ_BN * 2) + (((b0 >> 5) ^ t) << 6) + ((ch ^ t) << 4) + (s & 1) * 8;
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)p0);
        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t *)(p0 + 4 * (DQ_BN * 2)));
        typedef short i16x8 __attribute__((ext_vector_type(8)));
        const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        return __builtin_bit_cast(V8, v);
    }
};

// A through registers, for rows that the direct loads do not take (2-byte
// aligned, or a ragged m-contiguous extent): 16-byte pieces by unaligned
// vector loads, into the direct loads' LDS layout.
template <typename T, int BM, bool KCONT, int NW>
struct RegOperand {
    typedef PipeOperandH<T, BM, KCONT, NW, 16> Lay;
    typedef T V8 __attribute__((ext_vector_type(8)));
    typedef V8 __attribute__((aligned(2))) V8u;
    V8 r[Lay::LOADS];
    const T *g;
    int64_t ld;
    int mn0, ext, wave, lane;

    __device__ __forceinline__ void init(const T *p, int64_t l, int m0, int e, int w, int ln)
    {
        g = p;
        ld = l;
        mn0 = m0;
        ext = e;
        wave = w;
        lane = ln;
    }
    __device__ __forceinline__ void load(int k0, int Kl)
    {
#pragma unroll
        for (int i = 0; i < Lay::LOADS; ++i) {
            const int rbase = (i * NW + wave) * Lay::ROWS_PER_LOAD;
            const T *src;
            int valid;
            if constexpr (KCONT) {
                const int row = rbase + (lane >> 3), c = (lane & 7) ^ ((row >> 1) & 7);
                src = g + (int64_t)(mn0 + row) * ld + k0 + c * 8;
                valid = mn0 + row < ext ? Kl - k0 - c * 8 : 0;
            } else {
                const int k = rbase + lane / (Lay::ROW_BYTES / 16), p = lane % (Lay::ROW_BYTES / 16);
                const int col = mn0 + ((p >> 2) ^ Lay::swz(k)) * 32 + (p & 3) * 8;
                src = g + (int64_t)(k0 + k) * ld + col;
                valid = k0 + k < Kl ? ext - col : 0;
            }
            if (valid >= 8) {
                r[i] = *(const V8u *)src;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) r[i][e] = e < valid ? src[e] : (T)0.f;
            }
        }
    }
    __device__ __forceinline__ void store(lds_char_t *st) const
    {
#pragma unroll
        for (int i = 0; i < Lay::LOADS; ++i)
            *(__attribute__((address_space(3))) V8 *)(st + (i * NW + wave) * 1024 + lane * 16) = r[i];
    }
};

// DIRECT: A by direct loads (4-byte aligned rows, an m-contiguous extent of
// whole 16-byte pieces), else through registers.
template <typename T, int FB, bool TA, bool DIRECT, int BM, int WM, int WN>
__global__ __launch_bounds__(64 * (BM / WM) * (DQ_BN / WN), 2) void dq_gemm_kernel(MxGemmParams p)
{
    constexpr int WAVES_N = DQ_BN / WN, NW = (BM / WM) * WAVES_N;
    constexpr int TM = WM / 32, TN = WN / 32, KPW = DQ_BK / 16;
    typedef PipeOperandH<T, BM, !TA, NW, 16> OpA;
    typedef RegOperand<T, BM, !TA, NW> RegA;
    typedef DqOperand<T, FB, NW> OpB;
    typedef T V8 __attribute__((ext_vector_type(8)));
    constexpr int SA = 3, SR = 3;                      // stages of A and of raw B
    constexpr int LOADS = (DIRECT ? OpA::LOADS : 0) + OpB::LOADS;
    constexpr int A_AT = 0, B_AT = SA * OpA::BYTES, R_AT = B_AT + 2 * OpB::BYTES;
    constexpr int SMEM = R_AT + SR * OpB::RAW_BYTES;
    static_assert(SMEM <= 160 * 1024 && NW * kEpiBytes<WN> <= SMEM, "LDS");
    __shared__ __attribute__((aligned(1024))) char smem_raw[SMEM];
    lds_char_t *smem = (lds_char_t *)smem_raw;

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm0 = (wave / WAVES_N) * WM, wn0 = (wave % WAVES_N) * WN;
    int bid, split, k_begin, Kl, tm, tn;
    split_of(p.g, bid, split, k_begin, Kl);
    tile_coords(bid, p.g, tm, tn);
    const int m0 = tm * BM, n0 = tn * DQ_BN;
    const int nk = (Kl + DQ_BK - 1) / DQ_BK, krem = Kl - (nk - 1) * DQ_BK;
    const int blk0 = (n0 % MX_GROUP) / 32;

    OpA ga;
    RegA ra;
    OpB gb;
    const T *A = (const T *)p.g.A + (TA ? (int64_t)k_begin * p.g.lda : (int64_t)k_begin);
    if constexpr (DIRECT) ga.init(A, p.g.lda, m0, p.g.M, wave, lane);
    else ra.init(A, p.g.lda, m0, p.g.M, wave, lane);
    gb.init(p, k_begin, n0, wave, lane);

    auto a_at = [&](int s) { return smem + A_AT + (s % SA) * OpA::BYTES; };
    auto b_at = [&](int s) { return smem + B_AT + (s & 1) * OpB::BYTES; };
    auto r_at = [&](int s) { return smem + R_AT + (s % SR) * OpB::RAW_BYTES; };
    auto issue_a = [&](int s) {
        if constexpr (DIRECT) {
            if (s == nk - 1 && krem < DQ_BK) ga.issue_tail(a_at(s), wave, lane, krem);
            else ga.issue(a_at(s), wave);
        }
    };
    auto issue_r = [&](int s) {
        if (s == nk - 1 && krem < DQ_BK) gb.offsets(krem);
        gb.issue(r_at(s));
    };
    auto convert = [&](int s) { gb.convert(r_at(s), b_at(s), blk0, s == nk - 1 ? krem : DQ_BK); };

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    // prologue: raw slabs 0 .. SR-1, A slabs 0 .. SA-2, slab 0 converted
#pragma unroll
    for (int s = 0; s < SR; ++s)
        if (s < nk) issue_r(s);
#pragma unroll
    for (int s = 0; s < SA - 1; ++s)
        if (s < nk) issue_a(s);
    if constexpr (!DIRECT) {
        ra.load(0, Kl);
        ra.store(a_at(0));
        if (nk > 1) ra.load(DQ_BK, Kl);
    }
    wait_vmcnt<0>();
    __syncthreads();
    convert(0);

    for (int kt = 0; kt < nk; ++kt) {
        // A's slab kt and raw slab kt+1 (loaded two steps ago) have landed, slab
        // kt is converted, and every wave is done with A's slab kt-1, raw slab
        // kt and B's slab kt-1
        if (kt + 2 < nk) wait_vmcnt<LOADS>();
        else wait_vmcnt<0>();
        __syncthreads();
        if (kt + SA - 1 < nk) issue_a(kt + SA - 1);
        if (kt + SR < nk) issue_r(kt + SR);
        if constexpr (!DIRECT) {
            if (kt + 1 < nk) ra.store(a_at(kt + 1));
            if (kt + 2 < nk) ra.load((kt + 2) * DQ_BK, Kl);
        }
        const lds_char_t *sa = a_at(kt), *sb = b_at(kt);
        V8 fa[KPW][TM], fb[KPW][TN];
#pragma unroll
        for (int s = 0; s < KPW; ++s) {
#pragma unroll
            for (int i = 0; i < TM; ++i) fa[s][i] = ga.frag(sa, wm0 + 32 * i, s, lane);
#pragma unroll
            for (int j = 0; j < TN; ++j) fb[s][j] = gb.frag(sb, wn0 + 32 * j, s);
        }
        if (kt + 1 < nk) convert(kt + 1);
#pragma unroll
        for (int s = 0; s < KPW; ++s)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = mfma_32x32x16(fa[s][i], fb[s][j], acc[i][j]);
    }

    __syncthreads();  // every wave is done with the ring
    store_tile<TM, TN>(p, smem + wave * kEpiBytes<WN>, acc, m0 + wm0, n0 + wn0, lane, split);
}

template <typename T, int FB, bool TA, bool DIRECT, int BM, int WM, int WN>
hipError_t launch_dq(const MxGemmParams &p, hipStream_t s)
{
    const unsigned nwg = (unsigned)p.g.tiles_m * (unsigned)p.g.tiles_n * (unsigned)p.g.splits;
    MxGemmParams arg = p;
    void *args[] = {&arg};
    return hipLaunchKernel((const void *)&dq_gemm_kernel<T, FB, TA, DIRECT, BM, WM, WN>, dim3(nwg),
                           dim3(64 * (BM / WM) * (DQ_BN / WN)), args, 0, s);
}

}  // namespace

// [config][format][transA][direct]
#define DG_DQ4(T, FB, BM, WM, WN)                                                                   \
    {{launch_dq<T, FB, false, false, BM, WM, WN>, launch_dq<T, FB, false, true, BM, WM, WN>},       \
     {launch_dq<T, FB, true, false, BM, WM, WN>, launch_dq<T, FB, true, true, BM, WM, WN>}}
#define DG_DQ12(T, BM, WM, WN)                                                                      \
    {DG_DQ4(T, MX_FP4, BM, WM, WN), DG_DQ4(T, MX_FP8, BM, WM, WN), DG_DQ4(T, MX_INT8, BM, WM, WN)}
template <typename T>
mx_launch_fn dq_launcher_of(int config, int format, int ta, int direct)
{
    static const mx_launch_fn table[][3][2][2] = {
        DG_DQ12(T, 32, 32, 32),
        DG_DQ12(T, 128, 64, 32),
        DG_DQ12(T, 256, 64, 64),
    };
    return table[config][format][ta][direct];
}

mx_launch_fn dq_gemm_launcher(int type, int config, int format, int ta, int direct)
{
    return type == ELEM_F16 ? dq_launcher_of<_Float16>(config, format, ta, direct)
                            : dq_launcher_of<__bf16>(config, format, ta, direct);
}

}  // namespace dg
