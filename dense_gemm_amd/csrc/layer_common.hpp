// Shared by the kernels of a layer's products (fused epilogues, grouped by
// expert, weight gradients): their parameters, the epilogue's arithmetic, and
// which tile of which group a workgroup takes.
//
//   forward    z = alpha * acc + bias;        C = act(z) + beta * R
//   gradient   h = alpha * acc + beta * R;    C = h * act'(Z)
//   weights    C = alpha * acc + beta * C
// z (forward) or h (gradient) is written to `keep` when that is given.  Sums and
// the epilogue are fp32, with one rounding of each output.
#pragma once

#include "gemm_common.hpp"
#include "layer_ranges.hpp"

namespace dg {

enum { LAYER_FORWARD = 0, LAYER_GRAD = 1, LAYER_WEIGHTS = 2 };

struct LayerParams {
    const void *A, *B;
    int64_t lda, ldb, strideB;      // strideB: from a group's B to the next (elements)
    // forward, gradient: A holds M rows, the groups' B is K x N (or N x K).
    // weights: A and B hold K rows, a group's C is M x N.
    int32_t M, N, K;
    float alpha, beta;
    int32_t kind, act;
    const int32_t *offsets;         // groups + 1 row offsets on the device; NULL: one group of all rows
    int32_t groups;
    const void *bias;
    int64_t stride_bias;
    const void *Z;                  // gradient: the activation's input
    int64_t ldz;
    const void *R;                  // weights: C itself, or NULL for beta = 0
    int64_t ldr;
    void *keep;
    int64_t ldk;
    void *C;
    int64_t ldc, strideC;           // strideC: weights, from a group's C to the next (else 0)
    int32_t ctype;                  // element of C, R, Z, keep and bias: 0 fp32, 1 fp16, 2 bf16
    int32_t tiles_m, tiles_n, group_m;
    int32_t past_caches;            // outputs too large for the caches
    int32_t splits;                 // K ranges, a grid dimension; with more than one the raw sums go to ws
    float *ws;                      // [splits][groups][M][N], and weights: [splits][groups][M] behind them
    float *dbias;                   // weights: [groups][M], or NULL
};

#ifdef __HIPCC__

// Phi(-a) / exp(-a^2 / 2), a >= 0, for 16-bit results: half of erfc(z) exp(z^2), z = a /
// sqrt 2, as a polynomial in t = 1 / (1 + 0.44 z), fitted here to the least largest
// relative error over 0 <= z <= 9: 5.2e-6, a thousandth of a bf16 step also far out on
// gelu's negative side (gelu()'s approximation, of one degree less, has an absolute
// error of 1.5e-7, 4e-4 of gelu at -4).  fp32 results take the device library's erfcf.
__device__ __forceinline__ float tail_ratio(float a)
{
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.31112698f, a, 1.f));
    float poly = __builtin_fmaf(t, -0.073042706f, 0.17529286f);
    poly = __builtin_fmaf(t, poly, 0.020407932f);
    poly = __builtin_fmaf(t, poly, 0.13176741f);
    poly = __builtin_fmaf(t, poly, 0.12129223f);
    poly = __builtin_fmaf(t, poly, 0.12427969f);
    return poly * t;
}
// exp(-a^2 / 2)
__device__ __forceinline__ float gauss(float a) { return __builtin_amdgcn_exp2f(a * -0.72134752f * a); }

// act(x) of the forward pass.  gelu(x) = x Phi(x) = max(x, 0) - |x| Phi(-|x|), so that the
// negative side keeps its relative accuracy; |x| is cut at 16, where Phi(-|x|) is zero
// in fp32 and an infinite |x| would not be.
template <bool EXACT>
__device__ __forceinline__ float layer_act(int act, float x)
{
    const float m = x < 0.f ? 0.f : x;               // NaN stays
    if (act == ACT_RELU) return m;
    if (act == ACT_GELU) {
        const float a = __builtin_fminf(__builtin_fabsf(x), 16.f);
        const float q = EXACT ? 0.5f * erfcf(a * 0.70710678118654752f) : tail_ratio(a) * gauss(a);
        return __builtin_fmaf(-a, q, m);
    }
    return x;
}

// h * act'(x).  relu chooses h or 0 (an infinite or NaN h does not pass a unit
// that is off; a NaN x gives NaN).  gelu'(x) = Phi(x) + x phi(x), which is s for
// x < 0 and 1 - s for x >= 0 with s = Phi(-|x|) - |x| phi(x).
template <bool EXACT>
__device__ __forceinline__ float layer_act_grad(int act, float h, float x)
{
    if (act == ACT_RELU) return x > 0.f ? h : (x <= 0.f ? 0.f : x);
    if (act == ACT_GELU) {
        const float a = __builtin_fabsf(x), cut = __builtin_fminf(a, 16.f) * 0.39894228040143268f;
        const float s = EXACT ? __builtin_fmaf(-cut, expf(-0.5f * a * a), 0.5f * erfcf(a * 0.70710678118654752f))
                              : gauss(a) * (tail_ratio(a) - cut);
        return h * (x >= 0.f ? 1.f - s : s);
    }
    return h;
}

// W consecutive elements of a row, by 16-byte accesses that need no more than the
// element's alignment (the GPU takes misaligned vectors); where only n < W exist, one
// by one, and the others are 0.
template <typename T, int W>
__device__ __forceinline__ auto load_raw(const T *x, int n)
{
    constexpr int PER = (int)(16 / sizeof(T)) < W ? (int)(16 / sizeof(T)) : W;
    typedef T V __attribute__((ext_vector_type(PER)));
    typedef V __attribute__((aligned(sizeof(T)))) Vu;
    typedef T VW __attribute__((ext_vector_type(W)));
    VW v = (VW)(T)0.f;
    if (n >= W) {
#pragma unroll
        for (int c = 0; c < W / PER; ++c) {
            const V y = *(const Vu *)(x + c * PER);
#pragma unroll
            for (int e = 0; e < PER; ++e) v[c * PER + e] = y[e];
        }
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e)
            if (e < n) v[e] = x[e];
    }
    return v;
}

template <typename T, int W>
__device__ __forceinline__ void load_row(const T *x, float (&v)[W], int n)
{
    const auto y = load_raw<T, W>(x, n);
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = (float)y[e];
}

template <typename T, int W, bool NT = false>
__device__ __forceinline__ void store_row(T *x, const float (&v)[W], int n)
{
    constexpr int PER = (int)(16 / sizeof(T)) < W ? (int)(16 / sizeof(T)) : W;
    typedef T V __attribute__((ext_vector_type(PER)));
    typedef V __attribute__((aligned(sizeof(T)))) Vu;
    if (n >= W) {
#pragma unroll
        for (int c = 0; c < W / PER; ++c) {
            V y;
#pragma unroll
            for (int e = 0; e < PER; ++e) y[e] = (T)v[c * PER + e];
            if constexpr (NT) __builtin_nontemporal_store(y, (Vu *)(x + c * PER));
            else *(Vu *)(x + c * PER) = y;
        }
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e)
            if (e < n) x[e] = (T)v[e];
    }
}

// The tile a workgroup works on, with its group's matrices.
struct LayerTile {
    int group;
    int rows;            // rows of the group (forward, gradient) or of C (weights)
    int m0, n0;
    int64_t row0;        // first row of the group in the matrices of rows
    int64_t out0;        // the same for C's rows (weights: 0, a group's C stands by itself)
    int k0, k_len;       // this split's part of the sum
};

// What W columns of a row of C need beside the sums, fetched ahead of them and kept
// in C's type: Z of the gradient, else R.  (A gradient's R is read when it is
// needed: both ahead take more registers than the largest tile leaves.)
template <typename TC, int W>
struct LayerAux {
    typedef TC V __attribute__((ext_vector_type(W)));
    V x;
    __device__ __forceinline__ static V residual(const LayerParams &p, const LayerTile &t, int row, int col, int n)
    {
        return load_raw<TC, W>((const TC *)p.R + t.group * p.strideC + (t.out0 + row) * p.ldr + col, n);
    }
    __device__ __forceinline__ void fetch(const LayerParams &p, const LayerTile &t, int row, int col, int n = W)
    {
        x = (V)(TC)0.f;
        if (p.Z) x = load_raw<TC, W>((const TC *)p.Z + (t.out0 + row) * p.ldz + col, n);
        else if (p.R) x = residual(p, t, row, col, n);
    }
};

// The epilogue of W columns col .. of row `row`, n of which exist: v holds the sums.
// NT: stores that do not stay in the caches.
template <typename TC, int W, bool NT = false>
__device__ __forceinline__ void layer_finish(const LayerParams &p, const LayerTile &t, int row, int col,
                                             float (&v)[W], const LayerAux<TC, W> &aux, const float (&bias)[W], int n = W)
{
    constexpr bool EXACT = sizeof(TC) == 4;
    const int64_t out = t.out0 + row;
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = __builtin_fmaf(p.alpha, v[e], bias[e]);
    if (p.kind == LAYER_GRAD && p.R) {
        const auto r = LayerAux<TC, W>::residual(p, t, row, col, n);
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = __builtin_fmaf(p.beta, (float)r[e], v[e]);
    }
    if (p.keep) store_row<TC, W, NT>((TC *)p.keep + out * p.ldk + col, v, n);
    if (p.kind == LAYER_GRAD) {
        if (p.act == ACT_GELU) {
#pragma unroll
            for (int e = 0; e < W; ++e) {
                v[e] = layer_act_grad<EXACT>(ACT_GELU, v[e], (float)aux.x[e]);
                if (EXACT) __builtin_amdgcn_sched_barrier(0);    // erfcf's registers one at a time
            }
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] = layer_act_grad<EXACT>(ACT_RELU, v[e], (float)aux.x[e]);
        }
    } else if (p.act == ACT_GELU) {
#pragma unroll
        for (int e = 0; e < W; ++e) {
            v[e] = layer_act<EXACT>(ACT_GELU, v[e]);
            if (EXACT) __builtin_amdgcn_sched_barrier(0);
        }
    } else if (p.act == ACT_RELU) {
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = layer_act<EXACT>(ACT_RELU, v[e]);
    }
    if (p.kind != LAYER_GRAD && p.R) {
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = __builtin_fmaf(p.beta, (float)aux.x[e], v[e]);
    }
    store_row<TC, W, NT>((TC *)p.C + t.group * p.strideC + out * p.ldc + col, v, n);
}

// The bias of W columns of a group.
template <typename TC, int W>
__device__ __forceinline__ void layer_bias(const LayerParams &p, int group, int col, float (&b)[W], int n = W)
{
    if (p.bias) {
        load_row<TC, W>((const TC *)p.bias + group * p.stride_bias + col, b, n);
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e) b[e] = 0.f;
    }
}

// The raw sums of a split's W columns.
template <int W>
__device__ __forceinline__ void layer_partial(const LayerParams &p, const LayerTile &t, int row, int col,
                                              const float (&v)[W], int n = W)
{
    float *w = p.ws + (((int64_t)blockIdx.y * p.groups + t.group) * p.M + row) * p.N + col;
    store_row<float, W>(w, v, n);
}

// One column's sum for the bias's gradient: a split's goes behind the splits' sums of
// the product, [splits][groups][M].
__device__ __forceinline__ void layer_dbias(const LayerParams &p, int group, int m, float v)
{
    const int64_t at = (int64_t)group * p.M + m, gm = (int64_t)p.groups * p.M;
    if (p.splits > 1) {
        p.ws[p.splits * gm * p.N + blockIdx.y * gm + at] = v;
        return;
    }
    if (p.beta != 0.f) v = __builtin_fmaf(p.beta, p.dbias[at], v);
    p.dbias[at] = v;
}

// First row and rows of group g.  Offsets outside 0 .. total and descending ones
// are brought back, so that no offset leads outside the matrices.
__device__ __forceinline__ void group_rows(const LayerParams &p, int g, int total, int &begin, int &rows)
{
    int b = p.offsets[g], e = p.offsets[g + 1];
    b = b < 0 ? 0 : (b > total ? total : b);
    e = e < b ? b : (e > total ? total : e);
    begin = b;
    rows = e - b;
}

// Workgroup ids go to the 8 XCDs in turn; give each XCD a contiguous range of
// the `nwg` tiles, so that the tiles resident on it share rows and columns.
__device__ __forceinline__ int xcd_contiguous(int bid, int nwg)
{
    const int xcd = bid & 7, local = bid >> 3, per = nwg >> 3, rem = nwg & 7;
    return xcd * per + (xcd < rem ? xcd : rem) + local;
}

// Tile `in` of a group with tiles_m x tiles_n: group_m tile rows are walked
// together, column by column.
__device__ __forceinline__ void walk_tiles(int in, int tiles_m, int tiles_n, int group_m, int &tm, int &tn)
{
    const int gsz = group_m * tiles_n, g = in / gsz, first = g * group_m;
    const int rows = tiles_m - first < group_m ? tiles_m - first : group_m;
    const int r = in - g * gsz;
    tm = first + r % rows;
    tn = r / rows;
}

// Tile `id` (a workgroup's, in launch order), or false where there are fewer tiles.  The
// host does not know how many rows a group has: the launch holds one workgroup for every
// tile there can be, and every wave counts the groups' tiles (64 groups at a time, a lane
// each) to find its own (one wave of a workgroup for all, through LDS, is 2% slower with 14
// decoding experts).
__device__ __forceinline__ bool layer_tile(const LayerParams &p, int bm, int bn, int id, LayerTile &t)
{
    t.group = 0;
    t.row0 = 0;
    if (p.kind == LAYER_WEIGHTS) {
        // Every group goes over all XCDs, in a multiple of 8 workgroups, and where groups are
        // long the one with most rows first: a group's tiles take as long as it has rows, so that
        // a group to an XCD, or a long one at the end, would leave the others idle (8 uneven
        // groups of 2048 rows on average, 5632 x 2048 on the 256 tile: 583 us, 375 with this; equal
        // groups 371).  Finding the order takes every wave a microsecond: 32 uneven groups
        // of 2048 rows 388 us, 476 as they come (2048 x 1408), of 512 rows 147 and 150, of 128
        // rows 104 and 90; 64 groups of 128 rows (1031 x 517) 73 and 60.
        const int per = p.tiles_m * p.tiles_n, slots = (per + 7) & ~7, slot = id / slots;
        id -= slot * slots;
        if (id >= per) return false;
        id = xcd_contiguous(id, per);
        t.group = slot;
        int begin = 0, n = p.K;
        if (p.offsets && p.groups > 1 && p.groups <= 64 && p.K >= 1024 * p.groups) {
            const int lane = threadIdx.x & 63;
            int b = 0, m = 0, rank = 0;
            if (lane < p.groups) group_rows(p, lane, p.K, b, m);
            // (rows and, among equals, the group, in one word; lanes past the groups come last)
            const uint32_t key = lane < p.groups ? ((uint32_t)(m < 0x1ffffff ? m : 0x1ffffff) << 6 | (63 - lane)) + 1 : 0;
            for (int g = 0; g < p.groups; g += 8)
#pragma unroll
                for (int u = 0; u < 8; ++u) rank += (uint32_t)__builtin_amdgcn_readlane(key, g + u) > key;
            t.group = __ffsll((unsigned long long)__ballot(rank == slot)) - 1;
            begin = __builtin_amdgcn_readlane(b, t.group);
            n = __builtin_amdgcn_readlane(m, t.group);
        } else if (p.offsets) {
            group_rows(p, slot, p.K, begin, n);
            begin = __builtin_amdgcn_readfirstlane(begin);
            n = __builtin_amdgcn_readfirstlane(n);
        }
        int tm, tn;
        walk_tiles(id, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
        t.m0 = tm * bm;
        t.n0 = tn * bn;
        t.rows = p.M;
        t.out0 = 0;
        t.row0 = begin;
        t.k0 = 0;
        t.k_len = n;
        if (p.splits > 1) range_of(n, p.splits, (int)blockIdx.y, t.k0, t.k_len);
        return true;
    }
    t.out0 = t.row0;
    t.k0 = 0;
    t.k_len = p.K;
    int tiles_m, first = 0;                     // of the group, and its first tile row
    if (p.offsets == nullptr) {
        tiles_m = p.tiles_m;
        t.rows = p.M;
        if (id >= tiles_m * p.tiles_n) return false;
        id = xcd_contiguous(id, tiles_m * p.tiles_n);
        if (p.splits > 1) range_of(p.K, p.splits, (int)blockIdx.y, t.k0, t.k_len);
    } else {
        // (no group is counted with more tile rows than the launch has workgroups for,
        // so that no offsets, ascending or not, let the sums overflow)
        const int lane = threadIdx.x & 63, limit = gridDim.x / p.tiles_n;
        int b, n;                               // of the group that a lane looked at last
        auto tiles_of = [&](int g) {
            b = n = 0;
            if (g < p.groups) group_rows(p, g, p.M, b, n);
            const int x = (n + bm - 1) / bm;
            return x < limit ? x : limit;
        };
        auto scan = [&](int x) {                // inclusive sums over the lanes: within rows of 16, then over them
            x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);
            x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
            x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
            x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
            x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);
            x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);
            return x;
        };
        int sum = scan(tiles_of(lane)), total = __builtin_amdgcn_readlane(sum, 63);
        const int sum0 = sum, total0 = total, b0 = b, n0 = n;
        for (int base = 64; base < p.groups && total < limit; base += 64) {
            sum = scan(tiles_of(base + lane));
            total += __builtin_amdgcn_readlane(sum, 63);
        }
        if (total > limit) total = limit;
        if (id >= total * p.tiles_n) return false;
        id = xcd_contiguous(id, total * p.tiles_n);
        const int row = id / p.tiles_n;         // tile row, counted over all groups
        int base = 0, before = 0;
        sum = sum0;
        b = b0;
        n = n0;
        for (int upto = total0; row >= upto && base + 64 < p.groups;) {
            base += 64;
            before = upto;
            sum = scan(tiles_of(base + lane));
            upto += __builtin_amdgcn_readlane(sum, 63);
        }
        const uint64_t past = __ballot(before + sum > row);
        if (past == 0) return false;
        const int l = __ffsll((unsigned long long)past) - 1;
        t.group = base + l;
        const int upto = before + __builtin_amdgcn_readlane(sum, l);
        first = l == 0 ? before : before + __builtin_amdgcn_readlane(sum, l - 1);
        tiles_m = upto - first;
        t.row0 = t.out0 = __builtin_amdgcn_readlane(b, l);
        t.rows = __builtin_amdgcn_readlane(n, l);
    }
    int tm, tn;
    walk_tiles(id - first * p.tiles_n, tiles_m, p.tiles_n, p.group_m, tm, tn);
    t.m0 = tm * bm;
    t.n0 = tn * bn;
    return t.m0 < t.rows;
}

#endif

}  // namespace dg
