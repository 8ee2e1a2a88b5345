// Host side of the block-scaled (MX) operators: argument checks, kernel
// choice and launches on the caller's stream.  The C ABI is declared in
// include/dense_gemm.h.
#include "../../include/dense_gemm.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_tile.hpp"

namespace dg {
launch_fn scale_launcher(int dtype);
launch_fn splitk_reduce_launcher(int dtype);
int launch_status(hipError_t err);
mx_launch_fn mx_gemm_launcher(int config, int format_a, bool exact);
mx_launch_fn dq_gemm_launcher(int type, int config, int format, int ta, int direct);
}  // namespace dg

namespace {

using dg::MxGemmParams;
using dg::MxParams;

constexpr int64_t kMaxDim = 0x7fffffff;

bool is_elem(int t) { return t == DG_ELEM_F32 || t == DG_ELEM_F16 || t == DG_ELEM_BF16; }
bool is_format(int f) { return f == DG_MXFP4 || f == DG_MXFP8 || f == DG_MXINT8; }
bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t elem_size(int t) { return t == DG_ELEM_F32 ? 4 : 2; }

int64_t row_bytes(int format, int64_t cols) { return dg::mx_groups(cols) * dg::mx_group_bytes(format); }

// An MX matrix's elements: 16-byte aligned rows that hold whole groups.
bool bad_q(const void *Q) { return Q == nullptr || !aligned(Q, 16); }
bool bad_ldq(int64_t ldq, int format, int64_t cols) { return ldq < row_bytes(format, cols) || ldq % 16 != 0; }
// Its scales: 8 bytes per row and group.
bool bad_s(const void *S) { return S == nullptr || !aligned(S, 8); }

// The dense library's dtype whose C has the element type.
int c_dtype(int type) { return type == DG_ELEM_F32 ? DG_F32 : type == DG_ELEM_F16 ? DG_F16_F32ACC : DG_BF16_F32ACC; }

// C's rows start on 4-byte boundaries: 16-byte pieces (as in the dense
// kernels' epilogue).
bool c_rows4(const void *C, int64_t ldc, int type) { return aligned(C, 4) && ldc * elem_size(type) % 4 == 0; }

// 256 rows of an operand within the tiled kernels' 32-bit byte offsets.
bool offsets_fit(int64_t ld_bytes) { return 256 * ld_bytes < ((int64_t)1 << 31); }

// ---- the kernels of dg_gemm_mx ------------------------------------------------
struct MxFamily {
    const char *name;
    int bm, bn, group_m;
    bool tiled;          // 32-bit row offsets
};
const MxFamily kMx[] = {
    {"mx_16x16_rows", 16, 16, 1, false},
    {"mx_32x16_rows", 32, 16, 1, false},
    {"mx_64x64_tile", 64, 64, 4, true},
    {"mx_128x128_tile", 128, 128, 4, true},
    {"mx_256x256_tile", 256, 256, 4, true},
};
constexpr int kNumMx = sizeof(kMx) / sizeof(kMx[0]);

bool mx_supports(int k, int64_t M, int64_t N, int64_t lda, int64_t ldb)
{
    const MxFamily &f = kMx[k];
    const int64_t tm = ceil_div(M, f.bm), tn = ceil_div(N, f.bn);
    if (!f.tiled) return tm <= 65535 && tn * 512 < ((int64_t)1 << 32);
    return offsets_fit(lda) && offsets_fit(ldb) && tm * tn < (1 << 22);
}

// The kernel by its time (us) under a model of each: a fixed part, and a part
// per slab (128 k, or 256 k of two mxfp4 operands) for as many rounds of tiles
// as the compute units need (and C's way out at 4 TB/s for the 64 x 64 tile).
// Fitted to back-to-back times; over 40 shapes with a bf16 C (M 1 to 8192, N 65 to
// 8192, K 67 to 8192) the choice is 0.4% slower than the fastest kernel by
// geometric mean, 14% at the worst (4138 x 901 x 291).  A 64 x 64 tile's units
// share about 270 tiles a round, a 128 x 128 one's 212 (two fit a unit, at less
// than twice the speed), and a 256 x 256 one's 256, whose last round costs 0.82
// when partly filled.  The row kernels read B once per 16 (or 32) rows of A and their
// own rows of A for every 16 columns.  Measured on both sides of the choice
// (M x N x K, mxfp8 times mxfp4): 16 x 8192 x 8192 rows 15.1, tile 17.9 us;
// 32 x 8192 x 8192 rows 22.2, tile 18.0; 64 x 2048 x 2048 rows 5.1, tile 6.9;
// 512 x 5632 x 2048 64-tile 13.0, 128-tile 13.4; 1024 x 8192 x 8192 128-tile
// 58.9, 256-tile 80.1; mxfp4 both, 2048 x 8192 x 4096 128-tile 42.9, 256-tile
// 37.7.  `exact` (mxfp8 with an fp32 C) takes two matrix instructions for one on the
// tiled kernels: 32 x 8192 x 8192 rows 23, 64-tile 31; 512 x 5632 x 2048 64-tile
// 17.4, 128-tile 19.7; 1024 x 8192 x 8192 128-tile 102, 64-tile 139; 4096^3 256-tile
// 100, 128-tile 106.
int mx_choose(bool a4, bool exact, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb)
{
    const double slabs = (double)ceil_div(K, a4 ? 256 : 128);
    auto tiles = [&](int64_t b) { return (double)ceil_div(M, b) * (double)ceil_div(N, b); };
    auto at_least_1 = [](double x) { return x > 1 ? x : 1.; };
    // a row workgroup's start costs as much as 600 k
    const double nk = (double)ceil_div(N, 16) * ((double)K + 600), mb = (double)M * (double)N * 2e-6;
    const double t256 = tiles(256), full = (double)(int64_t)(t256 / 256);
    const double cost[kNumMx] = {
        2.5 + (1.6e-6 + (a4 ? 0.05e-6 : 0.1e-6) * (double)(M < 16 ? M : 16)) * (double)ceil_div(M, 16) * nk,
        2.7 + 5.0e-6 * (double)ceil_div(M, 32) * nk,
        3.1 + slabs * (a4 ? 0.28 : exact ? 0.42 : 0.23) * at_least_1(tiles(64) / (exact ? 430 : 270)) + mb / 4,
        5.8 + slabs * (a4 ? 0.50 : exact ? 0.70 : 0.36) * at_least_1(tiles(128) / 212),
        9.0 + slabs * (a4 ? 1.4 : exact ? 2.6 : 1.2) * (full + (t256 > full * 256 ? (full > 0 ? 0.82 : 1.) : 0.)),
    };
    int best = -1;
    for (int k = 0; k < kNumMx; ++k)
        if (mx_supports(k, M, N, lda, ldb) && (best < 0 || cost[k] < cost[best])) best = k;
    return best;
}

// ---- the kernels of dg_gemm_dq -------------------------------------------------
struct DqTile {
    const char *name;
    int bm, bn;
    double fixed, slab;      // us: the fixed part, and a slab of 64 k
    int resident;            // workgroups that fit a compute unit (LDS)
    double share;            // of a slab's time, for each of them
};
const DqTile kDq[] = {
    {"dq_32x128_tile", 32, 128, 3.0, 0.50, 4, 0.45},
    {"dq_64x128_tile", 64, 128, 3.0, 0.60, 3, 0.58},
    {"dq_128x128_tile", 128, 128, 4.0, 0.74, 2, 0.635},
    {"dq_256x256_tile", 256, 256, 10.0, 1.38, 1, 1.0},   // A by direct loads only
};
constexpr int kNumDq = sizeof(kDq) / sizeof(kDq[0]);

// K ranges of `splits` (each a multiple of 64 but the last).
int64_t dq_chunk(int64_t K, int splits) { return ceil_div(ceil_div(K, splits), 64) * 64; }

// Tile and K ranges by their time (us) under a model fitted to back-to-back
// times of 21 shapes: a fixed part; a part per slab for as many rounds as the
// workgroups need, a round longer once a compute unit's workgroups fill its
// LDS bandwidth (`share` of a slab each); and for more than one range the
// second launch and the partials' way to memory and back at a large copy's 5
// TB/s.  `splits` > 0 fixes the ranges.  Over 32 shapes (M 8 to 8192, N 700 to
// 6144, K 1024 to 16384) the choice is 3.4% slower than the fastest tile and
// ranges by geometric mean, 25% at the worst (64 x 5632 x 2048).  Measured on both
// sides (M x N x K, us): 512 x 2048 x 5632 in 4 ranges 26.5, in one 54.1; 1024^3 in one range
// 11.8, in two 16; 4096 x 2048 x 16384 256-tile in two ranges 241, in one 345,
// 128-tile in one 291; 5632 x 2048 x 16384 256-tile in one range 354, in two 416;
// 4096^3 256-tile 108, 128-tile 130.
void dq_choose(int64_t M, int64_t N, int64_t K, bool direct, int splits, int *tile, int *ranges)
{
    double best = 1e300;
    const double out = (double)M * (double)N;
    const int fixed_splits[] = {splits}, tried[] = {1, 2, 3, 4, 6, 8, 12, 16};
    const int *list = splits > 0 ? fixed_splits : tried;
    const int n = splits > 0 ? 1 : (int)(sizeof(tried) / sizeof(tried[0]));
    for (int k = 0; k < kNumDq; ++k) {
        if (k == 3 && !direct) continue;
        const double tiles = (double)ceil_div(M, kDq[k].bm) * (double)ceil_div(N, kDq[k].bn);
        for (int i = 0; i < n; ++i) {
            const int64_t chunk = dq_chunk(K, list[i]), s = ceil_div(K, chunk);
            // ranges of at least 4 slabs, and no more partials than 256 MiB, where the choice is free
            if (splits == 0 && s > 1 && (chunk < 256 || (double)s * out * 4 > 268435456.0)) continue;
            const double w = tiles * (double)s / 256, full = (double)(int64_t)(w / kDq[k].resident);
            auto round = [&](double wgs) { return kDq[k].share * wgs > 1 ? kDq[k].share * wgs : 1.; };
            const double rest = w - full * kDq[k].resident;
            const double last = rest > 0 ? (k == 3 && full > 0 ? 0.82 : round(rest)) : 0.;
            const double rounds = full * round(kDq[k].resident) + last;
            // (with every unit at work on the largest tile the clock drops)
            const double slab = kDq[k].slab * (direct ? 1. : 1.2) * (k == 3 && w > 0.9 ? 1.15 : 1.);
            double t = kDq[k].fixed + (double)(chunk / 64) * slab * rounds;
            if (s > 1) t += 3.0 + (double)s * (0.4 + out * 8 / 5e6);
            if (t < best) {
                best = t;
                *tile = k;
                *ranges = (int)s;
            }
        }
    }
}

}  // namespace

extern "C" {

int64_t dg_mx_row_bytes(dg_mx_t format, int64_t cols)
{
    if (!is_format(format)) return -1;
    if (cols < 0 || cols > kMaxDim) return -2;
    return row_bytes(format, cols);
}

int64_t dg_mx_scale_bytes(int64_t lds, int64_t cols)
{
    if (lds < 0 || lds > kMaxDim) return -1;
    if (cols < 0 || cols > kMaxDim) return -2;
    return 8 * lds * dg::mx_groups(cols);
}

int dg_mx_quantize(dg_op_t transX, int64_t rows, int64_t cols, const void *X, int64_t ldx, dg_elem_t type,
                   dg_mx_t format, void *Q, int64_t ldq, void *S, int64_t lds, void *stream)
{
    if (transX != DG_OP_N && transX != DG_OP_T) return -1;
    if (rows < 0 || rows > kMaxDim) return -2;
    if (cols < 0 || cols > kMaxDim) return -3;
    const bool any = rows > 0 && cols > 0;
    if (!is_elem(type)) return -6;
    if (any && (X == nullptr || !aligned(X, elem_size(type)))) return -4;
    const int64_t inner = transX == DG_OP_T ? rows : cols;
    if (ldx < (inner > 1 ? inner : 1)) return -5;
    if (!is_format(format)) return -7;
    if (any && bad_q(Q)) return -8;
    if (bad_ldq(ldq, format, cols)) return -9;
    if (any && bad_s(S)) return -10;
    if (lds < rows) return -11;
    if (!any) return DG_OK;
    MxParams p = {};
    p.X = X;
    p.Q = (uint8_t *)Q;
    p.S = (uint8_t *)S;
    p.ldx = ldx;
    p.ldq = ldq;
    p.lds = lds;
    p.rows = rows;
    p.cols = cols;
    p.trans = transX;
    p.type = type;
    p.format = format;
    return dg::launch_status(dg::launch_mx_quantize(p, (hipStream_t)stream));
}

int dg_mx_dequantize(int64_t rows, int64_t cols, dg_mx_t format, const void *Q, int64_t ldq, const void *S,
                     int64_t lds, void *X, int64_t ldx, dg_elem_t type, void *stream)
{
    if (rows < 0 || rows > kMaxDim) return -1;
    if (cols < 0 || cols > kMaxDim) return -2;
    const bool any = rows > 0 && cols > 0;
    if (!is_format(format)) return -3;
    if (any && bad_q(Q)) return -4;
    if (bad_ldq(ldq, format, cols)) return -5;
    if (any && bad_s(S)) return -6;
    if (lds < rows) return -7;
    if (!is_elem(type)) return -10;
    if (any && (X == nullptr || !aligned(X, elem_size(type)))) return -8;
    if (ldx < (cols > 1 ? cols : 1)) return -9;
    if (!any) return DG_OK;
    MxParams p = {};
    p.Y = X;
    p.Q = (uint8_t *)Q;
    p.S = (uint8_t *)S;
    p.ldy = ldx;
    p.ldq = ldq;
    p.lds = lds;
    p.rows = rows;
    p.cols = cols;
    p.type = type;
    p.format = format;
    return dg::launch_status(dg::launch_mx_dequantize(p, (hipStream_t)stream));
}

int dg_act_checkpoint(int64_t rows, int64_t cols, const void *Z, int64_t ldz, void *H, int64_t ldh, dg_elem_t type,
                      dg_epilogue_t activation, dg_mx_t format, void *Q, int64_t ldq, void *S, int64_t lds, void *stream)
{
    if (rows < 0 || rows > kMaxDim) return -1;
    if (cols < 0 || cols > kMaxDim) return -2;
    const bool any = rows > 0 && cols > 0;
    if (!is_elem(type)) return -7;
    if (any && (Z == nullptr || !aligned(Z, elem_size(type)))) return -3;
    if (ldz < (cols > 1 ? cols : 1)) return -4;
    if (any && (H == nullptr || !aligned(H, elem_size(type)))) return -5;
    if (ldh < (cols > 1 ? cols : 1) || (H == Z && any && ldh != ldz)) return -6;
    if (activation != DG_EPI_RELU && activation != DG_EPI_GELU && activation != DG_EPI_RELU_POSITIVE) return -8;
    if (format != DG_MXFP8 && format != DG_MXINT8) return -9;
    if (any && bad_q(Q)) return -10;
    if (bad_ldq(ldq, format, cols)) return -11;
    if (any && bad_s(S)) return -12;
    if (lds < rows) return -13;
    if (!any) return DG_OK;
    MxParams p = {};
    p.X = Z;
    p.Y = H;
    p.Q = (uint8_t *)Q;
    p.S = (uint8_t *)S;
    p.ldx = ldz;
    p.ldy = ldh;
    p.ldq = ldq;
    p.lds = lds;
    p.rows = rows;
    p.cols = cols;
    p.type = type;
    p.format = format;
    p.act = activation == DG_EPI_GELU ? DG_EPI_GELU : DG_EPI_RELU;
    p.positive = activation == DG_EPI_RELU_POSITIVE;
    return dg::launch_status(dg::launch_act_checkpoint(p, (hipStream_t)stream));
}

size_t dg_act_backward_workspace_size(int64_t rows, int64_t cols)
{
    if (rows <= 0 || cols <= 0 || rows > kMaxDim || cols > kMaxDim) return 0;
    return (size_t)dg::act_backward_slices(rows, cols, true) * (size_t)cols * 4;
}

int dg_act_backward(int64_t rows, int64_t cols, const void *dH, int64_t ldh, dg_mx_t format, const void *Q, int64_t ldq,
                    const void *S, int64_t lds, void *dZ, int64_t ldz, dg_elem_t type, dg_epilogue_t activation,
                    float *dbias, void *workspace, size_t workspace_bytes, void *stream)
{
    if (rows < 0 || rows > kMaxDim) return -1;
    if (cols < 0 || cols > kMaxDim) return -2;
    const bool any = rows > 0 && cols > 0;
    if (!is_elem(type)) return -12;
    if (any && (dH == nullptr || !aligned(dH, elem_size(type)))) return -3;
    if (ldh < (cols > 1 ? cols : 1)) return -4;
    if (format != DG_MXFP8 && format != DG_MXINT8) return -5;
    if (any && bad_q(Q)) return -6;
    if (bad_ldq(ldq, format, cols)) return -7;
    if (any && bad_s(S)) return -8;
    if (lds < rows) return -9;
    if (any && (dZ == nullptr || !aligned(dZ, elem_size(type)))) return -10;
    if (ldz < (cols > 1 ? cols : 1) || (dZ == dH && any && ldz != ldh)) return -11;
    if (activation != DG_EPI_RELU && activation != DG_EPI_GELU) return -13;
    if (dbias && !aligned(dbias, 4)) return -14;
    if (cols == 0) return DG_OK;
    if (dbias && rows > 0) {
        if (workspace == nullptr || !aligned(workspace, 16)) return -15;
        if (workspace_bytes < dg_act_backward_workspace_size(rows, cols)) return -16;
    }
    if (rows == 0 && !dbias) return DG_OK;
    MxParams p = {};
    p.X = dH;
    p.Y = dZ;
    p.Q = (uint8_t *)Q;
    p.S = (uint8_t *)S;
    p.ldx = ldh;
    p.ldy = ldz;
    p.ldq = ldq;
    p.lds = lds;
    p.rows = rows;
    p.cols = cols;
    p.type = type;
    p.format = format;
    p.act = activation;
    p.dbias = dbias;
    p.ws = (float *)workspace;
    p.band = dg::act_backward_band(rows, cols, dbias != nullptr);
    p.slices = rows > 0 ? dg::act_backward_slices(rows, cols, dbias != nullptr) : 0;   // no rows: the sums are zero
    return dg::launch_status(dg::launch_act_backward(p, (hipStream_t)stream));
}

int dg_gemm_mx_with_kernel(int64_t M, int64_t N, int64_t K, float alpha, dg_mx_t formatA, const void *A, int64_t lda,
                           const void *SA, int64_t ldsa, dg_mx_t formatB, const void *B, int64_t ldb, const void *SB,
                           int64_t ldsb, float beta, void *C, int64_t ldc, dg_elem_t type, const void *bias,
                           dg_epilogue_t epilogue, void *stream, int kernel)
{
    if (M < 0 || M > kMaxDim) return -1;
    if (N < 0 || N > kMaxDim) return -2;
    if (K < 0 || K > kMaxDim - dg::MX_GROUP) return -3;
    const bool out = M > 0 && N > 0, reads = out && K > 0 && alpha != 0.f;
    if (formatA != DG_MXFP4 && formatA != DG_MXFP8) return -5;
    if (reads && bad_q(A)) return -6;
    if (bad_ldq(lda, formatA, K)) return -7;
    if (reads && bad_s(SA)) return -8;
    if (ldsa < M) return -9;
    if (formatB != DG_MXFP4) return -10;
    if (reads && bad_q(B)) return -11;
    if (bad_ldq(ldb, formatB, K)) return -12;
    if (reads && bad_s(SB)) return -13;
    if (ldsb < N) return -14;
    if (!is_elem(type)) return -18;
    if (out && (C == nullptr || !aligned(C, elem_size(type)))) return -16;
    if (ldc < (N > 1 ? N : 1)) return -17;
    if (bias && !aligned(bias, elem_size(type))) return -19;
    if (epilogue != DG_EPI_NONE && epilogue != DG_EPI_RELU && epilogue != DG_EPI_GELU) return -20;
    if (!out) return DG_OK;
    if (kernel != DG_KERNEL_AUTO && (kernel < 0 || kernel >= kNumMx)) return DG_ERR_UNSUPPORTED;

    MxGemmParams p = {};
    p.g.A = A;
    p.g.B = B;
    p.g.C = C;
    p.g.lda = lda;
    p.g.ldb = ldb;
    p.g.ldc = ldc;
    p.g.M = (int32_t)M;
    p.g.N = (int32_t)N;
    p.g.K = (int32_t)(dg::mx_groups(K) * dg::MX_GROUP);   // rows hold whole groups, zeros past K
    p.g.alpha = alpha;
    p.g.beta = beta;
    p.g.splits = 1;
    p.g.bias = bias;
    p.g.act = epilogue;
    p.g.batch = 1;
    p.SA = (const uint8_t *)SA;
    p.SB = (const uint8_t *)SB;
    p.ldsa = ldsa;
    p.ldsb = ldsb;
    p.ctype = type;
    if (!reads) return dg::launch_status(dg::scale_launcher(c_dtype(type))(p.g, (hipStream_t)stream));
    const bool exact = formatA == DG_MXFP8 && type == DG_ELEM_F32;
    if (kernel == DG_KERNEL_AUTO) kernel = mx_choose(formatA == DG_MXFP4, exact, M, N, K, lda, ldb);
    if (kernel < 0 || !mx_supports(kernel, M, N, lda, ldb)) return DG_ERR_UNSUPPORTED;
    const MxFamily &f = kMx[kernel];
    p.g.tiles_m = (int32_t)ceil_div(M, f.bm);
    p.g.tiles_n = (int32_t)ceil_div(N, f.bn);
    p.g.group_m = f.group_m;
    return dg::launch_status(dg::mx_gemm_launcher(kernel, formatA, exact)(p, (hipStream_t)stream));
}

int dg_gemm_mx(int64_t M, int64_t N, int64_t K, float alpha, dg_mx_t formatA, const void *A, int64_t lda, const void *SA,
               int64_t ldsa, dg_mx_t formatB, const void *B, int64_t ldb, const void *SB, int64_t ldsb, float beta,
               void *C, int64_t ldc, dg_elem_t type, const void *bias, dg_epilogue_t epilogue, void *stream)
{
    return dg_gemm_mx_with_kernel(M, N, K, alpha, formatA, A, lda, SA, ldsa, formatB, B, ldb, SB, ldsb, beta, C, ldc,
                                  type, bias, epilogue, stream, DG_KERNEL_AUTO);
}

int dg_gemm_mx_select(dg_mx_t formatA, int64_t M, int64_t N, int64_t K)
{
    if (formatA != DG_MXFP4 && formatA != DG_MXFP8) return -1;
    if (M < 0 || M > kMaxDim) return -2;
    if (N < 0 || N > kMaxDim) return -3;
    if (K < 0 || K > kMaxDim - dg::MX_GROUP) return -4;
    const int k = mx_choose(formatA == DG_MXFP4, false, M, N, K, row_bytes(formatA, K), row_bytes(DG_MXFP4, K));
    return k < 0 ? DG_ERR_UNSUPPORTED : k;
}

const char *dg_gemm_mx_kernel_name(int kernel) { return kernel >= 0 && kernel < kNumMx ? kMx[kernel].name : nullptr; }

int dg_gemm_dq_choose(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || M > kMaxDim) return -1;
    if (N < 0 || N > kMaxDim) return -2;
    if (K < 0 || K > kMaxDim) return -3;
    if (M == 0 || N == 0 || K == 0) return 1;
    int tile = 0, ranges = 1;
    dq_choose(M, N, K, true, 0, &tile, &ranges);
    return ranges;
}

int dg_gemm_dq_select(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || M > kMaxDim) return -1;
    if (N < 0 || N > kMaxDim) return -2;
    if (K < 0 || K > kMaxDim) return -3;
    int tile = 0, ranges = 1;
    if (M > 0 && N > 0 && K > 0) dq_choose(M, N, K, true, 0, &tile, &ranges);
    return tile;
}

const char *dg_gemm_dq_kernel_name(int kernel) { return kernel >= 0 && kernel < kNumDq ? kDq[kernel].name : nullptr; }

int dg_gemm_dq(dg_op_t transA, int64_t M, int64_t N, int64_t K, float alpha, const void *A, int64_t lda,
               dg_elem_t typeA, dg_mx_t formatB, const void *B, int64_t ldb, const void *SB, int64_t ldsb, float beta,
               void *C, int64_t ldc, dg_elem_t typeC, int splits, void *workspace, size_t workspace_bytes, void *stream)
{
    return dg_gemm_dq_with_kernel(transA, M, N, K, alpha, A, lda, typeA, formatB, B, ldb, SB, ldsb, beta, C, ldc, typeC,
                                  splits, workspace, workspace_bytes, stream, DG_KERNEL_AUTO);
}

int dg_gemm_dq_with_kernel(dg_op_t transA, int64_t M, int64_t N, int64_t K, float alpha, const void *A, int64_t lda,
                           dg_elem_t typeA, dg_mx_t formatB, const void *B, int64_t ldb, const void *SB, int64_t ldsb,
                           float beta, void *C, int64_t ldc, dg_elem_t typeC, int splits, void *workspace,
                           size_t workspace_bytes, void *stream, int kernel)
{
    if (transA != DG_OP_N && transA != DG_OP_T) return -1;
    if (M < 0 || M > kMaxDim) return -2;
    if (N < 0 || N > kMaxDim) return -3;
    if (K < 0 || K > kMaxDim - 64) return -4;
    const bool out = M > 0 && N > 0, reads = out && K > 0 && alpha != 0.f;
    if (reads && (A == nullptr || !aligned(A, 2))) return -6;
    const int64_t inner = transA == DG_OP_T ? M : K;
    if (lda < (inner > 1 ? inner : 1)) return -7;
    if (typeA != DG_ELEM_F16 && typeA != DG_ELEM_BF16) return -8;
    if (!is_format(formatB)) return -9;
    if (reads && bad_q(B)) return -10;
    if (bad_ldq(ldb, formatB, N)) return -11;
    if (reads && bad_s(SB)) return -12;
    if (ldsb < K) return -13;
    if (typeC != typeA && typeC != DG_ELEM_F32) return -17;
    if (out && (C == nullptr || !aligned(C, elem_size(typeC)))) return -15;
    if (ldc < (N > 1 ? N : 1)) return -16;
    if (splits < 0 || splits > 4096) return -18;
    if (!out) return DG_OK;
    if (kernel != DG_KERNEL_AUTO && (kernel < 0 || kernel >= kNumDq)) return DG_ERR_UNSUPPORTED;

    MxGemmParams p = {};
    p.g.A = A;
    p.g.B = B;
    p.g.C = C;
    p.g.lda = lda;
    p.g.ldb = ldb;
    p.g.ldc = ldc;
    p.g.M = (int32_t)M;
    p.g.N = (int32_t)N;
    p.g.K = (int32_t)K;
    p.g.alpha = alpha;
    p.g.beta = beta;
    p.g.c_vec = c_rows4(C, ldc, typeC);
    p.g.splits = 1;
    p.g.batch = 1;
    p.SB = (const uint8_t *)SB;
    p.ldsb = ldsb;
    p.ctype = typeC;
    const int cd = c_dtype(typeC);
    if (!reads) return dg::launch_status(dg::scale_launcher(cd)(p.g, (hipStream_t)stream));

    const int direct = aligned(A, 4) && lda % 2 == 0 && offsets_fit(lda * 2) && (transA == DG_OP_N || M % 8 == 0);
    int k = 0;
    // (the choice of ranges is dg_gemm_dq_choose's, which knows no alignment)
    if (splits == 0) dq_choose(M, N, K, true, 0, &k, &splits);
    dq_choose(M, N, K, direct, splits, &k, &splits);
    if (kernel != DG_KERNEL_AUTO) k = kernel;
    if (k == 3 && !direct) return DG_ERR_UNSUPPORTED;
    const int64_t tm = ceil_div(M, kDq[k].bm), tn = ceil_div(N, kDq[k].bn), chunk = dq_chunk(K, splits);
    if (tm * tn * splits >= (1 << 22)) return DG_ERR_UNSUPPORTED;    // a launch of fewer than 2^31 threads
    if (splits > 1) {
        if (workspace == nullptr || !aligned(workspace, 16)) return -19;
        if ((size_t)splits * (size_t)M * (size_t)N * 4 > workspace_bytes) return -20;
        p.g.splits = splits;
        p.g.k_chunk = (int32_t)chunk;
        p.g.ws = (float *)workspace;
    }
    p.g.tiles_m = (int32_t)tm;
    p.g.tiles_n = (int32_t)tn;
    p.g.group_m = 4;
    int rc = dg::launch_status(dg::dq_gemm_launcher(typeA, k, formatB, transA, direct)(p, (hipStream_t)stream));
    if (rc == DG_OK && splits > 1) rc = dg::launch_status(dg::splitk_reduce_launcher(cd)(p.g, (hipStream_t)stream));
    return rc;
}

}  // extern "C"
