// Host side of a layer's products: argument checks, kernel choice and launches on
// the caller's stream.  The C ABI is declared in include/dense_gemm.h.
#include "../../include/dense_gemm.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "layer_common.hpp"

namespace dg {
int launch_status(hipError_t err);
const void *layer_kernel_f32(int config, int variant);
const void *layer_kernel_f16(int config, int variant);
const void *layer_kernel_bf16(int config, int variant);
hipError_t launch_layer_join(const LayerParams &p, hipStream_t s);
hipError_t launch_layer_colsum(const LayerParams &p, int type, hipStream_t s);
}  // namespace dg

namespace {

using dg::LayerParams;

// Row and column counts leave room for a tile past the end.
constexpr int64_t kMaxDim = 0x7fffffff, kMaxTiled = kMaxDim - 1024;
constexpr int kMaxGroups = 65535;      // a grid dimension

bool is_dtype(int d) { return d >= DG_F32 && d <= DG_BF16_F32OUT; }
// Operand and output elements: 0 fp32, 1 fp16, 2 bf16.
int operand_type(int d) { return d == DG_F32 ? 0 : d == DG_F16_F32ACC || d == DG_F16_F32OUT ? 1 : 2; }
int output_type(int d) { return d == DG_F16_F32ACC ? 1 : d == DG_BF16_F32ACC ? 2 : 0; }
int64_t bytes_of(int type) { return type == 0 ? 4 : 2; }
bool bad_ptr(const void *p, int64_t align) { return p == nullptr || (uintptr_t)p % (uintptr_t)align != 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t max1(int64_t x) { return x > 1 ? x : 1; }

// How a kernel loads its operands.  ANY: the operands that the direct loads do not
// take through registers (three entries of the kernel tables, A, B or both).
// ROWS, STREAM: few rows (bn is that of a B stored N x K); STREAM with direct loads.
enum Loads { ANY, DIRECT, ROWS, STREAM };
struct LayerFamily {
    const char *name;
    int config;          // in the kernel tables
    int bm, bn, group_m, threads;
    Loads loads;
};
const LayerFamily kLayer[] = {
    {"layer_64x64_any", 0, 64, 64, 4, 256, ANY},
    {"layer_128x128_any", 3, 128, 128, 4, 256, ANY},
    {"layer_64x64_deep", 6, 64, 64, 4, 256, DIRECT},
    {"layer_64x64", 7, 64, 64, 4, 256, DIRECT},
    {"layer_128x128_deep", 8, 128, 128, 4, 512, DIRECT},
    {"layer_128x128", 9, 128, 128, 4, 256, DIRECT},
    {"layer_256x256", 10, 256, 256, 4, 512, DIRECT},
    {"layer_16_rows", 11, 16, 16, 8, 512, ROWS},
    {"layer_16_rows_stream", 12, 16, 16, 8, 512, STREAM},
};
constexpr int kNumLayer = sizeof(kLayer) / sizeof(kLayer[0]);
enum { K_ANY_64, K_ANY_128, K_64_DEEP, K_64, K_128_DEEP, K_128, K_256, K_ROWS, K_STREAM };

// What the choice of a kernel looks at.
struct LayerShape {
    int kind, type;
    bool tb, ragged;
    int64_t groups, M, N, K;      // as LayerParams
    bool out32;                   // C is fp32
    bool direct_a, direct_b;      // the direct loads take the operand
    bool direct() const { return direct_a && direct_b; }
};

// The direct loads' 16-byte pieces lie at whole multiples of 16 bytes from a row's
// start, which has to be 4-byte aligned, and 256 rows lie within 32-bit byte offsets.
bool direct_ok(const void *x, int64_t ld, int64_t stride, int64_t bytes)
{
    return ((uintptr_t)x & 3) == 0 && ld * bytes % 4 == 0 && stride * bytes % 4 == 0 && 256 * ld * bytes < ((int64_t)1 << 31);
}

// Tiles are powers of two wide.
int log2_of(int x) { return __builtin_ctz((unsigned)x); }
int64_t tiles_of(int64_t x, int b) { return (x + b - 1) >> log2_of(b); }
int bn_of(const LayerFamily &f, const LayerShape &s) { return f.loads == ROWS && !s.tb ? 64 : f.bn; }

// The most tiles a launch can have: each group that has rows ends in a partial tile
// (weights: a multiple of 8 for each group).
int64_t most_tiles(const LayerShape &s, const LayerFamily &f)
{
    const int64_t tn = tiles_of(s.N, bn_of(f, s));
    if (s.kind == dg::LAYER_WEIGHTS) return s.groups * ((tiles_of(s.M, f.bm) * tn + 7) & ~(int64_t)7);
    const int64_t used = s.ragged && s.groups < s.M ? s.groups : s.ragged ? s.M : 1;
    return ((s.M + used * (f.bm - 1)) >> log2_of(f.bm)) * tn;
}

bool supports(int k, const LayerShape &s)
{
    const LayerFamily &f = kLayer[k];
    if (s.M > kMaxTiled || s.N > kMaxTiled || s.K > kMaxTiled) return false;
    const bool dw = s.kind == dg::LAYER_WEIGHTS;
    if ((f.loads == DIRECT || f.loads == STREAM) && !s.direct()) return false;
    if (f.loads == STREAM && (dw || !s.tb)) return false;
    if (s.type == 0 && (k == K_128_DEEP || k == K_256)) return false;
    // the row kernels' columns of a B stored K x N go four together
    if (f.loads == ROWS && (dw || (!s.tb && s.N < 4))) return false;
    // a launch holds fewer than 2^32 threads
    return most_tiles(s, f) * f.threads < ((int64_t)1 << 32);
}

// A kernel's time (us): fixed + (tile + slab * (slabs of 64 summed indices)) for as many
// rounds as the tiles need, `share` of them a round, but no less than the weights'
// megabytes times `read`; + C's megabytes times `out`.  Fitted to the times, replayed
// in a graph, of 12182 random problems (1 to 16384 rows, 32 to 6000 columns and summed
// indices, 0 to 64 groups, aligned and not, all types).  On 8763 others of these sizes the
// choice, ranges included, is 3.2% slower than the fastest kernel and ranges by geometric mean,
// 19% at the 95th of a hundred, 3.2 times at the worst (64 groups with half a row each, K = 43);
// on 873 with 6000 to 32768 columns or summed indices, which no fit saw, 7.3%, 33% and 2.1 times.
// Both sides of some choices (bf16, B stored N x K, M x N x K, us): 24 x 2048 x 5632 stream
// 8.8, 64 deep in 6 ranges and their join 11.6, in one 18.9; 512 x 5632 x 2048 128 deep 22,
// 64 deep 27; 16384 x 5632 x 2048 256 343, 128 388.
struct LayerTime {
    double fixed, tile, slab, share, out, read;
};
const LayerTime kTime16[kNumLayer] = {
    {6.68, 1.12, 0.581, 466, 0.168, 0.226}, {19.5, 2.46, 1.04, 366, 0.256, 0.217}, {7.27, 1.33, 0.205, 187, 0.011, 0.193},
    {6.39, 0.969, 0.486, 467, 0.210, 0.209}, {10.7, 3.51, 0.414, 158, 0.165, 0.207}, {16.2, 2.28, 0.879, 342, 0.276, 0.198},
    {26.8, 3.28, 1.3, 163, 0.301, 0.257}, {4.29, 0.05, 0.203, 150, 1.867, 0.160},
    {3.58, 0.421, 0.0436, 155, 2.0, 0.146},
};
const LayerTime kTime32[kNumLayer] = {
    {7.73, 0, 1.396, 256, 0.124, 0.271}, {19.3, 0, 5.0, 256, 0.1, 0.503}, {7.5, 0, 1.11, 256, 0.471, 0.304},
    {8.03, 0, 1.086, 256, 0.233, 0.282}, {}, {21.2, 0, 4.06, 256, 0.152, 0.382},
    {}, {4.41, 0.05, 0.385, 141, 0.9, 0.161}, {3.7, 0.398, 0.124, 194, 2.0, 0.153},
};
// K_ROWS with a B stored N x K, which it takes where its rows are not aligned.
const LayerTime kTimeRowsT = {4.1, 0.0874, 0.225, 293, 2.0, 0.361};

// A split sum's second launch and its partials' way out and back.
constexpr double kJoin = 2.9, kJoinMb = 0.45;

size_t workspace_bytes_of(int64_t groups, int64_t M, int64_t N, int splits)
{
    if (groups <= 0 || M <= 0 || N <= 0 || splits <= 1) return 0;
    return (size_t)splits * (size_t)groups * (size_t)M * (size_t)(N + 1) * 4;     // and a bias's gradient
}

// The kernel, and with *splits = 0 the K ranges, of least time; a forced kernel or
// number of ranges stays (but groups of rows have one).  More than one range has to
// gain a tenth, and the workspace holds those that are chosen.  The few-rows kernel's
// ranges hold 512 bytes of a row or more.  On 500 random problems of 1 to 96 rows the choice is
// 3.2% slower than the fastest by geometric mean, 17% at the 95th of a hundred, 42% at the
// worst; with ranges of any length 4.3, 18 and 72%; with that kernel in one range only 11.5, 46
// and 89% (1 x 2048 x 5632 fp32, B stored K x N: 14 us, and 20 by the tile then chosen).
int choose(const LayerShape &s, int kernel, int *splits, size_t ws_bytes = SIZE_MAX)
{
    const bool dw = s.kind == dg::LAYER_WEIGHTS;
    const double groups = dw ? (double)s.groups : 1, mb = groups * (double)s.M * (double)s.N * 4e-6;      // in fp32
    const double K = dw && s.ragged ? (double)s.K / (double)s.groups : (double)s.K;
    const double used = (double)(s.groups < s.M ? s.groups : s.M);
    const double weights = dw ? 0 : used * (double)s.N * K * (s.type == 0 ? 4e-6 : 2e-6);
    if (s.ragged && !dw) *splits = 1;      // groups of rows are not split
    double best = 1e300;
    int k_best = -1, n_best = 1;
    for (int k = kernel == DG_KERNEL_AUTO ? 0 : kernel; k < (kernel == DG_KERNEL_AUTO ? kNumLayer : kernel + 1); ++k) {
        if (k < 0 || k >= kNumLayer || !supports(k, s)) continue;
        const LayerFamily &f = kLayer[k];
        const LayerTime &m = s.type == 0 ? kTime32[k] : k == K_ROWS && s.tb ? kTimeRowsT : kTime16[k];
        // the tiles to expect: each group ends in half of one
        const double tn = (double)tiles_of(s.N, bn_of(f, s)), rows = (double)s.M / f.bm;
        const double tiles = dw ? groups * (double)tiles_of(s.M, f.bm) * tn
                                : !s.ragged ? (double)tiles_of(s.M, f.bm) * tn
                                            : (rows > used / 2 ? rows + used / 2 : used) * tn;
        static const int kRanges[] = {1, 2, 3, 4, 6, 8, 12, 16};
        const int many = *splits > 0 || f.loads == STREAM || tiles > 512 || K < 512 ? 1 : 8;
        for (int i = 0; i < many; ++i) {
            const int n = *splits > 0 ? *splits : kRanges[i];
            if (i > 0 && f.loads == ROWS && K * (s.type == 0 ? 4 : 2) < 512. * n) break;
            if (i > 0 && (64. * n > K || tiles * n > 1024 || workspace_bytes_of(s.groups, s.M, s.N, n) > ws_bytes)) break;
            const double slabs = K <= 64. * n ? 1 : K / n / 64;
            double rounds = tiles * n / m.share;
            // an fp32 tile keeps its unit's matrix cores busy: the last round is a whole one
            if (s.type == 0 && f.loads < ROWS && rounds < 4) rounds = (double)(int)(rounds + 0.999);
            if (rounds < 1) rounds = 1;
            const double tiled = (m.tile + m.slab * slabs) * rounds, read = m.read * weights;
            double t = m.fixed + (tiled > read ? tiled : read);
            t += n == 1 ? m.out * mb * (s.out32 ? 1 : 0.5) : kJoin + kJoinMb * mb * n + 0.1 * t;
            if (t < best) {
                best = t;
                k_best = k;
                n_best = n;
            }
        }
    }
    *splits = n_best;
    return k_best;
}

int launch(LayerParams &p, const LayerShape &s, int dtype, int kernel, int splits, void *ws, size_t ws_bytes, int ws_arg,
           hipStream_t stream)
{
    kernel = choose(s, kernel, &splits, ws == nullptr ? 0 : ws_bytes);
    if (kernel < 0) return DG_ERR_UNSUPPORTED;
    const LayerFamily &f = kLayer[kernel];
    p.splits = splits;
    p.ws = (float *)ws;
    if (p.splits > 1) {
        if (bad_ptr(ws, 16)) return -ws_arg;
        if (ws_bytes < workspace_bytes_of(p.groups, p.M, p.N, p.splits)) return -(ws_arg + 1);
    }
    p.tiles_m = (int32_t)ceil_div(p.M, f.bm);
    p.tiles_n = (int32_t)ceil_div(p.N, bn_of(f, s));
    p.group_m = f.group_m;
    p.past_caches = (double)(s.kind == dg::LAYER_WEIGHTS ? s.groups : 1) * (double)s.M * (double)s.N * (s.out32 ? 4 : 2) > 64e6;
    const int type = operand_type(dtype), variant = s.kind == dg::LAYER_WEIGHTS ? 2 : s.tb;
    // (an ANY kernel forced on operands that both could load directly takes both through registers)
    const int config = f.config + (f.loads != ANY || (!s.direct_a && s.direct_b) ? 0 : s.direct_a && !s.direct_b ? 1 : 2);
    const void *k = type == 0 ? dg::layer_kernel_f32(config, variant)
                              : type == 1 ? dg::layer_kernel_f16(config, variant) : dg::layer_kernel_bf16(config, variant);
    LayerParams arg = p;
    void *args[] = {&arg};
    hipError_t err = hipLaunchKernel(k, dim3((unsigned)most_tiles(s, f), (unsigned)p.splits), dim3((unsigned)f.threads), args,
                                     0, stream);
    if (err == hipSuccess && p.splits > 1) err = dg::launch_layer_join(p, stream);
    return dg::launch_status(err);
}

// The products over rows.  The arguments up to strideB (12) and from C (21) on stand
// at the same places in dg_gemm_fused and dg_gemm_act_grad; `p` brings those
// between them, checked by the caller from `between` on.
struct RowsCall {
    int transB;
    int64_t groups;
    const int32_t *offsets;
    int64_t M, N, K;
    float alpha;
    const void *A;
    int64_t lda;
    const void *B;
    int64_t ldb, strideB;
    void *C;
    int64_t ldc;
    int dtype, splits;
    void *workspace;
    size_t workspace_bytes;
    void *stream;
    int kernel;
    bool work() const { return M > 0 && N > 0 && groups > 0; }
};

// A matrix of rows that may be left out: -pos for its pointer, -(pos + 1) for its stride.
int check_rows(const void *x, int64_t ld, int64_t N, int64_t bytes, int pos)
{
    if (x == nullptr) return 0;
    return bad_ptr(x, bytes) ? -pos : ld < max1(N) ? -(pos + 1) : 0;
}

template <typename F>
int rows_product(const RowsCall &c, LayerParams &p, F between)
{
    if (c.transB != DG_OP_N && c.transB != DG_OP_T) return -1;
    if (c.groups < 0 || c.groups > kMaxGroups || (c.offsets == nullptr && c.groups != 1)) return -2;
    if (c.offsets != nullptr && bad_ptr(c.offsets, 4)) return -3;
    if (c.M < 0 || c.M > kMaxDim) return -4;
    if (c.N < 0 || c.N > kMaxDim) return -5;
    if (c.K < 0 || c.K > kMaxDim) return -6;
    if (!is_dtype(c.dtype)) return -23;
    const int64_t eb = bytes_of(operand_type(c.dtype)), cb = bytes_of(output_type(c.dtype));
    const bool reads = c.work() && c.K > 0 && c.alpha != 0.f;
    if (reads && bad_ptr(c.A, eb)) return -8;
    if (c.lda < max1(c.K)) return -9;
    if (reads && bad_ptr(c.B, eb)) return -10;
    if (c.ldb < max1(c.transB == DG_OP_T ? c.K : c.N)) return -11;
    if (c.strideB < 0) return -12;
    const int rc = between(cb);
    if (rc != 0) return rc;
    if (c.work() && bad_ptr(c.C, cb)) return -21;
    if (c.ldc < max1(c.N)) return -22;
    if (c.splits < 0 || c.splits > 4096) return -24;
    if (!c.work()) return DG_OK;
    p.A = c.A;
    p.B = c.B;
    p.lda = c.lda;
    p.ldb = c.ldb;
    p.strideB = c.strideB;
    p.M = (int32_t)c.M;
    p.N = (int32_t)c.N;
    p.K = reads ? (int32_t)c.K : 0;
    p.alpha = reads ? c.alpha : 0.f;
    p.offsets = c.offsets;
    p.groups = (int32_t)c.groups;
    if (p.beta == 0.f) p.R = nullptr;
    p.C = c.C;
    p.ldc = c.ldc;
    p.ctype = output_type(c.dtype);
    const LayerShape s = {p.kind, operand_type(c.dtype), c.transB == DG_OP_T, c.offsets != nullptr, c.groups, c.M, c.N, p.K, cb == 4,
                          direct_ok(c.A, c.lda, 0, eb), direct_ok(c.B, c.ldb, c.strideB, eb)};
    return launch(p, s, c.dtype, c.kernel, c.splits, c.workspace, c.workspace_bytes, 25, (hipStream_t)c.stream);
}

// An operand as a query of the choice knows it: by its address and row stride, or one
// that the direct loads take.
struct Operand {
    const void *x;
    int64_t ld;
};
constexpr Operand kAligned = {nullptr, 0};

// The choice for such operands, or -i (1 M, 2 N, 3 K, 4 transB, 5 dtype; 1 groups, 2
// rows, 3 M, 4 N, 5 dtype; 7 A's row stride, 9 B's).
int select_rows(int transB, int64_t groups, int64_t M, int64_t N, int64_t K, int dtype, bool ragged, int *splits,
                Operand A = kAligned, Operand B = kAligned)
{
    if (M < 0 || M > kMaxDim) return -1;
    if (N < 0 || N > kMaxDim) return -2;
    if (K < 0 || K > kMaxDim) return -3;
    if (transB != DG_OP_N && transB != DG_OP_T) return -4;
    if (!is_dtype(dtype)) return -5;
    if (A.ld < 0) return -7;
    if (B.ld < 0) return -9;
    const int64_t eb = bytes_of(operand_type(dtype));
    const LayerShape s = {dg::LAYER_FORWARD, operand_type(dtype), transB == DG_OP_T, ragged, max1(groups), max1(M), max1(N), K,
                          output_type(dtype) == 0, direct_ok(A.x, A.ld, 0, eb), direct_ok(B.x, B.ld, 0, eb)};
    const int k = choose(s, DG_KERNEL_AUTO, splits);
    return k < 0 ? DG_ERR_UNSUPPORTED : k;
}

int select_dw(int64_t groups, int64_t rows, int64_t M, int64_t N, int dtype, int *splits, Operand A = kAligned,
              Operand B = kAligned)
{
    if (groups < 0 || groups > kMaxGroups) return -1;
    if (rows < 0 || rows > kMaxDim) return -2;
    if (M < 0 || M > kMaxDim) return -3;
    if (N < 0 || N > kMaxDim) return -4;
    if (!is_dtype(dtype)) return -5;
    if (A.ld < 0) return -7;
    if (B.ld < 0) return -9;
    const int64_t eb = bytes_of(operand_type(dtype));
    const LayerShape s = {dg::LAYER_WEIGHTS, operand_type(dtype), false, groups > 1, max1(groups), max1(M), max1(N), rows,
                          output_type(dtype) == 0, direct_ok(A.x, A.ld, 0, eb), direct_ok(B.x, B.ld, 0, eb)};
    const int k = choose(s, DG_KERNEL_AUTO, splits);
    return k < 0 ? DG_ERR_UNSUPPORTED : k;
}

}  // namespace

extern "C" {

int dg_gemm_fused_with_kernel(dg_op_t transB, int64_t groups, const int32_t *offsets, int64_t M, int64_t N, int64_t K,
                              float alpha, const void *A, int64_t lda, const void *B, int64_t ldb, int64_t strideB,
                              const void *bias, int64_t strideBias, dg_epilogue_t epilogue, void *Z, int64_t ldz, float beta,
                              const void *R, int64_t ldr, void *C, int64_t ldc, dg_dtype_t dtype, int splits,
                              void *workspace, size_t workspace_bytes, void *stream, int kernel)
{
    const RowsCall c = {transB, groups, offsets, M, N, K, alpha, A, lda, B, ldb, strideB, C, ldc, dtype, splits, workspace,
                        workspace_bytes, stream, kernel};
    LayerParams p = {};
    p.kind = dg::LAYER_FORWARD;
    return rows_product(c, p, [&](int64_t cb) {
        if (bias != nullptr && bad_ptr(bias, cb)) return -13;
        if (strideBias < 0) return -14;
        if (epilogue != DG_EPI_NONE && epilogue != DG_EPI_RELU && epilogue != DG_EPI_GELU) return -15;
        if (int rc = check_rows(Z, ldz, N, cb, 16)) return rc;
        if (int rc = check_rows(R, ldr, N, cb, 19)) return rc;
        p.bias = bias;
        p.stride_bias = strideBias;
        p.act = epilogue;
        p.keep = Z;
        p.ldk = ldz;
        p.beta = beta;
        p.R = R;
        p.ldr = ldr;
        return 0;
    });
}

int dg_gemm_fused(dg_op_t transB, int64_t groups, const int32_t *offsets, int64_t M, int64_t N, int64_t K, float alpha,
                  const void *A, int64_t lda, const void *B, int64_t ldb, int64_t strideB, const void *bias,
                  int64_t strideBias, dg_epilogue_t epilogue, void *Z, int64_t ldz, float beta, const void *R, int64_t ldr,
                  void *C, int64_t ldc, dg_dtype_t dtype, int splits, void *workspace, size_t workspace_bytes, void *stream)
{
    return dg_gemm_fused_with_kernel(transB, groups, offsets, M, N, K, alpha, A, lda, B, ldb, strideB, bias, strideBias,
                                     epilogue, Z, ldz, beta, R, ldr, C, ldc, dtype, splits, workspace, workspace_bytes,
                                     stream, DG_KERNEL_AUTO);
}

int dg_gemm_act_grad_with_kernel(dg_op_t transB, int64_t groups, const int32_t *offsets, int64_t M, int64_t N, int64_t K,
                                 float alpha, const void *A, int64_t lda, const void *B, int64_t ldb, int64_t strideB,
                                 float beta, const void *R, int64_t ldr, void *H, int64_t ldh, dg_epilogue_t activation,
                                 const void *Z, int64_t ldz, void *C, int64_t ldc, dg_dtype_t dtype, int splits,
                                 void *workspace, size_t workspace_bytes, void *stream, int kernel)
{
    const RowsCall c = {transB, groups, offsets, M, N, K, alpha, A, lda, B, ldb, strideB, C, ldc, dtype, splits, workspace,
                        workspace_bytes, stream, kernel};
    LayerParams p = {};
    p.kind = dg::LAYER_GRAD;
    return rows_product(c, p, [&](int64_t cb) {
        if (int rc = check_rows(R, ldr, N, cb, 14)) return rc;
        if (int rc = check_rows(H, ldh, N, cb, 16)) return rc;
        if (activation != DG_EPI_RELU && activation != DG_EPI_GELU) return -18;
        if (c.work() && bad_ptr(Z, cb)) return -19;
        if (ldz < max1(N)) return -20;
        p.beta = beta;
        p.R = R;
        p.ldr = ldr;
        p.keep = H;
        p.ldk = ldh;
        p.act = activation;
        p.Z = Z;
        p.ldz = ldz;
        return 0;
    });
}

int dg_gemm_act_grad(dg_op_t transB, int64_t groups, const int32_t *offsets, int64_t M, int64_t N, int64_t K, float alpha,
                     const void *A, int64_t lda, const void *B, int64_t ldb, int64_t strideB, float beta, const void *R,
                     int64_t ldr, void *H, int64_t ldh, dg_epilogue_t activation, const void *Z, int64_t ldz, void *C,
                     int64_t ldc, dg_dtype_t dtype, int splits, void *workspace, size_t workspace_bytes, void *stream)
{
    return dg_gemm_act_grad_with_kernel(transB, groups, offsets, M, N, K, alpha, A, lda, B, ldb, strideB, beta, R, ldr, H,
                                        ldh, activation, Z, ldz, C, ldc, dtype, splits, workspace, workspace_bytes, stream,
                                        DG_KERNEL_AUTO);
}

int dg_gemm_dw_with_kernel(int64_t groups, const int32_t *offsets, int64_t rows, int64_t M, int64_t N, float alpha,
                           const void *A, int64_t lda, const void *B, int64_t ldb, float beta, void *C, int64_t ldc,
                           int64_t strideC, float *dbias, dg_dtype_t dtype, int splits, void *workspace,
                           size_t workspace_bytes, void *stream, int kernel)
{
    if (groups < 0 || groups > kMaxGroups || (offsets == nullptr && groups != 1)) return -1;
    if (offsets != nullptr && bad_ptr(offsets, 4)) return -2;
    if (rows < 0 || rows > kMaxDim) return -3;
    if (M < 0 || M > kMaxDim) return -4;
    if (N < 0 || N > kMaxDim) return -5;
    if (!is_dtype(dtype)) return -16;
    const int64_t eb = bytes_of(operand_type(dtype)), cb = bytes_of(output_type(dtype));
    const bool work = groups > 0 && M > 0 && N > 0, sums = dbias != nullptr && groups > 0 && M > 0;
    const bool reads = work && rows > 0 && alpha != 0.f;
    if ((reads || (sums && rows > 0)) && bad_ptr(A, eb)) return -7;
    if (lda < max1(M)) return -8;
    if (reads && bad_ptr(B, eb)) return -9;
    if (ldb < max1(N)) return -10;
    if (work && bad_ptr(C, cb)) return -12;
    if (ldc < max1(N)) return -13;
    if (strideC < 0 || (work && groups > 1 && strideC < (M - 1) * ldc + N)) return -14;
    if (dbias != nullptr && bad_ptr(dbias, 4)) return -15;
    if (splits < 0 || splits > 4096) return -17;
    LayerParams p = {};
    p.kind = dg::LAYER_WEIGHTS;
    p.A = A;
    p.B = B;
    p.lda = lda;
    p.ldb = ldb;
    p.M = (int32_t)M;
    p.N = (int32_t)N;
    p.K = (int32_t)rows;
    p.alpha = alpha;
    p.beta = beta;
    p.offsets = offsets;
    p.groups = (int32_t)groups;
    p.R = beta != 0.f ? C : nullptr;
    p.ldr = ldc;
    p.C = C;
    p.ldc = ldc;
    p.strideC = strideC;
    p.ctype = output_type(dtype);
    p.dbias = dbias;
    // the bias's gradient comes with the product, or by a pass of its own without one
    const bool alone = sums && !reads && (rows > 0 || !work);
    // (a launch of 512 threads for 64 columns holds fewer than 2^32)
    if (alone && (M > ((int64_t)1 << 28) || rows > kMaxTiled)) return DG_ERR_UNSUPPORTED;
    if (work) {
        LayerParams q = p;
        if (!reads) {
            q.K = 0;
            q.alpha = 0.f;
        }
        if (alone) q.dbias = nullptr;
        const LayerShape s = {p.kind, operand_type(dtype), false, offsets != nullptr, groups, M, N, q.K, cb == 4,
                              direct_ok(A, lda, 0, eb), direct_ok(B, ldb, 0, eb)};
        const int rc = launch(q, s, dtype, kernel, splits, workspace, workspace_bytes, 18, (hipStream_t)stream);
        if (rc != DG_OK) return rc;
    }
    return alone ? dg::launch_status(dg::launch_layer_colsum(p, operand_type(dtype), (hipStream_t)stream)) : DG_OK;
}

int dg_gemm_dw(int64_t groups, const int32_t *offsets, int64_t rows, int64_t M, int64_t N, float alpha, const void *A,
               int64_t lda, const void *B, int64_t ldb, float beta, void *C, int64_t ldc, int64_t strideC, float *dbias,
               dg_dtype_t dtype, int splits, void *workspace, size_t workspace_bytes, void *stream)
{
    return dg_gemm_dw_with_kernel(groups, offsets, rows, M, N, alpha, A, lda, B, ldb, beta, C, ldc, strideC, dbias, dtype,
                                  splits, workspace, workspace_bytes, stream, DG_KERNEL_AUTO);
}

int dg_gemm_fused_choose(int64_t M, int64_t N, int64_t K, dg_op_t transB, dg_dtype_t dtype)
{
    int splits = 0;
    const int k = select_rows(transB, 1, M, N, K, dtype, false, &splits);
    return k < 0 ? k : splits;
}

int dg_gemm_fused_choose_for(int64_t M, int64_t N, int64_t K, dg_op_t transB, dg_dtype_t dtype, const void *A, int64_t lda,
                             const void *B, int64_t ldb)
{
    int splits = 0;
    const int k = select_rows(transB, 1, M, N, K, dtype, false, &splits, {A, lda}, {B, ldb});
    return k < 0 ? k : splits;
}

int dg_gemm_fused_select(int64_t M, int64_t N, int64_t K, dg_op_t transB, dg_dtype_t dtype, int64_t groups, int splits)
{
    if (groups < 0 || groups > kMaxGroups) return -6;
    if (splits < 0 || splits > 4096) return -7;
    return select_rows(transB, groups, M, N, K, dtype, groups > 0, &splits);
}

int dg_gemm_dw_choose(int64_t groups, int64_t rows, int64_t M, int64_t N, dg_dtype_t dtype)
{
    int splits = 0;
    const int k = select_dw(groups, rows, M, N, dtype, &splits);
    return k < 0 ? k : splits;
}

int dg_gemm_dw_choose_for(int64_t groups, int64_t rows, int64_t M, int64_t N, dg_dtype_t dtype, const void *A, int64_t lda,
                          const void *B, int64_t ldb)
{
    int splits = 0;
    const int k = select_dw(groups, rows, M, N, dtype, &splits, {A, lda}, {B, ldb});
    return k < 0 ? k : splits;
}

int dg_gemm_dw_select(int64_t groups, int64_t rows, int64_t M, int64_t N, dg_dtype_t dtype, int splits)
{
    if (splits < 0 || splits > 4096) return -6;
    return select_dw(groups, rows, M, N, dtype, &splits);
}

size_t dg_layer_workspace_size(int64_t groups, int64_t M, int64_t N, int splits)
{
    return workspace_bytes_of(groups, M, N, splits);
}

const char *dg_layer_kernel_name(int kernel) { return kernel >= 0 && kernel < kNumLayer ? kLayer[kernel].name : nullptr; }

}  // extern "C"
