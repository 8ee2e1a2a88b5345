/*
 * dense_gemm.h -- C ABI of libdense_gemm_amd.so, a dense matrix multiply for
 * AMD Instinct MI355X (gfx950).
 *
 * The operation (one call):
 *
 *     C = alpha * op(A) * op(B) + beta * C
 *
 * the full SGEMM form given in "Optimizing GEMM on Apple's M5 from scratch,
 * Part 1", Introduction (whose own runs fix alpha = 1, beta = 0), with the
 * transpose variants of "Metal GEMM Kernels for LoRA Training on Apple
 * Silicon", section 2 ("GEMM structure": nn A[M,K] B[K,N], tn A[K,M]^T B[K,N],
 * nt A[M,K] B[N,K]^T; tt is the remaining combination).
 *
 * Layout.  Every matrix is row-major: element (i, j) of a stored matrix X is
 * X[i * ldX + j] (ld = row stride in elements).  op(A) is M x K and op(B) is
 * K x N:
 *   transA = DG_OP_N: A is stored M x K, lda >= max(1, K)
 *   transA = DG_OP_T: A is stored K x M, lda >= max(1, M)
 *   transB = DG_OP_N: B is stored K x N, ldb >= max(1, N)
 *   transB = DG_OP_T: B is stored N x K, ldb >= max(1, K)
 *   C is stored M x N, ldc >= max(1, N).
 * A sub-matrix is passed as a pointer to its first element plus the parent's
 * ld.  Elements outside the logical extents (padding between rows) are never
 * read and never written.
 *
 * Types (dtype):
 *   DG_F32         A, B, C are fp32; products and sums in fp32 on the fp32
 *                  matrix cores (full precision, no reduced-precision inputs).
 *   DG_F16_F32ACC  A, B, C are IEEE fp16; products are accumulated in fp32
 *                  (the fp16 matrix-core path with fp32 accumulators -- "Metal
 *                  GEMM Kernels for LoRA Training", section 1); the result
 *                  alpha*acc + beta*C is formed in fp32 (an fp16 C is widened
 *                  exactly) and rounded once to fp16, round-to-nearest-even,
 *                  overflow to +-Inf.
 *   DG_BF16_F32ACC A, B, C are bfloat16 (8 significant bits, fp32's exponent
 *                  range); as DG_F16_F32ACC otherwise: fp32 accumulation, one
 *                  round-to-nearest-even to bf16 at the end.  The page above
 *                  (section 1) has bf16 emulated on its GPU; gfx950 has a
 *                  native bf16 matrix-core instruction.
 *   DG_F16_F32OUT  A, B are fp16, C is fp32: the fp16 matrix-core path with
 *                  fp32 accumulators, and alpha*acc + beta*C (fp32 C read as
 *                  is) written to C in fp32 with no rounding to fp16 -- the
 *                  fp32-output variant of "Metal GEMM Kernels for LoRA
 *                  Training", section 4 (writing fp32 straight to device
 *                  memory), for callers that keep fp32 results (gradient
 *                  accumulation, a following fp32 reduction).
 *   DG_BF16_F32OUT A, B are bf16, C is fp32; as DG_F16_F32OUT otherwise.
 *   alpha and beta are fp32 for every type.  The bias of dg_gemm_ex has C's
 *   type.
 *
 * Special values of the arguments:
 *   M == 0 or N == 0       nothing is done (returns DG_OK).
 *   K == 0 or alpha == 0   C = beta * C; A and B are not read.
 *   beta == 0              C is write-only: its old contents (NaN included)
 *                          are not read.
 *
 * Pointers, ownership, execution:
 *   A, B, C are device pointers on the device that `stream` belongs to, owned
 *   by the caller; the library keeps no reference after the call returns.
 *   `stream` is a hipStream_t (NULL = the default stream).  The call enqueues
 *   the work and returns without waiting for it (asynchronous, like any
 *   kernel launch); it allocates no memory.  Calls are thread-safe.
 *   C must not overlap A or B (not checked).
 *
 * Errors (return value):
 *   DG_OK (0)          enqueued (or nothing to do).
 *   -i                 argument i (1-based, in the order of dg_gemm's
 *                      parameters) is invalid: transA/transB not 0 or 1,
 *                      M/N/K negative or above 2^31-1, ld below its minimum,
 *                      NULL pointer with a non-empty extent, unknown dtype.
 *                      Nothing is enqueued.
 *   DG_ERR_UNSUPPORTED the forced kernel cannot run this problem.
 *   DG_ERR_SCRATCH     (dg_gemm_splitk_noalloc) more partials than the
 *                      library's scratch holds.
 *   DG_ERR_HIP         a HIP call failed; dg_last_hip_error() returns its
 *                      hipError_t (per calling thread).
 */
#ifndef DENSE_GEMM_H
#define DENSE_GEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The enumerations are int-sized in both languages (C++ fixes the underlying
 * type, so that every int a caller passes is a value of the parameter's type
 * and the library's own range checks see it); the ABI passes them as int. */
#ifdef __cplusplus
#define DG_ENUM(name) enum name : int
#else
#define DG_ENUM(name) enum name
#endif

/* op(X): X as stored (N) or its transpose (T). */
typedef DG_ENUM(dg_op) { DG_OP_N = 0, DG_OP_T = 1 } dg_op_t;
/* Operand, accumulator and output types (see "Types" above). */
typedef DG_ENUM(dg_dtype) {
    DG_F32 = 0,          /* A, B, C fp32; fp32 accumulation            */
    DG_F16_F32ACC = 1,   /* A, B, C fp16; fp32 accumulation, fp16 out  */
    DG_BF16_F32ACC = 2,  /* A, B, C bf16; fp32 accumulation, bf16 out  */
    DG_F16_F32OUT = 3,   /* A, B fp16; fp32 accumulation, C fp32       */
    DG_BF16_F32OUT = 4   /* A, B bf16; fp32 accumulation, C fp32       */
} dg_dtype_t;
/* Epilogue activations of dg_gemm_ex (DG_EPI_RELU_POSITIVE: dg_act_checkpoint
 * only). */
typedef DG_ENUM(dg_epilogue) {
    DG_EPI_NONE = 0,
    DG_EPI_RELU = 1,
    DG_EPI_GELU = 2,
    DG_EPI_RELU_POSITIVE = 4
} dg_epilogue_t;
/* Element types of the plain matrices beside MX matrices. */
typedef DG_ENUM(dg_elem) { DG_ELEM_F32 = 0, DG_ELEM_F16 = 1, DG_ELEM_BF16 = 2 } dg_elem_t;
/* Formats of MX matrices (see "Block-scaled (MX) matrices" below). */
typedef DG_ENUM(dg_mx) { DG_MXFP4 = 0, DG_MXFP8 = 1, DG_MXINT8 = 2 } dg_mx_t;
#undef DG_ENUM

#define DG_OK 0
#define DG_ERR_UNSUPPORTED (-100)
#define DG_ERR_SCRATCH (-101)
#define DG_ERR_HIP (-200)

/* Kernel choice for dg_gemm_with_kernel: DG_KERNEL_AUTO lets the library pick. */
#define DG_KERNEL_AUTO (-1)

/* C = alpha * op(A) * op(B) + beta * C  (see above). */
int dg_gemm(dg_op_t transA, dg_op_t transB, int64_t M, int64_t N, int64_t K, float alpha,
            const void *A, int64_t lda, const void *B, int64_t ldb, float beta, void *C,
            int64_t ldc, dg_dtype_t dtype, void *stream);

/* Same as dg_gemm, but runs kernel `kernel` (an index into the library's
 * kernel table, see dg_kernel_count / dg_kernel_name) instead of the one the
 * library would pick; DG_KERNEL_AUTO behaves as dg_gemm.  Returns
 * DG_ERR_UNSUPPORTED (nothing enqueued) when that kernel does not handle the
 * problem's dtype, transposes, alignment or row strides (the pipelined
 * kernels address a tile's operands with 32-bit byte offsets, so they need
 * 256 rows of the stored A and of the stored B to span less than 2^31
 * bytes).  For tests and measurement. */
int dg_gemm_with_kernel(dg_op_t transA, dg_op_t transB, int64_t M, int64_t N, int64_t K,
                        float alpha, const void *A, int64_t lda, const void *B, int64_t ldb, float beta,
                        void *C, int64_t ldc, dg_dtype_t dtype, void *stream, int kernel);

/* Extended form: a fused bias + activation epilogue and strided batches.
 *
 *   for b in 0 .. batch-1:
 *     C_b = act(alpha * op(A_b) * op(B_b) + beta * C_b + bias)
 *     with A_b = A + b*strideA, B_b = B + b*strideB, C_b = C + b*strideC
 *     (strides in elements).
 *
 * The epilogue is the fusion of "From a C loop to a GPU kernel", section
 * "Fusion": a per-output bias is added and an elementwise activation applied
 * while the tile is still on chip, and the result is written once.  In a
 * row-major C the outputs of one feature are a column, so bias[j] is added to
 * every element of column j:
 *   x = alpha*acc + beta*C_in + bias[j]   (in fp32, one rounding at the end)
 *   epilogue DG_EPI_NONE: x;  DG_EPI_RELU: max(x, 0) (NaN stays NaN);
 *   DG_EPI_GELU: x * Phi(x) = x/2 * (1 + erf(x / sqrt(2))), the exact-erf
 *   form, Phi the standard normal distribution function.
 * The batch is the per-head offset of "Metal GEMM Kernels for LoRA Training",
 * section 8 (Q, K, V head-major, one GEMM per head at a fixed offset): one
 * call runs every head, so the heads together fill the GPU.
 *
 * Arguments (1-based positions, for the -i error codes):
 *   1-8, 10-11, 13-15, 20-21: as dg_gemm's transA, transB, M, N, K, alpha,
 *       A, lda, B, ldb, beta, C, ldc, dtype, stream.
 *   9 strideA, 12 strideB: >= 0 (0 reuses one matrix for every batch).
 *   16 strideC: >= 0; with batch > 1 the outputs must not overlap:
 *       strideC >= (M-1)*ldc + N.
 *   17 batch: 0 .. 65535 (0: nothing is done).
 *   18 bias: NULL (no bias) or N elements of C's type, contiguous, aligned
 *       to its element size, shared by every batch; caller-owned device
 *       memory.
 *   19 epilogue: DG_EPI_NONE, DG_EPI_RELU or DG_EPI_GELU.
 * Special values as dg_gemm; with K == 0 or alpha == 0 the result is
 * act(beta*C + bias) and A and B are not read.  Pointer rules, asynchrony and
 * errors as dg_gemm (nothing enqueued on error).  No allocation. */
int dg_gemm_ex(dg_op_t transA, dg_op_t transB, int64_t M, int64_t N, int64_t K, float alpha,
               const void *A, int64_t lda, int64_t strideA, const void *B, int64_t ldb,
               int64_t strideB, float beta, void *C, int64_t ldc, int64_t strideC,
               int64_t batch, const void *bias, dg_epilogue_t epilogue, dg_dtype_t dtype,
               void *stream);

/* dg_gemm_ex with a forced kernel, as dg_gemm_with_kernel (argument 22). */
int dg_gemm_ex_with_kernel(dg_op_t transA, dg_op_t transB, int64_t M, int64_t N, int64_t K,
                           float alpha, const void *A, int64_t lda, int64_t strideA, const void *B,
                           int64_t ldb, int64_t strideB, float beta, void *C, int64_t ldc,
                           int64_t strideC, int64_t batch, const void *bias,
                           dg_epilogue_t epilogue, dg_dtype_t dtype, void *stream, int kernel);

/* Split-K form of dg_gemm, for outputs too small to give every compute unit a
 * tile (skinny and low-rank products): K is cut into `splits` ranges (each a
 * multiple of 64 long except the last), each range's products are summed
 * into fp32 partials in `workspace`, and a second kernel forms
 * C = alpha * (sum of the partials, in increasing range order) + beta * C with
 * one rounding to the output type.  This is the split-K remedy of "Metal
 * GEMM Kernels for LoRA Training on Apple Silicon", section 5 (fp32 partials,
 * then a reduction).
 *   splits      1: exactly dg_gemm (workspace unused); 0: the library's
 *               choice (dg_gemm_splitk_choose); n > 1: at most n ranges (the
 *               range length is rounded up to a multiple of 64, so fewer
 *               ranges may result).  Invalid (-16): below 0 or above 4096.
 *   workspace   device memory of at least dg_gemm_splitk_workspace_size(M,
 *               N, splits) bytes, 16-byte aligned, owned by the caller, not
 *               read or written outside that size; its contents on return
 *               are unspecified.  Invalid (-17): NULL or misaligned when
 *               splits != 1 and the output is not empty.  Too small for the
 *               ranges actually used: -18.  Two calls that share a workspace
 *               must be ordered on one stream.
 * Otherwise as dg_gemm (arguments 1-15, same errors, asynchronous). */
int dg_gemm_splitk(dg_op_t transA, dg_op_t transB, int64_t M, int64_t N, int64_t K, float alpha,
                   const void *A, int64_t lda, const void *B, int64_t ldb, float beta, void *C,
                   int64_t ldc, dg_dtype_t dtype, void *stream, int splits, void *workspace,
                   size_t workspace_bytes);

/* Bytes of the library's own split-K scratch on each GPU (see
 * dg_gemm_splitk_noalloc). */
#define DG_SCRATCH_BYTES (16 * 1024 * 1024)

/* dg_gemm_splitk without a workspace and without any allocation, for callers
 * that cannot allocate device memory: code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc.  The fp32 partials go to a
 * device array inside the library, DG_SCRATCH_BYTES (16 MiB) on each GPU,
 * which the GPU holds from the library's load until the process ends.  The
 * call uses the K ranges dg_gemm_splitk would use for the same `splits` (0:
 * the library's choice; 1: no split, the scratch is not touched), computes
 * the same result with the same kernels, and enqueues the same work.
 *   Arguments 1-16: as dg_gemm_splitk's first 16 (same errors, -16 for
 *   splits below 0 or above 4096).
 *   DG_ERR_SCRATCH: the partials, splits * M * N * 4 bytes for the ranges
 *   used, exceed DG_SCRATCH_BYTES; nothing is enqueued (call dg_gemm_splitk
 *   with a workspace, or fewer splits).
 *   DG_ERR_HIP: looking up the scratch's device address failed (first call
 *   on a device only).
 * Every call on one GPU shares that GPU's scratch, and a call leaves its
 * partials there: calls that may overlap on one GPU (on different streams,
 * or from several host threads without ordering) race on it and must be
 * ordered by the caller, for example on one stream.  No memory is cleared:
 * the GEMM kernel writes every partial before the reduction reads it.
 * Asynchronous, like dg_gemm; calls no allocating routine. */
int dg_gemm_splitk_noalloc(dg_op_t transA, dg_op_t transB, int64_t M, int64_t N, int64_t K,
                           float alpha, const void *A, int64_t lda, const void *B, int64_t ldb,
                           float beta, void *C, int64_t ldc, dg_dtype_t dtype, void *stream,
                           int splits);

/* The number of K ranges dg_gemm_splitk uses when called with splits = 0
 * (1 when splitting does not pay), or a negative status for invalid
 * arguments (host logic only). */
int dg_gemm_splitk_choose(dg_op_t transA, dg_op_t transB, int64_t M, int64_t N, int64_t K,
                          dg_dtype_t dtype);

/* Bytes of workspace dg_gemm_splitk needs for `splits` K ranges (0 when
 * splits <= 1 or the output is empty). */
size_t dg_gemm_splitk_workspace_size(int64_t M, int64_t N, int splits);

/* The kernel dg_gemm would run for these arguments (host logic only, no GPU
 * call), or a negative status as dg_gemm would return it. */
int dg_select_kernel(dg_op_t transA, dg_op_t transB, int64_t M, int64_t N, int64_t K, const void *A,
                     int64_t lda, const void *B, int64_t ldb, const void *C, int64_t ldc,
                     dg_dtype_t dtype);

/* ---- Block-scaled (MX) matrices ------------------------------------------------
 *
 * An MX matrix of rows x cols holds each row in blocks of 32 elements (the
 * last one may be short).  A block has one scale 2^e and elements of 4 or 8
 * bits, after the OCP Microscaling Formats (MX) specification v1.0:
 *   DG_MXFP4   E2M1: +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}        emax = 2
 *   DG_MXFP8   E4M3: up to 448                              emax = 8
 *   DG_MXINT8  a signed integer in 64ths, -127 .. 127       emax = 0
 * Rounding (dg_mx_quantize, dg_act_checkpoint): with m the largest magnitude
 * of the block, e = max(floor(log2(m)) - emax, -127) (-127 for m = 0), and
 * each element is x / 2^e rounded to nearest even and saturated to the
 * format's largest.  A block that holds a NaN or an infinity gets a NaN
 * scale and zero elements: all of its values are then NaN.
 *
 * Storage, two buffers in device memory:
 *   Q  elements, row r at byte r * ldq; mxfp4 two elements to a byte, the
 *      even one in the low 4 bits.  A row holds whole groups of 256 elements
 *      (128 bytes of mxfp4, 256 of the others; dg_mx_row_bytes); elements at
 *      or past cols are zero (dg_gemm_mx relies on it: a matrix of fewer
 *      columns than were stored is one only if it ends at a multiple of 256).
 *      Q is 16-byte aligned, ldq a multiple of 16.
 *   S  scales, one byte e + 127 each (255: NaN); the scale of block b of row
 *      r is byte ((b / 8) * lds + r) * 8 + b % 8, so the 8 scales of a row's
 *      group lie together and a group's rows one after the other.  S is
 *      8-byte aligned, lds >= rows (dg_mx_scale_bytes).
 * A row takes the bytes of its whole groups: 136 (mxfp4) or 264 (8 bits) with
 * the scales, per 256 columns begun.  Short rows save little or nothing: 32
 * columns take 64 bytes in 16 bits, and 8-bit storage is the smaller from 133
 * columns on (mxfp4 from 69).
 * Rows r0 .. of a matrix are the matrix at Q + r0 * ldq and S + r0 * 8 with
 * the same ldq and lds; columns from a multiple of 256 on, at Q + (128 or
 * 256) * g and S + g * lds * 8.  Nothing outside a matrix's own rows and
 * groups is written; scales of blocks past cols within the last group are
 * written as 0.
 *
 * Pointers, streams, asynchrony and errors as dg_gemm: -i names an invalid
 * argument by its position (types and formats are checked before the pointers
 * whose alignment depends on them), and nothing is enqueued then.  Plain
 * matrices are aligned to their element.  Sizes are at most 2^31 - 1.  No call allocates memory, and no call keeps state: calls on
 * different streams do not interfere unless they share a workspace or an
 * output. */

/* Bytes of one row of Q, or -i. */
int64_t dg_mx_row_bytes(dg_mx_t format, int64_t cols);

/* Bytes of S for group stride lds, or -i. */
int64_t dg_mx_scale_bytes(int64_t lds, int64_t cols);

/* (Q, S) = op(X) in `format`.  op(X) is rows x cols; transX = DG_OP_T: X is
 * stored cols x rows.  ldx >= max(1, cols) (rows with transX).
 *   1 transX, 2 rows, 3 cols, 4 X, 5 ldx, 6 type, 7 format, 8 Q, 9 ldq, 10 S,
 *   11 lds, 12 stream. */
int dg_mx_quantize(dg_op_t transX, int64_t rows, int64_t cols, const void *X, int64_t ldx, dg_elem_t type,
                   dg_mx_t format, void *Q, int64_t ldq, void *S, int64_t lds, void *stream);

/* X = the values of (Q, S), rounded once to the element type (exact in fp32
 * and bf16 within their range; in fp16 for values that fp16 holds).
 *   1 rows, 2 cols, 3 format, 4 Q, 5 ldq, 6 S, 7 lds, 8 X, 9 ldx, 10 type,
 *   11 stream. */
int dg_mx_dequantize(int64_t rows, int64_t cols, dg_mx_t format, const void *Q, int64_t ldq, const void *S,
                     int64_t lds, void *X, int64_t ldx, dg_elem_t type, void *stream);

/* C = act(alpha * A B^T + beta * C + bias): A is M x K in DG_MXFP4 or
 * DG_MXFP8, B is N x K in DG_MXFP4, both with their blocks along K; C (and the
 * bias, N elements, NULL for none) of type `type`; the epilogue of dg_gemm_ex.
 * Products and sums on the scaled matrix cores with fp32 accumulators, one
 * rounding of the result.  The products of two DG_MXFP4 operands, those of a
 * DG_MXFP8 A when C is fp32, and those of the kernels for few rows of A are
 * summed to the fp32 rounding of each step of 64 or 128 k.  In the tiled kernels
 * with a DG_MXFP8 A and a 16-bit C the hardware adds 8 neighbouring k (from a
 * multiple of 8 on) at a time with each product cut, towards zero, by less than
 * 2^-13 of the largest magnitude among the 8: measured 2.5e-6 by norm on
 * normal data, 1.4e-5 where a few columns of A are eight times the others (C's
 * own rounding: 2e-4 fp16, 1.7e-3 bf16).  Sums that cancel keep that absolute
 * error; an fp32 C does not have it, at up to twice the time.
 *   M == 0 or N == 0: nothing is done; K == 0 or alpha == 0: A and B are not
 *   read, C = act(beta * C + bias); beta == 0: C is not read.
 *   DG_ERR_UNSUPPORTED: more tiles than a launch holds (2^22 of 256 x 256, edge
 *   tiles counted whole: from 2^30 rows of up to 256 columns or 2^19 x 2^19 on).
 *   1 M, 2 N, 3 K, 4 alpha, 5 formatA, 6 A, 7 lda (bytes), 8 SA, 9 ldsa,
 *   10 formatB, 11 B, 12 ldb (bytes), 13 SB, 14 ldsb, 15 beta, 16 C, 17 ldc,
 *   18 type, 19 bias, 20 epilogue, 21 stream. */
int dg_gemm_mx(int64_t M, int64_t N, int64_t K, float alpha, dg_mx_t formatA, const void *A, int64_t lda,
               const void *SA, int64_t ldsa, dg_mx_t formatB, const void *B, int64_t ldb, const void *SB,
               int64_t ldsb, float beta, void *C, int64_t ldc, dg_elem_t type, const void *bias,
               dg_epilogue_t epilogue, void *stream);

/* dg_gemm_mx with a forced kernel (argument 22; DG_KERNEL_AUTO: the
 * library's choice), for tests and measurement; DG_ERR_UNSUPPORTED when it
 * cannot run the problem.  The choice for packed operands and a 16-bit C
 * (DG_ERR_UNSUPPORTED when there is none; or -i: 1 formatA, 2 M, 3 N, 4 K), and
 * the kernels' names (NULL when out of range). */
int dg_gemm_mx_with_kernel(int64_t M, int64_t N, int64_t K, float alpha, dg_mx_t formatA, const void *A,
                           int64_t lda, const void *SA, int64_t ldsa, dg_mx_t formatB, const void *B, int64_t ldb,
                           const void *SB, int64_t ldsb, float beta, void *C, int64_t ldc, dg_elem_t type,
                           const void *bias, dg_epilogue_t epilogue, void *stream, int kernel);
int dg_gemm_mx_select(dg_mx_t formatA, int64_t M, int64_t N, int64_t K);
const char *dg_gemm_mx_kernel_name(int kernel);

/* C = alpha * op(A) B + beta * C: A is fp16 or bf16 (typeA), stored M x K or
 * K x M (transA); B is K x N in any MX format, its blocks along N; C of A's type
 * or fp32 (typeC).  The products of a backward pass: dX = dY W with W kept in
 * 4 bits (transA = DG_OP_N), dW = dY^T X with X kept in 8 bits (DG_OP_T).
 * B's values are brought to A's type (exact for a B that was rounded from a
 * matrix of that type; in fp16 others round, or overflow to infinity) and
 * multiplied on the 16-bit matrix cores with fp32 sums, one rounding of the
 * result.  Special values as dg_gemm.
 *   splits, workspace: as dg_gemm_splitk (0: the library's choice,
 *   dg_gemm_dq_choose; the workspace holds splits * M * N fp32 partials, see
 *   dg_gemm_splitk_workspace_size, and is needed only when more than one
 *   range results).
 *   DG_ERR_UNSUPPORTED: 2^22 tiles or more, times K ranges (an output of about
 *   2^34 elements in one range).
 *   1 transA, 2 M, 3 N, 4 K, 5 alpha, 6 A, 7 lda, 8 typeA, 9 formatB, 10 B,
 *   11 ldb (bytes), 12 SB, 13 ldsb, 14 beta, 15 C, 16 ldc, 17 typeC,
 *   18 splits, 19 workspace (NULL or not 16-byte aligned), 20
 *   workspace_bytes (too few), 21 stream. */
int dg_gemm_dq(dg_op_t transA, int64_t M, int64_t N, int64_t K, float alpha, const void *A, int64_t lda,
               dg_elem_t typeA, dg_mx_t formatB, const void *B, int64_t ldb, const void *SB, int64_t ldsb,
               float beta, void *C, int64_t ldc, dg_elem_t typeC, int splits, void *workspace,
               size_t workspace_bytes, void *stream);

/* The K ranges dg_gemm_dq uses with splits = 0, or -i (1 M, 2 N, 3 K). */
int dg_gemm_dq_choose(int64_t M, int64_t N, int64_t K);

/* dg_gemm_dq with a forced kernel (argument 22; DG_KERNEL_AUTO: the library's
 * choice), for tests and measurement; DG_ERR_UNSUPPORTED when it cannot run the
 * problem (the 256 x 256 tile: an A whose rows are not 4-byte aligned, whose lda
 * is odd or, with transA, whose M is not a multiple of 8).  The choice for an
 * aligned A with splits = 0 (or -i: 1 M, 2 N, 3 K), and the kernels' names (NULL
 * when out of range). */
int dg_gemm_dq_with_kernel(dg_op_t transA, int64_t M, int64_t N, int64_t K, float alpha, const void *A, int64_t lda,
                           dg_elem_t typeA, dg_mx_t formatB, const void *B, int64_t ldb, const void *SB,
                           int64_t ldsb, float beta, void *C, int64_t ldc, dg_elem_t typeC, int splits,
                           void *workspace, size_t workspace_bytes, void *stream, int kernel);
int dg_gemm_dq_select(int64_t M, int64_t N, int64_t K);
const char *dg_gemm_dq_kernel_name(int kernel);

/* H = act(Z) (relu or gelu, as the epilogues of dg_gemm_ex), and Z kept in 8
 * bits (DG_MXFP8 or DG_MXINT8) for dg_act_backward, in one pass.  H may be Z
 * itself (with ldh = ldz).  Under DG_EPI_RELU a z > 0 that rounds to zero has no
 * gradient in dg_act_backward: of normal data 1.1% of the positive z in
 * DG_MXINT8 (1.6% where one column in a hundred is eight times the others) and
 * 0.0005% in DG_MXFP8.  DG_EPI_RELU_POSITIVE keeps such a z as the format's least
 * positive element instead, so that the mask of z > 0 is kept exactly at the
 * same size; H and everything else are as under DG_EPI_RELU, and the backward
 * pass takes DG_EPI_RELU.
 *   1 rows, 2 cols, 3 Z, 4 ldz, 5 H, 6 ldh, 7 type, 8 activation, 9 format,
 *   10 Q, 11 ldq, 12 S, 13 lds, 14 stream. */
int dg_act_checkpoint(int64_t rows, int64_t cols, const void *Z, int64_t ldz, void *H, int64_t ldh,
                      dg_elem_t type, dg_epilogue_t activation, dg_mx_t format, void *Q, int64_t ldq, void *S,
                      int64_t lds, void *stream);

/* dZ = dH * act'(z) with z the values of (Q, S) (kept by dg_act_checkpoint or
 * dg_mx_quantize).  relu: dH where z > 0, else 0 (an infinite or NaN dH too);
 * gelu: dH times Phi(z) + z phi(z), off by at most 2e-6 of |dH| (the error
 * function as in the forward, 1.5e-7; in every element type).  Where z is NaN, dZ
 * is.
 * dZ may be dH itself (with ldz = ldh).  dbias (fp32, cols elements; NULL for
 * none) receives the column sums of dZ before its rounding, in a fixed order
 * of summation; it needs a workspace of dg_act_backward_workspace_size bytes
 * (16-byte aligned, caller-owned, contents unspecified on return).
 *   1 rows, 2 cols, 3 dH, 4 ldh, 5 format, 6 Q, 7 ldq, 8 S, 9 lds, 10 dZ,
 *   11 ldz, 12 type, 13 activation, 14 dbias, 15 workspace (NULL or
 *   misaligned while dbias is given), 16 workspace_bytes (too few), 17
 *   stream. */
int dg_act_backward(int64_t rows, int64_t cols, const void *dH, int64_t ldh, dg_mx_t format, const void *Q,
                    int64_t ldq, const void *S, int64_t lds, void *dZ, int64_t ldz, dg_elem_t type,
                    dg_epilogue_t activation, float *dbias, void *workspace, size_t workspace_bytes,
                    void *stream);
size_t dg_act_backward_workspace_size(int64_t rows, int64_t cols);

/* Number of kernels in the table, and a static name for kernel i (NULL when
 * i is out of range).  Names read "<dtype>_<tiles>_<variant>". */
int dg_kernel_count(void);
const char *dg_kernel_name(int kernel);

/* Output tile (rows x cols of C per workgroup) of kernel i; -1 if out of range. */
int dg_kernel_tile_m(int kernel);
int dg_kernel_tile_n(int kernel);

/* Static text for a status code.  An invalid argument is given by its position
 * and named for the dense products only; the lists above name those of the MX
 * calls. */
const char *dg_status_string(int status);

/* hipError_t of the calling thread's last DG_ERR_HIP (0 if none). */
int dg_last_hip_error(void);

/* Library version, major * 10000 + minor * 100 + patch. */
int dg_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_GEMM_H */
