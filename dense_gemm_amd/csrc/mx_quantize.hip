// Rounding to MX formats and back, and the activation passes that keep their
// input in 8 bits.  Elementwise work, bound by memory: each kernel makes one
// pass, 16 bytes or more per lane and access.
//
// Row kernels: a lane takes 8 consecutive elements of a row, so 4 lanes hold
// a block of 32 and the block's largest magnitude comes from two lane
// exchanges; a wave covers 512 columns of one row.  The scale byte is stored
// by one lane of the four.  At 32768 x 5632 (bf16): rounding to mxfp8 100 us
// (5.6 TB/s), to mxfp4 88 (5.3), back from mxfp8 101 (5.5); the checkpoint 158
// us with relu (5.9), 176 with gelu (5.3); the backward 169 with relu or gelu
// (5.5) and 184 with the column sums (5.0).  A plain copy of 1 GiB runs at 5.1
// TB/s on this card.  Stores stay ordinary ones: non-temporal stores of H, dZ
// and Y gain 3-25% when the pass is timed alone at this size and lose where the
// result is read next (checkpoint and the product on it, 2048 x 5632 by 2048:
// 64.6 us against 57.5).
#include "mx_common.hpp"

namespace dg {

namespace {

// Eight elements of a row as one 16-byte access (two for fp32).  Rows need
// only be aligned to their element: the GPU takes misaligned vector accesses
// to global memory, so odd row strides go the same way as aligned ones.
template <typename T> struct Eight {
    typedef T V8 __attribute__((ext_vector_type(8)));
    typedef V8 __attribute__((aligned(sizeof(T)))) V8u;
};

// Elements col .. col+7 of a row of n elements at `row` (zeros past n).
template <typename T>
__device__ __forceinline__ void load8(const T *row, int64_t col, int64_t n, float (&v)[8])
{
    if (col + 8 <= n) {
        const typename Eight<T>::V8 a = *(const typename Eight<T>::V8u *)(row + col);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)a[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = col + i < n ? (float)row[col + i] : 0.f;
    }
}

// One rounding to T (nothing for fp32).
template <typename T>
__device__ __forceinline__ void store8(T *row, int64_t col, int64_t n, const float (&v)[8])
{
    typename Eight<T>::V8 a;
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = (T)v[i];
    if (col + 8 <= n) {
        *(typename Eight<T>::V8u *)(row + col) = a;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < n) row[col + i] = a[i];
    }
}

// Largest magnitude of the 32 elements held by 4 neighbouring lanes, as bits.
__device__ __forceinline__ uint32_t block_amax(const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu;
        m = b > m ? b : m;
    }
    uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xb1, 0xf, 0xf, true);   // lane ^ 1
    m = o > m ? o : m;
    o = (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4e, 0xf, 0xf, true);            // lane ^ 2
    return o > m ? o : m;
}

// Codes and scale of the 8 elements a lane holds, col a multiple of 8.
template <int FORMAT, bool POSITIVE = false>
__device__ __forceinline__ void store_codes(const MxParams &p, int64_t row, int64_t col, const float (&v)[8])
{
    const uint32_t byte = mx_scale_byte(block_amax(v), FORMAT);
    const u32x2 q = mx_encode8<FORMAT, POSITIVE>(v, byte);
    uint8_t *qr = p.Q + row * p.ldq;
    if constexpr (FORMAT == MX_FP4) *(uint32_t *)(qr + col / 2) = q[0];
    else *(u32x2 *)(qr + col) = q;
    if ((threadIdx.x & 3) == 0)
        p.S[((col >> 8) * p.lds + row) * 8 + ((col >> 5) & 7)] = (uint8_t)byte;
}

template <int FORMAT>
__device__ __forceinline__ void load_codes(const MxParams &p, int64_t row, int64_t col, float (&v)[8])
{
    const uint8_t *qr = p.Q + row * p.ldq;
    u32x2 q = {0u, 0u};
    if constexpr (FORMAT == MX_FP4) q[0] = *(const uint32_t *)(qr + col / 2);
    else q = *(const u32x2 *)(qr + col);
    mx_decode8<FORMAT>(q, p.S[((col >> 8) * p.lds + row) * 8 + ((col >> 5) & 7)], v);
}

// The row kernels' places: item b is rows 4 * (b / chunks) .. +3 (one per
// wave) and columns 512 * (b % chunks) .. +511 (8 per lane).  The padding up
// to the next whole group is part of the stored row (zeros), so columns run to
// the group's end.  A workgroup takes every gridDim.x-th item (the grid is
// capped: a launch holds fewer than 2^32 threads).
__device__ __forceinline__ bool place(const MxParams &p, int64_t b, int64_t &row, int64_t &col)
{
    const int64_t chunks = (mx_groups(p.cols) + 1) / 2;
    row = (b / chunks) * 4 + (threadIdx.x >> 6);
    col = (b % chunks) * 512 + (threadIdx.x & 63) * 8;
    // whole groups of 32 lanes are in or out: a block's four lanes together
    return row < p.rows && col < mx_groups(p.cols) * MX_GROUP;
}

__host__ __device__ __forceinline__ int64_t row_items(const MxParams &p)
{
    return (mx_groups(p.cols) + 1) / 2 * ((p.rows + 3) / 4);
}

__host__ __device__ __forceinline__ int64_t trans_items(const MxParams &p)
{
    return (p.rows + 63) / 64 * mx_groups(p.cols);
}

template <typename T, int FORMAT>
__global__ __launch_bounds__(256) void mx_quantize_kernel(MxParams p)
{
    const int64_t n = row_items(p);
    for (int64_t b = blockIdx.x; b < n; b += gridDim.x) {
        int64_t row, col;
        if (!place(p, b, row, col)) continue;
        float v[8];
        load8<T>((const T *)p.X + row * p.ldx, col, p.cols, v);
        store_codes<FORMAT>(p, row, col, v);
    }
}

// X stored cols x rows: a workgroup rounds 256 k of 64 rows (one scale
// group) through LDS.  The tile is loaded 16 bytes a lane along the stored
// rows, as [256 k][64 n]; a thread then takes the 32 k of one block of one
// row: 16-bit elements by the transposing LDS read (four k of a lane's column
// at a time, where plain reads would take 32), fp32 one by one.  The codes go
// back through LDS, so that the stores write whole rows of 128 or 256 bytes.
// 32768 x 5632 bf16 to mxfp8: 122 us (4.6 TB/s), against 449 with 2-byte
// loads and each thread storing its own block.
template <typename T, int FORMAT>
__global__ __launch_bounds__(512) void mx_quantize_t_kernel(MxParams p)
{
    typedef __attribute__((address_space(3))) char lds_char;
    typedef __attribute__((address_space(3))) uint8_t lds_u8;
    typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
    typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
    typedef short i16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
    constexpr int V = 16 / sizeof(T);                    // elements of a load
    constexpr int LPR = 64 / V, RPP = 512 / LPR;         // lanes per k, k per pass
    constexpr int ROW = 64 * sizeof(T);                  // LDS bytes per k
    constexpr int QB = FORMAT == MX_FP4 ? 128 : 256;     // code bytes per row, QP in LDS
    constexpr int QP = QB + 16, QAT = 64 * QP;
    typedef T VT __attribute__((ext_vector_type(V)));
    typedef VT __attribute__((aligned(sizeof(T)))) VTu;
    static_assert(QAT + 64 * 8 <= MX_GROUP * ROW, "the codes fit the tile");
    __shared__ __attribute__((aligned(16))) char smem_raw[MX_GROUP * ROW];
    lds_char *smem = (lds_char *)smem_raw;
    const int64_t nb = (p.rows + 63) / 64, items = trans_items(p);
    const int tid = threadIdx.x, n = tid & 63, kq = tid >> 6;
    for (int64_t b = blockIdx.x; b < items; b += gridDim.x) {
        const int64_t n0 = (b % nb) * 64, k0 = (b / nb) * MX_GROUP;
        VT x[MX_GROUP / RPP];
#pragma unroll
        for (int i = 0; i < MX_GROUP / RPP; ++i) {
            const int64_t k = k0 + i * RPP + tid / LPR, nn = n0 + (tid % LPR) * V;
            const T *src = (const T *)p.X + k * p.ldx + nn;
            if (k < p.cols && nn + V <= p.rows) {
                x[i] = *(const VTu *)src;
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    T y = (T)0.f;
                    if (k < p.cols && nn + e < p.rows) y = src[e];
                    x[i][e] = y;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < MX_GROUP / RPP; ++i)
            *(lds_u32x4 *)(smem + (i * RPP + tid / LPR) * ROW + (tid % LPR) * 16) = __builtin_bit_cast(u32x4, x[i]);
        __syncthreads();
        float v[4][8];
        if constexpr (sizeof(T) == 2) {
            // in each 16-lane group, lanes 4t .. 4t+3 name k + t; a lane
            // receives its own column
            const lds_char *at = smem + (kq * 32 + ((n & 15) >> 2)) * ROW + (16 * (n >> 4) + 4 * (n & 3)) * 2;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const i16x4 q = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(at + 4 * j * ROW));
#pragma unroll
                for (int e = 0; e < 4; ++e) v[j >> 1][4 * (j & 1) + e] = (float)__builtin_bit_cast(T, (short)q[e]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                v[i >> 3][i & 7] = *(const __attribute__((address_space(3))) float *)(smem + (kq * 32 + i) * ROW + n * 4);
        }
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const uint32_t a = __builtin_bit_cast(uint32_t, v[i >> 3][i & 7]) & 0x7fffffffu;
            m = a > m ? a : m;
        }
        const uint32_t byte = mx_scale_byte(m, FORMAT);
        u32x2 o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = mx_encode8<FORMAT>(v[i], byte);
        __syncthreads();      // every thread has read its column
        lds_char *q = smem + n * QP + kq * (QB / 8);
        if constexpr (FORMAT == MX_FP4) {
            *(lds_u32x4 *)q = (u32x4){o[0][0], o[1][0], o[2][0], o[3][0]};
        } else {
            *(lds_u32x4 *)q = (u32x4){o[0][0], o[0][1], o[1][0], o[1][1]};
            *(lds_u32x4 *)(q + 16) = (u32x4){o[2][0], o[2][1], o[3][0], o[3][1]};
        }
        *(lds_u8 *)(smem + QAT + n * 8 + kq) = (uint8_t)byte;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 64 * QB / 16 / 512; ++i) {
            const int id = i * 512 + tid, row = id / (QB / 16), c = id % (QB / 16);
            if (n0 + row < p.rows)
                *(u32x4 *)(p.Q + (n0 + row) * p.ldq + k0 / MX_GROUP * QB + c * 16) = *(const lds_u32x4 *)(smem + row * QP + c * 16);
        }
        if (tid < 64 && n0 + tid < p.rows)
            *(u32x2 *)(p.S + ((k0 >> 8) * p.lds + n0 + tid) * 8) = *(const lds_u32x2 *)(smem + QAT + tid * 8);
        __syncthreads();      // the tile is free for the next item
    }
}

template <typename T, int FORMAT>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(MxParams p)
{
    const int64_t n = row_items(p);
    for (int64_t b = blockIdx.x; b < n; b += gridDim.x) {
        int64_t row, col;
        if (!place(p, b, row, col) || col >= p.cols) continue;
        float v[8];
        load_codes<FORMAT>(p, row, col, v);
        store8<T>((T *)p.Y + row * p.ldy, col, p.cols, v);
    }
}

// h = act(z) and z in 8 bits, one read of z.  H may be Z itself: a lane
// reads its elements before it writes them.  POSITIVE: see mx_encode8 (32768 x
// 5632 relu: mxfp8 157 us with and without, mxint8 161 and 158).
template <typename T, int FORMAT, bool POSITIVE>
__global__ __launch_bounds__(256) void act_checkpoint_kernel(MxParams p)
{
    const int64_t n = row_items(p);
    for (int64_t b = blockIdx.x; b < n; b += gridDim.x) {
        int64_t row, col;
        if (!place(p, b, row, col)) continue;
        float v[8];
        load8<T>((const T *)p.X + row * p.ldx, col, p.cols, v);
        store_codes<FORMAT, POSITIVE>(p, row, col, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = activate(p.act, v[i]);
        store8<T>((T *)p.Y + row * p.ldy, col, p.cols, v);
    }
}

// d * act'(z).  relu chooses instead of multiplying: d above zero, else 0
// whatever d is (an infinity or a NaN too), and NaN for a NaN z.  gelu = z Phi(z),
// its slope Phi(z) + z phi(z), with phi the normal density and Phi by the same
// approximation of erfc as the forward (Abramowitz & Stegun 7.1.26) on
// q = erfc(|z| / sqrt 2): Phi = 1 - q/2 for z >= 0 and q/2 below (its constants
// carry the 1/sqrt 2 and the 1/2).  exp(-z^2/2) serves both terms.  In z phi(z)
// z is clamped to 14, where the density has underflowed, so that an infinity
// gives 1 or 0 and not inf * 0 (a NaN comes through Phi).
__device__ __forceinline__ float act_gradient(int act, float z, float d)
{
    if (act == ACT_RELU) return z > 0.f ? d : (z <= 0.f ? 0.f : z);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f * 0.70710678f, __builtin_fabsf(z), 1.f));
    float poly = __builtin_fmaf(t, 0.5f * 1.061405429f, 0.5f * -1.453152027f);
    poly = __builtin_fmaf(t, poly, 0.5f * 1.421413741f);
    poly = __builtin_fmaf(t, poly, 0.5f * -0.284496736f);
    poly = __builtin_fmaf(t, poly, 0.5f * 0.254829592f);
    const float ex = __builtin_amdgcn_exp2f(z * z * -0.72134752f);   // 2^(-z^2/2 * log2 e)
    const float hq = poly * t * ex;
    const float cdf = z >= 0.f ? 1.f - hq : hq;
    return d * __builtin_fmaf(__builtin_amdgcn_fmed3f(z, -14.f, 14.f) * 0.3989422804014327f, ex, cdf);
}

// dZ = dH * act'(z8), and the column sums of dZ (before its rounding) into
// one row of partial sums per slice of rows.  Workgroup (c, s) takes 512
// columns and every slices-th band of rows from band s on; its eight waves take
// every eighth row of a band, one row at a time: what is in flight over the
// chip is then one stretch of memory that moves forward with the dispatch.  (With
// four rows' loads in flight per wave, or fewer workgroups that stay and stride
// over the rows, the streams spread: 32768 x 5632 with relu and no sums took
// 202-262 us against 168.)  The waves' sums meet in LDS, in wave order, so
// the sum's order is fixed.
template <typename T, int FORMAT>
__global__ __launch_bounds__(512) void act_backward_kernel(MxParams p)
{
    __shared__ float part[8][512];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t col = (int64_t)blockIdx.x * 512 + lane * 8;
    float sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = 0.f;
    if (col < p.cols) {
        for (int64_t r0 = (int64_t)blockIdx.y * p.band; r0 < p.rows; r0 += (int64_t)p.slices * p.band) {
            const int64_t end = r0 + p.band < p.rows ? r0 + p.band : p.rows;
#pragma unroll 1
            for (int64_t row = r0 + wave; row < end; row += 8) {
                float z[8], d[8];
                load8<T>((const T *)p.X + row * p.ldx, col, p.cols, d);
                load_codes<FORMAT>(p, row, col, z);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    d[i] = act_gradient(p.act, z[i], d[i]);
                    sum[i] += d[i];
                }
                store8<T>((T *)p.Y + row * p.ldy, col, p.cols, d);
            }
        }
    }
    if (!p.dbias) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) part[wave][lane * 8 + i] = sum[i];
    __syncthreads();
    const int64_t gc = (int64_t)blockIdx.x * 512 + threadIdx.x;
    if (gc < p.cols) {
        float t = part[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < 8; ++w) t += part[w][threadIdx.x];
        p.ws[(int64_t)blockIdx.y * p.cols + gc] = t;
    }
}

// dbias = the slices' partial sums in increasing order: 16 threads a column
// (each every 16th slice), then those 16 sums in order.
__global__ __launch_bounds__(256) void column_sum_kernel(const float *ws, float *dbias, int64_t cols, int slices)
{
    __shared__ float part[16][17];
    const int c = threadIdx.x & 15, q = threadIdx.x >> 4;
    for (int64_t c0 = (int64_t)blockIdx.x * 16; c0 < cols; c0 += (int64_t)gridDim.x * 16) {
        const int64_t col = c0 + c;
        float s = 0.f;
        if (col < cols)
#pragma unroll 8
            for (int i = q; i < slices; i += 16) s += ws[(int64_t)i * cols + col];
        part[q][c] = s;
        __syncthreads();
        if (q == 0 && col < cols) {
            for (int i = 1; i < 16; ++i) s += part[i][c];
            dbias[col] = s;
        }
        __syncthreads();
    }
}

template <typename... Args>
hipError_t launch(const void *f, dim3 grid, dim3 block, hipStream_t s, Args... a)
{
    void *args[] = {&a...};
    return hipLaunchKernel(f, grid, block, args, 0, s);
}

typedef void (*kernel_fn)(MxParams);

// Workgroups for n items of work (2^22 at most: 2^31 threads of 512).
dim3 grid_for(int64_t n) { return dim3((unsigned)(n < (1 << 22) ? n : (1 << 22))); }

template <typename T, int F>
kernel_fn quantize_fn(const MxParams &p)
{
    return p.trans ? mx_quantize_t_kernel<T, F> : mx_quantize_kernel<T, F>;
}
template <typename T, int F>
kernel_fn dequantize_fn(const MxParams &)
{
    return mx_dequantize_kernel<T, F>;
}
template <typename T, int F>
kernel_fn checkpoint_fn(const MxParams &p)
{
    return p.positive ? act_checkpoint_kernel<T, F, true> : act_checkpoint_kernel<T, F, false>;
}
template <typename T, int F>
kernel_fn backward_fn(const MxParams &)
{
    return act_backward_kernel<T, F>;
}

#define DG_BY_FORMAT8(fn, T) (p.format == MX_FP8 ? fn<T, MX_FP8>(p) : fn<T, MX_INT8>(p))
#define DG_BY_FORMAT(fn, T)                                                                        \
    (p.format == MX_FP4 ? fn<T, MX_FP4>(p) : p.format == MX_FP8 ? fn<T, MX_FP8>(p) : fn<T, MX_INT8>(p))
#define DG_BY_TYPE(by, fn) \
    (p.type == ELEM_F32 ? by(fn, float) : p.type == ELEM_F16 ? by(fn, _Float16) : by(fn, __bf16))

}  // namespace

hipError_t launch_mx_quantize(const MxParams &p, hipStream_t s)
{
    return launch((const void *)DG_BY_TYPE(DG_BY_FORMAT, quantize_fn), grid_for(p.trans ? trans_items(p) : row_items(p)),
                  dim3(p.trans ? 512 : 256), s, p);
}

hipError_t launch_mx_dequantize(const MxParams &p, hipStream_t s)
{
    return launch((const void *)DG_BY_TYPE(DG_BY_FORMAT, dequantize_fn), grid_for(row_items(p)), dim3(256), s, p);
}

hipError_t launch_act_checkpoint(const MxParams &p, hipStream_t s)
{
    return launch((const void *)DG_BY_TYPE(DG_BY_FORMAT8, checkpoint_fn), grid_for(row_items(p)), dim3(256), s, p);
}

// Rows of a band of the backward: 32 (four a wave) where that leaves four
// workgroups per compute unit; else 16 for the column sums, which halves the
// partial sums, or 8.  Bands of 8 / 16 / 32, fp16, relu, with the sums: 512 x 5632
// 7.6 / 7.4 / 8.3 us, 2048^2 8.4 / 7.7 / 9.4, 8192 x 5632 49 / 44 / 41, 32768 x 5632
// 207 / 186 / 182; without: 512 x 5632 4.0 / 4.6 / 5.8, 2048^2 4.7 / 5.0 / 6.0.
int act_backward_band(int64_t rows, int64_t cols, bool sums)
{
    const int64_t chunks = (cols + 511) / 512;
    if ((rows + 31) / 32 * chunks >= 1024) return 32;
    return sums && (rows + 15) / 16 * chunks >= 256 ? 16 : 8;
}

// Row slices: a band each, up to 4096 (the grid's second dimension and the
// workspace stay small) and to a grid of 2^22 workgroups (2^31 threads).
int act_backward_slices(int64_t rows, int64_t cols, bool sums)
{
    const int64_t chunks = (cols + 511) / 512, band = act_backward_band(rows, cols, sums);
    int64_t s = (rows + band - 1) / band;
    if (s > 4096) s = 4096;
    if (s > (1 << 22) / chunks) s = (1 << 22) / chunks;
    return s < 1 ? 1 : (int)s;
}

hipError_t launch_act_backward(const MxParams &p, hipStream_t s)
{
    if (p.slices > 0) {
        const dim3 grid((unsigned)((p.cols + 511) / 512), (unsigned)p.slices);
        const hipError_t e = launch((const void *)DG_BY_TYPE(DG_BY_FORMAT8, backward_fn), grid, dim3(512), s, p);
        if (e != hipSuccess || !p.dbias) return e;
    }
    return launch((const void *)&column_sum_kernel, grid_for((p.cols + 15) / 16), dim3(256), s,
                  (const float *)p.ws, p.dbias, p.cols, (int)p.slices);
}

}  // namespace dg
