// Block-scaled (MX) matrices on gfx950: the formats, and the parameters the
// MX kernels share with the host side.  Not part of the public ABI.
//
// A row is cut into blocks of 32 elements along its length.  A block has one
// scale 2^e, kept as the byte e + 127 (255: NaN), and elements of 4 or 8 bits:
//   mxfp4   E2M1: +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}, two to a byte, the even
//           element in the low half;
//   mxfp8   E4M3: up to 448;
//   mxint8  a signed integer in 64ths, up to 127/64.
// Rounding x to a block: e = max(floor(log2(max |x|)) - emax, -127), emax the
// exponent of the format's largest element (2, 8, 0), and each element is
// x / 2^e to nearest even, saturated.  A power-of-two scale makes x / 2^e
// exact, so the only rounding is the element's own.  A block that holds a NaN
// or an infinity gets the scale NaN, so that the loss shows in every use.
//
// Storage: Q[row][groups * 256 elements] (zeros past the last column) and
// S[group][row][8]: the 8 scale bytes of a row's 256-element group side by
// side and the rows of a group together, so that the rows of a tile read one
// contiguous run per 256 k.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_common.hpp"

namespace dg {

enum { MX_FP4 = 0, MX_FP8 = 1, MX_INT8 = 2 };      // dg_mx_t
enum { ELEM_F32 = 0, ELEM_F16 = 1, ELEM_BF16 = 2 };  // dg_elem_t

constexpr int MX_GROUP = 256;   // elements of a scale group (8 blocks of 32)

__host__ __device__ __forceinline__ int64_t mx_groups(int64_t cols) { return (cols + MX_GROUP - 1) / MX_GROUP; }
__host__ __device__ __forceinline__ int64_t mx_group_bytes(int format) { return format == MX_FP4 ? 128 : 256; }

// Elementwise MX kernels (quantise, dequantise, activation forward and
// backward).  Row strides of X, Y in elements; of Q in bytes; of S's groups
// in rows (8 bytes each).
struct MxParams {
    const void *X;        // input: quantise, checkpoint (z), backward (dH)
    void *Y;              // output: dequantise, checkpoint (h), backward (dZ)
    uint8_t *Q;
    uint8_t *S;
    int64_t ldx, ldy, ldq, lds;
    int64_t rows, cols;
    int32_t trans;        // quantise: X is stored cols x rows
    int32_t type;         // ELEM_*
    int32_t format;       // MX_*
    int32_t act;          // ACT_RELU, ACT_GELU
    int32_t positive;     // checkpoint: z above zero is kept above zero
    float *dbias;         // backward: column sums of dZ (NULL: none)
    float *ws;            // backward: partial column sums, [slices][cols]
    int32_t slices, band; // row slices of the backward's launch, rows of a band (8, 16 or 32)
};

hipError_t launch_mx_quantize(const MxParams &p, hipStream_t s);
hipError_t launch_mx_dequantize(const MxParams &p, hipStream_t s);
hipError_t launch_act_checkpoint(const MxParams &p, hipStream_t s);
hipError_t launch_act_backward(const MxParams &p, hipStream_t s);
int act_backward_band(int64_t rows, int64_t cols, bool sums);
int act_backward_slices(int64_t rows, int64_t cols, bool sums);

#ifdef __HIPCC__

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 2^(byte - 127): byte 0 is the subnormal 2^-127, byte 255 is NaN.
__device__ __forceinline__ float mx_scale(uint32_t byte)
{
    const uint32_t bits = byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23;
    return __builtin_bit_cast(float, bits);
}

// The scale byte of a block whose largest magnitude has the bits `amax` (an
// fp32 pattern without sign; NaN patterns compare above infinity's).  The
// exponent field is floor(log2) + 127 of a normal value; subnormals and zero
// come out at the least scale.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax, int format)
{
    const int emax = format == MX_FP4 ? 2 : format == MX_FP8 ? 8 : 0;
    const int f = (int)(amax >> 23);
    if (f == 255) return 255;
    return f > emax ? (uint32_t)(f - emax) : 0u;
}

// Eight consecutive elements of a block in the format's code, `byte` the
// block's scale: 4 bytes (mxfp4, in o[0]) or 8.  NaN blocks store zeros.
// POSITIVE (8 bits): what lies above zero stays above it, as the least positive
// element where it would round to zero.
template <int FORMAT, bool POSITIVE = false>
__device__ __forceinline__ u32x2 mx_encode8(const float (&v)[8], uint32_t byte)
{
    u32x2 o = {0u, 0u};
    if (byte == 255) return o;
    if constexpr (FORMAT == MX_FP4) {
        // the hardware conversion divides by the scale, rounds to nearest
        // even and saturates
        const float sc = mx_scale(byte);
        uint32_t w = 0;
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], sc, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], sc, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], sc, 2);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], sc, 3);
        o[0] = w;
    } else if constexpr (FORMAT == MX_FP8) {
        // the conversion would turn values past 448 into NaN: clamp first
        const int e = 127 - (int)byte;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = __builtin_amdgcn_fmed3f(__builtin_amdgcn_ldexpf(v[i], e), -448.f, 448.f);
            if (POSITIVE && v[i] > 0.f) x[i] = __builtin_fmaxf(x[i], 0x1p-9f);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int w = 0;
            w = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h], x[4 * h + 1], w, false);
            w = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h + 2], x[4 * h + 3], w, true);
            o[h] = (uint32_t)w;
        }
    } else {
        const int e = 6 + 127 - (int)byte;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float x = __builtin_amdgcn_fmed3f(__builtin_rintf(__builtin_amdgcn_ldexpf(v[i], e)), -127.f, 127.f);
            if (POSITIVE && v[i] > 0.f) x = __builtin_fmaxf(x, 1.f);
            o[i >> 2] |= ((uint32_t)(int)x & 255u) << (8 * (i & 3));
        }
    }
    return o;
}

// The eight values that codes q stand for, in fp32.
template <int FORMAT>
__device__ __forceinline__ void mx_decode8(u32x2 q, uint32_t byte, float (&v)[8])
{
    const float sc = mx_scale(byte);
    if constexpr (FORMAT == MX_FP4) {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], 1.f, 0);
        const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], 1.f, 1);
        const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], 1.f, 2);
        const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[0], 1.f, 3);
        v[0] = a[0] * sc; v[1] = a[1] * sc; v[2] = b[0] * sc; v[3] = b[1] * sc;
        v[4] = c[0] * sc; v[5] = c[1] * sc; v[6] = d[0] * sc; v[7] = d[1] * sc;
    } else if constexpr (FORMAT == MX_FP8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            v[4 * h + 0] = __builtin_amdgcn_cvt_f32_fp8((int)q[h], 0) * sc;
            v[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8((int)q[h], 1) * sc;
            v[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8((int)q[h], 2) * sc;
            v[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8((int)q[h], 3) * sc;
        }
    } else {
        // the scale of one 64th: 2^-133 at the least, an exact subnormal
        const float s64 = sc * 0.015625f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)((int32_t)(q[i >> 2] << (24 - 8 * (i & 3))) >> 24) * s64;
    }
}

#endif

}  // namespace dg
