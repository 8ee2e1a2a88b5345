// Few rows (single tokens, a decoding batch, a few tokens an expert): the product is
// bound by reading the weights once.
//
// A workgroup takes 16 rows of A and a strip of columns; its NWV waves share out the
// summed index in steps of KS (32 of 16 bits, 16 of fp32) and their sums meet in LDS in
// wave order.  Weights and rows come from global memory into fragments with no barrier
// before the end, so that every wave keeps several steps of loads in flight.  The weights
// are the matrix instruction's row operand: register e of lane l belongs to weight column
// 4 * (l / 16) + e of the fragment and to row l % 16 of A.
// Measured (bf16, weights stored N x K, in a graph): 1 x 5632 x 2048 with gelu 7.0 us, 3.3
// TB/s (the same strips by 64-byte pieces, layer_16_rows, 7.9); 14 experts of 5632 x 2048
// 70 us, 4.6 TB/s.  24 rows are two strips of rows that read the weights twice, from L2 the
// second time: 24 x 2048 x 5632 8.8 us, bound by the wait for a chunk's loads.
// STREAM (4-byte aligned rows): B passes through LDS on its way, so that a load
// fetches 512 bytes in a row of it in place of 64 (probes of 5632 x 2048, 16 bits, read
// alone: 4.3 against 5.8 us; 2048 columns of 12 KB 4.5 against 7.0).
//   B stored N x K: 16 columns; lane l loads a step's k 8 * (l / 16) .. + 7 (fp32: 4)
//     of column l % 16, the fragment itself.
//   B stored K x N: 64 columns; lane l loads columns 4 * (l % 16) .. + 3 of the same
//     k's rows, 4 x 8 elements that are transposed in registers into four
//     fragments; fragment j holds columns 4 * (l % 16) + j.
//     1 x 5632 x 2048 9.4 us; 1 x 2048 x 5632 in ranges of K and their join 10.4 (24 rows 13.2).
// Any strides and alignment (the GPU takes misaligned vectors).
#pragma once

#include "gemm_pipe.hpp"
#include "layer_common.hpp"

namespace dg {

template <typename T> struct RowStep;
template <> struct RowStep<_Float16> {
    static constexpr int PER = 8;
    typedef f16x8 vec;
    __device__ static __forceinline__ f32x4 mfma(vec a, vec b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};
template <> struct RowStep<__bf16> {
    static constexpr int PER = 8;
    typedef bf16x8 vec;
    __device__ static __forceinline__ f32x4 mfma(vec a, vec b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <> struct RowStep<float> {
    static constexpr int PER = 4;
    typedef f32x4 vec;
    __device__ static __forceinline__ f32x4 mfma(vec a, vec b, f32x4 c)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
        return c;
    }
};

// The columns of a workgroup's strip.
constexpr int layer_rows_columns(bool tb) { return tb ? 16 : 64; }

template <typename T, bool TB, int NWV, bool STREAM>
__global__ __launch_bounds__(64 * NWV, 4) void layer_rows_kernel(LayerParams p)
{
    typedef RowStep<T> S;
    typedef typename S::vec vec;
    typedef vec __attribute__((aligned(sizeof(T)))) vecu;
    typedef T T4 __attribute__((ext_vector_type(4)));
    typedef T4 __attribute__((aligned(sizeof(T)))) T4u;
    constexpr int PER = S::PER, KS = 4 * PER, NF = TB ? 1 : 4, BN = layer_rows_columns(TB), OUT = 16 * BN;
    // steps whose loads are in flight together
    constexpr int U = STREAM ? 1 : TB ? 8 : 2;
    static_assert(TB || !STREAM, "STREAM: B stored N x K");
    constexpr int CHUNK = 16 * 512, RED = NWV * NF * 64 * 16;
    constexpr int SMEM = STREAM && NWV * CHUNK > RED ? NWV * CHUNK : RED;
    __shared__ __attribute__((aligned(1024))) char smem_raw[SMEM];
    typedef f32x4 red_t[NF][64];
    red_t *red = (red_t *)smem_raw;

    LayerTile t;
    if (!layer_tile(p, 16, BN, blockIdx.x, t)) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4;
    const int K = t.k_len, steps = K / KS;
    // this lane's row of A, and its column (or its first of four, moved back from the
    // matrix's end: columns that it then shares with its neighbour are not its own)
    const bool has = t.m0 + r < t.rows;
    const T *A = (const T *)p.A + (t.row0 + (has ? t.m0 + r : t.rows - 1)) * p.lda + t.k0 + PER * q;
    const T *B = (const T *)p.B + t.group * p.strideB;
    if constexpr (TB) {
        const int col = t.n0 + r < p.N ? t.n0 + r : p.N - 1;
        B += (int64_t)col * p.ldb + t.k0 + PER * q;
    } else {
        const int col = t.n0 + 4 * r < p.N - 4 ? t.n0 + 4 * r : p.N - 4;
        B += ((int64_t)t.k0 + PER * q) * p.ldb + col;
    }

    // what the epilogue reads, ahead of everything else where a thread has one output
    constexpr bool AHEAD = OUT <= 64 * NWV;
    float ahead_x = 0.f, ahead_bias = 0.f;
    if (AHEAD && p.splits <= 1 && (int)threadIdx.x < OUT && t.m0 + (int)threadIdx.x / BN < t.rows &&
        t.n0 + (int)threadIdx.x % BN < p.N) {
        const int row = t.m0 + (int)threadIdx.x / BN, col = t.n0 + (int)threadIdx.x % BN;
        auto fetch = [&](auto type) {
            typedef decltype(type) TC;
            LayerAux<TC, 1> aux;
            float bias[1];
            aux.fetch(p, t, row, col);
            layer_bias<TC, 1>(p, t.group, col, bias);
            ahead_x = (float)aux.x[0];
            ahead_bias = bias[0];
        };
        if (sizeof(T) == 2 && p.ctype != 0) fetch(T());
        else fetch(0.f);
    }

    f32x4 acc[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[f] = (f32x4){0.f, 0.f, 0.f, 0.f};

    auto products = [&](vec a, const vec (&b)[NF]) {
#pragma unroll
        for (int f = 0; f < NF; ++f) acc[f] = S::mfma(b[f], a, acc[f]);
    };
    // The wave's chunks of 8 steps, 512 bytes of each of the 16 columns, through its own
    // 8 KB of LDS: a direct load fetches two columns' 512 bytes, and the 16-byte piece
    // c of column i sits at c ^ i, so that fragment reads meet no bank twice.
    const int chunks = STREAM ? steps / 8 : 0;
    if constexpr (STREAM) {
        typedef __attribute__((address_space(3))) vec lds_vec_t;
        lds_char_t *mine = (lds_char_t *)smem_raw + wave * CHUNK;
        const char *base = (const char *)((const T *)p.B + t.group * p.strideB + (int64_t)t.n0 * p.ldb + t.k0);
        uint32_t off[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = 2 * i + (lane >> 5), col = t.n0 + c < p.N ? c : p.N - 1 - t.n0;
            off[i] = (uint32_t)((int64_t)col * p.ldb * (int)sizeof(T)) + (((lane & 31) ^ c) << 4);
        }
        // More than four rows of A come the same way, through registers and then the memory that
        // B's chunk has left: 64-byte pieces of them take 10.7 us, this 8.8 (24 x 2048 x 5632;
        // 14 experts 70.7 and 69.9; one token so 7.2, by pieces 6.8).  What a row that does not exist
        // reads is not stored.
        const int n = t.rows - t.m0;
        const bool few = n <= 4;
        const char *rows = (const char *)((const T *)p.A + (t.row0 + t.m0) * p.lda + t.k0);
        uint32_t aoff[8];
        if (!few) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int row = 2 * i + (lane >> 5);
                aoff[i] = (uint32_t)((int64_t)(row < n ? row : n - 1) * p.lda * (int)sizeof(T)) + ((lane & 31) << 4);
            }
        }
        // fragment u of a chunk in LDS, and the place of the pieces that a lane fetches of rows 2i
        int frag = r * 512 + ((q ^ r) << 4), piece = (lane >> 5) * 512 + (((lane & 31) ^ (lane >> 5)) << 4);
        auto b_of = [&](int u) { return *(const lds_vec_t *)(mine + (frag ^ (u << 6))); };
        for (int ch = wave; ch < chunks; ch += NWV) {
            const i32x4_rsrc rsrc = buffer_rsrc(base + (int64_t)ch * 512);
#pragma unroll
            for (int i = 0; i < 8; ++i) load_lds16(off[i], rsrc, (unsigned)(uintptr_t)(mine + i * 1024));
            // (opaque to the compiler, which would otherwise keep every address in a register)
            asm volatile("" : "+v"(frag), "+v"(piece));
            vec a[8];
            if (few) {
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    a[u] = (vec)(T)0.f;
                    if (has) a[u] = *(const vecu *)(A + ((int64_t)ch * 8 + u) * KS);
                }
                wait_vmcnt<0>();
                asm volatile("" ::: "memory");
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const vec f[1] = {b_of(u)};
                    products(a[u], f);
                }
            } else {
                vec b[8];
                const char *at = rows + (int64_t)ch * 512;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (2 * i < n) a[i] = *(const vecu *)(at + aoff[i]);
                wait_vmcnt<0>();
                asm volatile("" ::: "memory");
#pragma unroll
                for (int u = 0; u < 8; ++u) b[u] = b_of(u);
                __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): read before it is overwritten
                asm volatile("" ::: "memory");
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (2 * i < n) *(lds_vec_t *)(mine + (piece ^ (i << 5)) + i * 1024) = a[i];
                asm volatile("" ::: "memory");
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const vec f[1] = {b[u]};
                    products(b_of(u), f);        // A's now
                }
            }
            __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): read before it is overwritten
            asm volatile("" ::: "memory");
        }
    }
    // U steps at a time, their loads first
    for (int s0 = chunks * 8 + wave * U; s0 < steps; s0 += NWV * U) {
        vec a[U], b[U];
        T4 x[U][PER];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s0 + u >= steps) break;
            const int64_t k = (int64_t)(s0 + u) * KS;
            if constexpr (TB) {
                b[u] = *(const vecu *)(B + k);
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i) x[u][i] = *(const T4u *)(B + (k + i) * p.ldb);
            }
            a[u] = (vec)(T)0.f;
            if (has) a[u] = *(const vecu *)(A + k);
        }
        __builtin_amdgcn_sched_barrier(0);    // the loads stay ahead of the products
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s0 + u >= steps) break;
            vec f[NF];
            if constexpr (TB) {
                f[0] = b[u];
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < PER; ++i) f[j][i] = x[u][i][j];
            }
            products(a[u], f);
        }
    }
    // the last, partial step, element by element
    if (K % KS != 0 && wave == NWV - 1) {
        const int64_t k = (int64_t)steps * KS;
        const int left = K - steps * KS - PER * q;
        vec a, f[NF];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool in = i < left;
            if constexpr (TB) {
                f[0][i] = in ? B[k + i] : (T)0.f;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j][i] = in ? B[(k + i) * p.ldb + j] : (T)0.f;
            }
            a[i] = in && has ? A[k + i] : (T)0.f;
        }
        products(a, f);
    }

    if constexpr (STREAM) __syncthreads();       // the chunks' memory is the sums' now
#pragma unroll
    for (int f = 0; f < NF; ++f) red[wave][f][lane] = acc[f];
    __syncthreads();
    auto finish = [&](auto type) {
        typedef decltype(type) TC;
        for (int o = threadIdx.x; o < OUT; o += 64 * NWV) {
            const int c = o % BN, m = o / BN, row = t.m0 + m;
            const int lc = TB ? c : c >> 2, f = TB ? 0 : c & 3;       // weight column of the fragment
            int col = t.n0 + c;
            if constexpr (!TB) {
                // of this fragment column's four, moved back at the end
                const int first = t.n0 + 4 * lc;
                if (first > p.N - 4) col = p.N - 4 + f < first ? p.N : p.N - 4 + f;
            }
            if (row >= t.rows || col >= p.N) continue;
            LayerAux<TC, 1> aux;
            float bias[1], v[1] = {0.f};
            if constexpr (AHEAD) {
                aux.x[0] = (TC)ahead_x;
                bias[0] = ahead_bias;
            } else if (p.splits <= 1) {       // (TC is their type then; a split's sums meet them in the join)
                aux.fetch(p, t, row, col);
                layer_bias<TC, 1>(p, t.group, col, bias);
            }
#pragma unroll
            for (int w = 0; w < NWV; ++w) v[0] += red[w][f][(lc >> 2) * 16 + m][lc & 3];
            if (p.splits > 1) layer_partial<1>(p, t, row, col, v);
            else layer_finish<TC, 1>(p, t, row, col, v, aux, bias);
        }
    };
    if (sizeof(T) == 2 && p.ctype != 0 && p.splits <= 1) finish(T());
    else finish(0.f);
}

}  // namespace dg
