// q4.hpp -- products with 4-bit weights: C[r][n] = sum over groups of k of
// scale[n][group] * sum over k of A[r][k] * (code[n][k] - 8).
//
// The codes are whole numbers of -8 .. 7, exact in every input type, so they go
// into the matrix instructions as they are; a group's sum is scaled and added
// in fp32.  The weights are never rounded to the input type, and a group costs
// one fma per output in place of one multiplication per weight.
//
// Bound by the bytes of the codes while an expert has few rows: every wave
// streams its own part of them from HBM to registers, with no LDS between.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "expert_rows.hpp"

namespace tg {

// Packed layout.  A block is 16 n by 128 k: 1 KiB of codes, one 16-byte load a
// lane.  Word s of lane l holds the codes of n = l % 16 and the eight k =
// 32 s + 8 (l / 16) .. + 7: the lane's operand of the 16x16x32 matrix
// instruction of k step s (fp32: eight 16x16x4 instructions, element e of every
// lane to instruction e).  Blocks of one n tile follow each other along k, n
// tiles and then experts outside.  The scales come after all codes, 16 n
// together: [expert][n tile][group][16].  Past N and K: weight 0, scale 0.
constexpr int kQ4N = 16, kQ4K = 128;

struct Q4Shape {
    int64_t n_tiles, k_blocks, groups;     // groups of a packed row: k_blocks * 128 / group
    int64_t codes, bytes;                   // bytes of all codes, of codes and scales
};
inline Q4Shape q4_shape(int64_t experts, int64_t N, int64_t K, int64_t group, int64_t esz) {
    Q4Shape s;
    s.n_tiles = (N + kQ4N - 1) / kQ4N;
    s.k_blocks = (K + kQ4K - 1) / kQ4K;
    s.groups = s.k_blocks * (kQ4K / group);
    s.codes = experts * s.n_tiles * s.k_blocks * 1024;
    s.bytes = s.codes + experts * s.n_tiles * s.groups * kQ4N * esz;
    return s;
}

// Where element e (0 .. 7) of a lane's eight sits in its word, and how it is
// stored, is chosen for the cheapest way back to the input type:
//  * f16: code e in bits 4 (e / 2) + 16 (e % 2), as it is: a shift and a mask
//    give two codes in the low bits of two halves, or-ing 0x6400 makes them
//    1024 + code exactly, and a packed subtraction of 1032 ends it: 11
//    instructions for eight.
//  * bf16, f32: code e in bits 4 e, its top bit turned, which makes it the
//    two's complement of code - 8; v_cvt_off_f32_i4 turns one into fp32 (value
//    / 16, exactly) in one instruction.  The factor 16 goes into the group's fma.
template <int DT>
TG_HD int q4_bit(int e) { return DT == DT_F16 ? 4 * (e / 2) + 16 * (e % 2) : 4 * e; }
template <int DT>
TG_HD uint32_t q4_stored(uint32_t code) { return DT == DT_F16 ? code : code ^ 8u; }

// One thread a word: grid-stride over the words of the packed codes, then the
// scales (as raw values of ESZ bytes).
template <int DT>
__global__ __launch_bounds__(256) void q4_pack_kernel(const uint8_t *__restrict__ codes, int64_t ld_codes,
                                                      int64_t stride_codes,
                                                      const typename ElemOf<DT>::type *__restrict__ scales,
                                                      int64_t ld_scales, int64_t stride_scales, Q4Shape s,
                                                      int64_t experts, int64_t N, int64_t K, int group,
                                                      uint32_t *__restrict__ packed) {
    typedef typename ElemOf<DT>::type T;
    const int64_t step = (int64_t)gridDim.x * 256, first = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t words = s.codes / 4;
    for (int64_t i = first; i < words; i += step) {
        const int word = (int)(i % 4), lane = (int)(i / 4 % 64);
        const int64_t block = i / 256, kb = block % s.k_blocks, tile = block / s.k_blocks;
        const int64_t n = tile % s.n_tiles * kQ4N + lane % 16, g = tile / s.n_tiles;
        const int64_t k0 = kb * kQ4K + 32 * word + 8 * (lane / 16);
        uint32_t v = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            uint32_t code = 8;
            if (n < N && k0 + e < K) {
                const uint32_t byte = codes[g * stride_codes + n * ld_codes + (k0 + e) / 2];
                code = e % 2 ? byte >> 4 : byte & 15u;
            }
            v |= q4_stored<DT>(code) << q4_bit<DT>(e);
        }
        packed[i] = v;
    }
    T *out = reinterpret_cast<T *>(reinterpret_cast<char *>(packed) + s.codes);
    const int64_t count = experts * s.n_tiles * s.groups * kQ4N;
    const int64_t groups_in = (K + group - 1) / group;
    for (int64_t i = first; i < count; i += step) {
        const int64_t q = i / kQ4N % s.groups, tile = i / kQ4N / s.groups;
        const int64_t n = tile % s.n_tiles * kQ4N + i % kQ4N, g = tile / s.n_tiles;
        out[i] = n < N && q < groups_in ? scales[g * stride_scales + n * ld_scales + q] : (T)0.0f;
    }
}

// Eight codes of a word as a matrix operand: 16 bytes (16-bit types), or eight
// floats.  Q4_UNIT is what one unit of the operand stands for.
template <int DT> struct Q4Unit { static constexpr float value = 16.0f; };
template <> struct Q4Unit<DT_F16> { static constexpr float value = 1.0f; };

__device__ __forceinline__ void q4_floats(uint32_t w, float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __builtin_amdgcn_cvt_off_f32_i4((int)(w >> (4 * e)));
}
template <int DT>
__device__ __forceinline__ u32x4 q4_operand(uint32_t w) {
    u32x4 v;
    if constexpr (DT == DT_F16) {
        typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
        const f16x2 off = {(_Float16)1032.0f, (_Float16)1032.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, ((w >> (4 * i)) & 0x000f000fu) | 0x64006400u) - off);
    } else {
        float f[8];
        q4_floats(w, f);
#pragma unroll
        for (int i = 0; i < 4; ++i)      // the high halves of two exact values
            v[i] = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, f[2 * i + 1]),
                                         __builtin_bit_cast(uint32_t, f[2 * i]), 0x07060302u);
    }
    return v;
}

struct Q4Params {
    const char *A;
    const char *codes, *scales;     // of the pack
    char *C;
    const int32_t *offsets;
    int64_t lda, ldc;
    int64_t k_blocks, groups;       // of a packed row
    int experts, rows, N, K, n_tiles;
    int c_f32;                      // C is fp32 (else the input type)
};

// A workgroup takes one n tile of one expert; its waves split K (blocks w,
// w + W, ...) and add their sums in LDS, wave by wave in order.  Weights are the
// matrix instruction's first operand, so lane l holds C[row l % 16][n 4 (l / 16)
// .. + 3]: four neighbours in a row of C, one store.  MT row tiles of 16 at a
// time; more rows take further passes over the codes (from L2).
template <int DT, int GROUP, int MT>
__global__ __launch_bounds__(MT == 4 ? 512 : 1024) void q4_kernel(Q4Params p) {
    typedef typename ElemOf<DT>::type T;
    constexpr int E = (int)sizeof(T);
    constexpr int PIECES = DT == DT_F32 ? 2 : 1;    // 16-byte loads for a lane's eight k of a row
    constexpr int PER = 16 / E;
    extern __shared__ f32x4 q4_lds[];                // [waves][MT][64]
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // the same in every lane of a wave
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    const int g = blockIdx.y, tile = blockIdx.x;
    const RowSpan span = rows_of(p.offsets, g, p.experts, p.rows);
    const int n0 = tile * kQ4N + 4 * (lane / 16);
    const bool wide = p.ldc % 4 == 0 && reinterpret_cast<uintptr_t>(p.C) % 16 == 0;
    const bool dead = g == p.experts || p.K == 0;    // zeros
    const int64_t at = (int64_t)g * p.n_tiles + tile;
    const u32x4 *codes = reinterpret_cast<const u32x4 *>(p.codes) + at * p.k_blocks * 64 + lane;
    const T *scales = reinterpret_cast<const T *>(p.scales) + at * p.groups * kQ4N + 4 * (lane / 16);
    for (int r0 = span.lo; r0 < span.hi; r0 += 16 * MT) {
        f32x4 acc[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[i] = f32x4{0, 0, 0, 0};
        if (!dead) {
            const int rows = span.hi - r0 < 16 * MT ? span.hi - r0 : 16 * MT;
            const rsrc_t ra = make_rsrc(p.A + (int64_t)r0 * p.lda * E);
            int voff[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int r = 16 * i + lane % 16;
                voff[i] = r < rows ? (int)(r * (int)p.lda + 8 * (lane / 16)) * E : kOutOfRange;
            }
            // one block of 128 k; TAIL: K ends in it (A past K is +0, so that a NaN
            // behind a row's end meets no weight)
            auto block = [&](int kb, auto tail) {
                constexpr bool TAIL = decltype(tail)::value;
                const u32x4 w = codes[(int64_t)kb * 64];
                f32x4 sum[MT];
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int k0 = kb * kQ4K + 32 * s;
                    u32x4 a[MT][PIECES];
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int h = 0; h < PIECES; ++h) {
                            if constexpr (TAIL) {
                                const int left = p.K - (k0 + 8 * (lane / 16) + PER * h);
                                a[i][h] = bload16_n<E>(ra, voff[i] + 16 * h, k0 * E,
                                                       left < 0 || voff[i] == kOutOfRange ? 0 : left);
                            } else {
                                a[i][h] = bload16(ra, voff[i] + 16 * h, k0 * E);
                            }
                        }
                    if (32 * s % GROUP == 0) {
#pragma unroll
                        for (int i = 0; i < MT; ++i) sum[i] = f32x4{0, 0, 0, 0};
                    }
                    if constexpr (DT == DT_F32) {
                        float f[8];
                        q4_floats(w[s], f);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
#pragma unroll
                            for (int i = 0; i < MT; ++i) {
                                const uint32_t x = a[i][e / 4][e % 4];
                                sum[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(f[e], __builtin_bit_cast(float, x), sum[i],
                                                                              0, 0, 0);
                            }
                    } else {
                        const u32x4 b = q4_operand<DT>(w[s]);
#pragma unroll
                        for (int i = 0; i < MT; ++i) mfma_chunk<DT>(b, a[i][0], sum[i]);
                    }
                    if ((32 * s + 32) % GROUP == 0) {
                        typedef T t4 __attribute__((ext_vector_type(4)));
                        const t4 q = *reinterpret_cast<const t4 *>(scales + (int64_t)(k0 / GROUP) * kQ4N);
#pragma unroll
                        for (int i = 0; i < MT; ++i)
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                acc[i][v] = __builtin_fmaf((float)q[v], Q4Unit<DT>::value * sum[i][v], acc[i][v]);
                    }
                }
            };
            const int full = p.K / kQ4K;
            int kb = wave;
            for (; kb < full; kb += waves) block(kb, std::false_type{});
            if (kb < p.k_blocks) block(kb, std::true_type{});
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) q4_lds[(wave * MT + i) * 64 + lane] = acc[i];
        __syncthreads();
        for (int i = wave; i < MT; i += waves) {
            f32x4 v = q4_lds[i * 64 + lane];
            for (int w = 1; w < waves; ++w) v += q4_lds[(w * MT + i) * 64 + lane];
            const int r = r0 + 16 * i + lane % 16;
            if (r < span.hi && n0 < p.N) store4<DT>(p.C, (int64_t)r * p.ldc + n0, p.N - n0, p.c_f32, wide, v);
        }
        __syncthreads();
    }
}

}  // namespace tg
