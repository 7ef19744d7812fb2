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
// tiles and then experts outside.  The scales come after all codes, a block's
// together: [expert][n tile][block][n / 4 of 4][group of the block][n % 4], so that a
// lane finds those of its four outputs side by side.  Past N and K: weight 0, scale 0.
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
//  * f16: code e in bits 4 (e / 2) + 16 (e % 2), as it is: a mask leaves two codes in
//    the low four or the next four bits of two halves, or-ing 0x6400 makes them 1024 +
//    code or 1024 + 16 code exactly, and a packed subtraction of 1032, or a
//    multiplication by 1 / 16 less 72, ends it: 9 instructions for eight.
//  * bf16, f32: code e in bits 4 e, its top bit turned, which makes it the
//    two's complement of code - 8; v_cvt_off_f32_i4 turns four bits into fp32 (value /
//    16, exactly).  The factor 16 is applied to the finished sum: 15 instructions for
//    eight bf16.
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
        const int per = kQ4K / group;                       // groups of a block
        const int64_t block = i / (kQ4N * per), in = i % (kQ4N * per), tile = block / s.k_blocks;
        const int64_t q = block % s.k_blocks * per + in / 4 % per;
        const int64_t n = tile % s.n_tiles * kQ4N + in / (4 * per) * 4 + in % 4, g = tile / s.n_tiles;
        out[i] = n < N && q < groups_in ? scales[g * stride_scales + n * ld_scales + q] : (T)0.0f;
    }
}

// Eight codes of a word as a matrix operand: 16 bytes (16-bit types), or eight
// floats.  Q4Unit is what one unit of the operand stands for.
template <int DT> struct Q4Unit { static constexpr float value = 16.0f; };
template <> struct Q4Unit<DT_F16> { static constexpr float value = 1.0f; };

__device__ __forceinline__ void q4_floats(uint32_t w, float (&f)[8]) {
    // v_cvt_off_f32_i4 reads the low four bits of its source, whose upper half or top
    // byte the instruction selects itself: three shifts for eight codes.  The empty asm
    // keeps a shift of a shift apart.
    uint32_t x = w >> 4;
    asm("" : "+v"(x));
    auto cvt = [](uint32_t v) { return __builtin_amdgcn_cvt_off_f32_i4((int)v); };
    f[0] = cvt(w);
    f[1] = cvt(x);
    f[2] = cvt(w >> 8);
    f[3] = cvt(x >> 8);
    f[4] = cvt(w >> 16);
    f[5] = cvt(x >> 16);
    f[6] = cvt(w >> 24);
    f[7] = cvt(x >> 24);
}
template <int DT>
__device__ __forceinline__ u32x4 q4_operand(uint32_t w) {
    u32x4 v;
    if constexpr (DT == DT_F16) {
        typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
        const f16x2 off = {(_Float16)1032.0f, (_Float16)1032.0f};
        const f16x2 sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f}, off16 = {(_Float16)72.0f, (_Float16)72.0f};
        // one v_and_or_b32 each: a literal at most would fit the instruction, so the
        // two are kept in registers
        uint32_t low = 0x000f000fu, high = 0x00f000f0u, one = 0x64006400u;
        asm("" : "+s"(low), "+s"(high), "+v"(one));
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const uint32_t x = i == 0 ? w : w >> 8;
            v[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, (x & low) | one) - off);
            v[i + 1] = __builtin_bit_cast(
                uint32_t, __builtin_elementwise_fma(__builtin_bit_cast(f16x2, (x & high) | one), sixteenth, -off16));
        }
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

// A workgroup takes NT neighbouring n tiles of one expert; its waves split K
// (blocks w, w + W, ...) and add their sums in LDS, in wave order.  Weights are the
// matrix instruction's first operand, so lane l holds C[row l % 16][n 4 (l / 16)
// .. + 3]: four neighbours in a row of C, one store.  It takes 16 rows; an expert's further
// rows have workgroups of their own (row_slot), which read the codes again, from cache.
// (Two or four row tiles a workgroup, to turn the codes into operands once for them, were
// slower for every number of rows: 64 rows of 4096 x 4096 bf16 13.9 and 23.8 us against 9.4;
// 2048 rows, K 8192, N 4096, 570 and 632 against 380.)
//
// The codes, scales and activations of the next block are in flight while a block
// is multiplied.  Activations are loaded as they lie, 256 bytes of a row by 16
// lanes (fp32: 512 by 32), and cross to the lanes that need them through LDS of
// the wave's own, in 16-byte units whose place in a row is XORed with the row so
// that 16 rows meet distinct banks (64 rows of 8192 x 8192 bf16, 64 a workgroup: 43 us, 65
// when each lane loads its own operands, 64 bytes of 16 rows an instruction; at 16 rows the
// two are equal).
//
// Measured: one token through 4096 x 4096 bf16 5.5 us, a launch and its latency; 16 rows
// through 8192 x 8192 f16 10.6 us (3.4 TB/s; the codes alone, neither multiplied nor
// scaled, took 9.2), 64 rows bf16 27.7; 64 rows over 24 of 64 experts of 2048 x 2048 bf16
// 15.1 us (3.5 TB/s, 2.8 us of it for turning codes into bf16); 37 rows through 1001 x 4100
// fp32 11.7 us, the latency of its few workgroups.
template <int DT>
struct Q4Rows {
    typedef typename ElemOf<DT>::type T;
    static constexpr int E = (int)sizeof(T), PER = 16 / E;
    static constexpr int ROW = kQ4K / PER;             // 16-byte units of a block's row: 16 or 32
    static constexpr int RPI = 64 / ROW;               // rows of a load: 4 or 2
    static constexpr int LOADS = 16 / RPI;             // loads of a row tile
    static constexpr int PIECES = DT == DT_F32 ? 2 : 1;    // units of a lane's eight k
    static constexpr int LDS = 16 * ROW;               // units of a wave's region

    rsrc_t ra;
    int voff, lda, rows, K, lane;
    u32x4 *lds;
    __device__ __forceinline__ void init(const char *A, int64_t lda_, int rows_, int K_, int lane_, u32x4 *lds_) {
        ra = make_rsrc(A);
        lda = (int)lda_;
        rows = rows_;
        K = K_;
        lane = lane_;
        lds = lds_;
        voff = (lane / ROW * lda + lane % ROW * PER) * E;
        // rows that are never loaded
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            if (i * RPI >= rows) lds[i * 64 + lane] = u32x4{0, 0, 0, 0};
    }
    // TAIL: K ends in the block (past it +0, so that a NaN behind a row's end meets no weight)
    template <bool TAIL>
    __device__ __forceinline__ void load(int kb, u32x4 (&a)[LOADS]) const {
#pragma unroll
        for (int d = 0; d < LOADS; ++d) {
            const int r0 = RPI * d;
            if (r0 >= rows) continue;
            const int soff = (r0 * lda + kb * kQ4K) * E;
            const bool in = r0 + lane / ROW < rows;
            if constexpr (TAIL) {
                const int left = K - (kb * kQ4K + lane % ROW * PER);
                a[d] = bload16_n<E>(ra, voff, soff, in && left > 0 ? left : 0);
            } else {
                a[d] = bload16(ra, in ? voff : kOutOfRange, soff);
            }
        }
    }
    __device__ __forceinline__ void stage(const u32x4 (&a)[LOADS]) const {
#pragma unroll
        for (int d = 0; d < LOADS; ++d) {
            const int r = RPI * d + lane / ROW;
            if (RPI * d < rows) lds[r * ROW + (lane % ROW ^ r)] = a[d];
        }
    }
    // Activations pass from lane to lane between stage and read.  A wave's LDS operations
    // take effect in program order, which this keeps: nothing else tells the compiler that a
    // lane reads what another has stored (the fences are of a wave alone: no instruction).
    __device__ __forceinline__ static void order() {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
    // unit h of this lane's eight k of step s, row lane % 16
    __device__ __forceinline__ u32x4 read(int s, int h) const {
        const int r = lane % 16, unit = 4 * PIECES * s + PIECES * (lane / 16) + h;
        return lds[r * ROW + (unit ^ r)];
    }
};

template <int DT, int GROUP, int NT>
struct Q4Block {
    using Rows = Q4Rows<DT>;
    typedef typename ElemOf<DT>::type T;
    typedef T t4 __attribute__((ext_vector_type(4)));
    static constexpr int SCALES = kQ4K / GROUP;
    u32x4 w[NT];
    t4 q[NT][SCALES];           // loaded together
    u32x4 a[Rows::LOADS];

    template <bool TAIL>
    __device__ __forceinline__ void load(const u32x4 *const (&codes)[NT], const T *const (&scales)[NT], const Rows &rows,
                                         int kb) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            w[t] = codes[t][(int64_t)kb * 64];
            const t4 *from = reinterpret_cast<const t4 *>(scales[t] + (int64_t)kb * (SCALES * kQ4N));
#pragma unroll
            for (int g = 0; g < SCALES; ++g) q[t][g] = from[g];
        }
        rows.template load<TAIL>(kb, a);
    }
    __device__ __forceinline__ void multiply(const Rows &rows, f32x4 (&acc)[NT]) {
        Rows::order();          // the block before has been read
        rows.stage(a);
        Rows::order();
        f32x4 sum[NT];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            u32x4 x[Rows::PIECES];
#pragma unroll
            for (int h = 0; h < Rows::PIECES; ++h) x[h] = rows.read(s, h);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (32 * s % GROUP == 0) sum[t] = f32x4{0, 0, 0, 0};
                if constexpr (DT == DT_F32) {
                    float f[8];
                    q4_floats(w[t][s], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t y = x[e / 4][e % 4];
                        sum[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(f[e], __builtin_bit_cast(float, y), sum[t], 0, 0, 0);
                    }
                } else {
                    mfma_chunk<DT>(q4_operand<DT>(w[t][s]), x[0], sum[t]);
                }
                if ((32 * s + 32) % GROUP == 0) {
                    const t4 c = q[t][32 * s / GROUP];
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[t][v] = __builtin_fmaf((float)c[v], sum[t][v], acc[t][v]);
                }
            }
        }
    }
};

// Waves of a workgroup at most: their LDS regions are 64 KiB together.
template <int DT>
constexpr int q4_waves() {
    const int fit = 65536 / (Q4Rows<DT>::LDS * 16);
    return fit < 8 ? fit : 8;
}

template <int DT, int GROUP, int NT>
__global__ __launch_bounds__(512) void q4_kernel(Q4Params p) {
    using Block = Q4Block<DT, GROUP, NT>;
    using Rows = Q4Rows<DT>;
    typedef typename Block::T T;
    extern __shared__ u32x4 q4_lds[];                // [waves][Rows::LDS], then the sums [waves][NT][64]
    static_assert(Rows::LDS >= NT * 64, "the sums fit the waves' regions");
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // the same in every lane of a wave
    const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
    const bool wide = p.ldc % 4 == 0 && reinterpret_cast<uintptr_t>(p.C) % 16 == 0;
    const int tile = blockIdx.x * NT;
    int g;
    RowSpan span;
    if (!row_slot<16>(p.offsets, p.experts, p.rows, slot_of(p.experts), g, span)) return;
    const bool dead = g == p.experts || p.K == 0;    // zeros
    const int n0 = tile * kQ4N + 4 * (lane / 16);
    const u32x4 *codes[NT];
    const T *scales[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        // past the last tile: the last one again, for columns that are not stored
        const int64_t at = (int64_t)g * p.n_tiles + (tile + t < p.n_tiles ? tile + t : p.n_tiles - 1);
        codes[t] = reinterpret_cast<const u32x4 *>(p.codes) + at * p.k_blocks * 64 + lane;
        scales[t] = reinterpret_cast<const T *>(p.scales) + at * p.groups * kQ4N + 4 * (kQ4K / GROUP) * (lane / 16);
    }
    const int r0 = span.lo;
    f32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[t] = f32x4{0, 0, 0, 0};
    if (!dead) {
        Rows rows;
        const int count = __builtin_amdgcn_readfirstlane(span.hi - r0);
        rows.init(p.A + (int64_t)r0 * p.lda * Rows::E, p.lda, count, p.K, lane, q4_lds + wave * Rows::LDS);
        const int full = p.K / kQ4K;
        int kb = wave;
        if (kb < full) {
            Block b, n;
            b.template load<false>(codes, scales, rows, kb);
            for (;;) {
                if (kb + waves < full) n.template load<false>(codes, scales, rows, kb + waves);
                b.multiply(rows, acc);
                kb += waves;
                if (kb >= full) break;
                if (kb + waves < full) b.template load<false>(codes, scales, rows, kb + waves);
                n.multiply(rows, acc);
                kb += waves;
                if (kb >= full) break;
            }
        }
        if (kb < p.k_blocks) {
            Block b;
            b.template load<true>(codes, scales, rows, kb);
            b.multiply(rows, acc);
        }
    }
    __syncthreads();
    f32x4 *sums = reinterpret_cast<f32x4 *>(q4_lds);
#pragma unroll
    for (int t = 0; t < NT; ++t) sums[(wave * NT + t) * 64 + lane] = acc[t];
    __syncthreads();
    for (int t = wave; t < NT; t += waves) {
        f32x4 v = sums[t * 64 + lane];
        for (int w = 1; w < waves; ++w) v += sums[(w * NT + t) * 64 + lane];
        const int r = r0 + lane % 16, n = n0 + 16 * t;
        v *= Q4Unit<DT>::value;
        if (r < span.hi && n < p.N) store4<DT>(p.C, (int64_t)r * p.ldc + n, p.N - n, p.c_f32, wide, v);
    }
}

}  // namespace tg
