/*
 * tile_gemm_experts.h -- C ABI of the operators of a mixture-of-experts layer
 * on the MI355X (gfx950), next to the dense contraction of tile_gemm.h.
 *
 * A router sends each of `tokens` tokens to `top_k` of `experts` experts.  The
 * layer sorts the (token, choice) entries by expert, lays the tokens' rows out
 * in that order, multiplies every expert's rows by that expert's weights, and
 * sums the results back per token with the router's weights:
 *
 *   sort     entry e = t * top_k + j  ->  row(e), offsets
 *   gather   rows[row(e)] = x[t]
 *   grouped  C[r] = A[r] . B[g]           for the rows r of expert g
 *   q4       C[r] = A[r] . W[g]^T         W in 4 bits, one scale per group of k
 *   combine  out[t] = sum_j weights[t][j] * y[row(t * top_k + j)]
 *
 * and backwards
 *
 *   combine's gradient   d_y[row(e)] = weights[t][j] * d_out[t],
 *                        d_w[t][j]   = <d_out[t], y[row(e)]>      (combine_grad)
 *   gather's gradient    d_x[t]      = sum_j d_rows[row(e)]       (combine, weights NULL)
 *   the product's        d_A[r]      = d_C[r] . B[g]^T            (grouped, transposed 1)
 *                        d_B[g]      = A[rows of g]^T . d_C[rows of g]   (grouped_wgrad)
 *
 * Conventions (those of tile_gemm.h, and)
 *  - Matrices are row-major; leading dimensions and strides count ELEMENTS.
 *    dtype is the type of the inputs; c_dtype that of the product's result:
 *    TG_F32, or dtype.  Sums are held in fp32; a 16-bit result is rounded once,
 *    to nearest even.
 *  - No alignment requirement beyond the element size, except where stated.
 *  - Row tables.  row_of_entry holds row(e) for an entry that has an expert,
 *    and the complement ~row (negative) for one that has none: an entry whose
 *    id is outside 0 .. experts - 1 (-1 marks a choice that a capacity limit
 *    dropped).  Those entries' rows come after every expert's.  entry_of_row is
 *    the inverse: the entry of each row, complemented for rows without an expert.
 *    Both are contiguous.  offsets[g] is the first row of expert g (offsets[0] is 0)
 *    and offsets[experts] the number of rows that have one; they must not decrease.
 *    Tables live in device memory and are not checked on the host.  The kernels
 *    clamp what they read to the rows there are, so a wrong table gives wrong
 *    results and no access outside the operands.
 *  - Rows without an expert: gather writes zeros there, combine does not read
 *    them (a NaN there goes nowhere), combine_grad writes zeros into their row
 *    of d_y and their d_w, the products write zeros into their rows of C.  An
 *    expert without a row costs nothing in `grouped` and `q4`; its d_B is zeros.
 *  - tokens, rows or an extent of 0: what there is to write is written (zeros
 *    where a sum is empty), else nothing is launched; TG_OK.
 *  - The caller owns every buffer.  Outputs must not overlap inputs or each
 *    other (checked: TG_ERR_INVALID_ARG).  Calls only launch kernels on
 *    `stream`: no allocation, no memset, no synchronisation, so they can be
 *    captured into a HIP graph.  Results are bitwise reproducible: no atomics.
 *  - TG_ERR_UNSUPPORTED: no visible gfx950 device; tokens * top_k of 2^31 or
 *    more (the sort: 2^31 - 2^24); more than TILE_GEMM_MAX_EXPERTS experts; in the products, rows or an
 *    extent above 2^30, a leading dimension at which a block's tile would span
 *    2^31 bytes, a result of 2^24 tiles or more, K of 2^30 bytes (4-bit products);
 *    a group size that is not built.
 *
 * These entry points were added beside version 11 of tile_gemm.h, whose structs
 * and calls they leave as they are; they have a version of their own.
 */
#ifndef TILE_GEMM_EXPERTS_H
#define TILE_GEMM_EXPERTS_H

#include <stdint.h>

#include "tile_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TILE_GEMM_EXPERTS_VERSION 2    /* 2: the plan queries */
#define TILE_GEMM_MAX_EXPERTS 2048

int tile_gemm_experts_version(void);

/*
 * Sort the entries by expert: equal experts by entry, entries without an
 * expert last.  ids: tokens x top_k (row stride ld_ids >= top_k), int32.
 * offsets: experts + 1; entry_of_row and row_of_entry: tokens * top_k.
 * workspace: 4-byte aligned device memory of at least the size that
 * tile_gemm_expert_sort_workspace_size gives (may be 0: then NULL will do).
 */
tg_status tile_gemm_expert_sort_workspace_size(int64_t tokens, int64_t top_k, int64_t experts, int64_t *bytes);
tg_status tile_gemm_expert_sort(int64_t tokens, int64_t top_k, int64_t experts, const int32_t *ids, int64_t ld_ids,
                                int32_t *offsets, int32_t *entry_of_row, int32_t *row_of_entry,
                                void *workspace, int64_t workspace_bytes, void *stream);

/* rows[row(e)] = x[t] for every entry e = t * top_k + j; x: tokens x cols,
 * rows: tokens * top_k x cols, both of `dtype`.  Each row of x is read once. */
tg_status tile_gemm_expert_gather(int64_t tokens, int64_t top_k, int64_t cols, tg_dtype dtype, const void *x,
                                  int64_t ldx, const int32_t *row_of_entry, void *rows, int64_t ldr, void *stream);

/* out[t] = sum over j of weights[t][j] * y[row(t * top_k + j)], j increasing,
 * over the entries that have an expert; weights (fp32, tokens x top_k, row
 * stride ld_w) NULL: every weight 1 (the gradient of gather). */
tg_status tile_gemm_expert_combine(int64_t tokens, int64_t top_k, int64_t cols, tg_dtype dtype, const void *y,
                                   int64_t ldy, const int32_t *row_of_entry, const float *weights, int64_t ld_w,
                                   void *out, int64_t ldo, void *stream);

/* The gradient of combine: d_y (tokens * top_k x cols) and d_w (fp32, tokens x
 * top_k, row stride ld_dw) from d_out (tokens x cols), y and the weights. */
tg_status tile_gemm_expert_combine_grad(int64_t tokens, int64_t top_k, int64_t cols, tg_dtype dtype,
                                        const void *d_out, int64_t ldo, const void *y, int64_t ldy,
                                        const int32_t *row_of_entry, const float *weights, int64_t ld_w,
                                        void *d_y, int64_t ldd, float *d_w, int64_t ld_dw, void *stream);

/*
 * C[r] = A[r] . B[g] for the rows r in [offsets[g], offsets[g + 1]) of every
 * expert g.  A: rows x K; C: rows x N.  transposed 0: B[g] is K x N, element
 * (k, n) at B[g * strideB + k * ldb + n]; transposed 1: N x K, (k, n) at
 * B[g * strideB + n * ldb + k].  offsets may be NULL for one expert (it has
 * every row).
 */
tg_status tile_gemm_grouped(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, const void *A,
                            int64_t lda, const void *B, int64_t ldb, int64_t strideB, int transposed, void *C,
                            int64_t ldc, tg_dtype c_dtype, const int32_t *offsets, void *stream);

/*
 * C[g] = A[rows of g]^T . D[rows of g] for every expert g: A rows x M, D rows
 * x N, C[g] M x N at C + g * strideC (strideC >= (M - 1) * ldc + N for more
 * than one expert).  Zeros for an expert without a row.
 */
tg_status tile_gemm_grouped_wgrad(int64_t experts, int64_t rows, int64_t M, int64_t N, tg_dtype dtype, const void *A,
                                  int64_t lda, const void *D, int64_t ldd, void *C, int64_t ldc, int64_t strideC,
                                  tg_dtype c_dtype, const int32_t *offsets, void *stream);

/*
 * 4-bit weights.  W[g] is N x K; element (n, k) is (code - 8) * scale, its
 * code four bits of byte codes[g * stride_codes + n * ld_codes + k / 2] (the
 * lower four for even k), its scale scales[g * stride_scales + n * ld_scales +
 * k / group], of `dtype`.  group: 32, 64 or 128.
 *
 * tile_gemm_pack_q4 lays codes and scales out once, in the order in which the
 * product's lanes take them; packed is caller-owned, 16-byte aligned, at least
 * tile_gemm_q4_packed_size bytes: roundup(N, 16) * roundup(K, 128) / 2 bytes of
 * codes for each expert, then the scales.  dtype is part of the layout.
 *
 * tile_gemm_q4: C[r] = A[r] . W[g]^T for the rows of every expert g, A rows x K
 * of the dtype of the pack.  The codes enter the products as whole numbers and
 * a group's sum is scaled in fp32, so the weights are never rounded.  offsets
 * may be NULL for one expert.
 */
tg_status tile_gemm_q4_packed_size(int64_t experts, int64_t N, int64_t K, int64_t group, tg_dtype dtype,
                                   int64_t *bytes);
tg_status tile_gemm_pack_q4(int64_t experts, int64_t N, int64_t K, int64_t group, tg_dtype dtype,
                            const uint8_t *codes, int64_t ld_codes, int64_t stride_codes, const void *scales,
                            int64_t ld_scales, int64_t stride_scales, void *packed, int64_t packed_bytes,
                            void *stream);
tg_status tile_gemm_q4(int64_t experts, int64_t rows, int64_t N, int64_t K, int64_t group, tg_dtype dtype,
                       const void *A, int64_t lda, const void *packed, void *C, int64_t ldc, tg_dtype c_dtype,
                       const int32_t *offsets, void *stream);

/*
 * The kernel and grid a product would be launched with (pure host arithmetic on
 * sizes and types; no device is needed).  The arguments are the calls' own and
 * are refused as they are there; rows, N or M of 0: kernel TG_EXPERTS_NOTHING.
 */
typedef enum {
    TG_EXPERTS_NOTHING = 0,
    TG_EXPERTS_STREAM = 1,     /* weights streamed to registers, the waves of a workgroup split K */
    TG_EXPERTS_TILES = 2,      /* block tiles through LDS */
    TG_EXPERTS_NARROW = 3,     /* the weights' gradient of an extent below 8 */
    TG_EXPERTS_Q4 = 4          /* 4-bit weights */
} tg_experts_kernel;

typedef struct {
    int kernel;                /* tg_experts_kernel */
    int tile_m, tile_n;        /* rows and columns of the result a workgroup holds at a time */
    int pieces;                /* 1: short last tile rows and part-filled rounds in quarters of the tile */
    int pipeline;              /* tiles: 1: fragments a K tile ahead in registers */
    int waves;                 /* of a workgroup */
    int past_caches;           /* tiles: 1: whole tiles are stored past the caches */
    int pad_;
    int64_t workgroups;
    int64_t row_tiles;         /* tiles of rows one workgroup takes in turn at most, however the rows are split */
} tg_experts_plan_info;

tg_status tile_gemm_grouped_plan(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, int transposed,
                                 tg_dtype c_dtype, tg_experts_plan_info *out);
tg_status tile_gemm_grouped_wgrad_plan(int64_t experts, int64_t rows, int64_t M, int64_t N, tg_dtype dtype,
                                       tg_dtype c_dtype, tg_experts_plan_info *out);
tg_status tile_gemm_q4_plan(int64_t experts, int64_t rows, int64_t N, int64_t K, int64_t group, tg_dtype dtype,
                            tg_dtype c_dtype, tg_experts_plan_info *out);

#ifdef __cplusplus
}
#endif

#endif /* TILE_GEMM_EXPERTS_H */
