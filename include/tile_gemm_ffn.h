/*
 * tile_gemm_ffn.h -- C ABI of the operators of a feed-forward block on the MI355X
 * (gfx950), next to the dense contraction of tile_gemm.h and the operators of a
 * mixture-of-experts layer of tile_gemm_experts.h: what stands inside the block whose
 * products those compute.
 *
 *   gated        u = A . Bg,  v = A . Bu,  h = act(u) * v, per expert or for all rows
 *   gated_grad   d_h = D . B,  d_u = d_h * v * act'(u),  d_v = d_h * act(u),  h again
 *   gate, gate_grad   the same two from u and v (and d_h) that another call gave
 *   adapters     t = s[g] (x . A[g]),  y = x . W + t . B[g]: a projection shared by all
 *                rows, and beside it a low-rank adapter of each row's own
 *   adapters_wgrad   d_A[g] = x^T . d_t,  d_B[g] = t^T . d_y over the rows of adapter g
 *
 * The rest of the gated block's backward pass are products that are there: with the two
 * projections side by side (one matrix of K x 2N, or 2N x K, for an expert) and d_u, d_v
 * side by side too, d_x = [d_u d_v] . [Bg Bu]^T is tile_gemm_grouped, and their gradient
 * x^T . [d_u d_v] tile_gemm_grouped_wgrad.  The adapters' d_x = d_y . W^T + d_t . A[g]^T and
 * d_t = s[g] (d_y . B[g]^T) are tile_gemm_adapters on the same matrices, with N and K, A and B
 * exchanged and the other value of `transposed`.
 *
 * Conventions: those of tile_gemm_experts.h, and
 *  - Activations by the numbers of tile_gemm.h's fused tail: 0 none, 1 ReLU, 2 GELU (x Phi(x));
 *    3 is SiLU, x / (1 + e^-x).
 *  - Results are of dtype, except where a c_dtype is given; sums and the activation's
 *    argument are fp32.  t enters the second product in fp32 where rows are few (up to 64;
 *    up to 512 with at most 192 tiles of 64 x 64 in y; any number with N below 8), and rounded
 *    once to dtype (as T is) where there are more: how exact a row's y is goes by the rows and
 *    columns of its call, and in TG_F16 a t past 65504 is an infinity there, which y gets.
 *    A NaN or an infinity in a row, or in an adapter, reaches that row's, or that adapter's
 *    rows', results only.
 *  - transposed 0: matrices are inputs x outputs (Bg, Bu, W: K x N, an adapter's A: K x rank,
 *    B: rank x N); 1: outputs x inputs (N x K, rank x K, N x rank).
 *  - Rows without an expert get zeros in h, u, v and in d_u, d_v (u and v are not read
 *    there); rows without an adapter get y = x . W and t = 0.
 *  - Workspaces: 16-byte aligned device memory of the caller's, of at least the size that the
 *    query gives for the same arguments, free again when the call's work on `stream` is
 *    done.  Two calls that may run at the same time need one each.
 *  - Two outputs (U and V, dU and dV) may lie side by side in rows of one matrix.
 *  - TG_ERR_UNSUPPORTED: as in tile_gemm_experts.h; also, with an order and more rows than
 *    the streamed kernels take, x of 2^31 bytes or more.
 */
#ifndef TILE_GEMM_FFN_H
#define TILE_GEMM_FFN_H

#include <stdint.h>

#include "tile_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TILE_GEMM_FFN_VERSION 1

int tile_gemm_ffn_version(void);

/*
 * The gated pair: H[r] = act(A[r] . Bg[g]) * (A[r] . Bu[g]) for the rows r in [offsets[g],
 * offsets[g + 1]) of every expert g.  A: rows x K; B (Bg) and B_up (Bu): K x N, or N x K with
 * transposed 1, both at row stride ldb and strideB from expert to expert; H: rows x N.  U, V: the
 * two products (rows x N, row stride ldu), for the gradient; both NULL: not stored.  offsets
 * may be NULL for one expert.  workspace: optional (smaller than the query's size: not used);
 * with it K is split over more workgroups where there are few.
 */
tg_status tile_gemm_gated_workspace_size(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype,
                                         int transposed, int64_t *bytes);
tg_status tile_gemm_gated(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, const void *A,
                          int64_t lda, const void *B, const void *B_up, int64_t ldb, int64_t strideB, int transposed,
                          int activation, void *H, int64_t ldh, void *U, void *V, int64_t ldu, const int32_t *offsets,
                          void *workspace, int64_t workspace_bytes, void *stream);

/*
 * The gradient of the gate, from the gradient D (rows x K) of what the block gives and its down
 * projection: d_h = D . B[g], B K x N or, with transposed 1, N x K -- a down projection of N inputs
 * and K outputs stored inputs x outputs is transposed 1 here.  U, V: the forward call's.
 * dU, dV: rows x N at row stride lddu.  H (rows x N): act(u) * v once more, from U and V; NULL: not
 * written.
 */
tg_status tile_gemm_gated_grad(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, const void *D,
                               int64_t ldd, const void *B, int64_t ldb, int64_t strideB, int transposed,
                               int activation, const void *U, const void *V, int64_t ldu, void *dU, void *dV,
                               int64_t lddu, void *H, int64_t ldh, const int32_t *offsets, void *stream);

/*
 * The gate alone, of rows that another call gave (a projection with adapters, 4-bit
 * weights): H = act(U) * V, and from the gradient D of H (rows x N) dU = D * V * act'(U),
 * dV = D * act(U), and H once more (NULL: not written).
 */
tg_status tile_gemm_gate(int64_t rows, int64_t N, tg_dtype dtype, int activation, const void *U, const void *V,
                         int64_t ldu, void *H, int64_t ldh, void *stream);
tg_status tile_gemm_gate_grad(int64_t rows, int64_t N, tg_dtype dtype, int activation, const void *D, int64_t ldd,
                              const void *U, const void *V, int64_t ldu, void *dU, void *dV, int64_t lddu, void *H,
                              int64_t ldh, void *stream);

/*
 * Y[r] = X[r] . W + t[r] . B[g], t[r] = scales[g] * (X[r] . A[g]).  X: rows x K, Y: rows x N, W: K x N
 * (or N x K); A[g], B[g]: K x rank and rank x N (or rank x K and N x rank) at strideA, strideB.
 * scales: one fp32 an adapter, NULL: 1.  Adapter g has the positions offsets[g] .. offsets[g + 1] - 1
 * of the adapters' order, those from offsets[adapters] on have none; position p is row order[p]
 * of X, Y and T (order[p] or its complement: tile_gemm_expert_sort's entry_of_row, with one
 * choice a row, is such a table; it must hold every row once), or row p where order is NULL.
 * T (rows x rank, of dtype): t, for the gradients, where N is 0 too; NULL: not stored.
 */
tg_status tile_gemm_adapters_workspace_size(int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank,
                                            tg_dtype dtype, int transposed, int64_t *bytes);
tg_status tile_gemm_adapters(int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank, tg_dtype dtype,
                             const void *X, int64_t ldx, const void *W, int64_t ldw, const void *A, int64_t lda,
                             int64_t strideA, const void *B, int64_t ldb, int64_t strideB, int transposed,
                             const float *scales, void *Y, int64_t ldy, void *T, int64_t ldt, const int32_t *offsets,
                             const int32_t *order, void *workspace, int64_t workspace_bytes, void *stream);

/*
 * dA[g] = X^T . dT and dB[g] = T^T . dY over the rows of adapter g (K x rank and rank x N, or
 * transposed rank x K and N x rank), in c_dtype; zeros for an adapter without a row.  X, dY:
 * rows x K, rows x N; T, dT: rows x rank, what tile_gemm_adapters stored forward and backward.
 * strideA and strideB at least one matrix where there are several adapters.
 */
tg_status tile_gemm_adapters_wgrad_workspace_size(int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank,
                                                  tg_dtype dtype, int64_t *bytes);
tg_status tile_gemm_adapters_wgrad(int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank, tg_dtype dtype,
                                   const void *X, int64_t ldx, const void *dY, int64_t ldy, const void *T, int64_t ldt,
                                   const void *dT, int64_t lddt, void *dA, int64_t lda, int64_t strideA, void *dB,
                                   int64_t ldb, int64_t strideB, int transposed, tg_dtype c_dtype,
                                   const int32_t *offsets, const int32_t *order, void *workspace,
                                   int64_t workspace_bytes, void *stream);

/*
 * The kernel and grid of a call (pure host arithmetic on sizes and types; no device is
 * needed); rows or N of 0: kernel TG_FFN_NOTHING.  tile_gemm_gated's with the workspace
 * that its query asks for, tile_gemm_adapters' the product with W.
 */
typedef enum {
    TG_FFN_NOTHING = 0,
    TG_FFN_STREAM = 1,         /* weights streamed to registers */
    TG_FFN_TILES = 2           /* block tiles through LDS */
} tg_ffn_kernel;

typedef struct {
    int kernel;                /* tg_ffn_kernel */
    int tile_m, tile_n;        /* rows and columns of the result a workgroup holds */
    int pieces;                /* 1: short last tile rows and part-filled rounds in quarters of the tile */
    int pipeline;              /* tiles: 1: fragments a K tile ahead in registers */
    int waves;                 /* of a workgroup */
    int splits;                /* of K over workgroups, whose sums a second launch adds (1: none) */
    int pad_;
    int64_t workgroups;
} tg_ffn_plan_info;

tg_status tile_gemm_gated_plan(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, int transposed,
                               tg_ffn_plan_info *out);
tg_status tile_gemm_gated_grad_plan(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, int transposed,
                                    tg_ffn_plan_info *out);
tg_status tile_gemm_adapters_plan(int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank, tg_dtype dtype,
                                  int transposed, tg_ffn_plan_info *out);

#ifdef __cplusplus
}
#endif

#endif /* TILE_GEMM_FFN_H */
