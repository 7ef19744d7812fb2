// experts.hip -- the C ABI of the operators of a mixture-of-experts layer:
// argument checks, launches on the caller's stream, plan queries.  Declarations and
// contracts are in include/tile_gemm_experts.h.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "exchange.hpp"
#include "experts_plan.hpp"
#include "tile_gemm_experts.h"

using namespace tg;

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxExtent = int64_t(1) << 30;

bool known(tg_dtype t) { return t == TG_F32 || t == TG_BF16 || t == TG_F16; }
int size_of(tg_dtype t) { return t == TG_F32 ? 4 : 2; }
bool aligned(const void *p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
tg_status launched() { return hipGetLastError() == hipSuccess ? TG_OK : TG_ERR_LAUNCH; }

// Entries of a routing, tokens * top_k, or a refusal.
tg_status entries(int64_t tokens, int64_t top_k, int64_t &n) {
    if (tokens < 0 || top_k < 0) return TG_ERR_INVALID_ARG;
    if (tokens > kMaxRows || top_k > kMaxRows || tokens * top_k > kMaxRows) return TG_ERR_UNSUPPORTED;
    n = tokens * top_k;
    return TG_OK;
}

tg_status sort_arguments(int64_t tokens, int64_t top_k, int64_t experts, int64_t &n, SortShape &shape, int64_t &bytes) {
    if (experts < 1) return TG_ERR_INVALID_ARG;
    const tg_status st = entries(tokens, top_k, n);
    if (st != TG_OK) return st;
    // the places of a block's last entries are computed in 32 bits
    if (experts > TILE_GEMM_MAX_EXPERTS || n > kMaxRows - (int64_t(1) << 24)) return TG_ERR_UNSUPPORTED;
    shape = sort_shape(n, experts);
    bytes = shape.blocks > 1 ? (experts + 1) * shape.blocks * 4 : 0;
    return TG_OK;
}

tg_status sort(int64_t tokens, int64_t top_k, int64_t experts, const int32_t *ids, int64_t ld_ids, int32_t *offsets,
               int32_t *entry_of_row, int32_t *row_of_entry, void *workspace, int64_t workspace_bytes, void *stream) {
    int64_t n = 0, bytes = 0;
    SortShape shape;
    tg_status st = sort_arguments(tokens, top_k, experts, n, shape, bytes);
    if (st != TG_OK) return st;
    if (!offsets || (n > 0 && (!ids || !entry_of_row || !row_of_entry)) || ld_ids < top_k) return TG_ERR_INVALID_ARG;
    if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(entry_of_row, 4) || !aligned(row_of_entry, 4))
        return TG_ERR_INVALID_ARG;
    if (bytes > 0 && (!workspace || workspace_bytes < bytes || !aligned(workspace, 4))) return TG_ERR_INVALID_ARG;
    const Range r[5] = {span(ids, 1, tokens, top_k, ld_ids, 0, 4), span(offsets, 1, 1, experts + 1, 0, 0, 4),
                        span(entry_of_row, 1, 1, n, 0, 0, 4), span(row_of_entry, 1, 1, n, 0, 0, 4),
                        span(workspace, 1, 1, bytes, 0, 0, 1)};
    for (int i = 0; i < 5; ++i)
        for (int j = 0; j < i; ++j)
            if (overlaps(r[i], r[j])) return TG_ERR_INVALID_ARG;
    st = device_ok();
    if (st != TG_OK) return st;
    SortParams p;
    p.ids = ids;
    p.ld_ids = ld_ids;
    p.offsets = offsets;
    p.entry_of_row = entry_of_row;
    p.row_of_entry = row_of_entry;
    p.counts = static_cast<int32_t *>(workspace);
    p.n = (int)n;
    p.top_k = (int)top_k;
    p.experts = (int)experts;
    p.bits = 1;
    while ((int64_t(1) << p.bits) <= experts) ++p.bits;
    p.iters = shape.iters;
    p.blocks = (int)shape.blocks;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 grid((unsigned)shape.blocks), block((unsigned)shape.waves * 64);
    const unsigned keys = (unsigned)experts + 1;
    if (shape.blocks > 1) {
        hipLaunchKernelGGL(sort_count_kernel, grid, block, shape.waves * keys * 4, s, p);
        st = launched();
        if (st != TG_OK) return st;
    }
    const unsigned lds = (shape.waves + 2) * keys * 4;
    if (shape.iters == 1) hipLaunchKernelGGL(sort_place_kernel<1>, grid, block, lds, s, p);
    else if (shape.iters <= kSortOnce) hipLaunchKernelGGL(sort_place_kernel<kSortOnce>, grid, block, lds, s, p);
    else hipLaunchKernelGGL(sort_place_kernel<0>, grid, block, lds, s, p);
    return launched();
}

// One row-moving operand: rows x cols at row stride ld.
bool operand_ok(const void *p, int64_t rows, int64_t cols, int64_t ld, int esz) {
    return ld >= (cols > 1 ? cols : 1) && aligned(p, esz) && (p || rows == 0 || cols == 0);
}

tg_status gather(int64_t tokens, int64_t top_k, int64_t cols, tg_dtype dtype, const void *x, int64_t ldx,
                 const int32_t *row_of_entry, void *rows, int64_t ldr, void *stream) {
    int64_t n = 0;
    tg_status st = entries(tokens, top_k, n);
    if (st != TG_OK) return st;
    if (cols < 0 || !known(dtype)) return TG_ERR_INVALID_ARG;
    const int esz = size_of(dtype);
    if (!operand_ok(x, n, cols, ldx, esz) || !operand_ok(rows, n, cols, ldr, esz) || !aligned(row_of_entry, 4) ||
        (n > 0 && cols > 0 && !row_of_entry))
        return TG_ERR_INVALID_ARG;
    if (n == 0 || cols == 0) return TG_OK;
    const Range out = span(rows, 1, n, cols, ldr, 0, esz);
    if (overlaps(out, span(x, 1, tokens, cols, ldx, 0, esz)) || overlaps(out, span(row_of_entry, 1, 1, n, 0, 0, 4)))
        return TG_ERR_INVALID_ARG;
    st = device_ok();
    if (st != TG_OK) return st;
    const int group = row_group(cdiv(cols * esz, 16));
    const dim3 grid = token_grid(tokens, group);
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool past = store_past((n + tokens) * cols * esz);
#define TG_GATHER(DT, PAST, NARROW)                                                                                \
    hipLaunchKernelGGL((gather_kernel<DT, PAST, NARROW>), grid, dim3(256), 0, s,                                      \
                       static_cast<const ElemOf<DT>::type *>(x), ldx, row_of_entry,                                   \
                       static_cast<ElemOf<DT>::type *>(rows), ldr, (int)tokens, (int)top_k, cols, group)
#define TG_GATHER_AS(DT)                                         \
    if (past && group < 64) TG_GATHER(DT, true, true);           \
    else if (past) TG_GATHER(DT, true, false);                   \
    else if (group < 64) TG_GATHER(DT, false, true);             \
    else TG_GATHER(DT, false, false)
    // the bytes are moved as they are: one 16-bit kernel
    if (dtype == TG_F32) {
        TG_GATHER_AS(DT_F32);
    } else {
        TG_GATHER_AS(DT_F16);
    }
#undef TG_GATHER_AS
#undef TG_GATHER
    return launched();
}

// choices of a token taken together: the smallest of 1, 2, 4, 8 that holds them
int choices(int64_t top_k) { return top_k <= 1 ? 1 : (top_k <= 2 ? 2 : (top_k <= 4 ? 4 : 8)); }

template <int DT>
void launch_combine(const void *y, int64_t ldy, const int32_t *row_of_entry, const float *weights, int64_t ld_w,
                    void *out, int64_t ldo, int64_t tokens, int64_t top_k, int64_t cols, hipStream_t s) {
    typedef typename ElemOf<DT>::type T;
    // few choices: two chunks a thread, for as many loads in flight
    const int64_t chunks = cdiv(cols * (int64_t)sizeof(T), 16);
    const int group = row_group(choices(top_k) <= 2 ? cdiv(chunks, 2) : chunks);
    const dim3 grid = token_grid(tokens, group);
    const bool past = store_past((tokens * top_k + tokens) * cols * (int64_t)sizeof(T));
#define TG_COMBINE_AS(JB, U, PAST, NARROW)                                                                        \
    hipLaunchKernelGGL((combine_kernel<DT, JB, U, PAST, NARROW>), grid, dim3(256), 0, s, static_cast<const T *>(y), ldy, \
                       row_of_entry, weights, ld_w, static_cast<T *>(out), ldo, (int)tokens, (int)top_k, cols, group)
#define TG_COMBINE(JB, U)                                        \
    if (past && group < 64) TG_COMBINE_AS(JB, U, true, true);    \
    else if (past) TG_COMBINE_AS(JB, U, true, false);            \
    else if (group < 64) TG_COMBINE_AS(JB, U, false, true);      \
    else TG_COMBINE_AS(JB, U, false, false)
    switch (choices(top_k)) {
        case 1: TG_COMBINE(1, 2); break;
        case 2: TG_COMBINE(2, 2); break;
        case 4: TG_COMBINE(4, 1); break;
        default: TG_COMBINE(8, 1); break;
    }
#undef TG_COMBINE_AS
#undef TG_COMBINE
}

tg_status combine(int64_t tokens, int64_t top_k, int64_t cols, tg_dtype dtype, const void *y, int64_t ldy,
                  const int32_t *row_of_entry, const float *weights, int64_t ld_w, void *out, int64_t ldo,
                  void *stream) {
    int64_t n = 0;
    tg_status st = entries(tokens, top_k, n);
    if (st != TG_OK) return st;
    if (cols < 0 || !known(dtype)) return TG_ERR_INVALID_ARG;
    const int esz = size_of(dtype);
    if (!operand_ok(y, n, cols, ldy, esz) || !operand_ok(out, tokens, cols, ldo, esz) || !aligned(row_of_entry, 4) ||
        !aligned(weights, 4) || (weights && ld_w < top_k) || (n > 0 && cols > 0 && !row_of_entry))
        return TG_ERR_INVALID_ARG;
    if (tokens == 0 || cols == 0) return TG_OK;
    const Range to = span(out, 1, tokens, cols, ldo, 0, esz);
    if (overlaps(to, span(y, 1, n, cols, ldy, 0, esz)) || overlaps(to, span(row_of_entry, 1, 1, n, 0, 0, 4)) ||
        (weights && overlaps(to, span(weights, 1, tokens, top_k, ld_w, 0, 4))))
        return TG_ERR_INVALID_ARG;
    st = device_ok();
    if (st != TG_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (dtype) {
        case TG_F32: launch_combine<DT_F32>(y, ldy, row_of_entry, weights, ld_w, out, ldo, tokens, top_k, cols, s); break;
        case TG_BF16: launch_combine<DT_BF16>(y, ldy, row_of_entry, weights, ld_w, out, ldo, tokens, top_k, cols, s); break;
        case TG_F16: launch_combine<DT_F16>(y, ldy, row_of_entry, weights, ld_w, out, ldo, tokens, top_k, cols, s); break;
    }
    return launched();
}

template <int DT>
void launch_combine_grad(const void *d_out, int64_t ldo, const void *y, int64_t ldy, const int32_t *row_of_entry,
                         const float *weights, int64_t ld_w, void *d_y, int64_t ldd, float *d_w, int64_t ld_dw,
                         int64_t tokens, int64_t top_k, int64_t cols, hipStream_t s) {
    typedef typename ElemOf<DT>::type T;
    const int rows = row_group(cdiv(cols * (int64_t)sizeof(T), 16)), group = rows < 64 ? rows : 64;
    const dim3 grid = token_grid(tokens, group);
    const bool past = store_past((2 * tokens * top_k + tokens) * cols * (int64_t)sizeof(T));
#define TG_GRAD_AS(JB, PAST, NARROW)                                                                                \
    hipLaunchKernelGGL((combine_grad_kernel<DT, JB, PAST, NARROW>), grid, dim3(256), 0, s, static_cast<const T *>(d_out), \
                       ldo, static_cast<const T *>(y), ldy, row_of_entry, weights, ld_w, static_cast<T *>(d_y), ldd, d_w, \
                       ld_dw, (int)tokens, (int)top_k, cols, group)
#define TG_GRAD(JB)                                        \
    if (past && group < 64) TG_GRAD_AS(JB, true, true);    \
    else if (past) TG_GRAD_AS(JB, true, false);            \
    else if (group < 64) TG_GRAD_AS(JB, false, true);      \
    else TG_GRAD_AS(JB, false, false)
    switch (choices(top_k)) {
        case 1: TG_GRAD(1); break;
        case 2: TG_GRAD(2); break;
        case 4: TG_GRAD(4); break;
        default: TG_GRAD(8); break;
    }
#undef TG_GRAD
#undef TG_GRAD_AS
}

tg_status combine_grad(int64_t tokens, int64_t top_k, int64_t cols, tg_dtype dtype, const void *d_out, int64_t ldo,
                       const void *y, int64_t ldy, const int32_t *row_of_entry, const float *weights, int64_t ld_w,
                       void *d_y, int64_t ldd, float *d_w, int64_t ld_dw, void *stream) {
    int64_t n = 0;
    tg_status st = entries(tokens, top_k, n);
    if (st != TG_OK) return st;
    if (cols < 0 || !known(dtype)) return TG_ERR_INVALID_ARG;
    const int esz = size_of(dtype);
    if (!operand_ok(d_out, n, cols, ldo, esz) || !operand_ok(y, n, cols, ldy, esz) ||
        !operand_ok(d_y, n, cols, ldd, esz) || !aligned(row_of_entry, 4) || !aligned(weights, 4) || !aligned(d_w, 4) ||
        ld_w < top_k || ld_dw < top_k || (n > 0 && (!row_of_entry || !weights || !d_w)))
        return TG_ERR_INVALID_ARG;
    if (n == 0) return TG_OK;
    const Range in[4] = {span(d_out, 1, tokens, cols, ldo, 0, esz), span(y, 1, n, cols, ldy, 0, esz),
                         span(row_of_entry, 1, 1, n, 0, 0, 4), span(weights, 1, tokens, top_k, ld_w, 0, 4)};
    const Range to[2] = {span(d_y, 1, n, cols, ldd, 0, esz), span(d_w, 1, tokens, top_k, ld_dw, 0, 4)};
    if (overlaps(to[0], to[1])) return TG_ERR_INVALID_ARG;
    for (const Range &a : in)
        for (const Range &b : to)
            if (overlaps(a, b)) return TG_ERR_INVALID_ARG;
    st = device_ok();
    if (st != TG_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
#define TG_CALL(DT) \
    launch_combine_grad<DT>(d_out, ldo, y, ldy, row_of_entry, weights, ld_w, d_y, ldd, d_w, ld_dw, tokens, top_k, cols, s)
    switch (dtype) {
        case TG_F32: TG_CALL(DT_F32); break;
        case TG_BF16: TG_CALL(DT_BF16); break;
        case TG_F16: TG_CALL(DT_F16); break;
    }
#undef TG_CALL
    return launched();
}

// What the products of both kinds have in common.
tg_status product_sizes(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, tg_dtype c_dtype) {
    if (experts < 1 || rows < 0 || N < 0 || K < 0 || !known(dtype)) return TG_ERR_INVALID_ARG;
    if (c_dtype != TG_F32 && c_dtype != dtype) return TG_ERR_INVALID_ARG;
    if (experts > TILE_GEMM_MAX_EXPERTS || rows > kMaxExtent || N > kMaxExtent || K > kMaxExtent)
        return TG_ERR_UNSUPPORTED;
    return TG_OK;
}
tg_status product_arguments(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, tg_dtype c_dtype,
                            const int32_t *offsets) {
    const tg_status st = product_sizes(experts, rows, N, K, dtype, c_dtype);
    if (st == TG_ERR_INVALID_ARG || (!offsets && experts != 1) || !aligned(offsets, 4)) return TG_ERR_INVALID_ARG;
    return st;
}

// whether operands and result together exceed the last-level cache (GroupedParams::past)
bool past_caches(int64_t operand_bytes, int64_t result_bytes) {
    return operand_bytes + result_bytes > (int64_t(256) << 20);
}
bool grouped_past(int64_t experts, int64_t rows, int64_t N, int64_t K, int esz, int csz) {
    return past_caches((rows * K + experts * N * K) * esz, rows * N * csz);
}
bool wgrad_past(int64_t experts, int64_t rows, int64_t M, int64_t N, int esz, int csz) {
    return past_caches(rows * (M + N) * esz, experts * M * N * csz);
}

// A block's tile of an operand (256 rows of ld elements at most) is addressed
// in 31 bits from its first element.
bool tile_fits(int64_t ld, int esz) { return ld <= kMaxExtent && (256 * ld + 4096) * esz < (int64_t(1) << 31) - 65536; }

tg_status grouped(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, const void *A, int64_t lda,
                  const void *B, int64_t ldb, int64_t strideB, int transposed, void *C, int64_t ldc, tg_dtype c_dtype,
                  const int32_t *offsets, void *stream) {
    tg_status st = product_arguments(experts, rows, N, K, dtype, c_dtype, offsets);
    if (st != TG_OK) return st;
    if (transposed != 0 && transposed != 1) return TG_ERR_INVALID_ARG;
    const int esz = size_of(dtype), csz = size_of(c_dtype);
    const int64_t b_rows = transposed ? N : K, b_cols = transposed ? K : N;
    if (!operand_ok(A, rows, K, lda, esz) || !operand_ok(B, rows > 0 ? b_rows : 0, b_cols, ldb, esz) ||
        !operand_ok(C, rows, N, ldc, csz) || strideB < 0)
        return TG_ERR_INVALID_ARG;
    if (rows == 0 || N == 0) return TG_OK;
    const Range rc = span(C, 1, rows, N, ldc, 0, csz);
    if (overlaps(rc, span(A, 1, rows, K, lda, 0, esz)) ||
        overlaps(rc, span(B, experts, b_rows, b_cols, ldb, strideB, esz)) ||
        (offsets && overlaps(rc, span(offsets, 1, 1, experts + 1, 0, 0, 4))))
        return TG_ERR_INVALID_ARG;
    if (!tile_fits(lda, esz) || !tile_fits(ldb, esz) || !tile_fits(ldc, csz)) return TG_ERR_UNSUPPORTED;
    st = device_ok();
    if (st != TG_OK) return st;
    GroupedParams p = {};
    p.A = static_cast<const char *>(A);
    p.B = static_cast<const char *>(B);
    p.C = static_cast<char *>(C);
    p.offsets = offsets;
    p.lda = lda;
    p.ldb = ldb;
    p.ldc = ldc;
    p.sB = strideB;
    p.experts = (int)experts;
    p.rows = (int)rows;
    p.N = (int)N;
    p.K = (int)K;
    p.c_f32 = c_dtype == TG_F32;
    p.past = grouped_past(experts, rows, N, K, esz, csz);
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (dtype) {
        case TG_F32: return launch_grouped<DT_F32>(p, transposed != 0, s);
        case TG_BF16: return launch_grouped<DT_BF16>(p, transposed != 0, s);
        case TG_F16: return launch_grouped<DT_F16>(p, transposed != 0, s);
    }
    return TG_ERR_INTERNAL;
}

tg_status wgrad(int64_t experts, int64_t rows, int64_t M, int64_t N, tg_dtype dtype, const void *A, int64_t lda,
                const void *D, int64_t ldd, void *C, int64_t ldc, int64_t strideC, tg_dtype c_dtype,
                const int32_t *offsets, void *stream) {
    tg_status st = product_arguments(experts, rows, N, M, dtype, c_dtype, offsets);
    if (st != TG_OK) return st;
    const int esz = size_of(dtype), csz = size_of(c_dtype);
    if (!operand_ok(A, rows, M, lda, esz) || !operand_ok(D, rows, N, ldd, esz) || !operand_ok(C, M, N, ldc, csz) ||
        strideC < 0)
        return TG_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return TG_OK;
    if (experts > 1 && strideC < (M - 1) * ldc + N) return TG_ERR_INVALID_ARG;
    const Range rc = span(C, experts, M, N, ldc, strideC, csz);
    if (overlaps(rc, span(A, 1, rows, M, lda, 0, esz)) || overlaps(rc, span(D, 1, rows, N, ldd, 0, esz)) ||
        (offsets && overlaps(rc, span(offsets, 1, 1, experts + 1, 0, 0, 4))))
        return TG_ERR_INVALID_ARG;
    if (!tile_fits(lda, esz) || !tile_fits(ldd, esz) || !tile_fits(ldc, csz)) return TG_ERR_UNSUPPORTED;
    st = device_ok();
    if (st != TG_OK) return st;
    GroupedParams p = {};
    p.A = static_cast<const char *>(A);
    p.B = static_cast<const char *>(D);
    p.C = static_cast<char *>(C);
    p.offsets = offsets;
    p.lda = lda;
    p.ldb = ldd;
    p.ldc = ldc;
    p.sC = strideC;
    p.experts = (int)experts;
    p.rows = (int)rows;
    p.M = (int)M;
    p.N = (int)N;
    p.c_f32 = c_dtype == TG_F32;
    p.past = wgrad_past(experts, rows, M, N, esz, csz);
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (dtype) {
        case TG_F32: return launch_wgrad<DT_F32>(p, s);
        case TG_BF16: return launch_wgrad<DT_BF16>(p, s);
        case TG_F16: return launch_wgrad<DT_F16>(p, s);
    }
    return TG_ERR_INTERNAL;
}

tg_status q4_arguments(int64_t experts, int64_t N, int64_t K, int64_t group, tg_dtype dtype, Q4Shape &shape) {
    if (experts < 1 || N < 0 || K < 0 || group < 1 || !known(dtype)) return TG_ERR_INVALID_ARG;
    if (experts > TILE_GEMM_MAX_EXPERTS || N > kMaxExtent || K > kMaxExtent ||
        (group != 32 && group != 64 && group != 128))
        return TG_ERR_UNSUPPORTED;
    if (N > 0 && K > 0 && experts * ((N + 15) / 16) > (int64_t(1) << 50) / ((K + 127) / 128)) return TG_ERR_UNSUPPORTED;
    shape = q4_shape(experts, N, K, group, size_of(dtype));
    return TG_OK;
}

tg_status pack_q4(int64_t experts, int64_t N, int64_t K, int64_t group, tg_dtype dtype, const uint8_t *codes,
                  int64_t ld_codes, int64_t stride_codes, const void *scales, int64_t ld_scales, int64_t stride_scales,
                  void *packed, int64_t packed_bytes, void *stream) {
    Q4Shape shape;
    tg_status st = q4_arguments(experts, N, K, group, dtype, shape);
    if (st != TG_OK) return st;
    const int esz = size_of(dtype);
    const int64_t bytes = (K + 1) / 2, groups = cdiv(K, group);
    if (ld_codes < bytes || ld_scales < groups || stride_codes < 0 || stride_scales < 0 || !aligned(scales, esz))
        return TG_ERR_INVALID_ARG;
    if (N == 0 || K == 0) return TG_OK;
    if (!codes || !scales || !packed || !aligned(packed, 16) || packed_bytes < shape.bytes) return TG_ERR_INVALID_ARG;
    const Range to = span(packed, 1, 1, shape.bytes, 0, 0, 1);
    if (overlaps(to, span(codes, experts, N, bytes, ld_codes, stride_codes, 1)) ||
        overlaps(to, span(scales, experts, N, groups, ld_scales, stride_scales, esz)))
        return TG_ERR_INVALID_ARG;
    st = device_ok();
    if (st != TG_OK) return st;
    const int64_t blocks = cdiv(shape.codes / 4, 256);
    const dim3 grid((unsigned)(blocks < 16384 ? blocks : 16384));
    hipStream_t s = static_cast<hipStream_t>(stream);
#define TG_PACK(DT)                                                                                                 \
    hipLaunchKernelGGL((q4_pack_kernel<DT>), grid, dim3(256), 0, s, codes, ld_codes, stride_codes,                   \
                       static_cast<const ElemOf<DT>::type *>(scales), ld_scales, stride_scales, shape, experts, N, K, \
                       (int)group, static_cast<uint32_t *>(packed))
    switch (dtype) {
        case TG_F32: TG_PACK(DT_F32); break;
        case TG_BF16: TG_PACK(DT_BF16); break;
        case TG_F16: TG_PACK(DT_F16); break;
    }
#undef TG_PACK
    return launched();
}

tg_status q4(int64_t experts, int64_t rows, int64_t N, int64_t K, int64_t group, tg_dtype dtype, const void *A,
             int64_t lda, const void *packed, void *C, int64_t ldc, tg_dtype c_dtype, const int32_t *offsets,
             void *stream) {
    tg_status st = product_arguments(experts, rows, N, K, dtype, c_dtype, offsets);
    if (st != TG_OK) return st;
    Q4Shape shape;
    st = q4_arguments(experts, N, K, group, dtype, shape);
    if (st != TG_OK) return st;
    const int esz = size_of(dtype), csz = size_of(c_dtype);
    if (!operand_ok(A, rows, K, lda, esz) || !operand_ok(C, rows, N, ldc, csz)) return TG_ERR_INVALID_ARG;
    if (rows == 0 || N == 0) return TG_OK;
    if ((!packed && K > 0) || !aligned(packed, 16)) return TG_ERR_INVALID_ARG;
    const Range rc = span(C, 1, rows, N, ldc, 0, csz);
    if (overlaps(rc, span(A, 1, rows, K, lda, 0, esz)) || overlaps(rc, span(packed, 1, 1, shape.bytes, 0, 0, 1)) ||
        (offsets && overlaps(rc, span(offsets, 1, 1, experts + 1, 0, 0, 4))))
        return TG_ERR_INVALID_ARG;
    if (!tile_fits(lda, esz) || !tile_fits(ldc, csz) || K * esz >= (int64_t(1) << 30)) return TG_ERR_UNSUPPORTED;
    st = device_ok();
    if (st != TG_OK) return st;
    Q4Params p = {};
    p.A = static_cast<const char *>(A);
    p.codes = static_cast<const char *>(packed);
    p.scales = p.codes + shape.codes;
    p.C = static_cast<char *>(C);
    p.offsets = offsets;
    p.lda = lda;
    p.ldc = ldc;
    p.k_blocks = shape.k_blocks;
    p.groups = shape.groups;
    p.experts = (int)experts;
    p.rows = (int)rows;
    p.N = (int)N;
    p.K = (int)K;
    p.n_tiles = (int)shape.n_tiles;
    p.c_f32 = c_dtype == TG_F32;
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (dtype) {
        case TG_F32: return launch_q4<DT_F32>(p, (int)group, s);
        case TG_BF16: return launch_q4<DT_BF16>(p, (int)group, s);
        case TG_F16: return launch_q4<DT_F16>(p, (int)group, s);
    }
    return TG_ERR_INTERNAL;
}

tg_status answer(const ProductPlan &plan, bool past, tg_experts_plan_info *out) {
    if (!plan.fits()) return TG_ERR_UNSUPPORTED;
    *out = plan.info;
    out->past_caches = plan.info.kernel == TG_EXPERTS_TILES && past;
    return TG_OK;
}

tg_status grouped_plan(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, int transposed,
                       tg_dtype c_dtype, tg_experts_plan_info *out) {
    const tg_status st = product_sizes(experts, rows, N, K, dtype, c_dtype);
    if (st == TG_ERR_INVALID_ARG || (transposed != 0 && transposed != 1) || !out) return TG_ERR_INVALID_ARG;
    if (st != TG_OK) return st;
    *out = {};
    if (rows == 0 || N == 0) return TG_OK;
    const bool past = grouped_past(experts, rows, N, K, size_of(dtype), size_of(c_dtype));
    switch (dtype) {
        case TG_F32: return answer(plan_grouped<DT_F32>(transposed != 0, experts, rows, N, K), past, out);
        case TG_BF16: return answer(plan_grouped<DT_BF16>(transposed != 0, experts, rows, N, K), past, out);
        case TG_F16: return answer(plan_grouped<DT_F16>(transposed != 0, experts, rows, N, K), past, out);
    }
    return TG_ERR_INTERNAL;
}

tg_status wgrad_plan(int64_t experts, int64_t rows, int64_t M, int64_t N, tg_dtype dtype, tg_dtype c_dtype,
                     tg_experts_plan_info *out) {
    const tg_status st = product_sizes(experts, rows, N, M, dtype, c_dtype);
    if (st == TG_ERR_INVALID_ARG || !out) return TG_ERR_INVALID_ARG;
    if (st != TG_OK) return st;
    *out = {};
    if (M == 0 || N == 0) return TG_OK;
    const bool past = wgrad_past(experts, rows, M, N, size_of(dtype), size_of(c_dtype));
    switch (dtype) {
        case TG_F32: return answer(plan_wgrad<DT_F32>(experts, rows, M, N), past, out);
        case TG_BF16: return answer(plan_wgrad<DT_BF16>(experts, rows, M, N), past, out);
        case TG_F16: return answer(plan_wgrad<DT_F16>(experts, rows, M, N), past, out);
    }
    return TG_ERR_INTERNAL;
}

tg_status q4_plan(int64_t experts, int64_t rows, int64_t N, int64_t K, int64_t group, tg_dtype dtype, tg_dtype c_dtype,
                  tg_experts_plan_info *out) {
    tg_status st = product_sizes(experts, rows, N, K, dtype, c_dtype);
    if (st == TG_ERR_INVALID_ARG || !out) return TG_ERR_INVALID_ARG;
    if (st != TG_OK) return st;
    Q4Shape shape;
    st = q4_arguments(experts, N, K, group, dtype, shape);
    if (st != TG_OK) return st;
    *out = {};
    if (rows == 0 || N == 0) return TG_OK;
    switch (dtype) {
        case TG_F32: return answer(plan_q4<DT_F32>(experts, rows, N, K), false, out);
        case TG_BF16: return answer(plan_q4<DT_BF16>(experts, rows, N, K), false, out);
        case TG_F16: return answer(plan_q4<DT_F16>(experts, rows, N, K), false, out);
    }
    return TG_ERR_INTERNAL;
}

}  // namespace

// no exception leaves the library
#define TG_GUARD(call)            \
    try {                         \
        return call;              \
    } catch (...) {               \
        return TG_ERR_INTERNAL;   \
    }

extern "C" {

int tile_gemm_experts_version(void) { return TILE_GEMM_EXPERTS_VERSION; }

tg_status tile_gemm_expert_sort_workspace_size(int64_t tokens, int64_t top_k, int64_t experts, int64_t *bytes) {
    if (!bytes) return TG_ERR_INVALID_ARG;
    int64_t n = 0, b = 0;
    SortShape shape;
    const tg_status st = sort_arguments(tokens, top_k, experts, n, shape, b);
    if (st == TG_OK) *bytes = b;
    return st;
}

tg_status tile_gemm_expert_sort(int64_t tokens, int64_t top_k, int64_t experts, const int32_t *ids, int64_t ld_ids,
                                int32_t *offsets, int32_t *entry_of_row, int32_t *row_of_entry, void *workspace,
                                int64_t workspace_bytes, void *stream) {
    TG_GUARD(sort(tokens, top_k, experts, ids, ld_ids, offsets, entry_of_row, row_of_entry, workspace, workspace_bytes,
                  stream))
}

tg_status tile_gemm_expert_gather(int64_t tokens, int64_t top_k, int64_t cols, tg_dtype dtype, const void *x,
                                  int64_t ldx, const int32_t *row_of_entry, void *rows, int64_t ldr, void *stream) {
    TG_GUARD(gather(tokens, top_k, cols, dtype, x, ldx, row_of_entry, rows, ldr, stream))
}

tg_status tile_gemm_expert_combine(int64_t tokens, int64_t top_k, int64_t cols, tg_dtype dtype, const void *y,
                                   int64_t ldy, const int32_t *row_of_entry, const float *weights, int64_t ld_w,
                                   void *out, int64_t ldo, void *stream) {
    TG_GUARD(combine(tokens, top_k, cols, dtype, y, ldy, row_of_entry, weights, ld_w, out, ldo, stream))
}

tg_status tile_gemm_expert_combine_grad(int64_t tokens, int64_t top_k, int64_t cols, tg_dtype dtype,
                                        const void *d_out, int64_t ldo, const void *y, int64_t ldy,
                                        const int32_t *row_of_entry, const float *weights, int64_t ld_w, void *d_y,
                                        int64_t ldd, float *d_w, int64_t ld_dw, void *stream) {
    TG_GUARD(combine_grad(tokens, top_k, cols, dtype, d_out, ldo, y, ldy, row_of_entry, weights, ld_w, d_y, ldd, d_w,
                          ld_dw, stream))
}

tg_status tile_gemm_grouped(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, const void *A,
                            int64_t lda, const void *B, int64_t ldb, int64_t strideB, int transposed, void *C,
                            int64_t ldc, tg_dtype c_dtype, const int32_t *offsets, void *stream) {
    TG_GUARD(grouped(experts, rows, N, K, dtype, A, lda, B, ldb, strideB, transposed, C, ldc, c_dtype, offsets, stream))
}

tg_status tile_gemm_grouped_wgrad(int64_t experts, int64_t rows, int64_t M, int64_t N, tg_dtype dtype, const void *A,
                                  int64_t lda, const void *D, int64_t ldd, void *C, int64_t ldc, int64_t strideC,
                                  tg_dtype c_dtype, const int32_t *offsets, void *stream) {
    TG_GUARD(wgrad(experts, rows, M, N, dtype, A, lda, D, ldd, C, ldc, strideC, c_dtype, offsets, stream))
}

tg_status tile_gemm_q4_packed_size(int64_t experts, int64_t N, int64_t K, int64_t group, tg_dtype dtype,
                                   int64_t *bytes) {
    if (!bytes) return TG_ERR_INVALID_ARG;
    Q4Shape shape;
    const tg_status st = q4_arguments(experts, N, K, group, dtype, shape);
    if (st == TG_OK) *bytes = shape.bytes;
    return st;
}

tg_status tile_gemm_pack_q4(int64_t experts, int64_t N, int64_t K, int64_t group, tg_dtype dtype,
                            const uint8_t *codes, int64_t ld_codes, int64_t stride_codes, const void *scales,
                            int64_t ld_scales, int64_t stride_scales, void *packed, int64_t packed_bytes,
                            void *stream) {
    TG_GUARD(pack_q4(experts, N, K, group, dtype, codes, ld_codes, stride_codes, scales, ld_scales, stride_scales,
                     packed, packed_bytes, stream))
}

tg_status tile_gemm_q4(int64_t experts, int64_t rows, int64_t N, int64_t K, int64_t group, tg_dtype dtype,
                       const void *A, int64_t lda, const void *packed, void *C, int64_t ldc, tg_dtype c_dtype,
                       const int32_t *offsets, void *stream) {
    TG_GUARD(q4(experts, rows, N, K, group, dtype, A, lda, packed, C, ldc, c_dtype, offsets, stream))
}

tg_status tile_gemm_grouped_plan(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, int transposed,
                                 tg_dtype c_dtype, tg_experts_plan_info *out) {
    TG_GUARD(grouped_plan(experts, rows, N, K, dtype, transposed, c_dtype, out))
}

tg_status tile_gemm_grouped_wgrad_plan(int64_t experts, int64_t rows, int64_t M, int64_t N, tg_dtype dtype,
                                       tg_dtype c_dtype, tg_experts_plan_info *out) {
    TG_GUARD(wgrad_plan(experts, rows, M, N, dtype, c_dtype, out))
}

tg_status tile_gemm_q4_plan(int64_t experts, int64_t rows, int64_t N, int64_t K, int64_t group, tg_dtype dtype,
                            tg_dtype c_dtype, tg_experts_plan_info *out) {
    TG_GUARD(q4_plan(experts, rows, N, K, group, dtype, c_dtype, out))
}

}  // extern "C"
