// ffn.hip -- the C ABI of the operators of a feed-forward block: argument checks and
// launches on the caller's stream.  Declarations and contracts are in
// include/tile_gemm_ffn.h.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ffn.hpp"
#include "ffn_plan.hpp"
#include "tile_gemm_experts.h"
#include "tile_gemm_ffn.h"

using namespace tg;

namespace {

constexpr int64_t kMaxExtent = int64_t(1) << 30;

bool known(tg_dtype t) { return t == TG_F32 || t == TG_BF16 || t == TG_F16; }
int size_of(tg_dtype t) { return t == TG_F32 ? 4 : 2; }
bool aligned(const void *p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// rows x cols at row stride ld
bool operand_ok(const void *p, int64_t rows, int64_t cols, int64_t ld, int esz) {
    return ld >= (cols > 1 ? cols : 1) && aligned(p, esz) && (p || rows == 0 || cols == 0);
}
// A block's tile of an operand is addressed in 31 bits from its first element (as in the
// products of experts.hip).
bool tile_fits(int64_t ld, int esz) { return ld <= kMaxExtent && (256 * ld + 4096) * esz < (int64_t(1) << 31) - 65536; }

// No output overlaps another or an input; the first two are not compared with each other
// where they may lie side by side.
bool none_overlap(const Range *out, int outs, const Range *in, int ins, bool first_two = true) {
    for (int i = 0; i < outs; ++i) {
        for (int j = 0; j < i; ++j)
            if ((i > 1 || first_two) && overlaps(out[i], out[j])) return false;
        for (int j = 0; j < ins; ++j)
            if (overlaps(out[i], in[j])) return false;
    }
    return true;
}

// Whether two rows x cols matrices at the same row stride have no element in common: apart,
// or side by side in the same rows.
bool side_by_side(const void *a, const void *b, int64_t rows, int64_t cols, int64_t ld, int esz) {
    const Range x = span(a, 1, rows, cols, ld, 0, esz), y = span(b, 1, rows, cols, ld, 0, esz);
    if (!overlaps(x, y)) return true;
    const int64_t d = static_cast<int64_t>(x.lo < y.lo ? y.lo - x.lo : x.lo - y.lo), in = d % (ld * esz);
    return in >= cols * esz && in + cols * esz <= ld * esz;
}
tg_status sizes(int64_t groups, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, int transposed) {
    if (groups < 1 || rows < 0 || N < 0 || K < 0 || !known(dtype) || (transposed != 0 && transposed != 1))
        return TG_ERR_INVALID_ARG;
    if (groups > TILE_GEMM_MAX_EXPERTS || rows > kMaxExtent || N > kMaxExtent || K > kMaxExtent) return TG_ERR_UNSUPPORTED;
    return TG_OK;
}

bool no_device() {
    int n = 0;
    if (hipGetDeviceCount(&n) == hipSuccess && n > 0) return false;
    (void)hipGetLastError();
    return true;
}

Range table(const int32_t *p, int64_t n) { return p ? span(p, 1, 1, n, 0, 0, 4) : Range{0, 0}; }

bool past_caches(int64_t bytes) { return bytes > (int64_t(256) << 20); }

tg_status answer(const ProductPlan &plan, int splits, tg_ffn_plan_info *out) {
    if (!plan.fits()) return TG_ERR_UNSUPPORTED;
    *out = {};
    out->kernel = plan.info.kernel == TG_EXPERTS_STREAM ? TG_FFN_STREAM : TG_FFN_TILES;
    out->tile_m = plan.info.tile_m;
    out->tile_n = plan.info.tile_n;
    out->pieces = plan.info.pieces;
    out->pipeline = plan.info.pipeline;
    out->waves = plan.info.waves;
    out->splits = splits < 1 ? 1 : splits;
    out->workgroups = plan.info.workgroups;
    return TG_OK;
}

// ---- the gated pair -------------------------------------------------------------------------
GatedPlan gated_plan_of(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, int transposed) {
    const bool t = transposed != 0;
    return dtype == TG_F32    ? plan_gated<DT_F32>(t, experts, rows, N, K)
           : dtype == TG_BF16 ? plan_gated<DT_BF16>(t, experts, rows, N, K)
                              : plan_gated<DT_F16>(t, experts, rows, N, K);
}
tg_status gated_bytes(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, int transposed, int64_t *bytes) {
    const tg_status st = sizes(experts, rows, N, K, dtype, transposed);
    if (st != TG_OK) return st;
    *bytes = rows == 0 || N == 0 ? 0 : gated_workspace(gated_plan_of(experts, rows, N, K, dtype, transposed), rows, N);
    return *bytes < kNoMemory ? TG_OK : TG_ERR_UNSUPPORTED;
}
tg_status gated_plan(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, int transposed, bool grad,
                     tg_ffn_plan_info *out) {
    const tg_status st = sizes(experts, rows, N, K, dtype, transposed);
    if (st == TG_ERR_INVALID_ARG || !out) return TG_ERR_INVALID_ARG;
    if (st != TG_OK) return st;
    *out = {};
    if (rows == 0 || N == 0) return TG_OK;
    if (grad) {
        const bool t = transposed != 0;
        return answer(dtype == TG_F32    ? plan_gate_grad<DT_F32>(t, experts, rows, N, K)
                      : dtype == TG_BF16 ? plan_gate_grad<DT_BF16>(t, experts, rows, N, K)
                                         : plan_gate_grad<DT_F16>(t, experts, rows, N, K), 1, out);
    }
    const GatedPlan plan = gated_plan_of(experts, rows, N, K, dtype, transposed);
    return answer(plan.product, plan.splits, out);
}

tg_status gated(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, const void *A, int64_t lda,
                const void *B, const void *B_up, int64_t ldb, int64_t strideB, int transposed, int activation, void *H,
                int64_t ldh, void *U, void *V, int64_t ldu, const int32_t *offsets, void *workspace,
                int64_t workspace_bytes, void *stream) {
    tg_status st = sizes(experts, rows, N, K, dtype, transposed);
    if (st == TG_ERR_INVALID_ARG || activation < 0 || activation >= GATE_COUNT || (!offsets && experts != 1) ||
        !aligned(offsets, 4) || strideB < 0 || (U == nullptr) != (V == nullptr))
        return TG_ERR_INVALID_ARG;
    if (st != TG_OK) return st;
    const int esz = size_of(dtype);
    const int64_t b_rows = transposed ? N : K, b_cols = transposed ? K : N;
    if (!operand_ok(A, rows, K, lda, esz) || !operand_ok(B, rows > 0 ? b_rows : 0, b_cols, ldb, esz) ||
        !operand_ok(B_up, rows > 0 ? b_rows : 0, b_cols, ldb, esz) || !operand_ok(H, rows, N, ldh, esz) ||
        (U && (!operand_ok(U, rows, N, ldu, esz) || !operand_ok(V, rows, N, ldu, esz))) || !aligned(workspace, 16) ||
        workspace_bytes < 0)
        return TG_ERR_INVALID_ARG;
    if (rows == 0 || N == 0) return TG_OK;
    int64_t bytes = 0;
    st = gated_bytes(experts, rows, N, K, dtype, transposed, &bytes);
    if (st != TG_OK) return st;
    const bool use = workspace && bytes > 0 && workspace_bytes >= bytes;
    const Range out[4] = {U ? span(U, 1, rows, N, ldu, 0, esz) : Range{0, 0},
                          U ? span(V, 1, rows, N, ldu, 0, esz) : Range{0, 0}, span(H, 1, rows, N, ldh, 0, esz),
                          use ? span(workspace, 1, 1, bytes, 0, 0, 1) : Range{0, 0}};
    const Range in[4] = {span(A, 1, rows, K, lda, 0, esz), span(B, experts, b_rows, b_cols, ldb, strideB, esz),
                         span(B_up, experts, b_rows, b_cols, ldb, strideB, esz), table(offsets, experts + 1)};
    if (!none_overlap(out, 4, in, 4, false) || (U && !side_by_side(U, V, rows, N, ldu, esz))) return TG_ERR_INVALID_ARG;
    if (!tile_fits(lda, esz) || !tile_fits(ldb, esz) || !tile_fits(ldh, esz) || (U && !tile_fits(ldu, esz)))
        return TG_ERR_UNSUPPORTED;
    st = device_ok();
    if (st != TG_OK) return st;
    GatedParams p = {};
    p.A = static_cast<const char *>(A);
    p.B = static_cast<const char *>(B);
    p.Bu = static_cast<const char *>(B_up);
    p.C = static_cast<char *>(H);
    p.U = static_cast<char *>(U);
    p.V = static_cast<char *>(V);
    p.offsets = offsets;
    p.lda = lda;
    p.ldb = ldb;
    p.ldc = ldh;
    p.ldu = ldu;
    p.sB = strideB;
    p.experts = (int)experts;
    p.rows = (int)rows;
    p.N = (int)N;
    p.K = (int)K;
    p.act = activation;
    p.past = past_caches((rows * K + 2 * experts * N * K + rows * N * (U ? 3 : 1)) * esz);
    hipStream_t s = static_cast<hipStream_t>(stream);
    void *ws = use ? workspace : nullptr;
    switch (dtype) {
        case TG_F32: return launch_gated<DT_F32>(p, transposed != 0, ws, s);
        case TG_BF16: return launch_gated<DT_BF16>(p, transposed != 0, ws, s);
        case TG_F16: return launch_gated<DT_F16>(p, transposed != 0, ws, s);
    }
    return TG_ERR_INTERNAL;
}

tg_status gated_grad(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, const void *D, int64_t ldd,
                     const void *B, int64_t ldb, int64_t strideB, int transposed, int activation, const void *U,
                     const void *V, int64_t ldu, void *dU, void *dV, int64_t lddu, void *H, int64_t ldh,
                     const int32_t *offsets, void *stream) {
    tg_status st = sizes(experts, rows, N, K, dtype, transposed);
    if (st == TG_ERR_INVALID_ARG || activation < 0 || activation >= GATE_COUNT || (!offsets && experts != 1) ||
        !aligned(offsets, 4) || strideB < 0)
        return TG_ERR_INVALID_ARG;
    if (st != TG_OK) return st;
    const int esz = size_of(dtype);
    const int64_t b_rows = transposed ? N : K, b_cols = transposed ? K : N;
    if (!operand_ok(D, rows, K, ldd, esz) || !operand_ok(B, rows > 0 ? b_rows : 0, b_cols, ldb, esz) ||
        !operand_ok(U, rows, N, ldu, esz) || !operand_ok(V, rows, N, ldu, esz) || !operand_ok(dU, rows, N, lddu, esz) ||
        !operand_ok(dV, rows, N, lddu, esz) || (H && !operand_ok(H, rows, N, ldh, esz)))
        return TG_ERR_INVALID_ARG;
    if (rows == 0 || N == 0) return TG_OK;
    const Range out[3] = {span(dU, 1, rows, N, lddu, 0, esz), span(dV, 1, rows, N, lddu, 0, esz),
                          H ? span(H, 1, rows, N, ldh, 0, esz) : Range{0, 0}};
    const Range in[5] = {span(D, 1, rows, K, ldd, 0, esz), span(B, experts, b_rows, b_cols, ldb, strideB, esz),
                         span(U, 1, rows, N, ldu, 0, esz), span(V, 1, rows, N, ldu, 0, esz), table(offsets, experts + 1)};
    if (!none_overlap(out, 3, in, 5, false) || !side_by_side(dU, dV, rows, N, lddu, esz)) return TG_ERR_INVALID_ARG;
    if (!tile_fits(ldd, esz) || !tile_fits(ldb, esz) || !tile_fits(ldu, esz) || !tile_fits(lddu, esz) ||
        (H && !tile_fits(ldh, esz)))
        return TG_ERR_UNSUPPORTED;
    st = device_ok();
    if (st != TG_OK) return st;
    GatedParams p = {};
    p.A = static_cast<const char *>(D);
    p.B = static_cast<const char *>(B);
    p.U = const_cast<char *>(static_cast<const char *>(U));
    p.V = const_cast<char *>(static_cast<const char *>(V));
    p.dU = static_cast<char *>(dU);
    p.dV = static_cast<char *>(dV);
    p.C = static_cast<char *>(H);
    p.offsets = offsets;
    p.lda = ldd;
    p.ldb = ldb;
    p.ldc = ldh;
    p.ldu = ldu;
    p.lddu = lddu;
    p.sB = strideB;
    p.experts = (int)experts;
    p.rows = (int)rows;
    p.N = (int)N;
    p.K = (int)K;
    p.act = activation;
    p.past = past_caches((rows * K + experts * N * K + rows * N * (H ? 5 : 4)) * esz);
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (dtype) {
        case TG_F32: return launch_gate_grad<DT_F32>(p, transposed != 0, s);
        case TG_BF16: return launch_gate_grad<DT_BF16>(p, transposed != 0, s);
        case TG_F16: return launch_gate_grad<DT_F16>(p, transposed != 0, s);
    }
    return TG_ERR_INTERNAL;
}

// grad: D, dU, dV are there, and H may be NULL
tg_status gate(bool grad, int64_t rows, int64_t N, tg_dtype dtype, int activation, const void *D, int64_t ldd, const void *U,
               const void *V, int64_t ldu, void *dU, void *dV, int64_t lddu, void *H, int64_t ldh, void *stream) {
    tg_status st = sizes(1, rows, N, 0, dtype, 0);
    if (st == TG_ERR_INVALID_ARG || activation < 0 || activation >= GATE_COUNT) return TG_ERR_INVALID_ARG;
    if (st != TG_OK) return st;
    const int esz = size_of(dtype);
    if (!operand_ok(U, rows, N, ldu, esz) || !operand_ok(V, rows, N, ldu, esz) ||
        ((!grad || H) && !operand_ok(H, rows, N, ldh, esz)) ||
        (grad && (!operand_ok(D, rows, N, ldd, esz) || !operand_ok(dU, rows, N, lddu, esz) || !operand_ok(dV, rows, N, lddu, esz))))
        return TG_ERR_INVALID_ARG;
    if (rows == 0 || N == 0) return TG_OK;
    auto range = [&](const void *p, int64_t ld) { return p ? span(p, 1, rows, N, ld, 0, esz) : Range{0, 0}; };
    const Range out[3] = {range(dU, lddu), range(dV, lddu), range(H, ldh)};
    const Range in[3] = {range(D, ldd), range(U, ldu), range(V, ldu)};
    if (!none_overlap(out, 3, in, 3, false) || (grad && !side_by_side(dU, dV, rows, N, lddu, esz))) return TG_ERR_INVALID_ARG;
    if (!tile_fits(ldu, esz) || (grad && (!tile_fits(ldd, esz) || !tile_fits(lddu, esz))) || (H && !tile_fits(ldh, esz)))
        return TG_ERR_UNSUPPORTED;
    st = device_ok();
    if (st != TG_OK) return st;
    GatedParams p = {};
    p.A = static_cast<const char *>(D);
    p.U = const_cast<char *>(static_cast<const char *>(U));
    p.V = const_cast<char *>(static_cast<const char *>(V));
    p.dU = static_cast<char *>(dU);
    p.dV = static_cast<char *>(dV);
    p.C = static_cast<char *>(H);
    p.lda = ldd;
    p.ldu = ldu;
    p.lddu = lddu;
    p.ldc = ldh;
    p.rows = (int)rows;
    p.N = (int)N;
    p.act = activation;
    p.past = past_caches(rows * N * (grad ? (H ? 6 : 5) : 3) * esz);
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (dtype) {
        case TG_F32: return launch_gate<DT_F32>(p, grad, s);
        case TG_BF16: return launch_gate<DT_BF16>(p, grad, s);
        case TG_F16: return launch_gate<DT_F16>(p, grad, s);
    }
    return TG_ERR_INTERNAL;
}

// ---- adapters ---------------------------------------------------------------------------------
// with_t: t is computed, where N is 0 too
tg_status adapter_plan(int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank, tg_dtype dtype, int transposed,
                       bool with_t, AdapterPlan &plan) {
    const tg_status st = sizes(adapters, rows, N, K, dtype, transposed);
    if (st == TG_ERR_INVALID_ARG || rank < 0) return TG_ERR_INVALID_ARG;
    if (st != TG_OK) return st;
    if (rank > kMaxExtent) return TG_ERR_UNSUPPORTED;
    plan = {};
    if (rows == 0 || (N == 0 && !with_t)) return TG_OK;
    const bool t = transposed != 0;
    plan = dtype == TG_F32    ? plan_adapters<DT_F32>(t, adapters, rows, N, K, rank)
           : dtype == TG_BF16 ? plan_adapters<DT_BF16>(t, adapters, rows, N, K, rank)
                              : plan_adapters<DT_F16>(t, adapters, rows, N, K, rank);
    return plan.bytes < kNoMemory ? TG_OK : TG_ERR_UNSUPPORTED;
}

tg_status adapters(int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank, tg_dtype dtype, const void *X,
                   int64_t ldx, const void *W, int64_t ldw, const void *A, int64_t lda, int64_t strideA, const void *B,
                   int64_t ldb, int64_t strideB, int transposed, const float *scales, void *Y, int64_t ldy, void *T,
                   int64_t ldt, const int32_t *offsets, const int32_t *order, void *workspace, int64_t workspace_bytes,
                   void *stream) {
    AdapterPlan plan;
    tg_status st = adapter_plan(adapters, rows, N, K, rank, dtype, transposed, T != nullptr, plan);
    if (st != TG_OK) return st;
    const int esz = size_of(dtype);
    const int64_t any = rows > 0;
    auto stored = [&](const void *p, int64_t inputs, int64_t outputs, int64_t ld) {
        return transposed ? operand_ok(p, any * outputs, inputs, ld, esz) : operand_ok(p, any * inputs, outputs, ld, esz);
    };
    if (!operand_ok(X, rows, K, ldx, esz) || !stored(W, K, N, ldw) || !stored(A, K, rank, lda) || !stored(B, rank, N, ldb) ||
        !operand_ok(Y, rows, N, ldy, esz) || (T && !operand_ok(T, rows, rank, ldt, esz)) || strideA < 0 || strideB < 0 ||
        !aligned(scales, 4) || !aligned(offsets, 4) || !aligned(order, 4) || !aligned(workspace, 16))
        return TG_ERR_INVALID_ARG;
    // t does not depend on N
    if (rows == 0 || (N == 0 && (!T || rank == 0))) return TG_OK;
    if (!offsets || (plan.bytes > 0 && (!workspace || workspace_bytes < plan.bytes))) return TG_ERR_INVALID_ARG;
    auto range = [&](const void *p, int64_t n, int64_t inputs, int64_t outputs, int64_t ld, int64_t stride) {
        return transposed ? span(p, n, outputs, inputs, ld, stride, esz) : span(p, n, inputs, outputs, ld, stride, esz);
    };
    const Range out[3] = {span(Y, 1, rows, N, ldy, 0, esz), T ? span(T, 1, rows, rank, ldt, 0, esz) : Range{0, 0},
                          span(workspace, 1, plan.bytes > 0, plan.bytes, 0, 0, 1)};
    const Range in[7] = {span(X, 1, rows, K, ldx, 0, esz), range(W, 1, K, N, ldw, 0), range(A, adapters, K, rank, lda, strideA),
                         range(B, adapters, rank, N, ldb, strideB), table(offsets, adapters + 1), table(order, rows),
                         scales ? span(scales, 1, 1, adapters, 0, 0, 4) : Range{0, 0}};
    if (!none_overlap(out, 3, in, 7)) return TG_ERR_INVALID_ARG;
    if (!tile_fits(ldx, esz) || !tile_fits(ldw, esz) || !tile_fits(lda, esz) || !tile_fits(ldb, esz) || !tile_fits(ldy, esz) ||
        !tile_fits(rank, esz) || (T && !tile_fits(ldt, esz)))
        return TG_ERR_UNSUPPORTED;
    if (order && plan.form == ADAPTERS_TILES && rows * ldx * esz >= (int64_t(1) << 31) - 65536) return TG_ERR_UNSUPPORTED;
    if (N == 0 && no_device()) return TG_OK;       // y is empty, and no device holds a T
    st = device_ok();
    if (st != TG_OK) return st;
    AdapterParams p = {};
    p.A = static_cast<const char *>(X);
    p.B = static_cast<const char *>(W);
    p.C = static_cast<char *>(Y);
    p.T = static_cast<char *>(T);
    p.down = static_cast<const char *>(A);
    p.up = static_cast<const char *>(B);
    p.scales = scales;
    p.offsets = offsets;
    p.order = order;
    p.lda = ldx;
    p.ldb = ldw;
    p.ldc = ldy;
    p.ldt = ldt;
    p.ld_down = lda;
    p.s_down = strideA;
    p.ld_up = ldb;
    p.s_up = strideB;
    p.experts = (int)adapters;
    p.rows = (int)rows;
    p.N = (int)N;
    p.K = (int)K;
    p.rank = (int)rank;
    p.past = past_caches((rows * K + N * K + rows * N) * esz);
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (dtype) {
        case TG_F32: return launch_adapters<DT_F32>(p, transposed != 0, workspace, s);
        case TG_BF16: return launch_adapters<DT_BF16>(p, transposed != 0, workspace, s);
        case TG_F16: return launch_adapters<DT_F16>(p, transposed != 0, workspace, s);
    }
    return TG_ERR_INTERNAL;
}

tg_status adapters_plan(int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank, tg_dtype dtype, int transposed,
                        tg_ffn_plan_info *out) {
    AdapterPlan plan;
    const tg_status st = adapter_plan(adapters, rows, N, K, rank, dtype, transposed, false, plan);
    if (st == TG_ERR_INVALID_ARG || !out) return TG_ERR_INVALID_ARG;
    if (st != TG_OK) return st;
    *out = {};
    return rows == 0 || N == 0 ? TG_OK : answer(plan.product, plan.splits, out);
}

tg_status wgrad_plan(int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank, tg_dtype dtype,
                     AdapterGradPlan &plan) {
    const tg_status st = sizes(adapters, rows, N, K, dtype, 0);
    if (st == TG_ERR_INVALID_ARG || rank < 0) return TG_ERR_INVALID_ARG;
    if (st != TG_OK) return st;
    if (rank > kMaxExtent) return TG_ERR_UNSUPPORTED;
    plan = plan_adapters_wgrad(adapters, rows, N, K, rank, dtype == TG_F32);
    return plan.bytes < kNoMemory ? TG_OK : TG_ERR_UNSUPPORTED;
}

tg_status adapters_wgrad(int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank, tg_dtype dtype, const void *X,
                         int64_t ldx, const void *dY, int64_t ldy, const void *T, int64_t ldt, const void *dT, int64_t lddt,
                         void *dA, int64_t lda, int64_t strideA, void *dB, int64_t ldb, int64_t strideB, int transposed,
                         tg_dtype c_dtype, const int32_t *offsets, const int32_t *order, void *workspace,
                         int64_t workspace_bytes, void *stream) {
    AdapterGradPlan plan;
    tg_status st = wgrad_plan(adapters, rows, N, K, rank, dtype, plan);
    if (st == TG_ERR_INVALID_ARG || (transposed != 0 && transposed != 1) || (c_dtype != TG_F32 && c_dtype != dtype))
        return TG_ERR_INVALID_ARG;
    if (st != TG_OK) return st;
    const int esz = size_of(dtype), csz = size_of(c_dtype);
    const int64_t a_rows = transposed ? rank : K, a_cols = transposed ? K : rank, b_rows = transposed ? N : rank,
                  b_cols = transposed ? rank : N;
    if (!operand_ok(X, rows, K, ldx, esz) || !operand_ok(dY, rows, N, ldy, esz) || !operand_ok(T, rows, rank, ldt, esz) ||
        !operand_ok(dT, rows, rank, lddt, esz) || !operand_ok(dA, a_rows, a_cols, lda, csz) ||
        !operand_ok(dB, b_rows, b_cols, ldb, csz) || strideA < 0 || strideB < 0 || !aligned(offsets, 4) ||
        !aligned(order, 4) || !aligned(workspace, 16) ||
        (adapters > 1 && rank > 0 && ((K > 0 && strideA < (a_rows - 1) * lda + a_cols) ||
                                      (N > 0 && strideB < (b_rows - 1) * ldb + b_cols))))
        return TG_ERR_INVALID_ARG;
    if (rank == 0 || (N == 0 && K == 0)) return TG_OK;
    if (!offsets || (plan.bytes > 0 && (!workspace || workspace_bytes < plan.bytes))) return TG_ERR_INVALID_ARG;
    const Range out[3] = {span(dA, adapters, a_rows, a_cols, lda, strideA, csz),
                          span(dB, adapters, b_rows, b_cols, ldb, strideB, csz),
                          span(workspace, 1, plan.bytes > 0, plan.bytes, 0, 0, 1)};
    const Range in[6] = {span(X, 1, rows, K, ldx, 0, esz), span(dY, 1, rows, N, ldy, 0, esz),
                         span(T, 1, rows, rank, ldt, 0, esz), span(dT, 1, rows, rank, lddt, 0, esz),
                         table(offsets, adapters + 1), table(order, rows)};
    if (!none_overlap(out, 3, in, 6)) return TG_ERR_INVALID_ARG;
    st = device_ok();
    if (st != TG_OK) return st;
    AdapterGradParams p = {};
    p.L[0] = static_cast<const char *>(X);
    p.S[0] = static_cast<const char *>(dT);
    p.C[0] = static_cast<char *>(dA);
    p.ldl[0] = ldx;
    p.lds[0] = lddt;
    p.ldc[0] = lda;
    p.sC[0] = strideA;
    p.M[0] = (int)K;
    p.wide_first[0] = !transposed;
    p.L[1] = static_cast<const char *>(dY);
    p.S[1] = static_cast<const char *>(T);
    p.C[1] = static_cast<char *>(dB);
    p.ldl[1] = ldy;
    p.lds[1] = ldt;
    p.ldc[1] = ldb;
    p.sC[1] = strideB;
    p.M[1] = (int)N;
    p.wide_first[1] = transposed;
    p.offsets = offsets;
    p.order = order;
    p.adapters = (int)adapters;
    p.rows = (int)rows;
    p.rank = (int)rank;
    p.c_f32 = c_dtype == TG_F32;
    hipStream_t s = static_cast<hipStream_t>(stream);
    switch (dtype) {
        case TG_F32: return launch_adapters_wgrad<DT_F32>(p, workspace, s);
        case TG_BF16: return launch_adapters_wgrad<DT_BF16>(p, workspace, s);
        case TG_F16: return launch_adapters_wgrad<DT_F16>(p, workspace, s);
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

int tile_gemm_ffn_version(void) { return TILE_GEMM_FFN_VERSION; }

tg_status tile_gemm_gated_workspace_size(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype,
                                         int transposed, int64_t *bytes) {
    if (!bytes) return TG_ERR_INVALID_ARG;
    return gated_bytes(experts, rows, N, K, dtype, transposed, bytes);
}

tg_status tile_gemm_gated(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, const void *A,
                          int64_t lda, const void *B, const void *B_up, int64_t ldb, int64_t strideB, int transposed,
                          int activation, void *H, int64_t ldh, void *U, void *V, int64_t ldu, const int32_t *offsets,
                          void *workspace, int64_t workspace_bytes, void *stream) {
    TG_GUARD(gated(experts, rows, N, K, dtype, A, lda, B, B_up, ldb, strideB, transposed, activation, H, ldh, U, V, ldu,
                   offsets, workspace, workspace_bytes, stream))
}

tg_status tile_gemm_gated_grad(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, const void *D,
                               int64_t ldd, const void *B, int64_t ldb, int64_t strideB, int transposed,
                               int activation, const void *U, const void *V, int64_t ldu, void *dU, void *dV,
                               int64_t lddu, void *H, int64_t ldh, const int32_t *offsets, void *stream) {
    TG_GUARD(gated_grad(experts, rows, N, K, dtype, D, ldd, B, ldb, strideB, transposed, activation, U, V, ldu, dU, dV,
                        lddu, H, ldh, offsets, stream))
}

tg_status tile_gemm_gate(int64_t rows, int64_t N, tg_dtype dtype, int activation, const void *U, const void *V,
                         int64_t ldu, void *H, int64_t ldh, void *stream) {
    TG_GUARD(gate(false, rows, N, dtype, activation, nullptr, 0, U, V, ldu, nullptr, nullptr, 0, H, ldh, stream))
}

tg_status tile_gemm_gate_grad(int64_t rows, int64_t N, tg_dtype dtype, int activation, const void *D, int64_t ldd,
                              const void *U, const void *V, int64_t ldu, void *dU, void *dV, int64_t lddu, void *H,
                              int64_t ldh, void *stream) {
    TG_GUARD(gate(true, rows, N, dtype, activation, D, ldd, U, V, ldu, dU, dV, lddu, H, ldh, stream))
}

tg_status tile_gemm_adapters_workspace_size(int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank,
                                            tg_dtype dtype, int transposed, int64_t *bytes) {
    if (!bytes) return TG_ERR_INVALID_ARG;
    AdapterPlan plan;
    const tg_status st = adapter_plan(adapters, rows, N, K, rank, dtype, transposed, true, plan);
    if (st == TG_OK) *bytes = plan.bytes;
    return st;
}

tg_status tile_gemm_adapters(int64_t n_adapters, int64_t rows, int64_t N, int64_t K, int64_t rank, tg_dtype dtype,
                             const void *X, int64_t ldx, const void *W, int64_t ldw, const void *A, int64_t lda,
                             int64_t strideA, const void *B, int64_t ldb, int64_t strideB, int transposed,
                             const float *scales, void *Y, int64_t ldy, void *T, int64_t ldt, const int32_t *offsets,
                             const int32_t *order, void *workspace, int64_t workspace_bytes, void *stream) {
    TG_GUARD(adapters(n_adapters, rows, N, K, rank, dtype, X, ldx, W, ldw, A, lda, strideA, B, ldb, strideB, transposed,
                      scales, Y, ldy, T, ldt, offsets, order, workspace, workspace_bytes, stream))
}

tg_status tile_gemm_adapters_wgrad_workspace_size(int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank,
                                                  tg_dtype dtype, int64_t *bytes) {
    if (!bytes) return TG_ERR_INVALID_ARG;
    AdapterGradPlan plan;
    const tg_status st = wgrad_plan(adapters, rows, N, K, rank, dtype, plan);
    if (st == TG_OK) *bytes = plan.bytes;
    return st;
}

tg_status tile_gemm_adapters_wgrad(int64_t n_adapters, int64_t rows, int64_t N, int64_t K, int64_t rank, tg_dtype dtype,
                                   const void *X, int64_t ldx, const void *dY, int64_t ldy, const void *T, int64_t ldt,
                                   const void *dT, int64_t lddt, void *dA, int64_t lda, int64_t strideA, void *dB,
                                   int64_t ldb, int64_t strideB, int transposed, tg_dtype c_dtype,
                                   const int32_t *offsets, const int32_t *order, void *workspace,
                                   int64_t workspace_bytes, void *stream) {
    TG_GUARD(adapters_wgrad(n_adapters, rows, N, K, rank, dtype, X, ldx, dY, ldy, T, ldt, dT, lddt, dA, lda, strideA, dB,
                            ldb, strideB, transposed, c_dtype, offsets, order, workspace, workspace_bytes, stream))
}

tg_status tile_gemm_gated_plan(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, int transposed,
                               tg_ffn_plan_info *out) {
    TG_GUARD(gated_plan(experts, rows, N, K, dtype, transposed, false, out))
}

tg_status tile_gemm_gated_grad_plan(int64_t experts, int64_t rows, int64_t N, int64_t K, tg_dtype dtype, int transposed,
                                    tg_ffn_plan_info *out) {
    TG_GUARD(gated_plan(experts, rows, N, K, dtype, transposed, true, out))
}

tg_status tile_gemm_adapters_plan(int64_t adapters, int64_t rows, int64_t N, int64_t K, int64_t rank, tg_dtype dtype,
                                  int transposed, tg_ffn_plan_info *out) {
    TG_GUARD(adapters_plan(adapters, rows, N, K, rank, dtype, transposed, out))
}

}  // extern "C"
