"""Weights' gradients of an extent below 8: its waves share an expert's rows."""
import pytest
import torch

import tile_scheduled_dense_amd as tg
from tests import expert_ref as ref
from tests import test_gpu_experts as base
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("dt,experts,rows,spare,active,M,N,pad,skew", [
    ("bf16", 3, 700, 5, 2, 200, 3, 0, 0), ("f16", 2, 333, 0, 2, 7, 129, 1, 1), ("f32", 4, 1000, 1, 3, 5, 70, 2, 1),
    ("f32", 1, 129, 0, 1, 33, 4, 0, 0), ("bf16", 5, 60, 0, 1, 6, 7, 3, 0), ("f16", 1, 5000, 0, 1, 1, 1, 0, 0),
    ("bf16", 300, 900, 3, 100, 64, 1, 0, 1), ("f32", 2, 50, 50, 0, 7, 7, 0, 0), ("f16", 2, 4097, 0, 2, 2, 1000, 0, 0),
    ("bf16", 1, 0, 0, 0, 12, 5, 0, 0),
], ids=lambda v: str(v))
def test_values(dt, experts, rows, spare, active, M, N, pad, skew, out):
    if out == "f32" and dt == "f32":
        pytest.skip("the same case")
    o = dt if out == "same" else "f32"
    assert tg.tile_gemm_grouped_wgrad_plan(experts, rows + spare, M, N, dt, c_dtype=o)["kernel"] == "narrow"
    offsets = base.offsets_of(base.sizes_of(experts, rows, active, seed=rows))
    total = rows + spare
    A, D = base.normal(total, M, dtype=dt, seed=3), base.normal(total, N, dtype=dt, seed=4)
    A[offsets[-1]:] = float("nan")
    D[offsets[-1]:] = float("nan")
    want, absum = ref.wgrad(A, D, offsets)
    (Ad, lda), (Dd, ldd) = base.strided(A, pad, skew), base.strided(D, pad, skew)
    C = base.Out(M, N, ref.TYPES[o], pad, batch=experts, skew=skew)
    tg.tile_gemm_grouped_wgrad(experts, total, M, N, dt, Ad, lda, Dd, ldd, C.t, C.ld, C.stride,
                               torch.tensor(offsets, dtype=torch.int32).cuda(), c_dtype=o)
    ref.check(C.get().reshape(want.shape), want, rows, absum, o)


@pytest.mark.parametrize("M,N", [(3, 5), (2, 100), (64, 1)])
def test_many_rows_are_not_one_running_sum(M, N):
    """2^20 equal products: a workgroup has 1024 threads and gives 64 columns of the longer extent at most, so
    that rows go to 16 partial sums at least: 2^16 terms each, then 16, within 2 * (2^16 + 18) * 2^-24."""
    rows = 1 << 20
    A = torch.full((rows, M), 0.1, dtype=torch.bfloat16, device="cuda")
    D = torch.ones(rows, N, dtype=torch.bfloat16, device="cuda")
    C = torch.full((M, N), float("nan"), device="cuda")
    tg.tile_gemm_grouped_wgrad(1, rows, M, N, "bf16", A, M, D, N, C, N, M * N, None)
    want = rows * float(A[0, 0].double())
    assert float((C.double() - want).abs().max()) <= 2 * (2 ** 16 + 18) * 2.0 ** -24 * want
