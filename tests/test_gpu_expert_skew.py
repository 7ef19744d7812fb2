"""Products where one expert, or few, have the rows: the tables that a skewed router leaves."""
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


def splits(experts, rows):
    """Rows of each expert: all in the first, a middle, the last; one each and the rest in one; two neighbours."""
    for at in {0, experts // 2, experts - 1}:
        yield [rows * (g == at) for g in range(experts)]
    few = min(experts, rows)
    yield [(g < few) + (rows - few) * (g == experts // 3) for g in range(experts)]
    cut = rows // 3
    yield [cut * (g == experts // 2 - 1) + (rows - cut) * (g == experts // 2) for g in range(experts)]


@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("dt,experts,rows,spare,N,K", [
    ("f16", 64, 512, 0, 136, 264), ("bf16", 63, 99, 20, 136, 72), ("f32", 65, 300, 33, 72, 100), ("bf16", 2048, 4096, 17, 24, 40),
    ("f32", 130, 1000, 0, 40, 36), ("bf16", 2, 16, 15, 257, 65),
])
def test_streamed_products(dt, experts, rows, spare, N, K, transposed):
    total = rows + spare
    assert tg.tile_gemm_grouped_plan(experts, total, N, K, dt, c_dtype=dt, transposed=transposed)["kernel"] == "stream"
    A = base.normal(total, K, dtype=dt, seed=1)
    A[rows:] = float("nan")
    B = base.normal(experts, *((N, K) if transposed else (K, N)), dtype=dt, seed=2)
    Ad, Bd = A.cuda(), B.cuda()
    for sizes in splits(experts, rows):
        offsets = base.offsets_of(sizes)
        want, absum = ref.grouped(A, B, offsets, total, transposed)
        C = base.Out(total, N, ref.TYPES[dt])
        tg.tile_gemm_grouped(experts, total, N, K, dt, Ad, K, Bd, B.shape[2], N * K, C.t, N,
                             torch.tensor(offsets, dtype=torch.int32).cuda(), c_dtype=dt, transposed=transposed)
        ref.check(C.get(), want, K, absum, dt)
