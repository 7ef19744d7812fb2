"""T of tile_gemm_adapters without a column of y, on the GPU (t does not depend on N)."""
import pytest
import torch

from tests import ffn_ref as ref
from tests.gpu_util import need_gpu
from tests.test_gpu_ffn import AdapterCase

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("shuffled", [False, True])
@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("dt,adapters,rows,without,active,K,rank,pad", [
    ("bf16", 3, 1, 0, 1, 130, 8, 1), ("f16", 5, 40, 7, 4, 2050, 5, 1), ("f32", 41, 700, 21, 37, 264, 12, 8),
    ("bf16", 2, 900, 0, 2, 4104, 300, 1), ("bf16", 2, 20, 0, 2, 0, 8, 1), ("f32", 2, 20, 20, 0, 64, 3, 1)], ids=lambda v: str(v))
def test_t_without_a_column(dt, adapters, rows, without, active, K, rank, pad, transposed, shuffled):
    for exact in (True, False):
        c = AdapterCase(dt, adapters, rows, without, active, 0, K, rank, pad, 0, transposed, shuffled, exact)
        y, t = c.run()
        assert y.numel() == 0
        _, _, want, err = ref.adapters(c.x, c.w, c.a, c.b, c.scales, c.offsets, c.order, transposed, dt)
        if exact:
            assert float(want.abs().max()) <= 256
            assert torch.equal(t.double(), want)
        else:
            ref.check(t, want, err, dt, "t")
