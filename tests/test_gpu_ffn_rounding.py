"""y of rows beside a broken adapter is rounded once, on the GPU.

A tile of rows of several adapters leaves an adapter's infinities out of the product and adds them
to its own rows afterwards.  The other columns of those rows are x . W + t . B[g] in fp32 and rounded once: here
sums halfway between two neighbours of 16 bits, which x . W rounded by itself, and then the sum, miss.
"""
import pytest
import torch

import tile_scheduled_dense_amd as tg
from tests.gpu_util import need_gpu
from tests.test_gpu_ffn import AdapterCase, ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("what", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("shuffled", [False, True])
@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("dt,large", [("bf16", 256.0), ("f16", 2048.0)])
def test_rows_of_a_broken_adapter_are_rounded_once(dt, large, transposed, shuffled, what):
    rows, N, K, rank = 700, 136, 64, 4
    plan = tg.tile_gemm_adapters_plan(2, rows, N, K, rank, dt, transposed)
    assert plan["kernel"] == "tiles" and plan["tile_m"] == 128 and plan["splits"] == 1
    c = AdapterCase(dt, 2, rows, 0, 2, N, K, rank, 0, 0, transposed, shuffled, True, scaled=False)
    for m in (c.x, c.w, c.a, c.b):
        m.zero_()
    c.x[:, :2] = 1
    w, a, b = ((m.transpose(-1, -2) if transposed else m) for m in (c.w, c.a, c.b))
    w[0], w[1] = large, 1          # x . W = large + 1, halfway, rounded to large
    a[:, 0, 0] = 1                 # t = (1, 0, 0, 0)
    b[:, 0] = 2                    # y = large + 3, halfway, rounded to large + 4
    b[1, 0, 5] = what
    y, t = c.run()
    exact = torch.tensor(large + 3, dtype=torch.float64).to(y.dtype)
    assert float(exact) == large + 4
    own = torch.zeros(rows, dtype=torch.bool)
    own[ref.group_rows(c.offsets, 1, c.order)] = True
    assert 0 < int(own.sum()) < rows and c.offsets[1] % 128 != 0         # a tile has rows of both
    keep = torch.arange(N) != 5
    assert torch.equal(y[:, keep], exact.expand(rows, N - 1))
    assert torch.equal(y[~own, 5], exact.expand(int((~own).sum())))
    got = y[own, 5].float()
    assert bool(torch.isnan(got).all() if what != what else (got == what).all())
    assert torch.equal(t[:, 0].float(), torch.ones(rows))


@pytest.mark.parametrize("rows", [50, 700])
@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_zero_times_infinity_without_inputs(dt, rows, transposed):
    """K = 0: t is 0, and 0 times an adapter's infinity no number, in its own rows, whichever kernel takes them."""
    c = AdapterCase(dt, 3, rows, 9, 3, 136, 0, 4, 0, 0, transposed, True, True, scaled=False)
    b = c.b.transpose(-1, -2) if transposed else c.b
    b[1, 2, 5] = float("inf")
    y, t = c.run()
    own = torch.zeros(rows, dtype=torch.bool)
    own[ref.group_rows(c.offsets, 1, c.order)] = True
    assert 0 < int(own.sum()) < rows
    assert torch.isnan(y[own, 5]).all() and not t.any()
    assert not y[~own].any() and not y[:, torch.arange(136) != 5].any()
