"""Adapters of a narrow rank beside many rows, on the GPU: x . A[g] where A[g], stored inputs x outputs,
is narrower than a copy of the LDS ring (tests/test_ffn_bounds.py has the reach of the copies)."""
import pytest
import torch

import tile_scheduled_dense_amd as tg
from tests import ffn_ref as ref
from tests.gpu_util import need_gpu
from tests.test_gpu_ffn import AdapterCase

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


# dtype, adapters, rows, without, active, N, K, rank, pad
CASES = [
    ("bf16", 3, 700, 20, 3, 136, 97, 1, 0), ("bf16", 3, 700, 0, 3, 136, 34, 2, 0), ("f16", 2, 600, 7, 2, 264, 65, 3, 0),
    ("f16", 70, 700, 20, 60, 136, 102, 1, 0), ("f32", 3, 700, 20, 3, 136, 97, 1, 0), ("f32", 2, 600, 0, 2, 100, 34, 1, 0),
    ("bf16", 5, 4100, 100, 5, 2060, 1025, 1, 0), ("f32", 41, 1333, 21, 37, 264, 1025, 2, 0), ("f16", 3, 900, 0, 3, 72, 1031, 2, 3),
    ("bf16", 2, 700, 700, 0, 64, 40, 3, 0), ("bf16", 3, 700, 1, 2, 136, 0, 2, 0), ("bf16", 4, 600, 5, 4, 200, 130, 5, 0),
    ("f32", 4, 600, 5, 4, 200, 130, 7, 1), ("f16", 4, 600, 5, 4, 200, 2080, 4, 0),
]


@pytest.mark.parametrize("shuffled", [False, True])
@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("dt,adapters,rows,without,active,N,K,rank,pad", CASES, ids=lambda v: str(v))
def test_narrow_ranks(dt, adapters, rows, without, active, N, K, rank, pad, transposed, shuffled):
    assert tg.tile_gemm_adapters_plan(adapters, rows, N, K, rank, dt, transposed)["kernel"] == "tiles"
    for exact in (True, False):
        c = AdapterCase(dt, adapters, rows, without, active, N, K, rank, pad, 0, transposed, shuffled, exact, scaled=exact)
        y, t = c.run(save=exact or shuffled)
        dev = [m.cuda() for m in (c.x, c.w, c.a, c.b)]
        want, y_err, want_t, t_err = ref.adapters(*dev, c.scales, c.offsets, c.order, transposed, dt)
        if exact:
            assert float(want.abs().max() if want.numel() else 0) <= 256
            assert torch.equal(y.double(), want.cpu())
            assert torch.equal(t.double(), want_t.cpu())
        else:
            ref.check(y, want, y_err, dt, "y")
            if t is not None:
                ref.check(t, want_t, t_err, dt, "t")


def test_a_narrow_adapters_infinities_stay_its_own():
    """NaN in an adapter's A, and in the rows of no adapter: other rows are as without."""
    def case():
        return AdapterCase("bf16", 4, 700, 9, 4, 136, 97, 2, 0, 0, 0, True, False)

    c = case()
    whole, _ = c.run()
    c.a[1][50, 0] = float("nan")
    y, t = c.run()
    mine = ref.group_rows(c.offsets, 1, c.order)
    others = torch.ones(700, dtype=torch.bool)
    others[mine] = False
    assert torch.equal(y[others], whole[others]) and torch.isnan(y[mine]).all() and torch.isnan(t[mine][:, 0]).all()
    c = case()
    none = c.order[c.offsets[-1]:]
    c.x[none] = float("nan")
    y, t = c.run()
    live = torch.ones(700, dtype=torch.bool)
    live[none] = False
    assert torch.equal(y[live], whole[live]) and not t[none].any()
