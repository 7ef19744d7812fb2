"""tile_gemm_adapters without a column of y, on the CPU: T does not depend on N, so it is asked for like any
other result (tests/test_gpu_ffn_empty.py has its values)."""
import pytest
import torch

import tile_scheduled_dense_amd as tg
from tests.test_ffn_abi import ADAPT, INVALID, OK, call

NONE = dict(N=0, W=None, B=None, Y=None)


@pytest.mark.parametrize("dt,rows", [("bf16", 1), ("f16", 64), ("f32", 700), ("bf16", 8192)])
@pytest.mark.parametrize("transposed", [0, 1])
def test_t_has_its_sums_in_the_workspace(dt, rows, transposed):
    assert tg.tile_gemm_adapters_workspace_size(4, rows, 0, 4096, 8, dt, transposed=transposed) >= rows * 8 * 4
    assert tg.tile_gemm_adapters_workspace_size(4, rows, 0, 4096, 0, dt, transposed=transposed) == 0
    assert tg.tile_gemm_adapters_workspace_size(4, 0, 0, 4096, 8, dt, transposed=transposed) == 0
    assert tg.tile_gemm_adapters_plan(4, rows, 0, 4096, 8, dt, transposed)["kernel"] == "nothing"


@pytest.mark.parametrize("kw", [dict(workspace=None), dict(workspace_bytes=16), dict(offsets=None), dict(A=None), dict(X=None),
                                dict(ldt=7), dict(T=ADAPT["X"]), dict(T=ADAPT["workspace"])], ids=str)
def test_what_t_needs_is_checked(kw):
    assert call("tile_gemm_adapters", ADAPT, **{**NONE, **kw}) == INVALID


@pytest.mark.parametrize("kw", [dict(T=None, offsets=None, workspace=None), dict(rank=0, A=None, offsets=None, workspace=None),
                                dict(rows=0, X=None, T=None, offsets=None, workspace=None)], ids=str)
def test_nothing_is_needed_where_t_is_not_asked_for(kw):
    assert call("tile_gemm_adapters", ADAPT, **{**NONE, **kw}) == OK


def test_without_a_device_there_is_no_t():
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible")
    assert call("tile_gemm_adapters", ADAPT, **NONE) == OK


def test_sums_that_no_memory_holds_matter_where_t_is_asked_for():
    big = dict(NONE, rows=1 << 30, rank=1 << 30, lda=1 << 30, ldt=1 << 30, ldx=48)
    assert call("tile_gemm_adapters", ADAPT, **big, workspace_bytes=1 << 60) == tg.TG_ERR_UNSUPPORTED
    assert call("tile_gemm_adapters", ADAPT, **{**big, "T": None, "workspace": None}) == OK
