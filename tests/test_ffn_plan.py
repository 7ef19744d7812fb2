"""The plan queries of a feed-forward block's operators (include/tile_gemm_ffn.h) on the CPU: refusals, and
the kernel that each case of tests/ffn_cases.py is there for."""
import ctypes

import pytest

import tile_scheduled_dense_amd as tg
from tests import ffn_cases as cases

OK, INVALID, UNSUPPORTED = tg.TG_OK, tg.TG_ERR_INVALID_ARG, tg.TG_ERR_UNSUPPORTED


def has(plan, want):
    assert {k: plan[k] for k in want} == want


@pytest.mark.parametrize("want,dt,sizes,spare,N,K,pad,skew,transposed", cases.GATED, ids=lambda v: str(v)[:30])
def test_gated(want, dt, sizes, spare, N, K, pad, skew, transposed):
    has(tg.tile_gemm_gated_plan(len(sizes), sum(sizes) + spare, N, K, dt, transposed), want)


@pytest.mark.parametrize("want,dt,sizes,spare,N,K,pad,skew,transposed", cases.GRAD, ids=lambda v: str(v)[:30])
def test_gated_grad(want, dt, sizes, spare, N, K, pad, skew, transposed):
    has(tg.tile_gemm_gated_grad_plan(len(sizes), sum(sizes) + spare, N, K, dt, transposed), want)


@pytest.mark.parametrize("want,dt,adapters,rows,without,N,K,rank,pad,skew,transposed", cases.ADAPTERS,
                         ids=lambda v: str(v)[:30])
def test_adapters(want, dt, adapters, rows, without, N, K, rank, pad, skew, transposed):
    has(tg.tile_gemm_adapters_plan(adapters, rows, N, K, rank, dt, transposed), want)


def test_a_split_asks_for_its_sums():
    for want, dt, sizes, spare, N, K, *_, transposed in cases.GATED:
        n, rows = len(sizes), sum(sizes) + spare
        splits = tg.tile_gemm_gated_plan(n, rows, N, K, dt, transposed)["splits"]
        size = tg.tile_gemm_gated_workspace_size(n, rows, N, K, dt, transposed=transposed)
        assert size == (splits * 2 * rows * N * 4 if splits > 1 else 0)
    for want, dt, adapters, rows, without, N, K, rank, _, _, transposed in cases.ADAPTERS:
        splits = tg.tile_gemm_adapters_plan(adapters, rows, N, K, rank, dt, transposed)["splits"]
        assert tg.tile_gemm_adapters_workspace_size(adapters, rows, N, K, rank, dt, transposed) >= (
            splits * rows * N * 4 if splits > 1 else rows * rank * 4)


@pytest.mark.parametrize("fn,args", [("tile_gemm_gated_plan", (4, 64, 32, 48, 1, 0)),
                                     ("tile_gemm_gated_grad_plan", (4, 64, 32, 48, 1, 0)),
                                     ("tile_gemm_adapters_plan", (4, 64, 32, 48, 8, 1, 0))])
def test_refusals(fn, args):
    info = tg.FfnPlanInfo()
    at = ctypes.byref(info)
    assert tg.tile_gemm_status(fn, *args, at) == OK and info.workgroups > 0
    assert tg.tile_gemm_status(fn, *args, None) == INVALID
    for i in range(len(args) - 2):
        assert tg.tile_gemm_status(fn, *args[:i], -1, *args[i + 1:], at) == INVALID
    assert tg.tile_gemm_status(fn, *args[:-2], 3, 0, at) == INVALID
    assert tg.tile_gemm_status(fn, *args[:-1], 2, at) == INVALID
    assert tg.tile_gemm_status(fn, 2049, *args[1:], at) == UNSUPPORTED
    assert tg.tile_gemm_status(fn, args[0], 0, *args[2:], at) == OK and info.kernel == 0
    assert tg.tile_gemm_status(fn, args[0], 64, 0, *args[3:], at) == OK and info.kernel == 0
