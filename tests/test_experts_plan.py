"""The plan queries of the expert products (include/tile_gemm_experts.h) on the CPU: refusals, and the
kernel that each case of tests/expert_cases.py is there for."""
import ctypes

import pytest

import tile_scheduled_dense_amd as tg
from tests import expert_cases as cases

OK, INVALID, UNSUPPORTED = tg.TG_OK, tg.TG_ERR_INVALID_ARG, tg.TG_ERR_UNSUPPORTED


def has(plan, **want):
    assert {k: plan[k] for k in want} == want


@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("dt,out,sizes,spare,N,K,pad,skew", cases.TILE256, ids=lambda v: str(v)[:30])
def test_products_on_the_largest_tile(dt, out, sizes, spare, N, K, pad, skew, transposed):
    plan = tg.tile_gemm_grouped_plan(len(sizes), sum(sizes) + spare, N, K, dt, c_dtype=out, transposed=transposed)
    has(plan, kernel="tiles", tile_m=256, tile_n=256, pieces=1, pipeline=1)


def test_the_largest_tile_is_stored_both_ways():
    past = {tg.tile_gemm_grouped_plan(len(s), sum(s) + x, N, K, dt, c_dtype=o)["past_caches"]
            for dt, o, s, x, N, K, _, _ in cases.TILE256}
    grad = {tg.tile_gemm_grouped_wgrad_plan(len(s), sum(s) + x, M, N, dt, c_dtype=o)["past_caches"]
            for dt, o, s, x, M, N, _, _ in cases.WGRAD256}
    assert past == grad == {0, 1}


@pytest.mark.parametrize("dt,out,sizes,spare,M,N,pad,skew", cases.WGRAD256, ids=lambda v: str(v)[:30])
def test_weight_gradients_on_the_largest_tile(dt, out, sizes, spare, M, N, pad, skew):
    plan = tg.tile_gemm_grouped_wgrad_plan(len(sizes), sum(sizes) + spare, M, N, dt, c_dtype=out)
    has(plan, kernel="tiles", tile_m=256, tile_n=256, pieces=0, pipeline=1)


@pytest.mark.parametrize("dt,experts,rows,spare,active,N,K,pad,skew,transposed", cases.STREAM8, ids=lambda v: str(v))
def test_streamed_weights_in_eight_waves(dt, experts, rows, spare, active, N, K, pad, skew, transposed):
    has(tg.tile_gemm_grouped_plan(experts, rows + spare, N, K, dt, transposed=transposed), kernel="stream", waves=8)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("tile,experts,rows,spare,active,N,K,pad", cases.Q4_TILES, ids=lambda v: str(v))
def test_tiles_of_4_bit_products(tile, experts, rows, spare, active, N, K, pad, dt, group):
    plan = tg.tile_gemm_q4_plan(experts, rows + spare, N, K, group, dt)
    has(plan, kernel="q4", tile_m=tile[0], tile_n=tile[1])


@pytest.mark.parametrize("rows,N,K", [(48, 4096, 4096), (64, 4096, 4096), (200, 1037, 1290), (64, 8192, 8192), (2048, 4096, 4096)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_many_rows_of_4_bit_weights_go_16_at_a_time(rows, N, K, dt):
    """32 or 64 rows a workgroup were slower than 16 and two column tiles at every size measured."""
    has(tg.tile_gemm_q4_plan(1, rows, N, K, 128, dt), tile_m=16, tile_n=32)


def test_small_tiles():
    """The tiles below the largest, by type and form."""
    has(tg.tile_gemm_grouped_plan(33, 5001, 1000, 257, "f16"), kernel="tiles", tile_m=128, pieces=0, pipeline=0)
    has(tg.tile_gemm_grouped_plan(4, 2048, 1024, 512, "f32"), kernel="tiles", tile_m=64, pieces=0, pipeline=1)
    has(tg.tile_gemm_grouped_wgrad_plan(33, 5001, 257, 1000, "f16"), kernel="tiles", tile_m=128, pipeline=0)
    has(tg.tile_gemm_grouped_wgrad_plan(2, 1464, 464, 96, "bf16"), kernel="tiles", tile_m=128, pipeline=1)
    has(tg.tile_gemm_grouped_wgrad_plan(4, 2048, 512, 1024, "f32"), kernel="tiles", tile_m=64, pipeline=1)
    has(tg.tile_gemm_grouped_wgrad_plan(2, 500, 3, 1024, "bf16"), kernel="narrow")
    has(tg.tile_gemm_q4_plan(1, 37, 1001, 4100, 32, "f32"), kernel="q4", tile_m=16, tile_n=16)


def test_a_product_of_nothing():
    nothing = dict(kernel="nothing", workgroups=0)
    has(tg.tile_gemm_grouped_plan(4, 0, 32, 48, "bf16"), **nothing)
    has(tg.tile_gemm_grouped_plan(4, 9, 0, 48, "bf16"), **nothing)
    has(tg.tile_gemm_grouped_wgrad_plan(4, 9, 0, 48, "bf16"), **nothing)
    has(tg.tile_gemm_q4_plan(4, 0, 32, 48, 32, "bf16"), **nothing)
    # a sum of nothing is written
    assert tg.tile_gemm_grouped_plan(4, 9, 32, 0, "bf16")["workgroups"] > 0
    assert tg.tile_gemm_grouped_wgrad_plan(4, 0, 32, 48, "bf16")["workgroups"] > 0


OUT = tg.ExpertsPlanInfo()
ARGS = {
    "tile_gemm_grouped_plan": dict(experts=4, rows=64, N=32, K=48, dtype=1, transposed=0, c_dtype=1),
    "tile_gemm_grouped_wgrad_plan": dict(experts=4, rows=64, M=48, N=32, dtype=1, c_dtype=0),
    "tile_gemm_q4_plan": dict(experts=4, rows=64, N=32, K=48, group=32, dtype=2, c_dtype=2),
}


def ask(fn, out=None, **kw):
    out = ctypes.byref(OUT) if out is None else out
    return int(getattr(tg._lib(), fn)(*{**ARGS[fn], **kw}.values(), out))


@pytest.mark.parametrize("fn", list(ARGS))
def test_plan_refusals(fn):
    assert ask(fn) == OK
    assert ask(fn, out=ctypes.POINTER(tg.ExpertsPlanInfo)()) == INVALID
    for kw in (dict(experts=0), dict(rows=-1), dict(N=-1), dict(dtype=3), dict(c_dtype=3), dict(dtype=0, c_dtype=1)):
        assert ask(fn, **kw) == INVALID, kw
    assert ask(fn, experts=2049) == UNSUPPORTED
    assert ask(fn, rows=(1 << 30) + 1) == UNSUPPORTED
    if fn == "tile_gemm_grouped_plan":
        assert ask(fn, transposed=2) == INVALID
    if fn == "tile_gemm_q4_plan":
        assert ask(fn, group=0) == INVALID and ask(fn, group=48) == UNSUPPORTED


def test_grids_past_one_dimension_are_refused():
    """A workgroup has 256 threads, a grid fewer than 2^32: tiles of 64 x 64 over 2^30 rows, or over 2048 wide
    gradients of 8 rows."""
    assert ask("tile_gemm_grouped_plan", experts=1, rows=1 << 30, N=8, K=8, dtype=0, c_dtype=0) == UNSUPPORTED
    assert ask("tile_gemm_grouped_plan", experts=1, rows=1 << 29, N=8, K=8, dtype=0, c_dtype=0) == OK
    assert ask("tile_gemm_grouped_wgrad_plan", experts=2048, M=8, N=1 << 20) == UNSUPPORTED
    assert ask("tile_gemm_grouped_wgrad_plan", experts=2048, M=8, N=1 << 19) == OK


@pytest.mark.parametrize("experts,rows,N,K,dt", [(64, 512, 768, 1024, "f16"), (64, 512, 512, 512, "f32"), (256, 2048, 256, 256, "bf16"),
                                                 (2048, 8192, 128, 128, "bf16"), (8, 32, 4096, 1024, "bf16")])
def test_streamed_rows_of_one_expert_are_not_one_workgroups(experts, rows, N, K, dt):
    """Which expert has the rows is known on the device alone: wherever they are, a workgroup takes one row tile."""
    for transposed in (0, 1):
        has(tg.tile_gemm_grouped_plan(experts, rows, N, K, dt, transposed=transposed), kernel="stream", row_tiles=1)


@pytest.mark.parametrize("experts,rows,N,K,dt", [(64, 256, 2048, 2048, "bf16"), (64, 1024, 2048, 2048, "f16"), (1, 2048, 4096, 4096, "bf16"),
                                                 (16, 128, 1024, 1024, "f32"), (4, 9000, 300, 512, "bf16")])
def test_rows_of_one_4_bit_expert_are_not_one_workgroups(experts, rows, N, K, dt):
    has(tg.tile_gemm_q4_plan(experts, rows, N, K, 128, dt), kernel="q4", row_tiles=1)


@pytest.mark.parametrize("dt,experts,M,N", [("bf16", 64, 100, 100), ("bf16", 64, 384, 384), ("f16", 33, 257, 1000),
                                                 ("f32", 9, 64, 64), ("bf16", 64, 512, 512)])
def test_weight_gradients_have_a_workgroup_a_tile(dt, experts, M, N):
    """Workgroups go to the eight XCDs in turn, so that tiles without gaps are even between them."""
    plan = tg.tile_gemm_grouped_wgrad_plan(experts, 1100 * experts, M, N, dt)
    tiles = -(-M // plan["tile_m"]) * -(-N // plan["tile_n"])
    has(plan, kernel="tiles", workgroups=experts * tiles)


@pytest.mark.parametrize("dt,experts,M,N,tile", [
    ("bf16", 16, 1024, 1024, 256), ("f16", 12, 1024, 1024, 128), ("bf16", 17, 1024, 1024, 128), ("bf16", 64, 512, 512, 256),
    ("bf16", 8, 1300, 1304, 128), ("bf16", 5, 2048, 2048, 128), ("bf16", 8, 2048, 4096, 256), ("f32", 16, 2048, 2048, 256),
    ("f32", 8, 2560, 2560, 64), ("f32", 4, 3600, 3840, 64),
])
def test_tile_of_a_weight_gradient_by_its_rounds(dt, experts, M, N, tile):
    """The largest tile is for rounds that it fills (times of both sides: experts_plan.hpp)."""
    has(tg.tile_gemm_grouped_wgrad_plan(experts, 1100 * experts, M, N, dt, c_dtype=dt), kernel="tiles", tile_m=tile)
