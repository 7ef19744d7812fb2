"""The kernels of the expert products that only larger sizes reach (tests/expert_cases.py), on values.

Whole numbers, compared bit for bit with products in 64 bits on the GPU; then normal inputs within the
bounds of tests/expert_ref.py.  Operands are padded with NaN, outputs start as NaN between guard values.
"""
import pytest
import torch

import tile_scheduled_dense_amd as tg
from tests import expert_cases as cases
from tests import expert_ref as ref
from tests import test_gpu_experts as base
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu
TYPES = ref.TYPES


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def operand(*shape, dtype, terms, whole, pad, skew, seed):
    """A tensor on the GPU, its rows padded with NaN, behind `skew` elements; whole: -1, 0 and 1, of which
    at most about 100 of every `terms` are not 0 (sums that 8 bits hold)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = shape[-1] + pad
    n = 1
    for extent in shape[:-1]:
        n *= extent
    buf = torch.full((skew + n * ld + 16,), float("nan"), dtype=TYPES[dtype], device="cuda")
    x = torch.as_strided(buf, shape, (*(shape[1] * ld,) * (len(shape) == 3), ld, 1), skew)
    if whole:
        v = torch.randint(-1, 2, shape, generator=g, device="cuda", dtype=torch.int8)
        v *= torch.rand(shape, generator=g, device="cuda") < 100 / max(terms, 100)
        x.copy_(v)
    else:
        x.copy_(torch.randn(shape, generator=g, device="cuda"))
    return x, buf[skew:], ld


def same(C, want, absum, terms, out, whole):
    got = C.get().cuda().reshape(want.shape)
    if whole:
        assert float(absum.max()) <= 256
        assert torch.equal(got.double(), want)
    else:
        b = 2 * (terms + 2) * 2.0 ** -24 * absum
        b = b + (want.abs() + b) * torch.finfo(TYPES[out]).eps / 2 + ref.TINY[out] / 2
        over = (got.double() - want).abs() - b
        assert float(over.max()) <= 0 and not torch.isnan(got).any()


@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("dt,out,sizes,spare,N,K,pad,skew", cases.TILE256, ids=lambda v: str(v)[:30])
def test_products_on_the_largest_tile(dt, out, sizes, spare, N, K, pad, skew, transposed):
    E, rows = len(sizes), sum(sizes) + spare
    plan = tg.tile_gemm_grouped_plan(E, rows, N, K, dt, c_dtype=out, transposed=transposed)
    assert (plan["tile_m"], plan["pieces"]) == (256, 1)
    first = base.offsets_of(sizes)
    off = torch.tensor(first, dtype=torch.int32).cuda()
    for whole in (True, False):
        a, A, lda = operand(rows, K, dtype=dt, terms=K, whole=whole, pad=pad, skew=skew, seed=1)
        b, B, ldb = operand(E, *((N, K) if transposed else (K, N)), dtype=dt, terms=0, whole=whole, pad=pad, skew=skew, seed=2)
        a[first[-1]:] = float("nan")
        C = base.Out(rows, N, TYPES[out], pad, skew=skew)
        tg.tile_gemm_grouped(E, rows, N, K, dt, A, lda, B, ldb, b.stride(0), C.t, C.ld, off, c_dtype=out,
                             transposed=transposed)
        want = torch.zeros(rows, N, dtype=torch.float64, device="cuda")
        absum = torch.zeros_like(want)
        for g in range(E):
            lo, hi = first[g], first[g + 1]
            if lo < hi:
                x, y = a[lo:hi].double(), (b[g].t() if transposed else b[g]).double().contiguous()
                want[lo:hi], absum[lo:hi] = x @ y, x.abs() @ y.abs()
        same(C, want, absum, K, out, whole)


@pytest.mark.parametrize("dt,out,sizes,spare,M,N,pad,skew", cases.WGRAD256, ids=lambda v: str(v)[:30])
def test_weight_gradients_on_the_largest_tile(dt, out, sizes, spare, M, N, pad, skew):
    E, rows = len(sizes), sum(sizes) + spare
    assert tg.tile_gemm_grouped_wgrad_plan(E, rows, M, N, dt, c_dtype=out)["tile_m"] == 256
    first = base.offsets_of(sizes)
    off = torch.tensor(first, dtype=torch.int32).cuda()
    for whole in (True, False):
        a, A, lda = operand(rows, M, dtype=dt, terms=max(sizes), whole=whole, pad=pad, skew=skew, seed=1)
        d, D, ldd = operand(rows, N, dtype=dt, terms=0, whole=whole, pad=pad, skew=skew, seed=2)
        a[first[-1]:] = float("nan")
        d[first[-1]:] = float("nan")
        C = base.Out(M, N, TYPES[out], pad, batch=E, skew=skew)
        tg.tile_gemm_grouped_wgrad(E, rows, M, N, dt, A, lda, D, ldd, C.t, C.ld, C.stride, off, c_dtype=out)
        want = torch.zeros(E, M, N, dtype=torch.float64, device="cuda")
        absum = torch.zeros_like(want)
        for g in range(E):
            x, y = a[first[g]:first[g + 1]].double().t().contiguous(), d[first[g]:first[g + 1]].double()
            want[g], absum[g] = x @ y, x.abs() @ y.abs()
        same(C, want, absum, max(sizes), out, whole)


@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("dt,experts,rows,spare,active,N,K,pad,skew,transposed", cases.STREAM8, ids=lambda v: str(v))
def test_streamed_weights_in_eight_waves(dt, experts, rows, spare, active, N, K, pad, skew, transposed, out):
    plan = tg.tile_gemm_grouped_plan(experts, rows + spare, N, K, dt, transposed=transposed)
    assert (plan["kernel"], plan["waves"]) == ("stream", 8)
    base.test_grouped(dt, experts, rows, spare, active, N, K, pad, skew, out, transposed)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt,out", [("bf16", "same"), ("f16", "f32")])
@pytest.mark.parametrize("tile,experts,rows,spare,active,N,K,pad", cases.Q4_TILES, ids=lambda v: str(v))
def test_tiles_of_4_bit_products(tile, experts, rows, spare, active, N, K, pad, dt, out, group):
    plan = tg.tile_gemm_q4_plan(experts, rows + spare, N, K, group, dt)
    assert (plan["tile_m"], plan["tile_n"]) == tile
    base.test_q4(dt, experts, rows, spare, active, N, K, group, pad, out)
