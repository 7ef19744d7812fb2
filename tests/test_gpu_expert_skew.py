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


@pytest.mark.parametrize("tile,dt,experts,rows,spare,N,K,group", [
    ((16, 16), "bf16", 64, 300, 0, 40, 300, 64), ((16, 16), "f32", 65, 200, 21, 33, 130, 32), ((16, 32), "f16", 130, 400, 0, 70, 140, 128),
    ((16, 16), "bf16", 64, 1400, 19, 70, 260, 32), ((16, 32), "f16", 63, 2500, 0, 70, 130, 64), ((16, 32), "bf16", 2048, 3000, 5, 20, 33, 32),
])
def test_4_bit_products(tile, dt, experts, rows, spare, N, K, group):
    total = rows + spare
    plan = tg.tile_gemm_q4_plan(experts, total, N, K, group, dt)
    assert (plan["tile_m"], plan["tile_n"]) == tile
    A = base.normal(total, K, dtype=dt, seed=1)
    A[rows:] = float("nan")
    g = torch.Generator().manual_seed(K)
    groups, width = -(-K // group), -(-K // 2)
    codes = torch.randint(0, 256, (experts, N, width), generator=g, dtype=torch.uint8)
    scales = (torch.rand(experts, N, groups, generator=g) + 0.5).to(ref.TYPES[dt])
    W = ref.q4_weights(codes, scales, N, K, group).transpose(1, 2).contiguous()
    packed = torch.empty(tg.tile_gemm_q4_packed_size(experts, N, K, group, dt), dtype=torch.uint8, device="cuda")
    tg.tile_gemm_pack_q4(experts, N, K, group, dt, codes.cuda(), width, N * width, scales.cuda(), groups, N * groups, packed)
    Ad = A.cuda()
    for sizes in splits(experts, rows):
        offsets = base.offsets_of(sizes)
        want, absum = ref.grouped(A, W, offsets, total)
        C = base.Out(total, N, ref.TYPES[dt])
        tg.tile_gemm_q4(experts, total, N, K, group, dt, Ad, K, packed, C.t, N,
                        torch.tensor(offsets, dtype=torch.int32).cuda(), c_dtype=dt)
        # a group's sum of whole codes is scaled once more than a plain product: one term more
        ref.check(C.get(), want, K + 1, absum, dt)
