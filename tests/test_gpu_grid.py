"""Calls whose workgroups do not fit one dimension of a grid (2^32 threads)."""
import pytest
import torch

import tile_scheduled_dense_amd as tg
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("past,want", [(-1, tg.TG_OK), (5, tg.TG_ERR_UNSUPPORTED)])
def test_batch_of_many_problems(past, want):
    """One workgroup a problem: every problem, or a refusal that leaves C alone."""
    plan = tg.tile_gemm_plan(1 << 20, 1, 1, 1, "f32")
    assert plan["grid"] == 1 << 20
    batch = (1 << 32) // plan["threads"] + past
    A = (torch.arange(batch, device="cuda") % 1021).float()
    B, C = A + 1, torch.full((batch,), -1.0, device="cuda")
    got = tg.tile_gemm_status("tile_gemm_strided_batched", batch, 1, 1, 1, tg.DTYPES["f32"], A.data_ptr(), 1, 1,
                              B.data_ptr(), 1, 1, C.data_ptr(), 1, 1, 1.0, 0.0, 0)
    torch.cuda.synchronize()
    assert got == want
    assert torch.equal(C, A * B if want == tg.TG_OK else torch.full_like(C, -1.0))


def test_pack_of_many_rows():
    """64 threads a row of B: more rows than one dimension of a grid holds."""
    K = (1 << 26) + 9
    B = (torch.arange(K, device="cuda") % 251).to(torch.bfloat16)
    ld = tg.tile_gemm_packed_b_ld(1, "bf16")
    packed = torch.full((K, ld), -1.0, dtype=torch.bfloat16, device="cuda")
    assert tg.tile_gemm_packed_b_size(1, K, 1, "bf16") == K * ld * 2
    tg.tile_gemm_pack_b(1, K, 1, "bf16", B, 1, K, packed)
    assert torch.equal(packed[:, 0], B)
    assert not packed[:, 1:].any()
