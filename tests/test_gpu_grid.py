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


@pytest.mark.parametrize("q4", [False, True])
def test_row_tiles_past_one_layer_of_the_grid(q4):
    """More than 32768 row tiles of 16: the grid has a second layer of them."""
    rows, E, N, K = 600011, 2, 7, 40
    offsets = [0, 300003, rows - 9]
    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    A = torch.randint(-2, 3, (rows, K), generator=g, device="cuda").to(torch.bfloat16)
    A[offsets[-1]:] = float("nan")
    C = torch.full((rows, N), float("nan"), device="cuda")
    if q4:
        codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        scales = torch.ones(E, N, 2, dtype=torch.bfloat16, device="cuda")
        W = (torch.stack([codes & 15, codes >> 4], dim=3).reshape(E, N, K).double() - 8).transpose(1, 2)
        packed = torch.empty(tg.tile_gemm_q4_packed_size(E, N, K, 32, "bf16"), dtype=torch.uint8, device="cuda")
        tg.tile_gemm_pack_q4(E, N, K, 32, "bf16", codes, K // 2, N * K // 2, scales, 2, 2 * N, packed)
        tg.tile_gemm_q4(E, rows, N, K, 32, "bf16", A, K, packed, C, N, off)
    else:
        assert tg.tile_gemm_grouped_plan(E, rows, N, K, "bf16")["kernel"] == "stream"
        B = torch.randint(-2, 3, (E, K, N), generator=g, device="cuda").to(torch.bfloat16)
        W = B.double()
        tg.tile_gemm_grouped(E, rows, N, K, "bf16", A, K, B, N, K * N, C, N, off)
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        assert torch.equal(C[lo:hi].double(), A[lo:hi].double() @ W[e].contiguous())
    assert not C[offsets[-1]:].any()
