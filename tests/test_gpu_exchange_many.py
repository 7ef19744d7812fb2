"""The token exchange on more tokens than one dimension of a grid holds in threads (2^32, at 16 threads a token)."""
import pytest
import torch

import tile_scheduled_dense_amd as tg
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def test_more_tokens_than_a_grid_is_wide():
    need_gpu()
    tokens = (1 << 28) + 77
    # one column, one choice: every seventh token without an expert, the others in reverse
    entry = torch.arange(tokens, dtype=torch.int32, device="cuda")
    row = tokens - 1 - entry
    row = torch.where(entry % 7 == 3, ~row, row)
    has = row >= 0
    at = torch.where(has, row, ~row)
    x = (entry % 2039).to(torch.float16)                # whole numbers, exact in 16 bits
    w = (entry % 2 + 1).float()
    zero = torch.zeros((), dtype=torch.float16, device="cuda")

    def empty(dtype=torch.float16):
        return torch.full((tokens,), -1, dtype=dtype, device="cuda")

    out = empty()
    tg.tile_gemm_expert_gather(tokens, 1, 1, "f16", x, 1, row, out, 1)
    assert torch.equal(out, torch.where(has, x, zero).flip(0))
    out.fill_(-1)
    tg.tile_gemm_expert_combine(tokens, 1, 1, "f16", x, 1, row, w, 1, out, 1)
    y = x.flip(0)                                       # y[row] by token: the row is the token's mirror
    assert torch.equal(out, torch.where(has, (y.float() * w).half(), zero))
    out.fill_(-1)
    d_w = empty(torch.float32)
    d = (entry % 31).to(torch.float16)
    tg.tile_gemm_expert_combine_grad(tokens, 1, 1, "f16", d, 1, x, 1, row, w, 1, out, 1, d_w, 1)
    assert torch.equal(out, torch.where(has, (d.float() * w).half(), zero).flip(0))
    assert torch.equal(d_w, torch.where(has, d.float() * y.float(), zero.float()))
    assert int(at[0]) == tokens - 1
