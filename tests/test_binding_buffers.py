"""What the binding takes for a buffer, and how it measures a workspace whose size the caller leaves out, on the
CPU: a tensor, any object with data_ptr (and numel and element_size), an address."""
import pytest
import torch

import tile_scheduled_dense_amd as tg

P = [0x100000000 + (i << 36) for i in range(12)]     # never dereferenced, far apart


class Buffer:
    """A buffer of another library: no nbytes."""

    def __init__(self, at, n, size):
        self.at, self.n, self.size = at, n, size

    def data_ptr(self):
        return self.at

    def numel(self):
        return self.n

    def element_size(self):
        return self.size


class Sized(Buffer):
    def nbytes(self):               # a method, as a storage has it
        return self.n * self.size


def test_bytes_of():
    assert tg._bytes_of(None) == 0 and tg._bytes_of(P[0]) == 0
    assert tg._bytes_of(torch.zeros(3, 5, dtype=torch.bfloat16)) == 30
    assert tg._bytes_of(torch.zeros(8, 8)[:, ::2]) == 8 * 4 * 4
    assert tg._bytes_of(Buffer(P[0], 10, 4)) == 40
    assert tg._bytes_of(Sized(P[0], 10, 4)) == 40


def test_addresses():
    t = torch.zeros(4)
    assert tg._addr(None) is None and tg._addr(P[0]) == P[0] and tg._addr(t) == t.data_ptr()
    assert tg._addr(Buffer(P[1], 1, 1)) == P[1]
    for bad in ("x", 1.5, [1]):
        with pytest.raises(TypeError):
            tg._addr(bad)


def calls(make):
    """Calls whose workspace or packed matrix has to be of a size; what each returns without a device is UNSUPPORTED,
    after every check, and INVALID_ARG if the buffer counts as too small."""
    n = tg.tile_gemm_expert_sort_workspace_size(100000, 2, 8)
    yield lambda: tg.tile_gemm_expert_sort(100000, 2, 8, P[0], 2, P[1], P[2], P[3], workspace=make(P[4], n))
    n = tg.tile_gemm_q4_packed_size(2, 64, 64, 32, "bf16")
    yield lambda: tg.tile_gemm_pack_q4(2, 64, 64, 32, "bf16", P[0], 32, 32 * 64, P[1], 2, 128, make(P[4], n))
    n = tg.tile_gemm_packed_b_size(1, 64, 64, "bf16")
    yield lambda: tg.tile_gemm_pack_b(1, 64, 64, "bf16", P[0], 64, 0, make(P[4], n))
    n = tg.tile_gemm_adapters_workspace_size(4, 64, 32, 48, 8, "bf16")
    yield lambda: tg.tile_gemm_adapters(4, 64, 32, 48, 8, "bf16", P[0], 48, P[1], 32, P[2], 8, 384, P[3], 32, 256, P[5], 32, P[6],
                                        make(P[4], n))
    n = tg.tile_gemm_adapters_wgrad_workspace_size(4, 300, 32, 48, 8, "bf16")
    yield lambda: tg.tile_gemm_adapters_wgrad(4, 300, 32, 48, 8, "bf16", P[0], 48, P[1], 32, P[2], 8, P[3], 8, P[5], 8, 384,
                                              P[6], 32, 256, P[7], make(P[4], n))


@pytest.mark.parametrize("make,status", [
    (lambda at, n: Buffer(at, -(-n // 4), 4), tg.TG_ERR_UNSUPPORTED), (lambda at, n: Sized(at, n, 1), tg.TG_ERR_UNSUPPORTED),
    (lambda at, n: Buffer(at, n - 1, 1), tg.TG_ERR_INVALID_ARG), (lambda at, n: at, tg.TG_ERR_INVALID_ARG)],
    ids=["elements", "nbytes is a method", "one byte short", "an address alone"])
def test_a_workspace_is_measured(make, status):
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible")
    for call in calls(make):
        with pytest.raises(tg.TileGemmError) as e:
            call()
        assert e.value.status == status
