"""Rows past 2^31 bytes from a matrix's first, on the GPU: through a table whose order is none of the rows' (few
rows, many, the adapters' gradients), and in the gate and its gradient.  Matrices are wide rows of which the operators use
the first few elements; nothing else may be written.
"""
import pytest
import torch

import tile_scheduled_dense_amd as tg
from tests import ffn_ref as ref
from tests.gpu_util import need_gpu
from tests.test_gpu_experts import normal
from tests.test_gpu_ffn import table

pytestmark = pytest.mark.gpu
FAR = 2 ** 31


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    torch.cuda.empty_cache()


class Wide:
    """rows x cols bf16 at a row stride that takes the last rows past 2^31 bytes; zeros elsewhere."""

    def __init__(self, rows, cols, ld, values=None):
        assert (rows - 1) * ld * 2 > FAR
        self.rows, self.cols, self.ld = rows, cols, ld
        self.t = torch.zeros(rows * ld, dtype=torch.bfloat16, device="cuda")
        self.view = torch.as_strided(self.t, (rows, cols), (ld, 1))
        if values is not None:
            self.view.copy_(values.cuda())

    def get(self):
        """The values; all else is still zero."""
        torch.cuda.synchronize()
        got = self.view.clone()
        self.view.zero_()
        assert not bool(self.t.any()), "a write outside the rows"
        return got.cpu()


def shuffle(rows, seed):
    return torch.randperm(rows, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("rows,N,kernel", [(400, 24, "few"), (400, 5, "few"), (600, 24, "many")])
def test_adapters_through_a_table(rows, N, kernel, transposed):
    """Few rows: x, y and t far; many: y and t (of x there may be 2^31 bytes then)."""
    K, rank, G, ld = 40, 4, 3, 3_000_000
    offsets, order = [0, rows // 3, rows // 3, rows - 10], shuffle(rows, 1)
    shape = (lambda i, o: (o, i)) if transposed else (lambda i, o: (i, o))
    x = normal(rows, K, dtype="bf16", seed=1)
    w = normal(*shape(K, N), dtype="bf16", seed=2, scale=K ** -0.5)
    a = normal(G, *shape(K, rank), dtype="bf16", seed=3, scale=K ** -0.5)
    b = normal(G, *shape(rank, N), dtype="bf16", seed=4)
    X = Wide(rows, K, ld, x) if kernel == "few" else None
    xd, ldx = (X.t, ld) if X else (x.cuda(), K)
    Y, T = Wide(rows, N, ld), Wide(rows, rank, ld)
    plan = tg.tile_gemm_adapters_plan(G, rows, N, K, rank, "bf16", transposed)
    assert (plan["tile_m"] <= 64) == (kernel == "few")          # few rows: 16 or 64 at a time, many: 128
    size = tg.tile_gemm_adapters_workspace_size(G, rows, N, K, rank, "bf16", transposed=transposed)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    tg.tile_gemm_adapters(G, rows, N, K, rank, "bf16", xd, ldx, w.cuda(), w.shape[1], a.cuda(), a.shape[2], K * rank, b.cuda(),
                          b.shape[2], rank * N, Y.t, ld, table(offsets), ws, order=table(order.tolist()), transposed=transposed,
                          T=T.t, ldt=ld)
    want, err, want_t, t_err = ref.adapters(x, w, a, b, None, offsets, order, transposed, "bf16")
    ref.check(Y.get(), want, err, "bf16", "y")
    ref.check(T.get(), want_t, t_err, "bf16", "t")


@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("rows", [200, 700])
def test_adapter_gradients_through_a_table(rows, transposed):
    """One chunk of an adapter's rows, and several."""
    K, N, rank, G, ld = 40, 24, 5, 3, FAR // 2 // (rows - 1) // 8 * 8 + 8
    offsets, order = [0, rows // 2, rows // 2, rows - 10], shuffle(rows, 2)
    mats = [normal(rows, n, dtype="bf16", seed=10 + i) for i, n in enumerate((K, N, rank, rank))]
    x, dy, t, d_t = mats
    wide = [Wide(rows, m.shape[1], ld, m) for m in mats]
    da = torch.full((G, rank, K) if transposed else (G, K, rank), float("nan"), device="cuda")
    db = torch.full((G, N, rank) if transposed else (G, rank, N), float("nan"), device="cuda")
    size = tg.tile_gemm_adapters_wgrad_workspace_size(G, rows, N, K, rank, "bf16")
    ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    tg.tile_gemm_adapters_wgrad(G, rows, N, K, rank, "bf16", *[v for m in wide for v in (m.t, ld)], da, da.shape[2], K * rank, db,
                                db.shape[2], rank * N, table(offsets), ws, order=table(order.tolist()), transposed=transposed)
    torch.cuda.synchronize()
    for got, L, S, flip, what in ((da, x, d_t, transposed, "d_a"), (db, dy, t, not transposed, "d_b")):
        want, absum, terms = ref.adapters_wgrad(L, S, offsets, order)
        if flip:
            want, absum = want.transpose(1, 2), absum.transpose(1, 2)
        ref.check(got, want, ref.sum_error(terms, absum), "f32", what)


def test_the_gate_and_its_gradient():
    rows, N, ld = 400, 37, 3_000_000
    u, v, d = (normal(rows, N, dtype="bf16", seed=s, scale=2.0) for s in (1, 2, 3))
    U, V, D = (Wide(rows, N, ld, m) for m in (u, v, d))
    H, dU, dV = (Wide(rows, N, ld) for _ in range(3))
    tg.tile_gemm_gate(rows, N, "bf16", U.t, V.t, ld, H.t, ld)
    h = H.get()
    tg.tile_gemm_gate_grad(rows, N, "bf16", D.t, ld, U.t, V.t, ld, dU.t, dV.t, ld, H=H.t, ldh=ld)
    zero, live = torch.zeros(rows, N, dtype=torch.float64), torch.ones(rows, dtype=torch.bool)
    for got in (h, H.get()):
        ref.check_gate_grad(dU.view.cpu(), dV.view.cpu(), got, d.double(), zero, 0, u, v, live, ref.SILU, "bf16")
    dU.get(), dV.get()


@pytest.mark.parametrize("rows,E,kernel", [(300, 8, "stream"), (20000, 2, "tiles")])
def test_the_gates_gradient_through_the_projection(rows, E, kernel):
    K, N = 40, 24
    assert tg.tile_gemm_gated_grad_plan(E, rows, N, K, "bf16")["kernel"] == kernel
    ld = FAR // 2 // (rows - 1) // 8 * 8 + 8
    offsets = [0] * (E - 1) + [rows // 3, rows - 5]
    d, b = normal(rows, K, dtype="bf16", seed=1), normal(E, K, N, dtype="bf16", seed=2, scale=K ** -0.5)
    u, v = (normal(rows, N, dtype="bf16", seed=s, scale=2.0) for s in (3, 4))
    D, U, V = (Wide(rows, m.shape[1], ld, m) for m in (d, u, v))
    H, dU, dV = (Wide(rows, N, ld) for _ in range(3))
    tg.tile_gemm_gated_grad(E, rows, N, K, "bf16", D.t, ld, b.cuda(), N, K * N, U.t, V.t, ld, dU.t, dV.t, ld, table(offsets),
                            H=H.t, ldh=ld)
    d[offsets[-1]:] = 0
    live = torch.arange(rows) < offsets[-1]
    d_h, _, s, _ = ref.gated(d, b, torch.zeros_like(b), offsets, 0)
    ref.check_gate_grad(dU.get(), dV.get(), H.get(), d_h, s, K, u, v, live, ref.SILU, "bf16")
