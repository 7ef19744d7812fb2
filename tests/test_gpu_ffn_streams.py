"""The adapters' calls on many rows (t, its join, tiles, K split, sums), at once on two streams with a workspace
each, and captured into two graphs that are replayed between eager calls: bit for bit the results of one call
after the other."""
import pytest
import torch

import tile_scheduled_dense_amd as tg
from tests.gpu_util import need_gpu
from tests.test_gpu_experts import normal
from tests.test_gpu_ffn import table

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


class Trained:
    """Forward, back and the gradients of adapters beside a projection, with T alone (N = 0) before them."""

    def __init__(self, dt, rows, N, K, rank, G, transposed, seed):
        self.args = (dt, rows, N, K, rank, G, transposed)
        make = lambda *s, i, scale=1.0: normal(*s, dtype=dt, seed=10 * seed + i, scale=scale).cuda()  # noqa: E731
        sh = (lambda i, o: (o, i)) if transposed else (lambda i, o: (i, o))
        self.x, self.d_y = make(rows, K, i=1), make(rows, N, i=2)
        self.w = make(*sh(K, N), i=3, scale=K ** -0.5)
        self.a, self.b = make(G, *sh(K, rank), i=4, scale=K ** -0.5), make(G, *sh(rank, N), i=5)
        self.off = table([rows * g // (G + 1) for g in range(G + 1)])
        self.order = table(torch.randperm(rows, generator=torch.Generator().manual_seed(seed)).tolist())
        like = lambda *s: torch.empty(*s, dtype=self.x.dtype, device="cuda")  # noqa: E731
        self.y, self.t, self.t0, self.d_x, self.d_t = like(rows, N), like(rows, rank), like(rows, rank), like(rows, K), like(rows, rank)
        self.d_a, self.d_b = torch.empty_like(self.a), torch.empty_like(self.b)
        size = max(tg.tile_gemm_adapters_workspace_size(G, rows, N, K, rank, dt, transposed=transposed),
                   tg.tile_gemm_adapters_workspace_size(G, rows, K, N, rank, dt, transposed=1 - transposed),
                   tg.tile_gemm_adapters_workspace_size(G, rows, 0, K, rank, dt, transposed=transposed),
                   tg.tile_gemm_adapters_wgrad_workspace_size(G, rows, N, K, rank, dt))
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        self.outs = [self.y, self.t, self.t0, self.d_x, self.d_t, self.d_a, self.d_b]

    def call(self, stream=None):
        dt, rows, N, K, rank, G, tr = self.args
        w, a, b = self.w, self.a, self.b
        kw = dict(order=self.order, stream=stream)
        tg.tile_gemm_adapters(G, rows, 0, K, rank, dt, self.x, K, None, w.shape[1], a, a.shape[2], K * rank, None, b.shape[2], 0,
                              None, 1, self.off, self.ws, transposed=tr, T=self.t0, ldt=rank, **kw)
        tg.tile_gemm_adapters(G, rows, N, K, rank, dt, self.x, K, w, w.shape[1], a, a.shape[2], K * rank, b, b.shape[2], rank * N,
                              self.y, N, self.off, self.ws, transposed=tr, T=self.t, ldt=rank, **kw)
        tg.tile_gemm_adapters(G, rows, K, N, rank, dt, self.d_y, N, w, w.shape[1], b, b.shape[2], rank * N, a, a.shape[2], K * rank,
                              self.d_x, K, self.off, self.ws, transposed=1 - tr, T=self.d_t, ldt=rank, **kw)
        tg.tile_gemm_adapters_wgrad(G, rows, N, K, rank, dt, self.x, K, self.d_y, N, self.t, rank, self.d_t, rank, self.d_a,
                                    a.shape[2], K * rank, self.d_b, b.shape[2], rank * N, self.off, self.ws, c_dtype=dt,
                                    transposed=tr, **kw)

    def spoil(self):
        for o in self.outs:
            o.fill_(-7)

    def keep(self):
        torch.cuda.synchronize()
        self.want = [o.clone() for o in self.outs]
        assert all(bool(torch.isfinite(o.float()).all()) for o in self.want)

    def same(self):
        return all(torch.equal(o, x) for o, x in zip(self.outs, self.want))


@pytest.mark.parametrize("dt,rows,N,K,rank,G,transposed", [
    ("bf16", 1100, 520, 2100, 24, 7, 1),         # 128 x 128 tiles, K split over workgroups
    ("f16", 900, 264, 1025, 3, 5, 0),            # a narrow A, a cut K tile
    ("f32", 1333, 264, 1030, 20, 6, 1), ("bf16", 2100, 2060, 6200, 40, 5, 0)])      # 256 x 256, K in two halves
def test_at_once_and_replayed(dt, rows, N, K, rank, G, transposed):
    both = [Trained(dt, rows, N, K, rank, G, transposed, seed) for seed in (1, 2)]
    for c in both:
        c.call()
        c.keep()
    sides = [torch.cuda.Stream() for _ in both]
    for c in both:
        c.spoil()
    torch.cuda.synchronize()
    for _ in range(3):                           # in flight together, call by call
        for c, s in zip(both, sides):
            c.call(stream=s)
    torch.cuda.synchronize()
    assert both[0].same() and both[1].same()
    graphs = []
    for c, s in zip(both, sides):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            c.call()
        graphs.append(graph)
    for _ in range(3):
        for c in both:
            c.spoil()
        torch.cuda.synchronize()
        graphs[0].replay()
        both[1].call(stream=sides[1])
        torch.cuda.synchronize()
        assert both[0].same() and both[1].same()
        both[0].spoil()
        both[1].spoil()
        torch.cuda.synchronize()
        graphs[1].replay()
        both[0].call(stream=sides[0])
        torch.cuda.synchronize()
        assert both[0].same() and both[1].same()
