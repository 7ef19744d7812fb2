"""Every kernel of a feed-forward block's operators on values, at the sizes of tests/ffn_cases.py
(whose plans tests/test_ffn_plan.py asserts), against 64 bits on the GPU; and what no size alone
shows: values that are not finite, tables that are wrong, streams, graphs, far rows, the operators one
after the other.
"""
import pytest
import torch

import tile_scheduled_dense_amd as tg
from tests import ffn_cases as cases
from tests import ffn_ref as ref
from tests.gpu_util import need_gpu
from tests.test_gpu_experts import Out, normal, offsets_of, strided
from tests.test_gpu_ffn import AdapterCase, scratch, table

pytestmark = pytest.mark.gpu
TYPES = ref.TYPES


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("save", [True, False])
@pytest.mark.parametrize("want,dt,sizes,spare,N,K,pad,skew,transposed", cases.GATED, ids=lambda v: str(v)[:40])
def test_gated(want, dt, sizes, spare, N, K, pad, skew, transposed, save):
    E, offsets = len(sizes), offsets_of(sizes)
    total = sum(sizes) + spare
    shape = (E, N, K) if transposed else (E, K, N)
    x = normal(total, K, dtype=dt, seed=1)
    bg, bu = (normal(*shape, dtype=dt, seed=s, scale=K ** -0.5) for s in (2, 3))
    x[offsets[-1]:] = float("nan")
    (xd, lda), (gd, ldb), (ud, _) = (strided(t, pad, skew) for t in (x, bg, bu))
    h, u, v = (Out(total, N, TYPES[dt], pad, skew=skew) for _ in range(3))
    ws, whole = scratch(tg.tile_gemm_gated_workspace_size(E, total, N, K, dt, transposed=transposed))
    kind = ref.SILU if save else ref.GELU
    tg.tile_gemm_gated(E, total, N, K, dt, xd, lda, gd, ud, ldb, shape[1] * ldb, h.t, h.ld, table(offsets), activation=kind,
                       transposed=transposed, U=u.t if save else None, V=v.t if save else None, ldu=u.ld, workspace=ws)
    x[offsets[-1]:] = 0
    ref.check_gated(h.get(), u.get() if save else None, v.get() if save else None, x.cuda(), bg.cuda(), bu.cuda(), offsets,
                    transposed, kind, dt)
    whole()


@pytest.mark.parametrize("want,dt,sizes,spare,N,K,pad,skew,transposed", cases.GRAD, ids=lambda v: str(v)[:40])
def test_gated_grad(want, dt, sizes, spare, N, K, pad, skew, transposed):
    E, offsets = len(sizes), offsets_of(sizes)
    total = sum(sizes) + spare
    shape = (E, N, K) if transposed else (E, K, N)
    d, b = normal(total, K, dtype=dt, seed=1), normal(*shape, dtype=dt, seed=2, scale=K ** -0.5)
    u, v = (normal(total, N, dtype=dt, seed=s, scale=2.0) for s in (3, 4))
    for t in (d, u, v):
        t[offsets[-1]:] = float("nan")
    (dd, ldd), (bd, ldb), (ud, ldu), (vd, _) = (strided(t, pad, skew) for t in (d, b, u, v))
    du, dv, h = (Out(total, N, TYPES[dt], pad, skew=skew) for _ in range(3))
    tg.tile_gemm_gated_grad(E, total, N, K, dt, dd, ldd, bd, ldb, shape[1] * ldb, ud, vd, ldu, du.t, dv.t, du.ld,
                            table(offsets), activation=ref.SILU, transposed=transposed, H=h.t, ldh=h.ld)
    d[offsets[-1]:] = 0
    live = (torch.arange(total) < offsets[-1]).cuda()
    b = b.cuda()
    d_h, _, s, _ = ref.gated(d.cuda(), b, torch.zeros_like(b), offsets, transposed)
    ref.check_gate_grad(du.get(), dv.get(), h.get(), d_h, s, K, u.cuda(), v.cuda(), live, ref.SILU, dt)


class LargeCase(AdapterCase):
    """References on the GPU."""

    def check(self, save=True):
        y, t = self.run(save=save)
        dev = [m.cuda() for m in (self.x, self.w, self.a, self.b)]
        want, y_err, want_t, t_err = ref.adapters(*dev, self.scales, self.offsets, self.order, self.tr, self.dt)
        ref.check(y, want, y_err, self.dt, "y")
        if t is not None:
            ref.check(t, want_t, t_err, self.dt, "t")


@pytest.mark.parametrize("shuffled", [False, True])
@pytest.mark.parametrize("want,dt,adapters,rows,without,N,K,rank,pad,skew,transposed", cases.ADAPTERS, ids=lambda v: str(v)[:40])
def test_adapters(want, dt, adapters, rows, without, N, K, rank, pad, skew, transposed, shuffled):
    LargeCase(dt, adapters, rows, without, adapters, N, K, rank, pad, skew, transposed, shuffled, False).check(save=shuffled)


@pytest.mark.parametrize("dt,rows,N,K,rank,adapters", [("bf16", 3000, 1200, 700, 40, 3), ("f16", 2600, 300, 2100, 130, 9),
                                                       ("f32", 1500, 520, 264, 20, 2), ("bf16", 700, 264, 130, 64, 300)])
def test_adapter_gradients_of_many_rows(dt, rows, N, K, rank, adapters):
    """Several chunks an adapter, several passes over the rank."""
    c = AdapterCase(dt, adapters, rows, 11, adapters, N, K, 1, 0, 0, 1, True, False)
    x, dy, t, d_t = (normal(rows, n, dtype=dt, seed=s) for s, n in enumerate((K, N, rank, rank)))
    da, db = Out(rank, K, torch.float32, batch=adapters), Out(N, rank, torch.float32, batch=adapters)
    ws, whole = scratch(tg.tile_gemm_adapters_wgrad_workspace_size(adapters, rows, N, K, rank, dt))
    tg.tile_gemm_adapters_wgrad(adapters, rows, N, K, rank, dt, x.cuda(), K, dy.cuda(), N, t.cuda(), rank, d_t.cuda(), rank,
                                da.t, K, rank * K, db.t, rank, N * rank, table(c.offsets), ws, order=table(c.order.tolist()),
                                transposed=1)
    for got, L, S, flip in ((da, x, d_t, True), (db, dy, t, False)):
        want, absum, terms = ref.adapters_wgrad(L.cuda(), S.cuda(), c.offsets, c.order)
        if flip:
            want, absum = want.transpose(1, 2), absum.transpose(1, 2)
        ref.check(got.get().reshape(want.shape), want, ref.sum_error(terms, absum), "f32", "gradient")
    whole()


# ---- the gate alone -------------------------------------------------------------------------
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,N,pad,skew", [(1, 1, 0, 0), (3, 7, 1, 1), (70, 264, 0, 0), (33, 1001, 3, 1), (5000, 2048, 0, 0)])
def test_gate(dt, rows, N, pad, skew):
    u, v, d = (normal(rows, N, dtype=dt, seed=s, scale=3.0) for s in (1, 2, 3))
    (ud, ldu), (vd, _), (dd, ldd) = (strided(t, pad, skew) for t in (u, v, d))
    for kind in (ref.NONE, ref.RELU, ref.GELU, ref.SILU):
        h, du, dv, h2 = (Out(rows, N, TYPES[dt], pad, skew=skew) for _ in range(4))
        tg.tile_gemm_gate(rows, N, dt, ud, vd, ldu, h.t, h.ld, activation=kind)
        tg.tile_gemm_gate_grad(rows, N, dt, dd, ldd, ud, vd, ldu, du.t, dv.t, du.ld, activation=kind, H=h2.t, ldh=h2.ld)
        zero, live = torch.zeros(rows, N, dtype=torch.float64), torch.ones(rows, dtype=torch.bool)
        first = h.get()
        ref.check_gate_grad(du.get(), dv.get(), first, d.double(), zero, 0, u, v, live, kind, dt)
        again = h2.get()
        assert torch.equal(first, again) or kind == ref.GELU or kind == ref.SILU
        ref.check_gate_grad(du.get(), dv.get(), again, d.double(), zero, 0, u, v, live, kind, dt)


@pytest.mark.parametrize("kind", [ref.NONE, ref.RELU, ref.GELU, ref.SILU])
def test_gate_of_large_and_special_values(kind):
    """The activations where their exponentials overflow and vanish, and a NaN that stays where it is."""
    u = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 30, -30, 100, -100, 1e4, -1e4, 3e38, -3e38, float("nan"), 1.0])
    v = torch.ones_like(u)
    h, du, dv = (torch.empty_like(u).cuda() for _ in range(3))
    n = u.numel()
    tg.tile_gemm_gate(1, n, "f32", u.cuda(), v.cuda(), n, h, n, activation=kind)
    tg.tile_gemm_gate_grad(1, n, "f32", v.cuda(), n, u.cuda(), v.cuda(), n, du, dv, n, activation=kind)
    f, d = ref.act(u[None].double(), kind)
    for got, want, err in ((h, f, ref.err_act(u[None].double(), f)), (dv, f, ref.err_act(u[None].double(), f)),
                           (du, d, ref.err_slope(u[None].double()))):
        got = got[None].cpu().double()
        # the slope of no activation is 1 whatever u is
        nan = torch.zeros_like(u[None], dtype=torch.bool) if want is d and kind == ref.NONE else torch.isnan(u[None])
        assert torch.equal(torch.isnan(got), nan), (kind, got)
        ok = ~torch.isnan(u[None])
        # below fp32's normal numbers a result may be flushed
        assert bool(((got - want).abs()[ok] <= (err + want.abs() * 2 ** -22 + 2.0 ** -126)[ok]).all()), (kind, got - want)


# ---- values that are not finite ---------------------------------------------------------------
@pytest.mark.parametrize("rows,K,N,shuffled", [(50, 200, 136, True), (300, 200, 136, False), (300, 1100, 520, True),
                                               (1100, 1100, 520, True), (900, 200, 520, False), (1807, 6200, 2307, True), (4200, 1024, 2060, True)])
@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("what", [float("inf"), float("nan")])
def test_an_adapter_of_infinities_reaches_its_own_rows_only(rows, K, N, shuffled, transposed, what):
    def case():
        return AdapterCase("bf16", 6, rows, 9, 6, N, K, 24, 0, 0, transposed, shuffled, False)

    whole, _ = case().run()
    c = case()
    rank_at = (3, 5) if transposed else (5, 3)        # one value of adapter 2's B: an input of the rank, an output
    c.b[2][rank_at] = what
    c.a[4][0, 0] = what                                # and of adapter 4's A: its whole t
    y, t = c.run()
    rows_of = {g: ref.group_rows(c.offsets, g, c.order) for g in (2, 4)}
    others = torch.ones(rows, dtype=torch.bool)
    others[rows_of[2]] = others[rows_of[4]] = False
    assert torch.equal(y[others], whole[others])
    col = 3
    assert not torch.isfinite(y[rows_of[2], col]).any()
    # B's other columns are summed otherwise than in a whole tile; t is the same
    keep = torch.arange(N) != col
    dev = [m.cuda() for m in (c.x, c.w, c.a, c.b)]
    want, err, *_ = ref.adapters(*dev, c.scales, c.offsets, c.order, transposed, "bf16")
    r = rows_of[2]
    e = err[r][:, keep].cpu()
    # one rounding of y more, where the left-out part is added to what was stored
    e = e + want[r][:, keep].cpu().abs() * 2.0 ** -8
    base = c.x[r].double() @ ref.dense(c.w, transposed)
    ref.check(y[r][:, keep], want[r][:, keep].cpu(), e + base[:, keep].abs() * 2.0 ** -8 + 2.0 ** -8, "bf16", "y of adapter 2")
    assert not torch.isfinite(t[rows_of[4]]).all() and torch.isfinite(t[others]).all()


@pytest.mark.parametrize("rows", [20, 300, 1500])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_row_of_nan_stays_its_own(rows, dt):
    """In every operator: x's row 7 is NaN, and no other row of a result changes."""
    K, N, G, rank = 264, 200, 3, 12
    c = AdapterCase(dt, G, rows, 0, G, N, K, rank, 0, 0, 0, True, False)
    good, t_good = c.run()
    c.x[7] = float("nan")
    bad, t_bad = c.run()
    other = torch.arange(rows) != 7
    assert torch.equal(bad[other], good[other]) and torch.equal(t_bad[other], t_good[other])
    assert torch.isnan(bad[7]).all()
    x, b = normal(rows, K, dtype=dt, seed=1), normal(1, K, N, dtype=dt, seed=2)
    outs = []
    for spoil in (False, True):
        if spoil:
            x[7] = float("nan")
        h, u, v = (Out(rows, N, TYPES[dt]) for _ in range(3))
        tg.tile_gemm_gated(1, rows, N, K, dt, x.cuda(), K, b.cuda(), b.cuda(), N, 0, h.t, N, U=u.t, V=v.t, ldu=N)
        du, dv = Out(rows, N, TYPES[dt]), Out(rows, N, TYPES[dt])
        tg.tile_gemm_gated_grad(1, rows, N, K, dt, x.cuda(), K, b.cuda(), N, 0, u.t, v.t, N, du.t, dv.t, N)
        outs.append([o.get() for o in (h, u, v, du, dv)])
    for a, b in zip(*outs):
        assert torch.equal(a[other], b[other]) and torch.isnan(b[7]).all()


# ---- tables that are wrong, far rows --------------------------------------------------------------
def test_wrong_tables_stay_inside():
    """Offsets and orders outside the rows are clamped; nothing else is written."""
    for offsets in ([-5, 3, 10 ** 9], [7, 2, 30], [2 ** 31 - 1, -2 ** 31, 4], [0, 40, 20]):
        off = table(offsets)
        for rows in (20, 60, 600):
            K, N, rank = 72, 264, 12
            x, w = normal(rows, K, dtype="bf16").cuda(), normal(2, K, N, dtype="bf16").cuda()
            h, u, v, du, dv = (Out(rows, N, torch.bfloat16) for _ in range(5))
            ws, whole = scratch(tg.tile_gemm_gated_workspace_size(2, rows, N, K, "bf16"))
            tg.tile_gemm_gated(2, rows, N, K, "bf16", x, K, w, w, N, K * N, h.t, N, off, U=u.t, V=v.t, ldu=N, workspace=ws)
            tg.tile_gemm_gated_grad(2, rows, N, K, "bf16", x, K, w, N, K * N, u.t, v.t, N, du.t, dv.t, N, off)
            for o in (h, u, v, du, dv):
                o.get()
            whole()
            a, b = normal(2, K, rank, dtype="bf16").cuda(), normal(2, rank, N, dtype="bf16").cuda()
            order = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows,), dtype=torch.int64).to(torch.int32).cuda()
            for table_ in (None, order):
                y, t = Out(rows, N, torch.bfloat16), Out(rows, rank, torch.bfloat16)
                ws, whole = scratch(tg.tile_gemm_adapters_workspace_size(2, rows, N, K, rank, "bf16"))
                tg.tile_gemm_adapters(2, rows, N, K, rank, "bf16", x, K, w, N, a, rank, K * rank, b, N, rank * N, y.t, N, off,
                                      ws, order=table_, T=t.t, ldt=rank)
                y.get(), t.get(), whole()
                da, db = Out(K, rank, torch.float32, batch=2), Out(rank, N, torch.float32, batch=2)
                ws, whole = scratch(tg.tile_gemm_adapters_wgrad_workspace_size(2, rows, N, K, rank, "bf16"))
                low = torch.zeros(rows, rank, dtype=torch.bfloat16, device="cuda")
                y = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
                tg.tile_gemm_adapters_wgrad(2, rows, N, K, rank, "bf16", x, K, y, N, low, rank, low, rank, da.t, rank, da.stride,
                                            db.t, N, db.stride, off, ws, order=table_)
                da.get(), db.get(), whole()


def test_far_rows_and_strides():
    """Row offsets past 2^31 bytes, in order and (few rows) through a table."""
    ld, K, N, rank = 16 * 1024 + 8, 40, 24, 4
    for rows in (60, 70000):
        wide = ld if rows > 1000 else 20_000_000 // rows * 4
        X = torch.zeros(rows * wide, dtype=torch.bfloat16, device="cuda")
        Y = torch.zeros(rows * wide, dtype=torch.bfloat16, device="cuda")
        x = normal(8, K, dtype="bf16", seed=1)
        torch.as_strided(X, (rows, K), (wide, 1))[-8:] = x.cuda()
        w, a, b = (normal(*s, dtype="bf16", seed=i) for i, s in enumerate(((K, N), (2, K, rank), (2, rank, N))))
        off = [0, rows - 8, rows]
        order = torch.arange(rows) if rows < 100 else None
        ws, _ = scratch(tg.tile_gemm_adapters_workspace_size(2, rows, N, K, rank, "bf16"))
        tg.tile_gemm_adapters(2, rows, N, K, rank, "bf16", X, wide, w.cuda(), N, a.cuda(), rank, K * rank, b.cuda(), N, rank * N,
                              Y, wide, table(off), ws, order=None if order is None else table(order.tolist()))
        torch.cuda.synchronize()
        got = torch.as_strided(Y, (rows, N), (wide, 1))
        want, err, *_ = ref.adapters(x, w, a[1:], b[1:], None, [0, 8], None, 0, "bf16")
        ref.check(got[-8:].cpu(), want, err, "bf16", "y")
        assert not got[:-8].any()
        Y.zero_()
        bg = normal(2, K, N, dtype="bf16", seed=7)
        tg.tile_gemm_gated(2, rows, N, K, "bf16", X, wide, bg.cuda(), bg.cuda(), N, K * N, Y, wide, table(off))
        torch.cuda.synchronize()
        ref.check_gated(got[-8:].cpu(), None, None, x, bg[1:], bg[1:], [0, 8], 0, ref.SILU, "bf16")
        assert not got[:-8].any()


# ---- the operators one after the other ------------------------------------------------------------
class Block:
    """A gated block whose three projections have adapters, trained: gate and up in one adapted
    projection, the gate, an adapted down projection; and back."""

    def __init__(self, rows=300, D=136, H=264, G=3, rank=12, dt="bf16"):
        self.dims, self.dt = (rows, D, H, G, rank), dt
        self.order = torch.randperm(rows, generator=torch.Generator().manual_seed(1))
        self.offsets = [0, rows // 3, rows // 3, rows - 20]
        make = lambda *s, seed, scale: normal(*s, dtype=dt, seed=seed, scale=scale).cuda()  # noqa: E731
        self.x, self.d_y = make(rows, D, seed=1, scale=1), make(rows, D, seed=2, scale=1)
        self.w1, self.a1, self.b1 = (make(2 * H, D, seed=3, scale=D ** -0.5), make(G, rank, D, seed=4, scale=D ** -0.5),
                                     make(G, 2 * H, rank, seed=5, scale=rank ** -0.5))
        self.w2, self.a2, self.b2 = (make(D, H, seed=6, scale=H ** -0.5), make(G, rank, H, seed=7, scale=H ** -0.5),
                                     make(G, D, rank, seed=8, scale=rank ** -0.5))
        self.scales = torch.tensor([0.5, 1.0, 2.0]).cuda()
        empty = lambda *s: torch.empty(*s, dtype=TYPES[dt], device="cuda")  # noqa: E731
        self.uv, self.h, self.y, self.t1, self.t2 = empty(rows, 2 * H), empty(rows, H), empty(rows, D), empty(rows, rank), empty(rows, rank)
        self.d_h, self.d_uv, self.d_x, self.dt1, self.dt2 = empty(rows, H), empty(rows, 2 * H), empty(rows, D), empty(rows, rank), empty(rows, rank)
        self.grads = [torch.empty(m.shape, device="cuda") for m in (self.a1, self.b1, self.a2, self.b2)]
        size = max(tg.tile_gemm_adapters_workspace_size(G, rows, n, k, rank, dt, transposed=t)
                   for n, k, t in ((2 * H, D, 1), (D, H, 1), (H, D, 0), (D, 2 * H, 0)))
        size = max(size, tg.tile_gemm_adapters_wgrad_workspace_size(G, rows, 2 * H, D, rank, dt),
                   tg.tile_gemm_adapters_wgrad_workspace_size(G, rows, D, H, rank, dt))
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        self.off, self.table = table(self.offsets), table(self.order.tolist())
        self.outs = [self.y, self.uv, self.h, self.d_x, self.d_uv, *self.grads]

    def adapted(self, x, w, a, b, y, t, N, K, transposed, **kw):
        rows, _, _, G, rank = self.dims
        tg.tile_gemm_adapters(G, rows, N, K, rank, self.dt, x, K, w, w.stride(0), a, a.stride(1), a.stride(0), b, b.stride(1),
                              b.stride(0), y, N, self.off, self.ws, order=self.table, scales=self.scales,
                              transposed=transposed, T=t, ldt=rank, **kw)

    def call(self, stream=None):
        rows, D, H, G, rank = self.dims
        s = dict(stream=stream)
        self.adapted(self.x, self.w1, self.a1, self.b1, self.uv, self.t1, 2 * H, D, 1, **s)
        u, v = self.uv, self.uv[:, H:]
        tg.tile_gemm_gate(rows, H, self.dt, u, v, 2 * H, self.h, H, **s)
        self.adapted(self.h, self.w2, self.a2, self.b2, self.y, self.t2, D, H, 1, **s)
        self.adapted(self.d_y, self.w2, self.b2, self.a2, self.d_h, self.dt2, H, D, 0, **s)
        tg.tile_gemm_gate_grad(rows, H, self.dt, self.d_h, H, u, v, 2 * H, self.d_uv, self.d_uv[:, H:], 2 * H, **s)
        self.adapted(self.d_uv, self.w1, self.b1, self.a1, self.d_x, self.dt1, D, 2 * H, 0, **s)
        ga1, gb1, ga2, gb2 = self.grads
        for N, K, x, d, t, d_t, ga, gb in ((2 * H, D, self.x, self.d_uv, self.t1, self.dt1, ga1, gb1),
                                           (D, H, self.h, self.d_y, self.t2, self.dt2, ga2, gb2)):
            tg.tile_gemm_adapters_wgrad(G, rows, N, K, rank, self.dt, x, K, d, N, t, rank, d_t, rank, ga, K, rank * K, gb, rank,
                                        N * rank, self.off, self.ws, order=self.table, transposed=1, **s)

    def plain(self):
        """The block in 64 bits, differentiated by torch (on the CPU)."""
        rows, D, H, G, rank = self.dims
        leaves = [m.cpu().double().requires_grad_() for m in (self.x, self.a1, self.b1, self.a2, self.b2)]
        x, a1, b1, a2, b2 = leaves
        w1, w2 = self.w1.cpu().double(), self.w2.cpu().double()
        which = torch.full((rows,), G)
        for g in range(G):
            which[self.order[self.offsets[g]:self.offsets[g + 1]]] = g

        def project(x, w, a, b):
            y = x @ w.t()
            for g in range(G):
                mine = (which == g).double()[:, None]
                y = y + mine * (float(self.scales[g]) * (x @ a[g].t()) @ b[g].t())
            return y

        uv = project(x, w1, a1, b1)
        y = project(torch.nn.functional.silu(uv[:, :H]) * uv[:, H:], w2, a2, b2)
        y.backward(self.d_y.cpu().double())
        return y.detach(), [leaf.grad for leaf in leaves]


def far(got, want):
    return float((got.cpu().double() - want).norm() / want.norm())


@pytest.mark.parametrize("rows,dt", [(300, "bf16"), (40, "bf16"), (300, "f32"), (7, "f16")])
def test_a_block_with_adapters_is_trained(rows, dt):
    """Roundings of independent elements add in squares: forward four (u and v, h, y; t) leave at most
    sqrt(5) half steps of the type in the 2-norm, and back twice as many sqrt(10), an error of the
    gate's argument doubled; fp32 sums of up to 528 terms stay below 1e-5."""
    b = Block(rows=rows, dt=dt)
    if rows < 30:
        b.offsets = [0, 2, 2, rows - 1]
        b.off = table(b.offsets)
    b.call()
    torch.cuda.synchronize()
    y, (d_x, *grads) = b.plain()
    half = torch.finfo(TYPES[dt]).eps / 2
    assert far(b.y, y) < 5 ** 0.5 * half + 1e-5
    for got, want in zip([b.d_x, *b.grads], [d_x, *grads]):
        assert far(got, want) < 2 * 10 ** 0.5 * half + 1e-5
    assert not b.grads[0][1].any() and not b.grads[1][1].any()         # an adapter without a row


def test_same_results_again_on_another_stream_and_in_a_graph():
    rows, D, H, E = 300, 136, 264, 4
    b = Block()
    w = [normal(E, D, H, dtype="bf16", seed=s, scale=D ** -0.5).cuda() for s in (21, 22)]
    w2 = normal(E, H, D, dtype="bf16", seed=23, scale=H ** -0.5).cuda()
    off = table([0, 20, 20, 200, 290])
    outs = [torch.empty(rows, H, dtype=torch.bfloat16, device="cuda") for _ in range(5)]
    few = torch.empty(16, 2048, dtype=torch.bfloat16, device="cuda")
    x16 = normal(16, 2048, dtype="bf16", seed=24).cuda()
    w16 = normal(2, 2048, 2048, dtype="bf16", seed=25, scale=2048 ** -0.5).cuda()
    size = tg.tile_gemm_gated_workspace_size(1, 16, 2048, 2048, "bf16")
    assert size > 0
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def call(stream=None):
        h, u, v, du, dv = outs
        b.call(stream)
        tg.tile_gemm_gated(E, rows, H, D, "bf16", b.x, D, w[0], w[1], H, D * H, h, H, off, U=u, V=v, ldu=H, stream=stream)
        tg.tile_gemm_gated_grad(E, rows, H, D, "bf16", b.d_y, D, w2, D, H * D, u, v, H, du, dv, H, off, transposed=1,
                                stream=stream)
        tg.tile_gemm_gated(1, 16, 2048, 2048, "bf16", x16, 2048, w16[0], w16[1], 2048, 0, few, 2048, workspace=ws, stream=stream)

    every = [*b.outs, *outs, few]
    call()
    torch.cuda.synchronize()
    want = [o.clone() for o in every]
    assert all(bool(torch.isfinite(o.float()).all()) for o in want)

    def spoil():
        for o in every:
            o.fill_(-7)
        torch.cuda.synchronize()

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(o, x) for o, x in zip(every, want))

    spoil()
    call()
    assert same()
    side = torch.cuda.Stream()
    spoil()
    call(stream=side)
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for _ in range(3):
        spoil()
        graph.replay()
        assert same()
        spoil()
        call()
        assert same()


def test_gradients_against_differences():
    """fp32 central differences of <d_y, block(x)> along random directions; the step's error is of second
    order in it (1e-2, third derivatives of order 1), the sums' 2^-24 times a few thousand terms over the step."""
    rows, D, H, E = 60, 24, 40, 3
    x, d_y = normal(rows, D, dtype="f32", seed=1).cuda(), normal(rows, D, dtype="f32", seed=2, scale=0.1).cuda()
    wg, wu = (normal(E, D, H, dtype="f32", seed=s, scale=D ** -0.5).cuda() for s in (3, 4))
    w2 = normal(E, H, D, dtype="f32", seed=5, scale=H ** -0.5).cuda()
    off = table([0, 25, 25, 60])

    def forward(x, wg, wu):
        h, u, v = (torch.empty(rows, H, device="cuda") for _ in range(3))
        tg.tile_gemm_gated(E, rows, H, D, "f32", x, D, wg, wu, H, D * H, h, H, off, U=u, V=v, ldu=H, activation=tg.ACT_GELU)
        y = torch.empty(rows, D, device="cuda")
        tg.tile_gemm_grouped(E, rows, D, H, "f32", h, H, w2, D, H * D, y, D, off)
        return (y.double() * d_y.double()).sum(), u, v

    _, u, v = forward(x, wg, wu)
    d_uv = torch.empty(rows, 2 * H, device="cuda")
    tg.tile_gemm_gated_grad(E, rows, H, D, "f32", d_y, D, w2, D, H * D, u, v, H, d_uv, d_uv[:, H:], 2 * H, off,
                            activation=tg.ACT_GELU, transposed=1)
    both = torch.cat([wg, wu], dim=2).contiguous()
    d_x, d_w = torch.empty(rows, D, device="cuda"), torch.empty(E, D, 2 * H, device="cuda")
    tg.tile_gemm_grouped(E, rows, D, 2 * H, "f32", d_uv, 2 * H, both, 2 * H, D * 2 * H, d_x, D, off, transposed=1)
    tg.tile_gemm_grouped_wgrad(E, rows, D, 2 * H, "f32", x, D, d_uv, 2 * H, d_w, 2 * H, D * 2 * H, off)
    step = 1e-2
    for i, (leaf, grad) in enumerate(((x, d_x), (wg, d_w[..., :H]), (wu, d_w[..., H:]))):
        direction = normal(*leaf.shape, dtype="f32", seed=30 + i).cuda()
        direction /= direction.norm()
        args = [x, wg, wu]
        args[i] = leaf + step * direction
        up = forward(*args)[0]
        args[i] = leaf - step * direction
        down = forward(*args)[0]
        got = float((grad.double() * direction.double()).sum())
        assert abs(float(up - down) / (2 * step) - got) < 20 * step ** 2 + 4096 * 2.0 ** -24 / step
