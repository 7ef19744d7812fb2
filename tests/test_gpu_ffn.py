"""The operators of a feed-forward block on the GPU, through the C ABI, against plain forms in 64
bits (tests/ffn_ref.py, which derives the bounds).

Inputs of small whole numbers have exact results in any order of summation and are compared bit
for bit.  Outputs lie between guard values, start as NaN, and rows are padded; what must not be
read (row padding, rows of no expert) is NaN.
"""
import pytest
import torch

import tile_scheduled_dense_amd as tg
from tests import ffn_ref as ref
from tests.gpu_util import need_gpu
from tests.test_gpu_experts import Out, ints, normal, offsets_of, sizes_of, strided

pytestmark = pytest.mark.gpu
TYPES = ref.TYPES


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def table(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def scratch(size):
    """A workspace of NaN between guards; `check` says whether the guards are whole."""
    buf = torch.full((size + 512,), 0xff, dtype=torch.uint8, device="cuda")

    def check():
        assert bool((buf[:256] == 0xff).all()) and bool((buf[256 + size:] == 0xff).all()), "a write outside the workspace"

    return (buf[256:256 + size] if size else None), check


def thin(t, share, seed=5):
    """All but a share of the values 0, so that sums of whole numbers stay small."""
    return t * (torch.rand(t.shape, generator=torch.Generator().manual_seed(seed)) < share).to(t.dtype)


# ---- the gated pair -----------------------------------------------------------------------
GATED = [
    # dtype, experts, rows, spare, active, N, K, pad, skew
    ("bf16", 1, 1, 0, 1, 64, 128, 0, 0), ("bf16", 1, 1, 0, 1, 1, 1, 0, 0), ("f16", 1, 3, 0, 1, 7, 9, 1, 1),
    ("f32", 1, 5, 0, 1, 3, 5, 2, 1), ("bf16", 8, 32, 0, 7, 256, 128, 0, 0), ("bf16", 3, 5, 2, 2, 72, 40, 0, 0),
    ("f16", 1, 48, 0, 1, 520, 1024, 0, 0), ("f32", 2, 17, 3, 1, 100, 1000, 0, 0), ("bf16", 1, 2, 0, 1, 40, 2056, 8, 0),
    ("bf16", 5, 700, 0, 4, 136, 264, 0, 0), ("f16", 3, 500, 0, 3, 200, 257, 0, 0), ("bf16", 2, 1000, 7, 2, 300, 72, 8, 0),
    ("f16", 1, 257, 0, 1, 258, 31, 0, 0), ("bf16", 2, 600, 0, 2, 520, 33, 0, 1), ("f32", 3, 400, 3, 3, 264, 100, 0, 0),
    ("f32", 2, 300, 0, 2, 129, 17, 1, 0), ("bf16", 4, 64, 4, 0, 40, 40, 0, 0), ("bf16", 2, 400, 0, 2, 96, 0, 0, 0),
    ("f32", 1, 200, 0, 1, 512, 64, 0, 0), ("bf16", 1, 300, 0, 1, 5, 64, 0, 0), ("f16", 90, 300, 9, 60, 72, 64, 0, 0),
]


def gated_case(dt, experts, rows, spare, active, N, K, pad, skew, transposed, kind, save, exact, split):
    offsets = offsets_of(sizes_of(experts, rows, active, seed=rows))
    total = rows + spare
    shape = (experts, N, K) if transposed else (experts, K, N)
    if exact:
        x = thin(ints(total, K, dtype=dt, low=-1, high=2, seed=1), min(1.0, 12 / max(K, 1)))
        bg, bu = (ints(*shape, dtype=dt, low=-1, high=2, seed=s) for s in (2, 3))
    else:
        x = normal(total, K, dtype=dt, seed=1)
        bg, bu = (normal(*shape, dtype=dt, seed=s, scale=max(K, 1) ** -0.5) for s in (2, 3))
    x[offsets[-1]:] = float("nan")
    xd, lda = strided(x, pad, skew)
    gd, ldb = strided(bg, pad, skew)
    ud, _ = strided(bu, pad, skew)
    h = Out(total, N, TYPES[dt], pad, skew=skew)
    u = Out(total, N, TYPES[dt], pad + (8 if pad else 0), skew=skew) if save else None
    v = Out(total, N, TYPES[dt], pad + (8 if pad else 0), skew=skew) if save else None
    ws, whole = scratch(tg.tile_gemm_gated_workspace_size(experts, total, N, K, dt, transposed=transposed) if split else 0)
    tg.tile_gemm_gated(experts, total, N, K, dt, xd, lda, gd, ud, ldb, shape[1] * ldb, h.t, h.ld,
                       table(offsets) if experts > 1 or spare else None, activation=kind, transposed=transposed,
                       U=u.t if save else None, V=v.t if save else None, ldu=u.ld if save else 0, workspace=ws)
    h, u, v = h.get(), u.get() if save else None, v.get() if save else None
    whole()
    x[offsets[-1]:] = 0
    if exact:
        want = ref.gated(x, bg, bu, offsets, transposed)
        f, _ = ref.act(want[0], kind)
        assert float((f * want[1]).abs().max() if want[0].numel() else 0) <= 256
        assert torch.equal(h.double(), f * want[1])
        if save:
            assert torch.equal(u.double(), want[0]) and torch.equal(v.double(), want[1])
    else:
        ref.check_gated(h, u, v, x, bg, bu, offsets, transposed, kind, dt)


@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("dt,experts,rows,spare,active,N,K,pad,skew", GATED, ids=lambda v: str(v))
def test_gated(dt, experts, rows, spare, active, N, K, pad, skew, transposed):
    args = (dt, experts, rows, spare, active, N, K, pad, skew, transposed)
    gated_case(*args, kind=ref.RELU, save=True, exact=True, split=True)
    gated_case(*args, kind=ref.NONE, save=False, exact=True, split=False)
    gated_case(*args, kind=ref.SILU, save=True, exact=False, split=True)
    gated_case(*args, kind=ref.GELU, save=False, exact=False, split=False)


def gate_grad_case(dt, experts, rows, spare, active, N, K, pad, skew, transposed, kind, with_h, exact):
    offsets = offsets_of(sizes_of(experts, rows, active, seed=rows))
    total = rows + spare
    shape = (experts, N, K) if transposed else (experts, K, N)
    if exact:
        d = thin(ints(total, K, dtype=dt, low=-1, high=2, seed=1), min(1.0, 12 / max(K, 1)))
        b = ints(*shape, dtype=dt, low=-1, high=2, seed=2)
        u, v = (ints(total, N, dtype=dt, low=-2, high=3, seed=s) for s in (3, 4))
    else:
        d = normal(total, K, dtype=dt, seed=1)
        b = normal(*shape, dtype=dt, seed=2, scale=max(K, 1) ** -0.5)
        u, v = (normal(total, N, dtype=dt, seed=s, scale=2.0) for s in (3, 4))
    for t in (d, u, v):
        t[offsets[-1]:] = float("nan")
    dd, ldd = strided(d, pad, skew)
    bd, ldb = strided(b, pad, skew)
    ud, ldu = strided(u, pad, skew)
    vd, _ = strided(v, pad, skew)
    du, dv = (Out(total, N, TYPES[dt], pad + (8 if pad else 0), skew=skew) for _ in range(2))
    h = Out(total, N, TYPES[dt], pad, skew=skew) if with_h else None
    tg.tile_gemm_gated_grad(experts, total, N, K, dt, dd, ldd, bd, ldb, shape[1] * ldb, ud, vd, ldu, du.t, dv.t, du.ld,
                            table(offsets) if experts > 1 or spare else None, activation=kind, transposed=transposed,
                            H=h.t if with_h else None, ldh=h.ld if with_h else 0)
    du, dv, h = du.get(), dv.get(), h.get() if with_h else None
    d[offsets[-1]:] = 0
    live = torch.arange(total) < offsets[-1]
    zeros = torch.zeros_like(b)
    d_h, _, s, _ = ref.gated(d, b, zeros, offsets, transposed)
    if exact:
        u, v = (torch.where(live[:, None], t.double(), 0) for t in (u, v))
        f, slope = ref.act(u, kind)
        assert float(d_h.abs().max() if d_h.numel() else 0) * 4 <= 256
        assert torch.equal(du.double(), d_h * v * slope) and torch.equal(dv.double(), d_h * f)
        assert h is None or torch.equal(h.double(), f * v)
    else:
        ref.check_gate_grad(du, dv, h, d_h, s, K, u, v, live, kind, dt)


@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("dt,experts,rows,spare,active,N,K,pad,skew", GATED, ids=lambda v: str(v))
def test_gated_grad(dt, experts, rows, spare, active, N, K, pad, skew, transposed):
    args = (dt, experts, rows, spare, active, N, K, pad, skew, transposed)
    gate_grad_case(*args, kind=ref.RELU, with_h=True, exact=True)
    gate_grad_case(*args, kind=ref.NONE, with_h=False, exact=True)
    gate_grad_case(*args, kind=ref.SILU, with_h=True, exact=False)
    gate_grad_case(*args, kind=ref.GELU, with_h=False, exact=False)


# ---- adapters -------------------------------------------------------------------------------
ADAPTERS = [
    # dtype, adapters, rows, without, active, N, K, rank, pad, skew
    ("bf16", 8, 1, 0, 1, 256, 512, 16, 0, 0), ("bf16", 1, 1, 1, 0, 8, 8, 8, 0, 0), ("f16", 2, 3, 1, 2, 7, 9, 3, 1, 1),
    ("f32", 3, 6, 2, 2, 5, 3, 1, 2, 1), ("bf16", 32, 64, 7, 20, 512, 1024, 32, 0, 0), ("f16", 5, 40, 0, 5, 1000, 264, 5, 0, 0),
    ("f32", 4, 33, 5, 3, 130, 257, 12, 0, 0), ("bf16", 3, 300, 0, 3, 264, 264, 16, 0, 0), ("f16", 4, 513, 50, 4, 520, 72, 64, 8, 0),
    ("bf16", 70, 700, 20, 60, 136, 96, 8, 0, 0), ("f16", 2, 260, 0, 2, 258, 31, 33, 0, 1), ("f32", 41, 400, 21, 37, 264, 101, 5, 0, 0),
    ("f32", 2, 130, 3, 1, 129, 64, 70, 1, 0), ("bf16", 2, 300, 100, 0, 96, 64, 4, 0, 0), ("bf16", 3, 200, 0, 2, 4, 64, 8, 0, 0),
    ("bf16", 2, 200, 0, 2, 64, 0, 8, 0, 0), ("f16", 2, 200, 0, 2, 64, 40, 0, 0, 0), ("bf16", 300, 520, 5, 200, 128, 64, 16, 0, 0),
    ("bf16", 2, 20, 0, 2, 64, 48, 300, 0, 0),
]


class AdapterCase:
    def __init__(self, dt, adapters, rows, without, active, N, K, rank, pad, skew, transposed, shuffled, exact, scaled=True):
        self.__dict__.update(dt=dt, adapters=adapters, rows=rows, N=N, K=K, rank=rank, pad=pad, skew=skew, tr=transposed)
        g = torch.Generator().manual_seed(rows + N)
        sizes = sizes_of(adapters, rows - without, active, seed=rows) if active else [0] * adapters
        self.offsets = offsets_of(sizes)
        self.order = torch.randperm(rows, generator=g) if shuffled else None

        def matrix(inputs, outputs, seed, scale=1.0, batch=None):
            shape = ([batch] if batch else []) + ([outputs, inputs] if transposed else [inputs, outputs])
            return ints(*shape, dtype=dt, low=-1, high=2, seed=seed) if exact else normal(*shape, dtype=dt, seed=seed, scale=scale)

        if exact:
            self.x = thin(ints(rows, K, dtype=dt, low=-1, high=2, seed=1), min(1.0, 6 / max(K, 1)))
        else:
            self.x = normal(rows, K, dtype=dt, seed=1)
        self.w = matrix(K, N, 2, max(K, 1) ** -0.5)
        self.a = matrix(K, rank, 3, max(K, 1) ** -0.5, adapters)
        self.b = matrix(rank, N, 4, max(rank, 1) ** -0.5, adapters)
        if exact:
            self.b = thin(self.b, min(1.0, 16 / max(rank, 1)))
        self.scales = None
        if scaled:
            self.scales = torch.randint(1, 3, (adapters,), generator=g).float() if exact else torch.rand(adapters, generator=g) + 0.5

    def run(self, save=True):
        c = self
        xd, ldx = strided(c.x, c.pad, c.skew)
        wd, ldw = strided(c.w, c.pad, c.skew)
        ad, lda = strided(c.a, c.pad, c.skew)
        bd, ldb = strided(c.b, c.pad, c.skew)
        y = Out(c.rows, c.N, TYPES[c.dt], c.pad, skew=c.skew)
        t = Out(c.rows, c.rank, TYPES[c.dt], c.pad + 1, skew=c.skew) if save and c.rank else None
        ws, whole = scratch(tg.tile_gemm_adapters_workspace_size(c.adapters, c.rows, c.N, c.K, c.rank, c.dt, transposed=c.tr))
        order = None
        if c.order is not None:        # some entries complemented, as the sort's table has them for rows without a group
            order = table(torch.where(torch.arange(c.rows) % 3 == 0, ~c.order, c.order).tolist())
        tg.tile_gemm_adapters(c.adapters, c.rows, c.N, c.K, c.rank, c.dt, xd, ldx, wd, ldw, ad, lda, c.a.shape[1] * lda, bd,
                              ldb, c.b.shape[1] * ldb, y.t, y.ld, table(c.offsets), ws, order=order,
                              scales=None if c.scales is None else c.scales.cuda(), transposed=c.tr, T=t.t if t else None,
                              ldt=t.ld if t else 0)
        y, t = y.get(), t.get() if t else None
        whole()
        return y, t


@pytest.mark.parametrize("shuffled", [False, True])
@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("dt,adapters,rows,without,active,N,K,rank,pad,skew", ADAPTERS, ids=lambda v: str(v))
def test_adapters(dt, adapters, rows, without, active, N, K, rank, pad, skew, transposed, shuffled):
    for exact in (True, False):
        c = AdapterCase(dt, adapters, rows, without, active, N, K, rank, pad, skew, transposed, shuffled, exact, scaled=exact or not shuffled)
        y, t = c.run(save=exact or not transposed)
        want, y_err, want_t, t_err = ref.adapters(c.x, c.w, c.a, c.b, c.scales, c.offsets, c.order, transposed, dt)
        if exact:
            assert float(want.abs().max() if want.numel() else 0) <= 256
            assert torch.equal(y.double(), want)
            assert t is None or torch.equal(t.double(), want_t)
        else:
            ref.check(y, want, y_err, dt, "y")
            if t is not None:
                ref.check(t, want_t, t_err, dt, "t")


@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("shuffled", [False, True])
@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("dt,adapters,rows,without,active,N,K,rank,pad,skew", ADAPTERS, ids=lambda v: str(v))
def test_adapters_wgrad(dt, adapters, rows, without, active, N, K, rank, pad, skew, transposed, shuffled, out):
    if out == "f32" and dt == "f32":
        pytest.skip("the same case")
    o = dt if out == "same" else "f32"
    c = AdapterCase(dt, adapters, rows, without, active, N, K, rank, pad, skew, transposed, shuffled, True)
    for exact in (True, False):
        if exact:
            x, dy, t, dt_ = (thin(ints(rows, n, dtype=dt, low=-1, high=2, seed=s), min(1.0, 100 / rows))
                             for s, n in enumerate((K, N, rank, rank)))
        else:
            x, dy, t, dt_ = (normal(rows, n, dtype=dt, seed=s) for s, n in enumerate((K, N, rank, rank)))
        if without:        # rows of no adapter take no part
            none = torch.arange(c.offsets[-1], rows)
            none = none if c.order is None else c.order[none]
            for m in (x, dy, t, dt_):
                m[none] = float("nan")
        dev = [strided(m, pad, skew) for m in (x, dy, t, dt_)]
        a_shape, b_shape = ((rank, K), (N, rank)) if transposed else ((K, rank), (rank, N))
        da, db = (Out(*s, TYPES[o], pad, batch=adapters, skew=skew) for s in (a_shape, b_shape))
        ws, whole = scratch(tg.tile_gemm_adapters_wgrad_workspace_size(adapters, rows, N, K, rank, dt))
        tg.tile_gemm_adapters_wgrad(adapters, rows, N, K, rank, dt, *[v for m in dev for v in m], da.t, max(da.ld, 1), da.stride, db.t,
                                    max(db.ld, 1), db.stride, table(c.offsets), ws,
                                    order=None if c.order is None else table(c.order.tolist()), c_dtype=o,
                                    transposed=transposed)
        if rank == 0:
            return
        for got, L, S, flip, what in ((da, x, dt_, transposed, "d_a"), (db, dy, t, not transposed, "d_b")):
            got = got.get().reshape(adapters, *(a_shape if what == "d_a" else b_shape))
            want, absum, terms = ref.adapters_wgrad(L, S, c.offsets, c.order)
            if flip:
                want, absum = want.transpose(1, 2), absum.transpose(1, 2)
            if exact:
                assert float(absum.max() if absum.numel() else 0) <= 256
                assert torch.equal(got.double(), want)
            else:
                ref.check(got, want, ref.sum_error(terms, absum), o, what)
        whole()
