"""The mixture-of-experts operators on the GPU, through the C ABI, against plain forms in 64 bits
(tests/expert_ref.py, which derives the bounds).

Inputs of small whole numbers have exact results in any order of summation, so they are compared
bit for bit: they pin addressing, masks, layouts and the order of rows.  Outputs lie between guard
values, start as NaN (what must be written shows), and rows are padded.
"""
import numpy as np
import pytest
import torch

import tile_scheduled_dense_amd as tg
from tests import expert_ref as ref
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu
TYPES = ref.TYPES
GUARD = 512


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


class Out:
    """A rows x cols output at row stride ld, NaN inside, guard values around and in the padding."""

    def __init__(self, rows, cols, dtype, pad=0, batch=1, skew=0):
        self.rows, self.cols, self.ld, self.batch = rows, cols, cols + pad, batch
        self.stride = rows * self.ld
        n = batch * self.stride
        self.buf = torch.full((n + 2 * GUARD + skew,), 77.0, dtype=dtype, device="cuda")
        self.t = self.buf[GUARD + skew:GUARD + skew + n]
        self.view().fill_(float("nan"))

    def view(self):
        return torch.as_strided(self.t, (self.batch, self.rows, self.cols), (self.stride, self.ld, 1))

    def get(self):
        torch.cuda.synchronize()
        res = self.view().clone()
        self.view().fill_(77.0)
        assert bool((self.buf == 77.0).all()), "a write outside the output"
        self.view().copy_(res)
        return res.cpu() if self.batch > 1 else res[0].cpu()


def strided(x, pad, skew=0):
    """x (rows x cols, or batched) on the GPU with padded rows of NaN; returns the tensor and its row stride."""
    ld = max(x.shape[-1] + pad, 1)
    buf = torch.full((*x.shape[:-1], ld), float("nan"), dtype=x.dtype)
    buf[..., :x.shape[-1]] = x
    flat = torch.cat([torch.zeros(skew, dtype=x.dtype), buf.reshape(-1), torch.full((16,), float("nan"), dtype=x.dtype)])
    return flat.cuda()[skew:], ld


def ints(*shape, dtype, low=-3, high=4, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(low, high, shape, generator=g).to(TYPES[dtype])


def normal(*shape, dtype, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(TYPES[dtype])


def routing(tokens, top_k, experts, dropped, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, experts, (tokens, top_k), generator=g)
    ids[torch.rand(tokens, top_k, generator=g) < dropped] = -1
    return ids.to(torch.int32)


def offsets_of(sizes):
    out = [0]
    for n in sizes:
        out.append(out[-1] + n)
    return out


# ---- sort ---------------------------------------------------------------------------------
@pytest.mark.parametrize("tokens,top_k,experts,dropped,pad", [
    (0, 2, 8, 0, 0), (1, 1, 1, 0, 0), (1, 1, 8, 1.0, 0), (16, 2, 8, 0, 0), (63, 1, 2, 0.5, 3), (1024, 1, 3, 0.1, 0),
    (1025, 1, 9, 0.1, 0), (333, 11, 64, 0.3, 2), (2048, 2, 129, 0, 0), (2049, 2, 129, 0.1, 0), (8192, 2, 8, 0, 0),
    (1999, 8, 129, 0.1, 0), (16384, 8, 256, 0.05, 0), (9000, 8, 511, 0, 1), (300, 3, 512, 0, 0),
    (5000, 4, 2048, 0.2, 0), (70000, 2, 1, 0.5, 0),
])
def test_sort(tokens, top_k, experts, dropped, pad):
    ids = routing(tokens, top_k, experts, dropped, seed=tokens + experts)
    if tokens > 3:
        ids[3, 0] = experts              # the first id outside
        ids[2, 0] = -2 ** 31
        ids[1, 0] = 2 ** 31 - 1
    wide = torch.full((tokens, top_k + pad), 5, dtype=torch.int32)
    wide[:, :top_k] = ids
    wide = wide.cuda()
    n = tokens * top_k
    buf = [torch.full((m + 64,), -99, dtype=torch.int32, device="cuda") for m in (experts + 1, n, n)]
    ws = torch.full((tg.tile_gemm_expert_sort_workspace_size(tokens, top_k, experts) // 4 + 64,), -99,
                    dtype=torch.int32, device="cuda")
    tg.tile_gemm_expert_sort(tokens, top_k, experts, wide if n else None, top_k + pad, *buf, workspace=ws)
    torch.cuda.synchronize()
    want = ref.sort(ids, experts)
    for b, w in zip(buf, want):
        got = b.cpu().tolist()
        assert got[:len(w)] == w and got[len(w):] == [-99] * 64
    assert ws.cpu()[-64:].tolist() == [-99] * 64


# ---- rows ---------------------------------------------------------------------------------
EXCHANGE = [
    # dtype, tokens, top_k, experts, cols, dropped, pad
    ("bf16", 16, 2, 8, 1024, 0.0, 0), ("bf16", 5, 1, 4, 1, 0.0, 0), ("f16", 7, 3, 4, 7, 0.4, 1),
    ("f32", 33, 8, 129, 1001, 0.1, 0), ("f32", 9, 4, 8, 3, 0.3, 2), ("bf16", 20, 11, 16, 520, 0.2, 3),
    ("f16", 40, 2, 8, 2048, 0.0, 8), ("bf16", 3, 2, 8, 4100, 0.5, 0), ("f32", 6, 2, 2, 64, 1.0, 0),
    ("bf16", 130, 5, 8, 65, 0.1, 5),
]


@pytest.mark.parametrize("dt,tokens,top_k,experts,cols,dropped,pad", EXCHANGE, ids=lambda v: str(v))
def test_exchange(dt, tokens, top_k, experts, cols, dropped, pad):
    ids = routing(tokens, top_k, experts, dropped, seed=cols)
    _, entry_of_row, row_of_entry = ref.sort(ids, experts)
    n = tokens * top_k
    has = [r >= 0 for r in row_of_entry]
    rows_dev = torch.tensor(row_of_entry, dtype=torch.int32).cuda()
    x = normal(tokens, cols, dtype=dt, seed=1)
    # gather: a copy, bit for bit; zeros where there is no expert
    xd, ldx = strided(x, pad)
    out = Out(n, cols, TYPES[dt], pad)
    tg.tile_gemm_expert_gather(tokens, top_k, cols, dt, xd, ldx, rows_dev, out.t, out.ld)
    want = torch.stack([x[e // top_k] if e >= 0 else torch.zeros_like(x[0]) for e in entry_of_row])
    assert torch.equal(out.get(), want)
    # combine, weighted and not; what lies in rows without an expert is NaN
    y = normal(n, cols, dtype=dt, seed=2)
    for r, e in enumerate(entry_of_row):
        if e < 0:
            y[r] = float("nan")
    yd, ldy = strided(y, pad)
    w = torch.rand(tokens, top_k, generator=torch.Generator().manual_seed(3))
    w[~torch.tensor(has).reshape(tokens, top_k)] = float("nan")
    wd, ld_w = strided(w, 1)
    y64, w64 = y.double(), w.double()
    for weights in (True, False):
        out = Out(tokens, cols, TYPES[dt], pad)
        tg.tile_gemm_expert_combine(tokens, top_k, cols, dt, yd, ldy, rows_dev, wd if weights else None,
                                    ld_w if weights else 0, out.t, out.ld)
        want, absum = torch.zeros(tokens, cols, dtype=torch.float64), torch.zeros(tokens, cols, dtype=torch.float64)
        for e in range(n):
            if has[e]:
                f = w64[e // top_k, e % top_k] if weights else 1.0
                want[e // top_k] += f * y64[row_of_entry[e]]
                absum[e // top_k] += (f * y64[row_of_entry[e]]).abs()
        ref.check(out.get(), want, top_k, absum, dt)
    # the gradient
    g = normal(tokens, cols, dtype=dt, seed=4)
    gd, ldg = strided(g, pad)
    d_y, d_w = Out(n, cols, TYPES[dt], pad), Out(tokens, top_k, torch.float32, 2)
    tg.tile_gemm_expert_combine_grad(tokens, top_k, cols, dt, gd, ldg, yd, ldy, rows_dev, wd, ld_w, d_y.t, d_y.ld,
                                     d_w.t, d_w.ld)
    g64 = g.double()
    want_y, want_w = torch.zeros(n, cols, dtype=torch.float64), torch.zeros(tokens, top_k, dtype=torch.float64)
    abs_w = torch.zeros_like(want_w)
    for e in range(n):
        if has[e]:
            t, j = e // top_k, e % top_k
            want_y[row_of_entry[e]] = w64[t, j] * g64[t]
            want_w[t, j] = (g64[t] * y64[row_of_entry[e]]).sum()
            abs_w[t, j] = (g64[t] * y64[row_of_entry[e]]).abs().sum()
    ref.check(d_y.get(), want_y, 1, want_y.abs(), dt)
    ref.check(d_w.get(), want_w, cols, abs_w, "f32")


@pytest.mark.parametrize("dt,cols", [("bf16", 2048), ("f32", 1023)])
def test_exchange_of_much_data(dt, cols):
    """More bytes than the caches hold (results are then stored past them); the same on the GPU in 64 bits."""
    T, k, E = 6001, 3, 8
    ids = routing(T, k, E, 0.1, 5).cuda()
    n = T * k
    offsets, entry, row = (torch.empty(m, dtype=torch.int32, device="cuda") for m in (E + 1, n, n))
    ws = torch.empty(tg.tile_gemm_expert_sort_workspace_size(T, k, E) // 4, dtype=torch.int32, device="cuda")
    tg.tile_gemm_expert_sort(T, k, E, ids, k, offsets, entry, row, workspace=ws)
    x, y, d = (normal(m, cols, dtype=dt, seed=i).cuda() for i, m in enumerate((T, n, T)))
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(1)).cuda()
    rows, out, d_y, d_w = Out(n, cols, TYPES[dt]), Out(T, cols, TYPES[dt]), Out(n, cols, TYPES[dt]), Out(T, k, torch.float32)
    tg.tile_gemm_expert_gather(T, k, cols, dt, x, cols, row, rows.t, cols)
    tg.tile_gemm_expert_combine(T, k, cols, dt, y, cols, row, w, k, out.t, cols)
    tg.tile_gemm_expert_combine_grad(T, k, cols, dt, d, cols, y, cols, row, w, k, d_y.t, cols, d_w.t, k)
    at = row.long().reshape(T, k)
    has = at >= 0
    at = torch.where(has, at, ~at)
    token = torch.arange(T, device="cuda")[:, None].expand(T, k)
    want = torch.zeros(n, cols, dtype=x.dtype, device="cuda")
    want[at[has]] = x[token[has]]
    assert torch.equal(rows.get(), want.cpu())
    f = torch.where(has, w, 0).double()
    picked = torch.where(has[..., None], y[at].double(), 0)
    ref.check(out.get(), (picked * f[..., None]).sum(1).cpu(), k, (picked.abs() * f[..., None]).sum(1).cpu(), dt)
    want = torch.zeros(n, cols, dtype=torch.float64, device="cuda")
    want[at.reshape(-1)] = (d.double()[:, None, :] * f[..., None]).reshape(n, cols)
    ref.check(d_y.get(), want.cpu(), 1, want.abs().cpu(), dt)
    prod = picked * d.double()[:, None, :]
    ref.check(d_w.get(), prod.sum(2).cpu(), cols, prod.abs().sum(2).cpu(), "f32")


def test_combine_gradient_against_differences():
    """<d_out, combine(w, y)> is linear in w and in y: a central difference of any step is its gradient."""
    T, k, D = 12, 3, 40
    ids = routing(T, k, 5, 0.2, 7)
    row = torch.tensor(ref.sort(ids, 5)[2], dtype=torch.int32).cuda()
    y, w, d = (normal(*s, dtype="f32", seed=i).cuda() for i, s in enumerate([(T * k, D), (T, k), (T, D)]))

    def loss(w, y):
        out = torch.empty(T, D, device="cuda")
        tg.tile_gemm_expert_combine(T, k, D, "f32", y, D, row, w, k, out, D)
        return float((out.double() * d.double()).sum())

    d_y, d_w = torch.empty(T * k, D, device="cuda"), torch.empty(T, k, device="cuda")
    tg.tile_gemm_expert_combine_grad(T, k, D, "f32", d, D, y, D, row, w, k, d_y, D, d_w, k)
    dir_w, dir_y = normal(T, k, dtype="f32", seed=8).cuda(), normal(T * k, D, dtype="f32", seed=9).cuda()
    # two losses of T * D terms of size ~ 3, each good to a few fp32 steps
    room = T * D * 3 * 16 * 2.0 ** -24
    assert abs((loss(w + dir_w, y) - loss(w - dir_w, y)) / 2 - float((d_w.double() * dir_w.double()).sum())) < room
    assert abs((loss(w, y + dir_y) - loss(w, y - dir_y)) / 2 - float((d_y.double() * dir_y.double()).sum())) < room


# ---- products -----------------------------------------------------------------------------
def sizes_of(experts, rows, active, seed):
    g = torch.Generator().manual_seed(seed)
    which = torch.randperm(experts, generator=g)[:active]
    sizes = torch.zeros(experts, dtype=torch.int64)
    if active:
        cuts = torch.randint(0, active, (rows,), generator=g)
        sizes[which] = torch.bincount(cuts, minlength=active)
    return sizes.tolist()


GROUPED = [
    # dtype, experts, rows, spare rows (of no expert), active, N, K, pad, skew
    ("bf16", 8, 32, 0, 7, 256, 128, 0, 0), ("bf16", 3, 5, 2, 2, 1, 1, 0, 0), ("f16", 4, 40, 3, 3, 7, 9, 1, 1),
    ("f32", 4, 50, 0, 4, 3, 5, 2, 1), ("f32", 2, 70, 5, 1, 130, 257, 0, 0), ("bf16", 5, 300, 0, 4, 136, 264, 0, 0),
    ("f16", 33, 500, 0, 29, 200, 257, 0, 0), ("bf16", 4, 1000, 7, 3, 300, 72, 8, 0), ("f16", 1, 257, 0, 1, 258, 31, 0, 0),
    ("bf16", 2, 600, 0, 2, 520, 33, 0, 1), ("f32", 3, 400, 3, 3, 264, 100, 0, 0), ("f32", 2, 300, 0, 2, 129, 17, 1, 0),
    ("bf16", 4, 64, 4, 0, 40, 40, 0, 0), ("bf16", 64, 128, 0, 50, 64, 96, 0, 0), ("f16", 2, 513, 0, 2, 256, 256, 0, 0),
    ("bf16", 3, 900, 0, 3, 512, 320, 0, 0), ("f32", 2, 520, 0, 2, 512, 64, 0, 0), ("bf16", 300, 700, 0, 200, 24, 24, 0, 0),
    ("bf16", 2, 50, 0, 2, 96, 0, 0, 0),
]


@pytest.mark.parametrize("transposed", [0, 1])
@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("dt,experts,rows,spare,active,N,K,pad,skew", GROUPED, ids=lambda v: str(v))
def test_grouped(dt, experts, rows, spare, active, N, K, pad, skew, out, transposed):
    if out == "f32" and dt == "f32":
        pytest.skip("the same case")
    o = dt if out == "same" else "f32"
    offsets = offsets_of(sizes_of(experts, rows, active, seed=rows))
    total = rows + spare
    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    for exact in (True, False):
        # whole numbers: a 16-bit result holds them up to 2^8 (bf16), so few terms are not 0
        if exact:
            A = ints(total, K, dtype=dt, low=-1, high=2, seed=1)
            B = ints(experts, *((N, K) if transposed else (K, N)), dtype=dt, low=-1, high=2, seed=2)
            A = A * (torch.rand(A.shape, generator=torch.Generator().manual_seed(5)) < 100 / max(K, 100)).to(A.dtype)
        else:
            A = normal(total, K, dtype=dt, seed=3)
            B = normal(experts, *((N, K) if transposed else (K, N)), dtype=dt, seed=4)
        A[offsets[-1]:] = float("nan")
        want, absum = ref.grouped(A, B, offsets, total, transposed)
        Ad, lda = strided(A, pad, skew)
        Bd, ldb = strided(B, pad, skew)
        C = Out(total, N, TYPES[o], pad, skew=skew)
        sB = B.shape[1] * ldb
        tg.tile_gemm_grouped(experts, total, N, K, dt, Ad, lda, Bd, ldb, sB, C.t, C.ld, off, c_dtype=o,
                             transposed=transposed)
        got = C.get()
        if exact:
            assert float(absum.max() if absum.numel() else 0) <= 256
            assert torch.equal(got.double(), want)
        else:
            ref.check(got, want, K, absum, o)


@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("dt,experts,rows,spare,active,N,K,pad,skew", GROUPED, ids=lambda v: str(v))
def test_wgrad(dt, experts, rows, spare, active, N, K, pad, skew, out):
    if out == "f32" and dt == "f32":
        pytest.skip("the same case")
    o = dt if out == "same" else "f32"
    offsets = offsets_of(sizes_of(experts, rows, active, seed=rows))
    total = rows + spare
    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    M = max(K, 1)
    for exact in (True, False):
        if exact:
            A, D = ints(total, M, dtype=dt, low=-1, high=2, seed=1), ints(total, N, dtype=dt, low=-1, high=2, seed=2)
            A = A * (torch.rand(A.shape, generator=torch.Generator().manual_seed(5)) < 100 / max(rows, 100)).to(A.dtype)
        else:
            A, D = normal(total, M, dtype=dt, seed=3), normal(total, N, dtype=dt, seed=4)
        A[offsets[-1]:] = float("nan")
        D[offsets[-1]:] = float("nan")
        want, absum = ref.wgrad(A, D, offsets)
        Ad, lda = strided(A, pad, skew)
        Dd, ldd = strided(D, pad, skew)
        C = Out(M, N, TYPES[o], pad, batch=experts, skew=skew)
        tg.tile_gemm_grouped_wgrad(experts, total, M, N, dt, Ad, lda, Dd, ldd, C.t, C.ld, C.stride, off, c_dtype=o)
        got = C.get().reshape(want.shape)
        if exact:
            assert float(absum.max() if absum.numel() else 0) <= 256
            assert torch.equal(got.double(), want)
        else:
            ref.check(got, want, rows, absum, o)


@pytest.mark.parametrize("form", ["nn", "nt", "tn"])
@pytest.mark.parametrize("dt,experts,rows,spare,N,K,pad", [
    # enough tiles for the largest ones, their pieces and a part-filled last round
    ("bf16", 5, 6500, 70, 2600, 200, 0), ("f16", 3, 7001, 0, 2307, 129, 1), ("f32", 6, 6400, 1, 2568, 72, 0),
    ("bf16", 80, 9000, 0, 2048, 64, 0),
], ids=lambda v: str(v))
def test_products_of_many_tiles(dt, experts, rows, spare, N, K, pad, form):
    offsets = offsets_of(sizes_of(experts, rows, experts - 1, seed=rows))
    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    total = rows + spare
    if form == "tn":
        M, N, total = 2 * K + 1600, N, total // 4
        offsets = [o // 4 for o in offsets]
        off = torch.tensor(offsets, dtype=torch.int32).cuda()
        experts = min(experts, 6)
        offsets, off = offsets[:experts + 1], off[:experts + 1]
        A, D = ints(total, M, dtype=dt, low=-1, high=2, seed=1), ints(total, N, dtype=dt, low=-1, high=2, seed=2)
        A[offsets[-1]:] = float("nan")
        want, _ = ref.wgrad(A, D, offsets)
        (Ad, lda), (Dd, ldd) = strided(A, pad), strided(D, pad)
        C = Out(M, N, torch.float32, pad, batch=experts)
        tg.tile_gemm_grouped_wgrad(experts, total, M, N, dt, Ad, lda, Dd, ldd, C.t, C.ld, C.stride, off)
    else:
        A, B = ints(total, K, dtype=dt, low=-1, high=2, seed=1), ints(experts, K, N, dtype=dt, low=-1, high=2, seed=2)
        A[offsets[-1]:] = float("nan")
        want, _ = ref.grouped(A, B, offsets, total)
        if form == "nt":
            B = B.transpose(1, 2).contiguous()
        (Ad, lda), (Bd, ldb) = strided(A, pad), strided(B, pad)
        C = Out(total, N, torch.float32, pad)
        tg.tile_gemm_grouped(experts, total, N, K, dt, Ad, lda, Bd, ldb, B.shape[1] * ldb, C.t, C.ld, off,
                             transposed=int(form == "nt"))
    assert torch.equal(C.get().double(), want)


@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
def test_products_larger_than_the_caches(dt, out):
    """Results stored past the caches, whole numbers against products in 64 bits on the GPU."""
    E, R, N, K = 3, 17000, 8192, 64
    offsets = [0, 5000, 5100, R]
    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    A, B = ints(R, K, dtype=dt, low=-1, high=2, seed=1).cuda(), ints(E, K, N, dtype=dt, low=-1, high=2, seed=2).cuda()
    C = torch.full((R, N), float("nan"), dtype=TYPES[out], device="cuda")
    tg.tile_gemm_grouped(E, R, N, K, dt, A, K, B, N, K * N, C, N, off, c_dtype=out)
    for g in range(E):
        lo, hi = offsets[g], offsets[g + 1]
        assert torch.equal(C[lo:hi].double(), A[lo:hi].double() @ B[g].double())
    C = torch.full((40, 1200, 3000), float("nan"), dtype=torch.float32, device="cuda")
    sizes = [13 * (g % 5) for g in range(40)]
    offsets = offsets_of(sizes)
    R = offsets[-1]
    A, D = ints(R, 1200, dtype=dt, low=-1, high=2, seed=3).cuda(), ints(R, 3000, dtype=dt, low=-1, high=2, seed=4).cuda()
    tg.tile_gemm_grouped_wgrad(40, R, 1200, 3000, dt, A, 1200, D, 3000, C, 3000, 1200 * 3000,
                               torch.tensor(offsets, dtype=torch.int32).cuda())
    for g in range(40):
        lo, hi = offsets[g], offsets[g + 1]
        assert torch.equal(C[g].double(), A[lo:hi].double().t().contiguous() @ D[lo:hi].double())


def test_grouped_nan_stays_in_its_row_and_column():
    """A NaN or an infinity in one row of A reaches that row alone; in one column of B, that column of its expert."""
    for dt in ("bf16", "f32"):
        for rows in (40, 700):
            offsets = [0, rows // 3, rows]
            A, B = normal(rows, 300, dtype=dt, seed=1), normal(2, 300, 260, dtype=dt, seed=2)
            A[5, 299] = float("nan")
            A[6, 0] = float("inf")
            B[1, 299, 259] = float("nan")
            C = Out(rows, 260, TYPES[dt])
            tg.tile_gemm_grouped(2, rows, 260, 300, dt, A.cuda(), 300, B.cuda(), 260, 300 * 260, C.t, 260,
                                 torch.tensor(offsets, dtype=torch.int32).cuda(), c_dtype=dt)
            bad = ~torch.isfinite(C.get())
            want = torch.zeros(rows, 260, dtype=torch.bool)
            want[5], want[6] = True, True
            want[offsets[1]:, 259] = True
            assert torch.equal(bad, want)


# ---- 4-bit weights ------------------------------------------------------------------------
Q4 = [
    # dtype, experts, rows, spare, active, N, K, group, pad
    ("bf16", 1, 1, 0, 1, 256, 256, 128, 0), ("bf16", 1, 1, 0, 1, 1, 1, 32, 0), ("f16", 1, 16, 0, 1, 100, 130, 64, 1),
    ("f32", 1, 37, 0, 1, 33, 260, 32, 3), ("bf16", 8, 20, 2, 5, 40, 384, 128, 0), ("f16", 3, 70, 0, 2, 17, 1000, 32, 0),
    ("f32", 2, 90, 1, 2, 16, 129, 64, 0), ("bf16", 2, 200, 0, 2, 48, 2100, 64, 5), ("f16", 1, 3, 0, 1, 31, 4200, 128, 0),
    ("f32", 4, 9, 0, 3, 20, 5, 128, 0), ("bf16", 5, 30, 3, 0, 20, 64, 32, 0), ("f16", 64, 130, 0, 40, 32, 256, 128, 0),
]


@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("dt,experts,rows,spare,active,N,K,group,pad", Q4, ids=lambda v: str(v))
def test_q4(dt, experts, rows, spare, active, N, K, group, pad, out):
    if out == "f32" and dt == "f32":
        pytest.skip("the same case")
    o = dt if out == "same" else "f32"
    offsets = offsets_of(sizes_of(experts, rows, active, seed=rows))
    total = rows + spare
    off = torch.tensor(offsets, dtype=torch.int32).cuda() if experts > 1 else None
    groups, width = -(-K // group), -(-K // 2)
    g = torch.Generator().manual_seed(K)
    codes = torch.randint(0, 256, (experts, N, width), generator=g, dtype=torch.uint8)
    wide = torch.full((experts, N, width + pad), 255, dtype=torch.uint8)
    wide[:, :, :width] = codes
    for exact in (True, False):
        if exact:      # few activations of one, scales of powers of two: every sum is held exactly
            A = (torch.rand(total, K, generator=g) < 3 / K).to(TYPES[dt])
            scales = 2.0 ** torch.randint(-1, 2, (experts, N, groups), generator=g).to(torch.float32)
            scales = scales.to(TYPES[dt])
        else:
            A = normal(total, K, dtype=dt, seed=3)
            scales = (torch.rand(experts, N, groups, generator=g) + 0.5).to(TYPES[dt])
        A[offsets[-1]:] = float("nan")
        W = ref.q4_weights(codes, scales, N, K, group)
        want, absum = ref.grouped(A, W.transpose(1, 2).contiguous(), offsets, total)
        packed = torch.full((tg.tile_gemm_q4_packed_size(experts, N, K, group, dt) + 256,), 170, dtype=torch.uint8,
                            device="cuda")
        sd, ld_s = strided(scales, pad)
        wd = wide.cuda()
        tg.tile_gemm_pack_q4(experts, N, K, group, dt, wd, width + pad, N * (width + pad), sd, ld_s, N * ld_s, packed,
                             packed_bytes=packed.numel() - 256)
        assert packed[-256:].tolist() == [170] * 256
        Ad, lda = strided(A, pad)
        C = Out(total, N, TYPES[o], pad)
        tg.tile_gemm_q4(experts, total, N, K, group, dt, Ad, lda, packed, C.t, C.ld, off, c_dtype=o)
        got = C.get()
        if exact and float(absum.max() if absum.numel() else 0) <= 64:
            assert torch.equal(got.double(), want)
        else:
            # a group's sum of whole codes is scaled once more than a plain product: one term more
            ref.check(got, want, K + 1, absum, o)


# ---- tables that are wrong, streams, graphs --------------------------------------------------
def test_wrong_tables_stay_inside():
    """Rows and offsets outside the operands are clamped or left out; nothing else is written."""
    T, k, D = 10, 2, 24
    x = normal(T, D, dtype="bf16").cuda()
    row = torch.tensor([0, 10 ** 9, -10 ** 9, 2 ** 31 - 1, -2 ** 31, 19, 20, -21] + [-1] * 12, dtype=torch.int32).cuda()
    w = torch.ones(T, k, device="cuda")
    rows, out, d_y = (Out(n, D, torch.bfloat16) for n in (T * k, T, T * k))
    d_w = Out(T, k, torch.float32)
    y = normal(T * k, D, dtype="bf16", seed=1).cuda()
    tg.tile_gemm_expert_gather(T, k, D, "bf16", x, D, row, rows.t, D)
    tg.tile_gemm_expert_combine(T, k, D, "bf16", y, D, row, w, k, out.t, D)
    tg.tile_gemm_expert_combine_grad(T, k, D, "bf16", x, D, y, D, row, w, k, d_y.t, D, d_w.t, k)
    assert torch.equal(rows.get()[19], x[2].cpu())
    assert torch.equal(out.get()[0], y[0].cpu()) and not torch.isnan(d_w.get()).any()
    d_y.get()
    for offsets in ([-5, 3, 10 ** 9], [7, 2, 30], [2 ** 31 - 1, -2 ** 31, 4], [0, 40, 20]):
        off = torch.tensor(offsets, dtype=torch.int32).cuda()
        for R in (20, 600):
            A, B = normal(R, 72, dtype="bf16").cuda(), normal(2, 72, 264, dtype="bf16").cuda()
            C, G = Out(R, 264, torch.bfloat16), Out(72, 264, torch.float32, batch=2)
            tg.tile_gemm_grouped(2, R, 264, 72, "bf16", A, 72, B, 264, 72 * 264, C.t, 264, off, c_dtype="bf16")
            tg.tile_gemm_grouped_wgrad(2, R, 72, 264, "bf16", A, 72, normal(R, 264, dtype="bf16").cuda(), 264, G.t, 264,
                                       G.stride, off)
            packed = torch.zeros(tg.tile_gemm_q4_packed_size(2, 264, 72, 32, "bf16"), dtype=torch.uint8, device="cuda")
            Q = Out(R, 264, torch.float32)
            tg.tile_gemm_q4(2, R, 264, 72, 32, "bf16", A, 72, packed, Q.t, 264, off)
            C.get(), G.get(), Q.get()


def layer(stream=None):
    """Every operator once, on fixed inputs; returns the call and its outputs."""
    T, k, E, D, H = 300, 2, 8, 264, 520
    ids = routing(T, k, E, 0.1, 3).cuda()
    n = T * k
    i32 = dict(dtype=torch.int32, device="cuda")
    offsets, entry, row = torch.empty(E + 1, **i32), torch.empty(n, **i32), torch.empty(n, **i32)
    ws = torch.empty(max(4, tg.tile_gemm_expert_sort_workspace_size(T, k, E)) // 4, **i32)
    x, w = normal(T, D, dtype="bf16", seed=1).cuda(), torch.rand(T, k, device="cuda")
    B = normal(E, D, H, dtype="bf16", seed=2, scale=D ** -0.5).cuda()
    rows, y, out = (torch.empty(*s, dtype=torch.bfloat16, device="cuda") for s in ((n, D), (n, H), (T, H)))
    d_y, d_w = torch.empty_like(y), torch.empty(T, k, device="cuda")
    d_rows, d_x, d_B = torch.empty_like(rows), torch.empty_like(x), torch.empty(E, D, H, device="cuda")
    codes = torch.randint(0, 256, (E, H, D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.ones(E, H, -(-D // 64), dtype=torch.bfloat16, device="cuda")
    packed = torch.empty(tg.tile_gemm_q4_packed_size(E, H, D, 64, "bf16"), dtype=torch.uint8, device="cuda")
    tg.tile_gemm_pack_q4(E, H, D, 64, "bf16", codes, D // 2, H * D // 2, scales, scales.shape[2], H * scales.shape[2],
                         packed)
    q = torch.empty(n, H, dtype=torch.bfloat16, device="cuda")

    def call(stream=None):
        s = dict(stream=stream)
        tg.tile_gemm_expert_sort(T, k, E, ids, k, offsets, entry, row, workspace=ws, **s)
        tg.tile_gemm_expert_gather(T, k, D, "bf16", x, D, row, rows, D, **s)
        tg.tile_gemm_grouped(E, n, H, D, "bf16", rows, D, B, H, D * H, y, H, offsets, c_dtype="bf16", **s)
        tg.tile_gemm_expert_combine(T, k, H, "bf16", y, H, row, w, k, out, H, **s)
        tg.tile_gemm_expert_combine_grad(T, k, H, "bf16", out, H, y, H, row, w, k, d_y, H, d_w, k, **s)
        tg.tile_gemm_grouped(E, n, D, H, "bf16", d_y, H, B, H, D * H, d_rows, D, offsets, c_dtype="bf16",
                             transposed=1, **s)
        tg.tile_gemm_grouped_wgrad(E, n, D, H, "bf16", rows, D, d_y, H, d_B, H, D * H, offsets, **s)
        tg.tile_gemm_expert_combine(T, k, D, "bf16", d_rows, D, row, None, 0, d_x, D, **s)
        tg.tile_gemm_q4(E, n, H, D, 64, "bf16", rows, D, packed, q, H, offsets, c_dtype="bf16", **s)

    return call, [offsets, entry, row, rows, y, out, d_y, d_w, d_rows, d_x, d_B, q]


def test_same_results_again_on_another_stream_and_in_a_graph():
    call, outs = layer()
    call()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    assert all(bool(torch.isfinite(w.float()).all()) for w in want)

    def spoil():
        for o in outs:
            o.fill_(-7)
        torch.cuda.synchronize()

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(o, w) for o, w in zip(outs, want))

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


def test_far_rows_and_strides():
    """Row offsets past 2^31 bytes: the last rows of a tall, widely strided A and C."""
    rows, K, N, ld = 70000, 40, 24, 16 * 1024 + 8
    A = torch.zeros(rows * ld, dtype=torch.bfloat16, device="cuda")
    a = normal(8, K, dtype="bf16", seed=1)
    at = torch.as_strided(A, (rows, K), (ld, 1))
    at[-8:] = a.cuda()
    B = normal(2, K, N, dtype="bf16", seed=2)
    C = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, rows - 8, rows], dtype=torch.int32).cuda()
    tg.tile_gemm_grouped(2, rows, N, K, "bf16", A, ld, B.cuda(), N, K * N, C, ld, off, c_dtype="bf16")
    torch.cuda.synchronize()
    got = torch.as_strided(C, (rows, N), (ld, 1))
    want, absum = ref.grouped(a, B[1:], [0, 8], 8)
    ref.check(got[-8:], want, K, absum, "bf16")
    assert not got[:-8].any()
