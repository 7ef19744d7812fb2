"""The operators of a feed-forward block, as measured work.

Two operators, each in its plain form (elementary torch operations in 32 bits,
rounded once at the end) and through this library's entry points:

gated     the gated pair of projections, per expert: u = x Wg, v = x Wu,
          h = act(u) * v (``tile_gemm_gated``), and its backward pass from the
          gradient of the block's result y = h W2: d_h = d_y W2^T,
          d_u = d_h v act'(u), d_v = d_h act(u) (``tile_gemm_gated_grad``),
          d_x = d_u Wg^T + d_v Wu^T (``tile_gemm_grouped``), the gradients of Wg
          and Wu (``tile_gemm_grouped_wgrad``).
adapters  a shared projection with a low-rank adapter of each row's own beside it:
          t = s[g] (x A[g]), y = x W + t B[g] (``tile_gemm_adapters``); backward
          the same call on the transposed matrices, and the gradients
          d_A[g] = x^T d_t, d_B[g] = t^T d_y over the rows of g
          (``tile_gemm_adapters_wgrad``).

Layouts.  transposed 0: a matrix is inputs x outputs; 1: outputs x inputs.  Wg and
Wu lie side by side, the gate first, along the outputs.  Rows of experts are in
expert order, those of no expert last.  Rows of adapters are in adapter order, those
without one last, or in any order (``shuffled``), with the table of their places in
adapter order.
"""
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
DEVICE = "cuda"


# ---- cases ----------------------------------------------------------------------
def listed():
    return [
        # one token through the gated pair of a small dense block, weights as a linear layer stores them
        dict(name="gated_token_bf16", op="gated", dtype="bf16", experts=1, active=1, rows=1, spare=0, N=2816, K=1024,
             activation="silu", transposed=1, grad=False),
        # a decoding batch spread over experts: every weight of those that are used is read once
        dict(name="gated_decode_bf16", op="gated", dtype="bf16", experts=8, active=7, rows=32, spare=0, N=2048, K=1024,
             activation="silu", transposed=0, grad=False),
        # a decoding batch through one wide dense block
        dict(name="gated_decode_f16", op="gated", dtype="f16", experts=1, active=1, rows=48, spare=0, N=8192, K=4096,
             activation="gelu", transposed=0, grad=False),
        # a prompt through a dense block
        dict(name="gated_prompt_bf16", op="gated", dtype="bf16", experts=1, active=1, rows=8192, spare=0, N=5632, K=2048,
             activation="silu", transposed=1, grad=False),
        # a training step of eight experts, forward and backward
        dict(name="gated_train_bf16", op="gated", dtype="bf16", experts=8, active=8, rows=16384, spare=0, N=2048, K=2048,
             activation="silu", transposed=0, grad=True),
        # many small experts, some without a row, rows of no expert, extents off every tile and off 16 bytes
        dict(name="gated_ragged_f16", op="gated", dtype="f16", experts=9, active=7, rows=2501, spare=13, N=1001, K=517,
             activation="gelu", transposed=0, grad=True),
        # a training step in fp32
        dict(name="gated_train_f32", op="gated", dtype="f32", experts=4, active=4, rows=2048, spare=0, N=1024, K=512,
             activation="silu", transposed=0, grad=True),
        # one request and its adapter beside a square projection
        dict(name="adapters_token_bf16", op="adapters", dtype="bf16", adapters=8, active=1, rows=1, without=0, N=4096,
             K=4096, rank=16, shuffled=False, transposed=1, grad=False),
        # a decoding batch of many requests in any order, some without an adapter
        dict(name="adapters_decode_bf16", op="adapters", dtype="bf16", adapters=32, active=20, rows=64, without=7, N=4096,
             K=4096, rank=32, shuffled=True, transposed=1, grad=False),
        # prompts of four requests
        dict(name="adapters_prompt_f16", op="adapters", dtype="f16", adapters=4, active=4, rows=8192, without=500, N=4096,
             K=4096, rank=64, shuffled=False, transposed=0, grad=False),
        # adapters trained beside a frozen projection, forward and backward
        dict(name="adapters_train_bf16", op="adapters", dtype="bf16", adapters=2, active=2, rows=8192, without=0, N=4096,
             K=2048, rank=16, shuffled=False, transposed=1, grad=True),
        # many adapters of few rows each, an odd rank, extents off every tile, fp32
        dict(name="adapters_ragged_f32", op="adapters", dtype="f32", adapters=41, active=37, rows=1333, without=21, N=771,
             K=1001, rank=5, shuffled=True, transposed=0, grad=True),
    ]


def _log_between(rng, low, high):
    """A whole number spread evenly over the logarithm, its ends among them."""
    x = low * (high / low) ** rng.random()
    return max(low, min(high, int(round(x))))


def draw(rng: random.Random):
    op = rng.choice(["gated", "adapters"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    grad = rng.random() < 0.5
    rows = _log_between(rng, 1, 16384)
    N, K = _log_between(rng, 64, 8192), _log_between(rng, 64, 8192)
    if rng.random() < 0.6:
        N, K = N // 8 * 8, K // 8 * 8
    # no more than the largest listed case; fp32 products take about ten times as long
    while rows * N * K > (16384 * 2048 * 2048 if dtype != "f32" else 4096 * 1024 * 1024):
        rows = (rows + 1) // 2
    if op == "gated":
        experts = rng.choice([1, 1, _log_between(rng, 2, 32)])
        while experts > 1 and experts * N * K > 32 * 2048 * 1024:
            experts = (experts + 1) // 2
        return dict(op=op, dtype=dtype, experts=experts, active=rng.randint(1, min(experts, rows)), rows=rows,
                    spare=rng.choice([0, 0, rng.randint(1, 100)]) if experts > 1 else 0, N=N, K=K,
                    activation=rng.choice(["silu", "silu", "gelu", "relu"]), transposed=rng.randint(0, 1), grad=grad)
    rank = rng.choice([8, 16, 32, 64, _log_between(rng, 1, 128)])
    adapters = _log_between(rng, 1, min(64, 2048 // rank))
    return dict(op=op, dtype=dtype, adapters=adapters, active=rng.randint(1, min(adapters, rows)), rows=rows,
                without=rng.choice([0, rng.randint(0, rows)]) if adapters > 1 else 0, N=N, K=K, rank=rank,
                shuffled=rng.random() < 0.5, transposed=rng.randint(0, 1), grad=grad)


# ---- inputs ---------------------------------------------------------------------
def _sizes(groups, active, rows, g):
    """Rows of each group: `active` of them have some, the split uneven."""
    chosen = torch.randperm(groups, generator=g)[:active].tolist()
    share = torch.rand(active, generator=g).add_(0.25).double()
    extra = (share / share.sum() * (rows - active)).floor().long().tolist()
    extra[0] += rows - active - sum(extra)
    sizes = [0] * groups
    for e, n in zip(chosen, extra):
        sizes[e] = 1 + n
    return sizes


def _inputs(case, seed):
    host = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    t = DTYPES[case["dtype"]]
    N, K = case["N"], case["K"]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32).mul_(scale).to(t)

    def matrix(groups, inputs, outputs, scale):
        shape = (outputs, inputs) if case["transposed"] else (inputs, outputs)
        w = torch.empty(groups, *shape, dtype=t, device=DEVICE)
        for e in range(groups):
            w[e] = normal(*shape, scale=scale)
        return w

    s = {}
    if case["op"] == "gated":
        E, R = case["experts"], case["rows"] + case["spare"]
        sizes = _sizes(E, case["active"], case["rows"], host)
        ids = [e for e in range(E) for _ in range(sizes[e])] + [E] * case["spare"]
        s["w"] = matrix(E, K, 2 * N, K ** -0.5)            # the gate's outputs, then the other's
        if case["grad"]:
            s["w2"] = matrix(E, N, K, N ** -0.5)
            s["d_y"] = normal(R, K, scale=0.1)
    else:
        G, R, r = case["adapters"], case["rows"], case["rank"]
        sizes = _sizes(G, case["active"], max(R - case["without"], case["active"]), host)
        ids = [e for e in range(G) for _ in range(sizes[e])]
        ids += [G] * (R - len(ids))
        s["w"] = matrix(1, K, N, K ** -0.5)[0]
        s["a"] = matrix(G, K, r, K ** -0.5)
        s["b"] = matrix(G, r, N, 0.3 * r ** -0.5)
        s["scales"] = torch.rand(G, generator=g, device=DEVICE).mul_(1.5).add_(0.5)
        if case["grad"]:
            s["d_y"] = normal(R, N, scale=0.1)
    s["x"] = normal(R, K)
    s["sizes"] = sizes
    s["offsets"] = torch.tensor([0] + sizes, dtype=torch.int32).cumsum(0).to(torch.int32).to(DEVICE)
    place = torch.tensor(ids)
    if case.get("shuffled"):
        place = place[torch.randperm(R, generator=host)]
        s["order"] = torch.sort(place, stable=True).indices.to(torch.int32).to(DEVICE)
    s["ids"] = place.to(DEVICE)                             # the group of each row; their number: none
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    import tile_scheduled_dense_amd as tg
    t = DTYPES[case["dtype"]]
    R, N, K, dt = s["x"].shape[0], case["N"], case["K"], case["dtype"]

    def empty(*shape, dtype=t):
        return torch.empty(*shape, dtype=dtype, device=DEVICE)

    def scratch(size):
        return empty(size, dtype=torch.uint8) if size else None

    if case["op"] == "gated":
        E, tr = case["experts"], case["transposed"]
        s["h"] = empty(R, N)
        s["workspace"] = scratch(tg.tile_gemm_gated_workspace_size(E, R, N, K, dt, transposed=tr))
        if case["grad"]:
            s["uv"], s["d_uv"] = empty(R, 2 * N), empty(R, 2 * N)
            s["d_x"], s["d_w"] = empty(R, K), torch.empty_like(s["w"])
        return s
    G, r, tr = case["adapters"], case["rank"], case["transposed"]
    s["y"] = empty(R, N)
    size = tg.tile_gemm_adapters_workspace_size(G, R, N, K, r, dt, transposed=tr)
    if case["grad"]:
        s["t"], s["d_t"], s["d_x"] = empty(R, r), empty(R, r), empty(R, K)
        s["d_a"], s["d_b"] = torch.empty_like(s["a"]), torch.empty_like(s["b"])
        size = max(size, tg.tile_gemm_adapters_workspace_size(G, R, K, N, r, dt, transposed=1 - tr),
                   tg.tile_gemm_adapters_wgrad_workspace_size(G, R, N, K, r, dt))
    s["workspace"] = scratch(size)
    return s


# ---- one pass -------------------------------------------------------------------
def run(s):
    gated = s["case"]["op"] == "gated"
    if own:
        return _own_gated(s) if gated else _own_adapters(s)
    return _plain_gated(s) if gated else _plain_adapters(s)


def _own_gated(s):
    import tile_scheduled_dense_amd as tg
    c = s["case"]
    E, R, N, K, t, tr = c["experts"], s["x"].shape[0], c["N"], c["K"], c["dtype"], c["transposed"]
    act = {"silu": tg.ACT_SILU, "gelu": tg.ACT_GELU, "relu": tg.ACT_RELU}[c["activation"]]
    offsets = s["offsets"] if E > 1 else None
    w = s["w"]
    up = w[:, N:] if tr else w[:, :, N:]
    ldb, stride = w.stride(1), w.stride(0)
    if not c["grad"]:
        tg.tile_gemm_gated(E, R, N, K, t, s["x"], K, w, up, ldb, stride, s["h"], N, offsets, activation=act, transposed=tr,
                           workspace=s["workspace"])
        return s["h"]
    u, v, d_u, d_v = s["uv"], s["uv"][:, N:], s["d_uv"], s["d_uv"][:, N:]
    tg.tile_gemm_gated(E, R, N, K, t, s["x"], K, w, up, ldb, stride, s["h"], N, offsets, activation=act, transposed=tr,
                       U=u, V=v, ldu=2 * N, workspace=s["workspace"])
    w2 = s["w2"]
    tg.tile_gemm_gated_grad(E, R, N, K, t, s["d_y"], K, w2, w2.stride(1), w2.stride(0), u, v, 2 * N, d_u, d_v, 2 * N,
                            offsets, activation=act, transposed=1 - tr)
    tg.tile_gemm_grouped(E, R, K, 2 * N, t, d_u, 2 * N, w, ldb, stride, s["d_x"], K, offsets, c_dtype=t, transposed=1 - tr)
    if tr:
        tg.tile_gemm_grouped_wgrad(E, R, 2 * N, K, t, d_u, 2 * N, s["x"], K, s["d_w"], ldb, stride, offsets, c_dtype=t)
    else:
        tg.tile_gemm_grouped_wgrad(E, R, K, 2 * N, t, s["x"], K, d_u, 2 * N, s["d_w"], ldb, stride, offsets, c_dtype=t)
    return dict(h=s["h"], d_uv=s["d_uv"], d_x=s["d_x"], d_w=s["d_w"])


def _own_adapters(s):
    import tile_scheduled_dense_amd as tg
    c = s["case"]
    G, R, N, K, r, t, tr = c["adapters"], c["rows"], c["N"], c["K"], c["rank"], c["dtype"], c["transposed"]
    w, a, b, order = s["w"], s["a"], s["b"], s.get("order")
    tg.tile_gemm_adapters(G, R, N, K, r, t, s["x"], K, w, w.stride(0), a, a.stride(1), a.stride(0), b, b.stride(1),
                          b.stride(0), s["y"], N, s["offsets"], s["workspace"], order=order, scales=s["scales"],
                          transposed=tr, T=s.get("t"), ldt=r)
    if not c["grad"]:
        return s["y"]
    tg.tile_gemm_adapters(G, R, K, N, r, t, s["d_y"], N, w, w.stride(0), b, b.stride(1), b.stride(0), a, a.stride(1),
                          a.stride(0), s["d_x"], K, s["offsets"], s["workspace"], order=order, scales=s["scales"],
                          transposed=1 - tr, T=s["d_t"], ldt=r)
    tg.tile_gemm_adapters_wgrad(G, R, N, K, r, t, s["x"], K, s["d_y"], N, s["t"], r, s["d_t"], r, s["d_a"],
                                a.stride(1), a.stride(0), s["d_b"], b.stride(1), b.stride(0), s["offsets"],
                                s["workspace"], order=order, c_dtype=t, transposed=tr)
    return dict(y=s["y"], d_x=s["d_x"], d_a=s["d_a"], d_b=s["d_b"])


def _cdf(u):
    return 0.5 * (1 + torch.erf(u * 0.5 ** 0.5))


def _act(u, kind):
    if kind == "relu":
        return torch.where(u > 0, u, 0)
    return u * _cdf(u) if kind == "gelu" else u / (1 + torch.exp(-u))


def _act_grad(u, kind):
    if kind == "relu":
        return (u > 0).to(u.dtype)
    if kind == "gelu":
        return _cdf(u) + u * torch.exp(-0.5 * u * u) * 0.3989422804014327
    e = torch.exp(-u.abs())
    sig = torch.where(u > 0, 1, e) / (1 + e)
    return sig * (1 + u * (1 - sig))


def _plain_gated(s):
    c = s["case"]
    E, N, t, ids = c["experts"], c["N"], DTYPES[c["dtype"]], s["ids"]
    n, most = ids.shape[0], max(s["sizes"])
    # every expert's rows in a block of its own, as many as the largest has, zeros behind them
    has = ids < E
    slot = torch.where(has, ids * most + torch.arange(n, device=ids.device) - s["offsets"].long()[ids], E * most)

    def spread(rows):
        blocks = torch.zeros(E * most + 1, rows.shape[1], device=rows.device)
        blocks[slot] = torch.where(has[:, None], rows.float(), 0)
        return blocks[:-1].reshape(E, most, -1)

    def back(blocks):
        flat = torch.nn.functional.pad(blocks.reshape(E * most, -1), (0, 0, 0, 1))
        return flat[slot]

    w = s["w"].float()
    w = w.transpose(1, 2).contiguous() if c["transposed"] else w
    x = spread(s["x"])
    uv = torch.bmm(x, w)
    u, v = uv[..., :N], uv[..., N:]
    act = _act(u, c["activation"])
    h = back(act * v).to(t)
    if not c["grad"]:
        return h
    w2 = s["w2"].float()
    w2 = w2.transpose(1, 2).contiguous() if c["transposed"] else w2
    d_h = torch.bmm(spread(s["d_y"]), w2.transpose(1, 2).contiguous())
    d_uv = torch.cat([d_h * v * _act_grad(u, c["activation"]), d_h * act], dim=2)
    d_x = torch.bmm(d_uv, w.transpose(1, 2).contiguous())
    d_w = torch.bmm(x.transpose(1, 2).contiguous(), d_uv)
    d_w = d_w.transpose(1, 2).contiguous() if c["transposed"] else d_w
    return dict(h=h, d_uv=back(d_uv).to(t), d_x=back(d_x).to(t), d_w=d_w.to(t))


def _plain_adapters(s):
    c = s["case"]
    G, R, r, t, ids = c["adapters"], c["rows"], c["rank"], DTYPES[c["dtype"]], s["ids"]
    w, a, b, x = s["w"].float(), s["a"].float(), s["b"].float(), s["x"].float()
    if c["transposed"]:
        w, a, b = w.t().contiguous(), a.transpose(1, 2).contiguous(), b.transpose(1, 2).contiguous()
    # every row with every adapter, all but its own scaled by 0
    mine = (ids[:, None] == torch.arange(G, device=ids.device)) * s["scales"]
    a_all, b_all = a.transpose(0, 1).reshape(-1, G * r), b.reshape(G * r, -1)

    def low(rows, into):
        return ((rows @ into).reshape(R, G, r) * mine[:, :, None]).reshape(R, G * r)

    low_x = low(x, a_all)
    y = (x @ w + low_x @ b_all).to(t)
    if not c["grad"]:
        return y
    d_y = s["d_y"].float()
    low_d = low(d_y, b_all.t().contiguous())
    d_x = d_y @ w.t().contiguous() + low_d @ a_all.t().contiguous()
    d_a = (x.t().contiguous() @ low_d).reshape(-1, G, r).transpose(0, 1)
    d_b = (low_x.t().contiguous() @ d_y).reshape(G, r, -1)
    if c["transposed"]:
        d_a, d_b = d_a.transpose(1, 2), d_b.transpose(1, 2)
    return dict(y=y, d_x=d_x.to(t), d_a=d_a.contiguous().to(t), d_b=d_b.contiguous().to(t))


# ---- the definition in 64 bits -----------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    N, K, kind = case["N"], case["K"], case.get("activation")

    def f64(m):
        """A matrix or several in 64 bits, inputs x outputs."""
        return m.double().transpose(-1, -2).contiguous() if case["transposed"] else m.double()

    def like(m):
        return m.transpose(-1, -2).contiguous() if case["transposed"] else m

    x, ids = s["x"].double(), s["ids"]
    if case["op"] == "gated":
        h = torch.zeros(x.shape[0], N, dtype=torch.float64, device=DEVICE)
        d_uv, d_x = torch.zeros(x.shape[0], 2 * N, dtype=torch.float64, device=DEVICE), torch.zeros_like(x)
        d_w = torch.zeros(case["experts"], K, 2 * N, dtype=torch.float64, device=DEVICE)
        for e, n in enumerate(s["sizes"]):
            if n == 0:
                continue
            at = (ids == e).nonzero()[:, 0]
            w = f64(s["w"][e])
            u, v = x[at] @ w[:, :N].contiguous(), x[at] @ w[:, N:].contiguous()
            if kind == "relu":
                f, df = u.clamp_min(0), (u > 0).double()
            elif kind == "gelu":
                phi = torch.special.ndtr(u)
                f, df = u * phi, phi + u * torch.exp(-u * u / 2) / (2 * torch.pi) ** 0.5
            else:
                sig = torch.sigmoid(u)
                f, df = u * sig, sig + u * sig * torch.sigmoid(-u)
            h[at] = f * v
            if case["grad"]:
                d_h = s["d_y"][at].double() @ f64(s["w2"][e]).t().contiguous()
                d_uv[at] = torch.cat([d_h * v * df, d_h * f], dim=1)
                d_x[at] = d_uv[at] @ w.t().contiguous()
                d_w[e] = x[at].t().contiguous() @ d_uv[at]
        return dict(h=h, d_uv=d_uv, d_x=d_x, d_w=like(d_w)) if case["grad"] else h
    w = f64(s["w"])
    y = x @ w
    if case["grad"]:
        d_y = s["d_y"].double()
        d_x = d_y @ w.t().contiguous()
        d_a = torch.zeros(case["adapters"], K, case["rank"], dtype=torch.float64, device=DEVICE)
        d_b = torch.zeros(case["adapters"], case["rank"], N, dtype=torch.float64, device=DEVICE)
    for e, n in enumerate(s["sizes"]):
        if n == 0:
            continue
        at = (ids == e).nonzero()[:, 0]
        a, b, scale = f64(s["a"][e]), f64(s["b"][e]), s["scales"][e].double()
        low = x[at] @ a * scale
        y[at] += low @ b
        if case["grad"]:
            d_low = d_y[at] @ b.t().contiguous() * scale
            d_x[at] += d_low @ a.t().contiguous()
            d_a[e] = x[at].t().contiguous() @ d_low
            d_b[e] = low.t().contiguous() @ d_y[at]
    return dict(y=y, d_x=d_x, d_a=like(d_a), d_b=like(d_b)) if case["grad"] else y


# ---- what a pass cannot do without --------------------------------------------------
def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}[case["dtype"]]
    N, K, R = case["N"], case["K"], case["rows"]
    if case["op"] == "gated":
        n = R + case["spare"]
        nbytes = (R * K + 2 * case["active"] * N * K + n * N) * size     # x, both projections; h
        flops = 4 * R * N * K
        if case["grad"]:
            # d_y and the down projection; u and v's gradients, x's and the projections'
            nbytes += (R * K + case["active"] * N * K + 2 * n * N + n * K + 2 * case["experts"] * N * K) * size
            flops += 10 * R * N * K
        return {"bytes": nbytes, "flops": flops}
    r, with_one = case["rank"], max(R - case["without"], case["active"])
    nbytes = (R * K + N * K + case["active"] * r * (N + K) + R * N) * size
    flops = 2 * R * N * K + 2 * with_one * r * (N + K)
    if case["grad"]:
        nbytes += (R * N + R * K + case["adapters"] * r * (N + K)) * size      # d_y; d_x, the adapters' gradients
        flops += 2 * R * N * K + 4 * with_one * r * (N + K)
    return {"bytes": nbytes, "flops": flops}
