"""The operators of a mixture-of-experts layer, as measured work.

Three operators, each in its plain form (elementary torch operations in 32
bits, rounded once at the end) and through this library's entry points:

exchange  tokens sorted by expert (``tile_gemm_expert_sort``), their rows laid
          out by expert (``_gather``), the experts' rows summed back with the
          router's weights (``_combine``), and the gradients of all of it
          (``_combine_grad``, and ``_combine`` without weights).
experts   one product per expert over that expert's rows
          (``tile_gemm_grouped``) and its gradients: with respect to the rows
          (the same call on the transposed weights) and to the weights
          (``tile_gemm_grouped_wgrad``).
q4        products with 4-bit weights and one scale per group along K
          (``tile_gemm_q4``), for one matrix or one matrix per expert.

Sort results.  Entry e = t * top_k + j is the j-th choice of token t.  Rows are
ordered by expert, equal experts by entry; entries without an expert (an id
outside the experts) come last.  ``offsets[g]`` is the first row of expert g
and ``offsets[experts]`` the number of rows that have one.  ``entry_of_row``
and ``row_of_entry`` are inverse to each other; entries without an expert, and
their rows, are held as their complement (negative).

4-bit weights.  Two codes a byte, the lower four bits first along K; the weight
is (code - 8) * scale of its group of ``group`` consecutive k.
"""
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
DEVICE = "cuda"


# ---- cases ----------------------------------------------------------------------
def listed():
    return [
        # one decoding step of a few sequences: latency is all that counts
        dict(name="exchange_decode_bf16", op="exchange", dtype="bf16", tokens=16, top_k=2, experts=8, cols=1024,
             dropped=0.0, grad=False),
        # a training step's batch, two experts a token, forward and backward
        dict(name="exchange_train_bf16", op="exchange", dtype="bf16", tokens=8192, top_k=2, experts=8, cols=2048,
             dropped=0.0, grad=True),
        # many experts, many choices, a tenth of them cut off by a capacity limit; odd sizes, fp32
        dict(name="exchange_dropped_f32", op="exchange", dtype="f32", tokens=1999, top_k=8, experts=129, cols=1001,
             dropped=0.1, grad=True),
        # decoding through the experts' weights: few rows, every weight read once
        dict(name="experts_decode_bf16", op="experts", dtype="bf16", out="bf16", experts=8, active=7, rows=32,
             N=4096, K=1024, forward=True, grad=False),
        # the up projection of a training step
        dict(name="experts_forward_bf16", op="experts", dtype="bf16", out="bf16", experts=8, active=8, rows=16384,
             N=4096, K=2048, forward=True, grad=False),
        # its two gradients
        dict(name="experts_backward_bf16", op="experts", dtype="bf16", out="bf16", experts=8, active=8, rows=16384,
             N=4096, K=2048, forward=False, grad=True),
        # many small experts, some without a row, extents off every tile and off 16 bytes, fp32 results
        dict(name="experts_ragged_f16", op="experts", dtype="f16", out="f32", experts=33, active=29, rows=5001,
             N=1000, K=257, forward=True, grad=True),
        # fp32 experts
        dict(name="experts_f32", op="experts", dtype="f32", out="f32", experts=4, active=4, rows=2048,
             N=1024, K=512, forward=True, grad=True),
        # one token through a square projection
        dict(name="q4_token_bf16", op="q4", dtype="bf16", out="bf16", experts=1, active=1, rows=1, N=4096, K=4096,
             group=128),
        # a decoding batch through a large matrix
        dict(name="q4_batch_f16", op="q4", dtype="f16", out="f16", experts=1, active=1, rows=16, N=8192, K=8192,
             group=64),
        # odd extents, small groups, fp32 activations and results
        dict(name="q4_ragged_f32", op="q4", dtype="f32", out="f32", experts=1, active=1, rows=37, N=1001, K=4100,
             group=32),
        # a decoding batch spread over 4-bit experts
        dict(name="q4_experts_bf16", op="q4", dtype="bf16", out="bf16", experts=64, active=24, rows=64, N=2048,
             K=2048, group=128),
    ]


def _log_between(rng, low, high):
    """A whole number spread evenly over the logarithm, its ends among them."""
    x = low * (high / low) ** rng.random()
    return max(low, min(high, int(round(x))))


def draw(rng: random.Random):
    op = rng.choice(["exchange", "experts", "q4"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "exchange":
        top_k = rng.randint(1, 8)
        cols = _log_between(rng, 64, 4096)
        if rng.random() < 0.5:
            cols = cols // 8 * 8
        most = 8192 * 2 * 2048 * 2 // (top_k * cols * (4 if dtype == "f32" else 2))
        return dict(op=op, dtype=dtype, tokens=_log_between(rng, 1, min(16384, most)), top_k=top_k,
                    experts=_log_between(rng, max(8, top_k), 256), cols=cols,
                    dropped=rng.choice([0.0, 0.0, 0.05, 0.3]), grad=rng.random() < 0.6)
    out = rng.choice([dtype, "f32"])
    if op == "experts":
        experts = _log_between(rng, 2, 64)
        rows = _log_between(rng, 1, 16384)
        N, K = _log_between(rng, 64, 4096), _log_between(rng, 64, 4096)
        if rng.random() < 0.6:
            N, K = N // 8 * 8, K // 8 * 8
        while rows * N * K > (16384 * 4096 * 2048 if dtype != "f32" else 16384 * 1024 * 1024):
            rows = (rows + 1) // 2
        forward = rng.random() < 0.6
        return dict(op=op, dtype=dtype, out=out, experts=experts,
                    active=rng.randint(1, min(experts, rows)), rows=rows, N=N, K=K,
                    forward=forward, grad=not forward or rng.random() < 0.4)
    experts = rng.choice([1, 1, _log_between(rng, 2, 64)])
    rows = _log_between(rng, 1, 64 if experts == 1 else 256)
    N, K = _log_between(rng, 64, 8192), _log_between(rng, 64, 8192)
    if rng.random() < 0.6:
        N, K = (N + 15) // 16 * 16, (K + 31) // 32 * 32
    while experts * N * K > 64 * 2048 * 2048:
        experts = (experts + 1) // 2
    return dict(op=op, dtype=dtype, out=out, experts=experts, active=rng.randint(1, min(experts, rows)), rows=rows,
                N=N, K=K, group=rng.choice([32, 64, 128]))


# ---- inputs ---------------------------------------------------------------------
def _sizes(case, g):
    """Rows of each expert: `active` of them have some, the split uneven."""
    E, active, rows = case["experts"], case["active"], case["rows"]
    chosen = torch.randperm(E, generator=g)[:active].tolist()
    share = torch.rand(active, generator=g).add_(0.25).double()
    extra = (share / share.sum() * (rows - active)).floor().long().tolist()
    extra[0] += rows - active - sum(extra)
    sizes = [0] * E
    for e, n in zip(chosen, extra):
        sizes[e] = 1 + n
    return sizes


def _offsets(sizes):
    out = [0]
    for n in sizes:
        out.append(out[-1] + n)
    return out


def _inputs(case, seed):
    host = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    t = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32).mul_(scale)

    s = {}
    if case["op"] == "exchange":
        T, k, E, D = case["tokens"], case["top_k"], case["experts"], case["cols"]
        # router scores with popular and unpopular experts
        logits = normal(T, E) + normal(E)
        top, ids = logits.topk(k, dim=1)
        weights = torch.softmax(top, dim=1)
        if case["dropped"]:
            cut = torch.rand(T, k, generator=g, device=DEVICE) < case["dropped"]
            ids = torch.where(cut, torch.full_like(ids, -1), ids)
        s["ids"] = ids.to(torch.int32).contiguous()
        s["weights"] = weights.contiguous()
        s["x"] = normal(T, D).to(t)
        s["y"] = normal(T * k, D).to(t)           # the experts' results, by row
        if case["grad"]:
            s["d_out"] = normal(T, D, scale=0.1).to(t)
            s["d_rows"] = normal(T * k, D, scale=0.1).to(t)
        return s
    sizes = _sizes(case, host)
    E, R, N, K = case["experts"], case["rows"], case["N"], case["K"]
    s["sizes"] = sizes
    s["offsets"] = torch.tensor(_offsets(sizes), dtype=torch.int32, device=DEVICE)
    s["a"] = normal(R, K).to(t)
    if case["op"] == "experts":
        s["b"] = torch.empty(E, K, N, dtype=t, device=DEVICE)
        for e in range(E):
            s["b"][e] = normal(K, N, scale=K ** -0.5).to(t)
        if case["grad"]:
            s["d"] = normal(R, N, scale=0.1).to(t)
        return s
    groups = (K + case["group"] - 1) // case["group"]
    s["codes"] = torch.randint(0, 256, (E, N, (K + 1) // 2), generator=g, device=DEVICE, dtype=torch.uint8)
    s["scales"] = (0.5 + torch.rand(E, N, groups, generator=g, device=DEVICE)).mul_(0.25 * K ** -0.5).to(t)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    import tile_scheduled_dense_amd as tg
    t = DTYPES[case["dtype"]]

    def empty(*shape, dtype=t):
        return torch.empty(*shape, dtype=dtype, device=DEVICE)

    if case["op"] == "exchange":
        T, k, E, D = case["tokens"], case["top_k"], case["experts"], case["cols"]
        s["offsets"] = empty(E + 1, dtype=torch.int32)
        s["entry_of_row"] = empty(T * k, dtype=torch.int32)
        s["row_of_entry"] = empty(T, k, dtype=torch.int32)
        s["workspace"] = empty(max(tg.tile_gemm_expert_sort_workspace_size(T, k, E), 4) // 4, dtype=torch.int32)
        s["rows"], s["out"] = empty(T * k, D), empty(T, D)
        if case["grad"]:
            s["d_x"], s["d_y"], s["d_w"] = empty(T, D), empty(T * k, D), empty(T, k, dtype=torch.float32)
        return s
    E, R, N, K = case["experts"], case["rows"], case["N"], case["K"]
    o = DTYPES[case["out"]]
    if case["op"] == "experts":
        if case["forward"]:
            s["c"] = empty(R, N, dtype=o)
        if case["grad"]:
            s["d_a"], s["d_b"] = empty(R, K, dtype=o), empty(E, K, N, dtype=o)
        return s
    s["c"] = empty(R, N, dtype=o)
    size = tg.tile_gemm_q4_packed_size(E, N, K, case["group"], case["dtype"])
    s["packed"] = empty(size, dtype=torch.uint8)
    codes, scales = s["codes"], s["scales"]
    tg.tile_gemm_pack_q4(E, N, K, case["group"], case["dtype"], codes, codes.stride(1), codes.stride(0), scales,
                         scales.stride(1), scales.stride(0), s["packed"])
    return s


# ---- one pass -------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"exchange": _own_exchange, "experts": _own_experts, "q4": _own_q4}[op](s)
    return {"exchange": _plain_exchange, "experts": _plain_experts, "q4": _plain_q4}[op](s)


def _own_exchange(s):
    import tile_scheduled_dense_amd as tg
    c = s["case"]
    T, k, E, D, t = c["tokens"], c["top_k"], c["experts"], c["cols"], c["dtype"]
    tg.tile_gemm_expert_sort(T, k, E, s["ids"], k, s["offsets"], s["entry_of_row"], s["row_of_entry"],
                             workspace=s["workspace"])
    tg.tile_gemm_expert_gather(T, k, D, t, s["x"], D, s["row_of_entry"], s["rows"], D)
    tg.tile_gemm_expert_combine(T, k, D, t, s["y"], D, s["row_of_entry"], s["weights"], k, s["out"], D)
    out = dict(offsets=s["offsets"], entry_of_row=s["entry_of_row"], row_of_entry=s["row_of_entry"],
               rows=s["rows"], out=s["out"])
    if c["grad"]:
        tg.tile_gemm_expert_combine_grad(T, k, D, t, s["d_out"], D, s["y"], D, s["row_of_entry"], s["weights"], k,
                                         s["d_y"], D, s["d_w"], k)
        tg.tile_gemm_expert_combine(T, k, D, t, s["d_rows"], D, s["row_of_entry"], None, 0, s["d_x"], D)
        out.update(d_y=s["d_y"], d_w=s["d_w"], d_x=s["d_x"])
    return out


def _own_experts(s):
    import tile_scheduled_dense_amd as tg
    c = s["case"]
    E, R, N, K, t, o = c["experts"], c["rows"], c["N"], c["K"], c["dtype"], c["out"]
    out = {}
    if c["forward"]:
        tg.tile_gemm_grouped(E, R, N, K, t, s["a"], K, s["b"], N, K * N, s["c"], N, s["offsets"], c_dtype=o)
        out["c"] = s["c"]
    if c["grad"]:
        tg.tile_gemm_grouped(E, R, K, N, t, s["d"], N, s["b"], N, K * N, s["d_a"], K, s["offsets"], c_dtype=o,
                             transposed=1)
        tg.tile_gemm_grouped_wgrad(E, R, K, N, t, s["a"], K, s["d"], N, s["d_b"], N, K * N, s["offsets"], c_dtype=o)
        out["d_a"], out["d_b"] = s["d_a"], s["d_b"]
    return out


def _own_q4(s):
    import tile_scheduled_dense_amd as tg
    c = s["case"]
    tg.tile_gemm_q4(c["experts"], c["rows"], c["N"], c["K"], c["group"], c["dtype"], s["a"], c["K"], s["packed"],
                    s["c"], c["N"], s["offsets"] if c["experts"] > 1 else None, c_dtype=c["out"])
    return s["c"]


def _plain_exchange(s):
    c = s["case"]
    T, k, E, t = c["tokens"], c["top_k"], c["experts"], DTYPES[c["dtype"]]
    ids = s["ids"].reshape(-1)
    key = torch.where((ids >= 0) & (ids < E), ids, torch.full_like(ids, E))
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.cumsum((key[None, :] == torch.arange(E, device=ids.device)[:, None]).sum(1), 0)
    order = torch.sort(key, stable=True).indices
    kept = key[order] < E
    row = torch.empty_like(order)
    row[order] = torch.arange(T * k, device=ids.device)
    has = key < E
    rows = torch.where(kept[:, None], s["x"][order // k], 0)
    w = torch.where(has, s["weights"].reshape(-1), 0)
    picked = torch.where(has[:, None], s["y"][row].float(), 0)
    out = (picked * w[:, None]).reshape(T, k, -1).sum(1)
    res = dict(offsets=offsets.int(), entry_of_row=torch.where(kept, order, ~order).int(),
               row_of_entry=torch.where(has, row, ~row).int().reshape(T, k), rows=rows, out=out.to(t))
    if c["grad"]:
        d_out = s["d_out"].float()
        d_y = torch.where(kept[:, None], d_out[order // k] * w[order][:, None], 0)
        d_w = (picked.reshape(T, k, -1) * d_out[:, None, :]).sum(2)
        d_x = torch.where(has[:, None], s["d_rows"][row].float(), 0).reshape(T, k, -1).sum(1)
        res.update(d_y=d_y.to(t), d_w=d_w, d_x=d_x.to(t))
    return res


def _plain_experts(s):
    c = s["case"]
    o = DTYPES[c["out"]]
    first = _offsets(s["sizes"])
    used = [(e, first[e], first[e + 1]) for e in range(c["experts"]) if first[e + 1] > first[e]]
    out = {}
    a, b = s["a"].float(), s["b"].float()
    if c["forward"]:
        res = torch.empty(c["rows"], c["N"], device=a.device)
        for e, lo, hi in used:
            res[lo:hi] = a[lo:hi] @ b[e]
        out["c"] = res.to(o)
    if c["grad"]:
        d = s["d"].float()
        d_a = torch.empty(c["rows"], c["K"], device=a.device)
        d_b = torch.zeros(c["experts"], c["K"], c["N"], device=a.device)
        for e, lo, hi in used:
            d_a[lo:hi] = d[lo:hi] @ b[e].t()
            d_b[e] = a[lo:hi].t() @ d[lo:hi]
        out["d_a"], out["d_b"] = d_a.to(o), d_b.to(o)
    return out


def _plain_q4(s):
    c = s["case"]
    K, group = c["K"], c["group"]
    first = _offsets(s["sizes"])
    a = s["a"].float()
    res = torch.empty(c["rows"], c["N"], device=a.device)
    for e in range(c["experts"]):
        lo, hi = first[e], first[e + 1]
        if lo == hi:
            continue
        codes = torch.stack([s["codes"][e] & 15, s["codes"][e] >> 4], dim=2).reshape(c["N"], -1)[:, :K]
        scales = s["scales"][e].float().repeat_interleave(group, dim=1)[:, :K]
        res[lo:hi] = a[lo:hi] @ ((codes.float() - 8) * scales).t()
    return res.to(DTYPES[c["out"]])


# ---- the definition in 64 bits -----------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "exchange":
        T, k, E = case["tokens"], case["top_k"], case["experts"]
        ids = s["ids"].cpu().reshape(-1).tolist()
        lists = [[] for _ in range(E + 1)]
        for entry, e in enumerate(ids):
            lists[e if 0 <= e < E else E].append(entry)
        offsets = _offsets([len(x) for x in lists[:E]])
        sorted_entries = [entry for x in lists for entry in x]
        n = offsets[-1]
        row_of = [0] * (T * k)
        for r, entry in enumerate(sorted_entries):
            row_of[entry] = r if r < n else -1 - r
        entry_of = [entry if r < n else -1 - entry for r, entry in enumerate(sorted_entries)]
        kept = torch.tensor(sorted_entries[:n], dtype=torch.int64, device=DEVICE)   # row r < n holds entry kept[r]
        token = torch.div(kept, k, rounding_mode="floor")
        x, y = s["x"].double(), s["y"].double()[:n]
        w = s["weights"].double().reshape(-1)[kept]
        rows = torch.zeros(T * k, case["cols"], dtype=torch.float64, device=DEVICE)
        rows[:n] = x[token]
        out = torch.zeros_like(x).index_add_(0, token, y * w[:, None])
        res = dict(offsets=torch.tensor(offsets, dtype=torch.int32, device=DEVICE),
                   entry_of_row=torch.tensor(entry_of, dtype=torch.int32, device=DEVICE),
                   row_of_entry=torch.tensor(row_of, dtype=torch.int32, device=DEVICE).reshape(T, k),
                   rows=rows, out=out)
        if case["grad"]:
            g = s["d_out"].double()[token]
            d_y = torch.zeros_like(rows)
            d_y[:n] = g * w[:, None]
            d_w = torch.zeros(T * k, dtype=torch.float64, device=DEVICE)
            d_w[kept] = (g * y).sum(1)
            d_x = torch.zeros_like(x).index_add_(0, token, s["d_rows"].double()[:n])
            res.update(d_y=d_y, d_w=d_w.reshape(T, k), d_x=d_x)
        return res
    bounds = [0]
    for n in s["sizes"]:
        bounds.append(bounds[-1] + n)
    a = s["a"].double()
    if case["op"] == "experts":
        res = {}
        if case["forward"]:
            res["c"] = torch.cat([a[bounds[e]:bounds[e + 1]] @ s["b"][e].double() for e in range(case["experts"])])
        if case["grad"]:
            d = s["d"].double()
            res["d_a"] = torch.cat([d[bounds[e]:bounds[e + 1]] @ s["b"][e].double().t().contiguous()
                                    for e in range(case["experts"])])
            res["d_b"] = torch.stack([a[bounds[e]:bounds[e + 1]].t().contiguous() @ d[bounds[e]:bounds[e + 1]]
                                      for e in range(case["experts"])])
        return res
    parts = []
    for e in range(case["experts"]):
        lo, hi = bounds[e], bounds[e + 1]
        raw = s["codes"][e].double()
        high = torch.floor(raw / 16)
        weight = torch.zeros(case["N"], 2 * raw.shape[1], dtype=torch.float64, device=DEVICE)
        weight[:, 0::2] = raw - 16 * high - 8
        weight[:, 1::2] = high - 8
        which = torch.arange(case["K"], device=DEVICE) // case["group"]
        weight = weight[:, :case["K"]] * s["scales"][e].double()[:, which]
        parts.append(a[lo:hi] @ weight.t().contiguous())
    return torch.cat(parts)


# ---- what a pass cannot do without --------------------------------------------------
def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}[case["dtype"]]
    if case["op"] == "exchange":
        T, k, E, D = case["tokens"], case["top_k"], case["experts"], case["cols"]
        token, rows = T * D * size, T * k * D * size
        small = T * k * 4
        # ids in, the two orders out; x and y read, rows and out written; the router's weights
        nbytes = 3 * small + 4 * (E + 1) + token + rows + rows + token + small
        flops = 2 * T * k * D
        if case["grad"]:
            nbytes += token + rows + rows + 2 * small      # d_out, y again for the backward pass; d_y, d_w
            nbytes += rows + token                         # d_rows; d_x
            flops += 4 * T * k * D
        return {"bytes": nbytes, "flops": flops}
    out = {"f32": 4, "bf16": 2, "f16": 2}[case["out"]]
    R, N, K, active = case["rows"], case["N"], case["K"], case["active"]
    if case["op"] == "experts":
        nbytes = active * K * N * size + 4 * (case["experts"] + 1)
        flops = 0
        if case["forward"]:
            nbytes += (R * N * out) + (R * K * size)
            flops += 2 * R * N * K
        if case["grad"]:
            nbytes += R * N * size + R * K * out + case["experts"] * K * N * out
            nbytes += 0 if case["forward"] else R * K * size
            flops += 4 * R * N * K
        return {"bytes": nbytes, "flops": flops}
    groups = (K + case["group"] - 1) // case["group"]
    return {"bytes": active * N * ((K + 1) // 2 + groups * size) + R * K * size + R * N * out,
            "flops": 2 * R * N * K}
