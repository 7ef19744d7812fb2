"""A mixture-of-experts layer on the library's operators: a training step and a decoding step.

The layer: a router picks `top_k` of `experts` for each token, each expert is a gated pair of
projections y = (silu(x W1) * (x W3)) W2, and the experts' results are summed with the router's
weights.  The step below runs forward and backward through

    sort -> gather -> the gated pair -> the product W2 -> combine   (tile_gemm_expert_*, _gated, _grouped)
    combine's gradient -> the gate's gradient -> transposed products, weights' gradients -> the
    gather's gradient                                               (tile_gemm_gated_grad, _grouped_wgrad)

and decoding runs the same layer with the three projections in 4 bits (tile_gemm_pack_q4 once,
tile_gemm_q4 each step, tile_gemm_gate between).  torch supplies memory and the router's softmax.

    python examples/expert_layer.py            # checks against plain torch, prints times
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tile_scheduled_dense_amd as tg  # noqa: E402

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Routing:
    """The expert order of one batch: offsets, and the row of every entry (token, choice)."""

    def __init__(self, tokens, top_k, experts, device="cuda"):
        self.shape = (tokens, top_k, experts)
        n = tokens * top_k
        self.offsets = torch.empty(experts + 1, dtype=I32, device=device)
        self.entry_of_row = torch.empty(n, dtype=I32, device=device)
        self.row_of_entry = torch.empty(n, dtype=I32, device=device)
        size = tg.tile_gemm_expert_sort_workspace_size(tokens, top_k, experts)
        self.workspace = torch.empty(size // 4, dtype=I32, device=device) if size else None

    def sort(self, ids):
        T, k, E = self.shape
        tg.tile_gemm_expert_sort(T, k, E, ids, k, self.offsets, self.entry_of_row, self.row_of_entry,
                                 workspace=self.workspace)

    def gather(self, x):
        T, k, _ = self.shape
        rows = torch.empty(T * k, x.shape[1], dtype=x.dtype, device=x.device)
        tg.tile_gemm_expert_gather(T, k, x.shape[1], "bf16", x, x.stride(0), self.row_of_entry, rows, rows.stride(0))
        return rows

    def combine(self, y, weights=None):
        T, k, _ = self.shape
        out = torch.empty(T, y.shape[1], dtype=y.dtype, device=y.device)
        tg.tile_gemm_expert_combine(T, k, y.shape[1], "bf16", y, y.stride(0), self.row_of_entry, weights, k, out,
                                    out.stride(0))
        return out

    def combine_grad(self, d_out, y, weights):
        T, k, _ = self.shape
        d_y, d_w = torch.empty_like(y), torch.empty(T, k, dtype=F32, device=y.device)
        tg.tile_gemm_expert_combine_grad(T, k, y.shape[1], "bf16", d_out, d_out.stride(0), y, y.stride(0),
                                         self.row_of_entry, weights, k, d_y, d_y.stride(0), d_w, k)
        return d_y, d_w

    def product(self, a, w, transposed=False):
        """a (rows x K) times every expert's w (K x N), or its transpose."""
        E, K, N = w.shape
        if transposed:
            K, N = N, K
        c = torch.empty(a.shape[0], N, dtype=BF16, device=a.device)
        tg.tile_gemm_grouped(E, a.shape[0], N, K, "bf16", a, a.stride(0), w, w.stride(1), w.stride(0), c, c.stride(0),
                             self.offsets, c_dtype="bf16", transposed=int(transposed))
        return c

    def gated(self, a, w1, w3):
        """silu(a w1) * (a w3) of every expert's rows, and the two products."""
        E, K, N = w1.shape
        h, u, v = (torch.empty(a.shape[0], N, dtype=BF16, device=a.device) for _ in range(3))
        size = tg.tile_gemm_gated_workspace_size(E, a.shape[0], N, K, "bf16")
        workspace = torch.empty(size, dtype=torch.uint8, device=a.device) if size else None
        tg.tile_gemm_gated(E, a.shape[0], N, K, "bf16", a, a.stride(0), w1, w3, w1.stride(1), w1.stride(0), h, N,
                           self.offsets, activation=tg.ACT_SILU, U=u, V=v, ldu=N, workspace=workspace)
        return h, u, v

    def gated_grad(self, d_y, w2, u, v):
        """The gradients of u and v from that of the rows' results."""
        E, N, K = w2.shape
        d_u, d_v = torch.empty_like(u), torch.empty_like(v)
        tg.tile_gemm_gated_grad(E, d_y.shape[0], N, K, "bf16", d_y, d_y.stride(0), w2, w2.stride(1), w2.stride(0), u, v, N,
                                d_u, d_v, N, self.offsets, activation=tg.ACT_SILU, transposed=1)
        return d_u, d_v

    def weight_grad(self, a, d):
        E = self.shape[2]
        g = torch.empty(E, a.shape[1], d.shape[1], dtype=F32, device=a.device)
        tg.tile_gemm_grouped_wgrad(E, a.shape[0], a.shape[1], d.shape[1], "bf16", a, a.stride(0), d, d.stride(0), g,
                                   g.stride(1), g.stride(0), self.offsets, c_dtype="f32")
        return g


def route(x, router, top_k):
    top, ids = (x.float() @ router).topk(top_k, dim=1)
    return ids.to(I32).contiguous(), torch.softmax(top, dim=1).contiguous()


def train_step(routing, x, router, w1, w3, w2, d_out, top_k):
    """Forward and backward; returns the output and the gradients of x, the router's weights, w1, w3, w2."""
    ids, weights = route(x, router, top_k)
    routing.sort(ids)
    rows = routing.gather(x)
    g, h1, h3 = routing.gated(rows, w1, w3)
    y = routing.product(g, w2)
    out = routing.combine(y, weights)
    d_y, d_w = routing.combine_grad(d_out, y, weights)
    d_h1, d_h3 = routing.gated_grad(d_y, w2, h1, h3)
    d_rows = routing.product(d_h1, w1, transposed=True) + routing.product(d_h3, w3, transposed=True)
    d_x = routing.combine(d_rows)
    return out, d_x, d_w, routing.weight_grad(rows, d_h1), routing.weight_grad(rows, d_h3), routing.weight_grad(g, d_y)


class Q4Weights:
    """Every expert's w (K x N) as packed 4-bit codes with one scale per `group` k."""

    def __init__(self, w, group=128):
        E, K, N = w.shape
        t = w.float().transpose(1, 2)                                   # experts x N x K
        G = -(-K // group)
        padded = torch.nn.functional.pad(t, (0, G * group - K)).reshape(E, N, G, group)
        self.scales = (padded.abs().amax(3) / 7).clamp_min(1e-8).to(BF16)
        codes = (padded / self.scales.float()[..., None]).round().clamp(-8, 7).add(8).to(torch.uint8)
        codes = torch.nn.functional.pad(codes.reshape(E, N, -1)[:, :, :K], (0, K % 2), value=8)
        self.codes = (codes[:, :, 0::2] | codes[:, :, 1::2] << 4).contiguous()
        self.shape, self.group = (E, K, N), group
        self.packed = torch.empty(tg.tile_gemm_q4_packed_size(E, N, K, group, "bf16"), dtype=torch.uint8, device=w.device)
        tg.tile_gemm_pack_q4(E, N, K, group, "bf16", self.codes, self.codes.stride(1), self.codes.stride(0), self.scales,
                             self.scales.stride(1), self.scales.stride(0), self.packed)

    def product(self, a, offsets):
        E, K, N = self.shape
        c = torch.empty(a.shape[0], N, dtype=BF16, device=a.device)
        tg.tile_gemm_q4(E, a.shape[0], N, K, self.group, "bf16", a, a.stride(0), self.packed, c, c.stride(0), offsets,
                        c_dtype="bf16")
        return c

    def dense(self):
        """The same weights in fp32, K x N per expert (for checks)."""
        E, K, N = self.shape
        c = torch.stack([self.codes & 15, self.codes >> 4], dim=3).reshape(E, N, -1)[:, :, :K].float() - 8
        return (c * self.scales.float().repeat_interleave(self.group, dim=2)[:, :, :K]).transpose(1, 2).contiguous()


def decode_step(routing, x, router, q1, q3, q2, top_k):
    ids, weights = route(x, router, top_k)
    routing.sort(ids)
    rows = routing.gather(x)
    h1, h3 = q1.product(rows, routing.offsets), q3.product(rows, routing.offsets)
    g = torch.empty_like(h1)
    tg.tile_gemm_gate(h1.shape[0], h1.shape[1], "bf16", h1, h3, h1.stride(0), g, g.stride(0), activation=tg.ACT_SILU)
    return routing.combine(q2.product(g, routing.offsets), weights)


def plain(x, router, w1, w3, w2, top_k):
    """The layer in fp32 torch, expert by expert."""
    ids, weights = route(x, router, top_k)
    out = torch.zeros(x.shape[0], w2.shape[2], device=x.device)
    for e in range(w1.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        h = x.float()[t]
        y = (torch.nn.functional.silu(h @ w1[e].float()) * (h @ w3[e].float())) @ w2[e].float()
        out.index_add_(0, t, y * weights[t, j][:, None])
    return out


def far(got, want):
    return float((got.float() - want.float()).norm() / want.float().norm())


def make(tokens, experts, cols, hidden, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    x = normal(tokens, cols).to(BF16)
    router = normal(cols, experts, scale=cols ** -0.5)
    w1, w3 = (normal(experts, cols, hidden, scale=cols ** -0.5).to(BF16) for _ in range(2))
    w2 = normal(experts, hidden, cols, scale=hidden ** -0.5).to(BF16)
    return x, router, w1, w3, w2, normal(tokens, cols, scale=0.1).to(BF16)


def main():
    top_k, experts, cols, hidden = 2, 8, 1024, 2048
    x, router, w1, w3, w2, d_out = make(4096, experts, cols, hidden)
    routing = Routing(x.shape[0], top_k, experts)
    out, d_x, d_w, d_w1, d_w3, d_w2 = train_step(routing, x, router, w1, w3, w2, d_out, top_k)
    want = plain(x, router, w1, w3, w2, top_k)
    print(f"training step: output {far(out, want):.1e} from plain fp32")
    q = [Q4Weights(w) for w in (w1, w3, w2)]
    few = x[:16].contiguous()
    decode = Routing(16, top_k, experts)
    got = decode_step(decode, few, router, *q, top_k)
    want = plain(few, router, *[w.dense() for w in q], top_k)
    print(f"decoding step, 4-bit weights: output {far(got, want):.1e} from plain fp32 on the same weights")
    for name, step in (("training step", lambda: train_step(routing, x, router, w1, w3, w2, d_out, top_k)),
                       ("decoding step", lambda: decode_step(decode, few, router, *q, top_k))):
        for _ in range(20):
            step()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(50):
            step()
        end.record()
        torch.cuda.synchronize()
        print(f"{name}: {start.elapsed_time(end) / 50:.3f} ms")


if __name__ == "__main__":
    main()
