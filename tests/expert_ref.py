"""Plain forms, in 64 bits on the CPU, of the operators of a mixture-of-experts layer, and the
bounds their results are held to.

Bounds.  An fp32 sum of n products, in any order, is within (n + 2) * 2^-24 * sum |a||b| of the
exact one where every operation rounds to nearest; the matrix instructions may truncate, which
doubles a step, so 2 * (n + 2) * 2^-24 * sum |a||b| it is.  A 16-bit result adds half a step of
its type, eps / 2 relative to the value (bf16 2^-8, fp16 2^-11), and half of the smallest
subnormal.
"""
from __future__ import annotations

import torch

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}


def bound(ref, terms, absum, dtype):
    """Largest |got - ref| allowed for sums of `terms` products with sum |a||b| = absum."""
    b = 2 * (terms + 2) * 2.0 ** -24 * absum
    t = TYPES[dtype]
    return b + (ref.abs() + b) * torch.finfo(t).eps / 2 + TINY[dtype] / 2


def check(got, ref, terms, absum, dtype):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape
    assert not torch.isnan(got).any(), "NaN in the result"
    over = (got - ref).abs() - bound(ref, terms, absum, dtype)
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, f"{worst:.3e} over the bound"


def sort(ids, experts):
    """offsets, entry_of_row, row_of_entry (int32 lists) of a tokens x top_k table of ids."""
    flat = ids.reshape(-1).tolist()
    order = sorted(range(len(flat)), key=lambda e: (flat[e] if 0 <= flat[e] < experts else experts, e))
    counts = [0] * (experts + 1)
    for e in flat:
        counts[e if 0 <= e < experts else experts] += 1
    offsets = [0]
    for c in counts[:experts]:
        offsets.append(offsets[-1] + c)
    n = offsets[-1]
    rows = [0] * len(flat)
    for r, e in enumerate(order):
        rows[e] = r if r < n else ~r
    return offsets, [e if r < n else ~e for r, e in enumerate(order)], rows


def grouped(A, B, offsets, rows, transposed=False):
    """C and sum |a||b|; B: experts x K x N (or N x K)."""
    A, B = A.detach().cpu().double(), B.detach().cpu().double()
    if transposed:
        B = B.transpose(1, 2).contiguous()
    C = torch.zeros(rows, B.shape[2], dtype=torch.float64)
    D = torch.zeros_like(C)
    for g in range(B.shape[0]):
        lo, hi = offsets[g], offsets[g + 1]
        C[lo:hi] = A[lo:hi] @ B[g]
        D[lo:hi] = A[lo:hi].abs() @ B[g].abs()
    return C, D


def wgrad(A, D, offsets):
    A, D = A.detach().cpu().double(), D.detach().cpu().double()
    E = len(offsets) - 1
    C = torch.zeros(E, A.shape[1], D.shape[1], dtype=torch.float64)
    S = torch.zeros_like(C)
    for g in range(E):
        a, d = A[offsets[g]:offsets[g + 1]], D[offsets[g]:offsets[g + 1]]
        C[g] = a.t().contiguous() @ d
        S[g] = a.abs().t().contiguous() @ d.abs()
    return C, S


def q4_weights(codes, scales, N, K, group):
    """experts x N x K in 64 bits; codes experts x N x ceil(K / 2) bytes."""
    c = codes.cpu().to(torch.int64)
    w = torch.stack([c % 16, c // 16], dim=3).reshape(c.shape[0], N, -1)[:, :, :K].double() - 8
    s = scales.detach().cpu().double().repeat_interleave(group, dim=2)[:, :, :K]
    return w * s
