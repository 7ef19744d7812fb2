"""Plain forms, in 64 bits, of the operators of a feed-forward block, and the bounds their
results are held to.

With e = 2^-24 (half a step of fp32): a sum of n products is within 2 (n + 2) e sum |a||b|
(tests/expert_ref.py).  The activations are evaluated in fp32 from functions of one step's error:

  act(u)    the logistic function s = 1 / (1 + E), E = e^-u: two roundings of E's exponent
            (2 |u| e relative in E), one step each of exp2 and the reciprocal, the sum's rounding:
            (2 |u| + 6) e relative, and SiLU's product one more.  GELU is within 2.4e-7 |u| of
            u Phi(u).  Together  err_f = (|f| (2 |u| + 8) + 5 |u|) e.
  act'(u)   SiLU: s (1 + u (1 - s)): the absolute error of s, at most 6 e for u > 0 and s (2 |u| + 5) e
            below, times |u|, whose product s u^2 stays below 1.  GELU: Phi within 2.4e-7, u phi(u)
            with an exponent of three roundings, |u|^3 phi(u) below 0.5.  Together
            err_d = (8 |u| + 16) e.

|act'| is at most 1.13, so an error of u enters act(u) with that factor.  Each product of the formulas
adds a rounding; a 16-bit result half a step of its type.
"""
from __future__ import annotations

import math

import torch

from tests.expert_ref import TINY, TYPES

E24 = 2.0 ** -24
NONE, RELU, GELU, SILU = range(4)


def act(u, kind):
    """act(u) and act'(u) in 64 bits."""
    if kind == RELU:
        return u.clamp_min(0), (u > 0).double()
    if kind == GELU:
        cdf = torch.special.ndtr(u)
        return u * cdf, cdf + u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)
    if kind == SILU:
        s = torch.sigmoid(u)
        return u * s, s + u * s * torch.sigmoid(-u)
    return u, torch.ones_like(u)


def err_act(u, f):
    return (f.abs() * (2 * u.abs() + 8) + 5 * u.abs()) * E24


def err_slope(u):
    return (8 * u.abs() + 16) * E24


def sum_error(n, absum):
    return 2 * (n + 2) * E24 * absum


def check(got, ref, error, dtype, what=""):
    """|got - ref| within `error` and one rounding to dtype."""
    t = TYPES[dtype]
    got = got.to(ref.device).double()
    assert got.shape == ref.shape
    assert not torch.isnan(got).any(), f"NaN in {what}"
    room = error + (ref.abs() + error) * torch.finfo(t).eps / 2 + TINY[dtype] / 2
    over = (got - ref).abs() - room
    worst = float(over.max()) if over.numel() else 0.0
    assert worst <= 0, f"{what}: {worst:.3e} over the bound"


def group_rows(offsets, g, order=None):
    at = torch.arange(offsets[g], offsets[g + 1])
    return at if order is None else order[at]


def dense(m, transposed):
    m = m.double()
    return m.transpose(-1, -2).contiguous() if transposed else m


def gated(x, bg, bu, offsets, transposed):
    """u, v and their sums |a||b|; zeros for rows of no expert."""
    x = x.double()
    out = [torch.zeros(x.shape[0], bg.shape[1 if transposed else 2], dtype=torch.float64, device=x.device) for _ in range(4)]
    for g in range(bg.shape[0]):
        lo, hi = offsets[g], offsets[g + 1]
        for i, b in enumerate((bg[g], bu[g])):
            w = dense(b, transposed)
            out[i][lo:hi] = x[lo:hi] @ w
            out[2 + i][lo:hi] = x[lo:hi].abs() @ w.abs()
    return out


def check_gated(got_h, got_u, got_v, x, bg, bu, offsets, transposed, kind, dtype):
    u, v, su, sv = gated(x, bg, bu, offsets, transposed)
    K = x.shape[1]
    eu, ev = sum_error(K, su), sum_error(K, sv)
    f, _ = act(u, kind)
    ef = 1.13 * eu + err_act(u, f)
    check(got_h, f * v, ef * (v.abs() + ev) + f.abs() * ev + 2 * E24 * (f * v).abs(), dtype, "h")
    if got_u is not None:
        check(got_u, u, eu, dtype, "u")
        check(got_v, v, ev, dtype, "v")


def check_gate_grad(d_u, d_v, h, d_h, s, K, u, v, live, kind, dtype):
    """d_h and its sum |a||b| s in 64 bits; u, v as stored; live: rows of an expert."""
    u, v = (torch.where(live[:, None], t.double(), 0) for t in (u, v))
    f, d = act(u, kind)
    e, ef, ed = sum_error(K, s), err_act(u, f), err_slope(u)
    want = d_h * v * d
    check(d_u, want, v.abs() * ((d.abs() + ed) * e + d_h.abs() * ed) + 3 * E24 * want.abs(), dtype, "d_u")
    want = d_h * f
    check(d_v, want, (f.abs() + ef) * e + d_h.abs() * ef + 2 * E24 * want.abs(), dtype, "d_v")
    if h is not None:
        check(h, f * v, ef * v.abs() + 2 * E24 * (f * v).abs(), dtype, "h")


def adapters(x, w, a, b, scales, offsets, order, transposed, dtype):
    """y, t and the errors they may have; t is taken with a rounding to dtype on its way."""
    x, w = x.double(), dense(w, transposed)
    K, rank = x.shape[1], a.shape[1 if transposed else 2]
    y, y_err = x @ w, sum_error(K, x.abs() @ w.abs())
    t = torch.zeros(x.shape[0], rank, dtype=torch.float64, device=x.device)
    t_err = torch.zeros_like(t)
    for g in range(a.shape[0]):
        at = group_rows(offsets, g, order).to(x.device)
        if at.numel() == 0:
            continue
        ag, bg, s = dense(a[g], transposed), dense(b[g], transposed), float(scales[g]) if scales is not None else 1.0
        t[at] = x[at] @ ag * s
        t_err[at] = sum_error(K, x[at].abs() @ ag.abs()) * abs(s) + E24 * t[at].abs()
        rounded = t_err[at] + (t[at].abs() + t_err[at]) * torch.finfo(TYPES[dtype]).eps / 2 + TINY[dtype] / 2
        y[at] += t[at] @ bg
        y_err[at] += rounded @ bg.abs() + sum_error(rank + 2, (t[at].abs() + rounded) @ bg.abs()) + E24 * y[at].abs()
    return y, y_err, t, t_err


def adapters_wgrad(x, s, offsets, order):
    """x^T s over every adapter's rows, and its sum |a||b| and number of terms."""
    x, s = x.double(), s.double()
    G = len(offsets) - 1
    c = torch.zeros(G, x.shape[1], s.shape[1], dtype=torch.float64, device=x.device)
    absum, terms = torch.zeros_like(c), torch.zeros(G, 1, 1, dtype=torch.float64, device=x.device)
    for g in range(G):
        at = group_rows(offsets, g, order).to(x.device)
        c[g] = x[at].t().contiguous() @ s[at]
        absum[g] = x[at].abs().t().contiguous() @ s[at].abs()
        terms[g] = at.numel()
    return c, absum, terms
