"""The dense feed-forward operators in FP64, and the bounds their BF16 outputs
are held to.

Bounds, per element. A product of n terms accumulated in FP32 from exact BF16
products is off by at most n 2^-24 of the sum of |terms| (one rounding per
addition; any order). Below, G, U, ... are such sums of absolute terms. An
output adds its own rounding to BF16: at most 2^-8 of its value (half a step:
torch.finfo(bfloat16).eps / 2 = 2^-8), or half the smallest subnormal.
"""
import math

import torch

EPS32 = 2.0 ** -24
EPSBF = 2.0 ** -8
TINY = 2.0 ** -133  # the smallest BF16 subnormal

ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
_C0, _C1 = math.sqrt(2.0 / math.pi), 0.044715


def act64(g, act):
    """act(g) and act'(g) in FP64."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-g * math.sqrt(0.5))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    s = torch.sigmoid(2 * _C0 * (g + _C1 * g ** 3))
    return g * s, s + g * s * (1 - s) * 2 * _C0 * (1 + 3 * _C1 * g * g)


def gated64(x, wg, wu, act):
    """(h, bound of the kernel's h). |act'| <= 1.13 and |act''| <= 1.2 for
    every activation here, |act(g)| <= |g|; act itself is evaluated in FP32
    with a few roundings: 16 units of 2^-24 relative to |g|."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    n = x.shape[1] + 1
    g, u = x @ wg.T, x @ wu.T
    eg = n * EPS32 * (x.abs() @ wg.abs().T)
    eu = n * EPS32 * (x.abs() @ wu.abs().T)
    a, _ = act64(g, act)
    ea = 1.13 * eg + 16 * EPS32 * g.abs()
    h = a * u
    err = ea * u.abs() + (a.abs() + ea) * eu + 2 * EPS32 * h.abs()
    return h, err + EPSBF * (h.abs() + err) + TINY


def gated_backward64(x, wg, wu, dh, act):
    """((dx, dwg, dwu), their bounds). dg and du carry the FP32 errors of g
    and u, then one rounding to BF16 as operands of the products; |act'| <=
    1.13, |act''| <= 1.2 (so act' of a g that is off by eg is off by at most
    1.2 eg); act' is evaluated in FP32: 16 units of 2^-24 of 1 + |g|."""
    x, wg, wu, dh = x.double(), wg.double(), wu.double(), dh.double()
    T, H = x.shape
    I = wg.shape[0]
    n = H + 1
    g, u = x @ wg.T, x @ wu.T
    eg = n * EPS32 * (x.abs() @ wg.abs().T)
    eu = n * EPS32 * (x.abs() @ wu.abs().T)
    a, da = act64(g, act)
    ea = 1.13 * eg + 16 * EPS32 * g.abs()
    eda = 1.2 * eg + 16 * EPS32 * (1 + g.abs())
    dg, du = dh * u * da, dh * a
    edg = dh.abs() * (eu * (da.abs() + eda) + u.abs() * eda) + 3 * EPS32 * dg.abs()
    edu = dh.abs() * ea + 2 * EPS32 * du.abs()
    edg = edg + EPSBF * (dg.abs() + edg) + TINY
    edu = edu + EPSBF * (du.abs() + edu) + TINY

    def out(v, e, terms, count):
        e = e + count * EPS32 * terms
        return v, e + EPSBF * (v.abs() + e) + TINY

    adg, adu = dg.abs() + edg, du.abs() + edu
    dx = out(dg @ wg + du @ wu, edg @ wg.abs() + edu @ wu.abs(),
             adg @ wg.abs() + adu @ wu.abs(), 2 * I + 1)
    dwg = out(dg.T @ x, edg.T @ x.abs(), adg.T @ x.abs(), T + 1)
    dwu = out(du.T @ x, edu.T @ x.abs(), adu.T @ x.abs(), T + 1)
    return (dx[0], dwg[0], dwu[0]), (dx[1], dwg[1], dwu[1])


def adapter64(x, w, a, b, scale, ids, residual):
    """(y, bound). v = scale (A x) carries the FP32 error of its sum and of
    the scaling, then one rounding to BF16 as an operand."""
    x, w = x.double(), w.double()
    T, K = x.shape
    y = x @ w.T
    terms = x.abs() @ w.abs().T
    err = torch.zeros_like(y)
    n = rank = 0
    if a is not None:
        n, rank = a.shape[:2]
    for i in range(n):
        rows = torch.nonzero(ids == i).flatten()
        if not len(rows):
            continue
        A, B, s = a[i].double(), b[i].double(), float(scale[i])
        v = s * (x[rows] @ A.T)
        ev = (K + 2) * EPS32 * abs(s) * (x[rows].abs() @ A.abs().T)
        ev = ev + EPSBF * (v.abs() + ev) + TINY
        y[rows] += v @ B.T
        err[rows] += ev @ B.abs().T
        terms[rows] += (v.abs() + ev) @ B.abs().T
    if residual is not None:
        y = y + residual.double()
        terms = terms + residual.double().abs()
    err = err + (K + rank + 2) * EPS32 * terms
    return y, err + EPSBF * (y.abs() + err) + TINY


def assert_within(got, want, bound, what):
    got = got.double()
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), f"{what}: not finite"
    off = (got - want).abs()
    bad = off > bound
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond their bound, worst "
                           f"{float((off / bound).max()):.3g} times")


def normal(shape, std, seed, device="cuda"):
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device=device) * std).to(torch.bfloat16)
