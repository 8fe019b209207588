"""The expert block's operators in 64 bits, and the tolerances of their kernels
(test code only).

Half a step of an output type is h = finfo.eps / 2 relative to the value (bf16
2^-8).  An fp32 sum of K products is off by at most K u S, S the sum of the
products' magnitudes, u = 2^-23 (the tensor core's adder may truncate, so a
whole step and not half of one).  Every tolerance below is h |value| for the
one rounding to the output's type plus the fp32 errors carried to it.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -23
BF = torch.finfo(torch.bfloat16).eps / 2
D = torch.float64


def act64(g, kind):
    """act(g), act'(g)."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = torch.special.ndtr(g)
    return g * c, c + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def product64(a, b):
    """a b^T and the bound of its fp32 error (a [n][K], b [m][K])."""
    a, b = a.to(D), b.to(D)
    return a @ b.T, a.shape[1] * U * (a.abs() @ b.abs().T)


def act_err(g):
    """Bound of the fp32 activation's own error, absolute, for act and act':
    the exponential (2 ulp, and its argument's rounding, |g| u, times the
    value), the division and the products; erf to 2 ulp of 1 times |g|."""
    return 8 * U * (1 + g.abs()) ** 2


def gate_up64(x, w, kind):
    """hid, its tolerance, gate_up, its tolerance."""
    gu, e = product64(x, w)
    g, u = gu.chunk(2, 1)
    eg, eu = e.chunk(2, 1)
    a, _ = act64(g, kind)
    hid = a * u
    # |act'| <= 1.13 for both activations
    tol = BF * hid.abs() * 1.01 + (1.13 * eg + act_err(g)) * (u.abs() + eu) + a.abs() * eu + 2.0 ** -126
    return hid, tol, gu, BF * gu.abs() * 1.01 + e


def down_bwd64(dy, w, gate_up, kind):
    """d_gate_up, its tolerance, hid, its tolerance."""
    dh, e = product64(dy, w.T)
    g, u = gate_up.to(D).chunk(2, 1)
    a, s = act64(g, kind)
    err = act_err(g)
    dg, du, hid = dh * u * s, dh * a, a * u
    tg = BF * dg.abs() * 1.01 + e * u.abs() * (s.abs() + err) + dh.abs() * u.abs() * err
    tu = BF * du.abs() * 1.01 + e * (a.abs() + err) + dh.abs() * err
    return torch.cat([dg, du], 1), torch.cat([tg, tu], 1), hid, BF * hid.abs() * 1.01 + u.abs() * err


def close(got, want, tol, what):
    got = got.to(D).cpu()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = (got - want).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} values off, first at "
        f"{bad.nonzero()[0].tolist()}: {got[bad][0].item()} for {want[bad][0].item()} "
        f"(allowed {tol.expand_as(bad)[bad][0].item()})")
