"""The norms after and before a block with its gate and residual scale, forward
and backward, against 64-bit values.

Tolerances: an output rounded to bf16 is off by half a step (2^-8 of the value)
plus the fp32 error before it.  A value of the kernels goes through at most
some 16 fp32 roundings besides its row's sums; a row's sums of H terms have
relative error H/256 + 16 steps at most (a thread adds at most 64 terms in turn
and the rest go over a tree), which 2^-16 of the terms' magnitudes covers up to
H = 16384; sums over T tokens are bounded by T 2^-23 of their magnitudes.
"""
from __future__ import annotations

import pytest
import torch

from block64 import BF, D, U, close

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
EPS = 1e-6
REL = 2.0 ** -16


def _ep():
    import combine_layout_gb300.moe_ep as ep
    return ep


def _inputs(T, H, post, gate, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(o=r(T, H).bfloat16(), res=(2 * r(T, H)).bfloat16(), w_post=1 + 0.2 * r(H) if post else None,
                gate=None if gate == "none" else 0.5 + 0.3 * r(T if gate == "token" else H), w_pre=1 + 0.2 * r(H),
                dr=r(T, H).bfloat16(), dy=r(T, H).bfloat16())


def _d(t):
    return None if t is None else t.to(D)


def _forward64(s, scale, gate):
    o, res, wp, g, wq = (_d(s[n]) for n in ("o", "res", "w_post", "gate", "w_pre"))
    g = 1.0 if g is None else g[:, None] if gate == "token" else g
    p = (o.pow(2).mean(1, keepdim=True) + EPS).rsqrt()
    u = o if wp is None else wp * o * p
    r = scale * res + g * u
    q = (r.pow(2).mean(1, keepdim=True) + EPS).rsqrt()
    mag = abs(scale) * res.abs() + (g * u).abs()
    return r, mag, wq * r * q, (wq * q).abs() * mag


def _dev(s):
    return {n: None if t is None else t.to(DEV) for n, t in s.items()}


SIZES = [(1, 8), (1, 7168), (3, 264), (200, 1024), (37, 4104), (5, 8200), (2, 16384), (700, 256)]
FORMS = [(True, "none", 1.0), (True, "channel", 0.75), (False, "token", 0.5), (True, "token", 1.0), (False, "none", 0.0)]


@pytest.mark.parametrize("post,gate,scale", FORMS)
@pytest.mark.parametrize("T,H", SIZES)
def test_forward(T, H, post, gate, scale):
    ep = _ep()
    grp = ep.moe_ep_create_group(1, 1, 1, 4, H)
    s = _inputs(T, H, post, gate)
    d = _dev(s)
    out, y = torch.zeros_like(d["o"]), torch.zeros_like(d["o"])
    ep.moe_ep_norm_residual(grp, d["o"], d["res"], d["w_post"], d["gate"], d["w_pre"], out, y, res_scale=scale,
                            gate_per_token=gate == "token", eps=EPS)
    r, rm, v, vm = _forward64(s, scale, gate)
    close(out, r, BF * r.abs() * 1.01 + REL * rm, "res_out")
    close(y, v, BF * v.abs() * 1.01 + REL * vm, "y")
    # either output alone, and in place, gives the same values
    o2, r2 = d["o"].clone(), d["res"].clone()
    ep.moe_ep_norm_residual(grp, o2, r2, d["w_post"], d["gate"], d["w_pre"], r2, o2, res_scale=scale,
                            gate_per_token=gate == "token", eps=EPS)
    assert torch.equal(r2, out) and torch.equal(o2, y)
    only = torch.zeros_like(y)
    ep.moe_ep_norm_residual(grp, d["o"], d["res"], d["w_post"], d["gate"], d["w_pre"], None, only, res_scale=scale,
                            gate_per_token=gate == "token", eps=EPS)
    assert torch.equal(only, y)
    ep.moe_ep_destroy_group(grp)


@pytest.mark.parametrize("post,gate,scale", FORMS)
@pytest.mark.parametrize("T,H", SIZES)
def test_backward(T, H, post, gate, scale):
    ep = _ep()
    grp = ep.moe_ep_create_group(1, 1, 1, 4, H)
    s = _inputs(T, H, post, gate, seed=1)
    d = _dev(s)
    work = torch.full((ep.moe_ep_norm_work_floats(grp),), float("nan"), device=DEV)
    nan = lambda t: None if t is None else torch.full(t.shape, float("nan"), dtype=t.dtype, device=DEV)  # noqa: E731
    out = dict(d_o=nan(s["o"]), dres=nan(s["o"]), dw_post=nan(s["w_post"]), dgate=nan(s["gate"]), dw_pre=nan(s["w_pre"]))

    def call(out):
        ep.moe_ep_norm_residual_backward(grp, d["o"], d["res"], d["w_post"], d["gate"], d["w_pre"], d["dr"], d["dy"],
                                         out["d_o"], out["dres"], out["dw_post"], out["dgate"], out["dw_pre"], work,
                                         res_scale=scale, gate_per_token=gate == "token", eps=EPS)

    call(out)
    again = {n: nan(t) for n, t in out.items()}
    call(again)
    for n, t in out.items():
        assert t is None or torch.equal(t, again[n]), n
    # 64 bits, by differentiating the forward formula
    leaf = {n: t.to(D).requires_grad_() for n, t in s.items() if t is not None and n not in ("dr", "dy")}
    r, _, y, _ = _forward64({**s, **leaf}, scale, gate)
    ((r * s["dr"].to(D)).sum() + (y * s["dy"].to(D)).sum()).backward()
    want = {n: leaf[m].grad for n, m in (("d_o", "o"), ("dres", "res"), ("dw_post", "w_post"), ("dgate", "gate"),
                                         ("dw_pre", "w_pre")) if m in leaf}
    # magnitudes: each gradient's terms taken without their signs
    with torch.no_grad():
        o, dr, dy, wq = (s[n].to(D) for n in ("o", "dr", "dy", "w_pre"))
        g = 1.0 if s["gate"] is None else s["gate"].to(D)[:, None] if gate == "token" else s["gate"].to(D)
        wp = None if not post else s["w_post"].to(D)
        p = (o.pow(2).mean(1, keepdim=True) + EPS).rsqrt()
        u = o if wp is None else wp * o * p
        rr, rm, _, _ = _forward64(s, scale, gate)
        q = (rr.pow(2).mean(1, keepdim=True) + EPS).rsqrt()
        n, nm, v = rr * q, rm * q, wq * dy
        # n's magnitude and its relative error enter twice
        dm = dr.abs() + q * (v.abs() + nm * (v.abs() * nm).mean(1, keepdim=True))
        tok = REL + T * U
        mag = dict(dres=abs(scale) * dm, dw_pre=(dy.abs() * nm).sum(0))
        du = (g if isinstance(g, float) else g.abs()) * dm
        if s["gate"] is not None:
            mag["dgate"] = (dm * u.abs()).sum(1 if gate == "token" else 0)
        if wp is None:
            mag["d_o"] = du
        else:
            m = (o * p).abs()
            z = du * wp.abs()
            mag["d_o"] = p * (z + m * (z * m).mean(1, keepdim=True))
            mag["dw_post"] = (du * m).sum(0)
    for name, t in want.items():
        half = BF if name in ("d_o", "dres") else 2.0 ** -24
        close(out[name], t, half * t.abs() * 1.01 + 4 * tok * mag[name], name)
    ep.moe_ep_destroy_group(grp)


def test_backward_against_differences():
    ep = _ep()
    T, H = 4, 64
    grp = ep.moe_ep_create_group(1, 1, 1, 4, H)
    s = _inputs(T, H, True, "channel", seed=5)
    d = _dev(s)
    work = torch.zeros(ep.moe_ep_norm_work_floats(grp), device=DEV)
    out = {n: torch.zeros_like(d[m]) for n, m in (("d_o", "o"), ("dres", "res"), ("dw_post", "w_post"),
                                                  ("dgate", "gate"), ("dw_pre", "w_pre"))}
    ep.moe_ep_norm_residual_backward(grp, d["o"], d["res"], d["w_post"], d["gate"], d["w_pre"], d["dr"], d["dy"],
                                     *(out[n] for n in ("d_o", "dres", "dw_post", "dgate", "dw_pre")), work,
                                     res_scale=0.5, eps=EPS)
    gen = torch.Generator().manual_seed(9)

    def loss(t):
        r, _, y, _ = _forward64(t, 0.5, "channel")
        return float((r * s["dr"].to(D)).sum() + (y * s["dy"].to(D)).sum())

    for name, m in (("d_o", "o"), ("dres", "res"), ("dw_post", "w_post"), ("dgate", "gate"), ("dw_pre", "w_pre")):
        v = torch.randn(s[m].shape, generator=gen, dtype=D)
        step = 1e-5
        want = (loss({**s, m: s[m].to(D) + step * v}) - loss({**s, m: s[m].to(D) - step * v})) / (2 * step)
        got = out[name].to(D).cpu()
        # one rounding of each value, all of the same sign at worst
        assert abs(float((got * v).sum()) - want) <= 2 * BF * float((got * v).abs().sum())
    ep.moe_ep_destroy_group(grp)


def test_optional_arguments_and_special_rows():
    ep = _ep()
    T, H = 6, 512
    grp = ep.moe_ep_create_group(1, 1, 1, 4, H)
    s = _inputs(T, H, True, "none", seed=3)
    s["res"][2] = 0                  # a row of zeros: y = 0, no division by zero
    s["res"][4] = 1e18               # squares stay finite in fp32
    d = _dev(s)
    y = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    ep.moe_ep_norm_residual(grp, None, d["res"], None, None, d["w_pre"], None, y, eps=EPS)
    r = s["res"].to(D)
    want = s["w_pre"].to(D) * r * (r.pow(2).mean(1, keepdim=True) + EPS).rsqrt()
    close(y, want, BF * want.abs() * 1.01 + REL * want.abs(), "y of the residual alone")
    assert bool((y[2] == 0).all())
    # a NaN stays in its row
    d["o"][1, 7] = float("nan")
    out = torch.zeros_like(y)
    ep.moe_ep_norm_residual(grp, d["o"], None, d["w_post"], None, None, out, None, eps=EPS)
    assert torch.isnan(out.float()).any(1).cpu().tolist() == [False, True] + [False] * 4
    # no tokens: weight gradients are zero, nothing else is written
    work = torch.zeros(ep.moe_ep_norm_work_floats(grp), device=DEV)
    dw = torch.full((H,), 3.0, device=DEV)
    ep.moe_ep_norm_residual_backward(grp, d["o"], d["res"], None, None, d["w_pre"], d["dr"], d["dy"], None, None,
                                     None, None, dw, work, num_tokens=0)
    assert bool((dw == 0).all())
    ep.moe_ep_norm_residual(grp, d["o"], d["res"], None, None, d["w_pre"], None, y, num_tokens=0)
    # one gradient alone: dy NULL leaves dres = scale * dr
    dres = torch.zeros_like(y)
    ep.moe_ep_norm_residual_backward(grp, None, d["res"], None, None, None, d["dr"], None, None, dres, None, None,
                                     None, work, res_scale=0.5)
    assert torch.equal(dres, (0.5 * d["dr"].float()).bfloat16())
    ep.moe_ep_destroy_group(grp)


def test_refusals():
    ep = _ep()
    H = 64
    grp = ep.moe_ep_create_group(1, 1, 1, 4, H)
    wide = ep.moe_ep_create_group(1, 1, 1, 4, 16392)
    z = torch.zeros((4, H), dtype=torch.bfloat16, device=DEV)
    big = torch.zeros((2, 16392), dtype=torch.bfloat16, device=DEV)
    w = torch.ones(H, device=DEV)
    buf = torch.zeros(9 * H, dtype=torch.bfloat16, device=DEV)
    bad = [
        lambda: ep.moe_ep_norm_residual(grp, z, z, None, None, None, None, None),          # no output
        lambda: ep.moe_ep_norm_residual(grp, None, None, None, None, w, None, z, num_tokens=4),
        lambda: ep.moe_ep_norm_residual(grp, None, z, w, None, w, None, z.clone()),        # w_post without o
        lambda: ep.moe_ep_norm_residual(grp, z, z, None, None, None, None, z.clone()),     # y without w_pre
        lambda: ep.moe_ep_norm_residual(grp, z, z, None, None, w, None, z.clone(), eps=-1.0),
        lambda: ep.moe_ep_norm_residual(grp, buf[: 4 * H].view(4, H), z, None, None, w, None, buf[H:5 * H].view(4, H)),
        lambda: ep.moe_ep_norm_residual(wide, big, None, None, None, None, big.clone(), None),
        lambda: ep.moe_ep_norm_residual_backward(grp, z, z, None, None, w, None, None, None, z.clone(), None, None, None,
                                                 torch.zeros(ep.moe_ep_norm_work_floats(grp), device=DEV)),
        lambda: ep.moe_ep_norm_residual_backward(grp, z, z, None, None, w, z, z, None, z.clone(), None, w, None,
                                                 torch.zeros(ep.moe_ep_norm_work_floats(grp), device=DEV)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ep.MoeEpError) as e:
            f()
        assert e.value.status == ep.MOE_EP_ERR_INVALID, i
    with pytest.raises(ValueError):
        ep.moe_ep_norm_residual(grp, z, z, None, None, w[:8], None, z.clone())
    with pytest.raises(ValueError):
        ep.moe_ep_norm_residual_backward(grp, z, z, None, None, w, z, z, None, z.clone(), None, None, None, w)
    ep.moe_ep_destroy_group(grp)
    ep.moe_ep_destroy_group(wide)
