"""The whole block -- norm, route, dispatch, feed-forward, combine, norm with the
residual -- forward and backward, against 64 bits by automatic differentiation,
and a decoding step of it captured into a CUDA graph.

Tolerance: a value of the forward pass goes through at most 7 roundings to bf16
(x, hid, y, o, h' and x_next, and the rows of d_x on the way back add 5 more: d_o,
the rows, d_gate_up, d_x, d_h), each off by at most 2^-8 of its value; in the
2-norm of a tensor of independent values they add up to less than their number
times 2^-8, and a norm or an activation passes a relative error on by a factor
below 2.
"""
from __future__ import annotations

import math

import pytest
import torch

from block64 import BF, D
from combine_layout_gb300 import synth

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
EPS = 1e-6


def _make(mode, T, E, k, H, F, seed=0, training=True, gate="channel", S=None):
    import combine_layout_gb300.moe_ep as ep
    from combine_layout_gb300.block import MoeBlock
    from combine_layout_gb300.pipeline import EpPipeline
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    w = dict(w_gate_up=(r(E, 2 * F, H) * H ** -0.5).bfloat16(), w_down=(r(E, H, F) * F ** -0.5).bfloat16(),
             w_in=1 + 0.1 * r(H), w_post=1 + 0.1 * r(H), w_next=1 + 0.1 * r(H),
             gate=0.5 + 0.1 * r(H) if gate == "channel" else None)
    h, router = r(T, H).bfloat16(), r(H, E) * H ** -0.5
    pipe = EpPipeline(mode, E, 1, S or T, H, k, device=DEV)
    d = {n: None if t is None else t.to(DEV) for n, t in w.items()}
    block = MoeBlock(pipe, d["w_gate_up"], d["w_down"], d["w_in"], d["w_post"], d["w_next"], d["gate"], res_scale=0.9,
                     eps=EPS, training=training)
    return ep, block, pipe, w, h, router, g


def _scores(router):
    return lambda x: torch.sigmoid(x.float() @ router)


def _norm64(v, w):
    return w * v * (v.pow(2).mean(1, keepdim=True) + EPS).rsqrt()


def _reference(h, w, idx, wk, E, k):
    """The block in 64 bits with the routing given: idx [T][k], wk [T][k]."""
    T = h.shape[0]
    x = _norm64(h, w["w_in"])
    o = torch.zeros_like(h)
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        g, u = (x[t] @ w["w_gate_up"][e].T).chunk(2, 1)
        y = (g * torch.sigmoid(g) * u) @ w["w_down"][e].T
        o = o.index_add(0, t, wk[t, j, None] * y)
    hn = 0.9 * h + w["gate"] * _norm64(o, w["w_post"])
    return hn, _norm64(hn, w["w_next"])


def _near(got, want, roundings, what):
    got = got.to(D).cpu()
    off = float((got - want).norm() / want.norm())
    assert math.isfinite(off) and off <= 2 * roundings * BF, f"{what}: {off / BF:.2f} half steps"


@pytest.mark.parametrize("mode,T,E,k,H,F", [(synth.MODE_HT, 50, 8, 2, 128, 72), (synth.MODE_LL, 33, 4, 3, 264, 64),
                                           (synth.MODE_HT, 1, 8, 4, 64, 32)])
def test_block_forward_and_backward(mode, T, E, k, H, F):
    ep, block, pipe, w, h, router, g = _make(mode, T, E, k, H, F)
    pipe.recv_x.fill_(float("nan"))
    h_dev, router_dev = h.to(DEV), router.to(DEV)
    out, x_next = block.forward(h_dev, _scores(router_dev))
    d_out, d_next = (torch.randn((T, H), generator=g).bfloat16() for _ in range(2))
    d_h = block.backward(d_out.to(DEV), d_next.to(DEV))
    torch.cuda.synchronize()
    idx, wk = pipe.topk_idx[:T].cpu().long(), pipe.topk_w[:T].cpu().to(D).requires_grad_()
    leaf = {n: t.to(D).requires_grad_() for n, t in w.items()}
    h64 = h.to(D).requires_grad_()
    hn, xn = _reference(h64, leaf, idx, wk, E, k)
    ((hn * d_out.to(D)).sum() + (xn * d_next.to(D)).sum()).backward()
    _near(out, hn.detach(), 5, "h'")
    _near(x_next, xn.detach(), 6, "x_next")
    _near(d_h, h64.grad, 12, "d_h")
    _near(block.d_topk_w[:T], wk.grad, 8, "d_topk_w")
    for n in ("gate_up", "down", "in", "post", "next"):
        _near(getattr(block, f"dw_{n}"), leaf[f"w_{n}"].grad, 12, f"dw_{n}")
    _near(block.dgate, leaf["gate"].grad, 8, "dgate")
    assert pipe.device_errors() == 0
    # a second backward pass adds the experts' weight gradients up
    once = block.dw_down.clone()
    block.backward(d_out.to(DEV), d_next.to(DEV), accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(block.dw_down, once * 2)
    pipe.close()


def test_decoding_step_in_a_graph():
    T, E, k, H, F = 4, 16, 2, 256, 128
    ep, block, pipe, w, h, router, g = _make(synth.MODE_LL, T, E, k, H, F, training=False, S=8)
    h_dev, router_dev = h.to(DEV), router.to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = [t.clone() for t in block.forward(h_dev, _scores(router_dev), stream=side)]
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, x_next = block.forward(h_dev, _scores(router_dev), stream=side)
    out.zero_()
    x_next.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(x_next, first[1])
    h_dev.copy_(h_dev.flip(0))                       # new tokens, other experts
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0].flip(0)) and torch.equal(x_next, first[1].flip(0))
    pipe.close()


def test_a_serving_block_has_no_backward():
    *_, h, router, g = (made := _make(synth.MODE_HT, 4, 4, 2, 64, 32, training=False))
    block, pipe = made[1], made[2]
    block.forward(h.to(DEV), _scores(router.to(DEV)))
    with pytest.raises(ValueError):
        block.backward(h.to(DEV), h.to(DEV))
    pipe.close()
