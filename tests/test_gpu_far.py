"""The expert block's calls where element offsets pass 32 bits: rows far into a
slotted layout, the last expert's gradient, the last tokens of a long batch.
Only the far rows hold data that is looked at.
"""
from __future__ import annotations

import pytest
import torch

from block64 import BF, D, U, close, gate_up64, product64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _ep():
    import combine_layout_gb300.moe_ep as ep
    return ep


def test_slots_beyond_32_bits():
    """8 experts x 40000 slots x 8192: the last expert's rows start at element 2.3e9."""
    ep = _ep()
    E, S, H, F, T = 8, 40000, 64, 4096, 20
    gen = torch.Generator().manual_seed(0)
    g = ep.moe_ep_create_group(0, E, 1, S, H)
    h = ep.moe_ep_create_handle(g, 1)
    idx = torch.full((T, 1), E - 1, dtype=torch.int32, device=DEV)
    ep.moe_ep_route(h, None, T, 1, idx)
    at = slice((E - 1) * S, (E - 1) * S + T)
    x = torch.zeros((E * S, H), dtype=torch.bfloat16, device=DEV)
    xr = torch.randn((T, H), generator=gen).bfloat16()
    x[at] = xr.to(DEV)
    w = (torch.randn((E, 2 * F, H), generator=gen) / 8).bfloat16()
    hid = torch.full((E * S, F), 7.0, dtype=torch.bfloat16, device=DEV)
    gu = torch.full((E * S, 2 * F), 7.0, dtype=torch.bfloat16, device=DEV)
    assert gu.numel() > 2 ** 31
    ep.moe_ep_ffn_gate_up(h, x, w.to(DEV), hid, gu)
    want, tol, wgu, tgu = gate_up64(xr, w[E - 1], "silu")
    close(hid[at], want, tol, "hid")
    close(gu[at], wgu, tgu, "gate_up")
    assert bool((gu[: (E - 1) * S] == 7).all()) and bool((gu[(E - 1) * S + T:] == 7).all())
    # back through them
    wd = (torch.randn((E, H, F), generator=gen) / 64).bfloat16()
    dgu = torch.full_like(gu, 7.0)
    dy = torch.zeros_like(x)
    dy[at] = torch.randn((T, H), generator=gen).bfloat16().to(DEV)
    ep.moe_ep_ffn_down_backward(h, dy, wd.to(DEV), gu, dgu)
    dx = torch.zeros_like(x)
    ep.moe_ep_ffn_gate_up_backward(h, dgu, w.to(DEV), dx)
    want, err = product64(dgu[at].cpu(), w[E - 1].T)
    close(dx[at], want, BF * want.abs() * 1.01 + err, "dx")
    assert bool((dgu[: (E - 1) * S] == 7).all())
    ep.moe_ep_destroy_handle(h)
    ep.moe_ep_destroy_group(g)


def test_gradients_beyond_32_bits():
    """9 experts' gradients of 16384 x 16384: the last starts at element 2.1e9."""
    ep = _ep()
    E, N, T = 9, 16384, 19
    gen = torch.Generator().manual_seed(1)
    g = ep.moe_ep_create_group(1, E, 1, T, 64)
    h = ep.moe_ep_create_handle(g, 1)
    idx = torch.full((T, 1), E - 1, dtype=torch.int32, device=DEV)
    ep.moe_ep_route(h, None, T, 1, idx)
    a, b = (torch.randn((T, N), generator=gen).bfloat16() for _ in range(2))
    dw = torch.full((E, N, N), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.moe_ep_ffn_weight_grad(h, a.to(DEV), b.to(DEV), dw)
    assert bool((dw[: E - 1] == 0).all())
    for rows in (slice(0, 64), slice(N - 64, N)):
        want, err = product64(a[:, rows].T.contiguous(), b.T.contiguous())
        close(dw[E - 1, rows], want, BF * want.abs() * 1.01 + err, "dw")
    ep.moe_ep_destroy_handle(h)
    ep.moe_ep_destroy_group(g)


def test_tokens_and_rows_beyond_32_bits():
    """The norms' and the combine's last of 140000 tokens x 16384."""
    ep = _ep()
    T, H, eps = 140000, 16384, 1e-6
    g = ep.moe_ep_create_group(1, 2, 1, T, H)
    o = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    o[-2:] = torch.randn((2, H), device=DEV).bfloat16()
    w = torch.ones(H, device=DEV)
    y = torch.full_like(o, 7.0)
    ep.moe_ep_norm_residual(g, None, o, None, None, w, None, y, eps=eps)
    r = o[-2:].cpu().to(D)
    want = r * (r.pow(2).mean(1, keepdim=True) + eps).rsqrt()
    close(y[-2:], want, (BF * 1.01 + 2.0 ** -16) * want.abs(), "y")
    assert bool((y[:-2] == 0).all())
    work = torch.zeros(ep.moe_ep_norm_work_floats(g), device=DEV)
    dw = torch.zeros(H, device=DEV)
    dy = torch.zeros_like(o)
    dy[-1] = 1.0
    ep.moe_ep_norm_residual_backward(g, None, o, None, None, w, None, dy, None, y, None, None, dw, work, eps=eps)
    n = want[1]
    close(dw, n, (2.0 ** -24 + 2.0 ** -16) * n.abs() + 2.0 ** -40, "dw_pre")
    q = (r[1].pow(2).mean() + eps).rsqrt()
    grad = q * (1 - n * n.mean())
    close(y[-1], grad, BF * 1.01 * grad.abs() + 2.0 ** -14 * q, "dres")
    # the combine's backward pass: one row a token
    h = ep.moe_ep_create_handle(g, 1)
    idx = torch.zeros((T, 1), dtype=torch.int32, device=DEV)
    ep.moe_ep_route(h, None, T, 1, idx)
    tw = torch.full((T, 1), 0.5, device=DEV)
    dtw = torch.full_like(tw, 7.0)
    ep.moe_ep_combine_backward(h, o, o, tw, y, dtw)
    assert torch.equal(y[-2:], (0.5 * o[-2:].float()).bfloat16())
    want = r.pow(2).sum(1, keepdim=True)
    close(dtw[-2:], want, H * U * want, "dw")
    assert bool((dtw[:-2] == 0).all())
    ep.moe_ep_destroy_handle(h)
    ep.moe_ep_destroy_group(g)


def test_addresses_off_16_bytes_are_refused():
    ep = _ep()
    g = ep.moe_ep_create_group(1, 2, 1, 4, 64)
    h = ep.moe_ep_create_handle(g, 1)
    ep.moe_ep_route(h, None, 4, 1, torch.zeros((4, 1), dtype=torch.int32, device=DEV))
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    off = bf(4 * 64 + 4)[4:].view(4, 64)             # 8 bytes into its storage
    w, hid, gate = bf(2, 64, 64), bf(4, 32), torch.ones(65, device=DEV)[1:]
    for f in (lambda: ep.moe_ep_ffn_gate_up(h, off, w, hid),
              lambda: ep.moe_ep_ffn_down(h, hid, bf(2, 64, 32), off),
              lambda: ep.moe_ep_ffn_weight_grad(h, off, hid, bf(2, 64, 32)),
              lambda: ep.moe_ep_combine_backward(h, off, bf(4, 64), torch.ones((4, 1), device=DEV), bf(4, 64),
                                                 torch.ones((4, 1), device=DEV)),
              lambda: ep.moe_ep_norm_residual(g, off, None, None, None, None, bf(4, 64), None),
              lambda: ep.moe_ep_norm_residual(g, bf(4, 64), None, None, gate, None, bf(4, 64), None)):
        with pytest.raises(ep.MoeEpError) as e:
            f()
        assert e.value.status == ep.MOE_EP_ERR_INVALID
    ep.moe_ep_destroy_handle(h)
    ep.moe_ep_destroy_group(g)


def test_combine_backward_refuses_other_tokens_than_routed():
    ep = _ep()
    g = ep.moe_ep_create_group(1, 2, 1, 4, 64)
    h = ep.moe_ep_create_handle(g, 2)
    with pytest.raises(ep.MoeEpError):
        ep.moe_ep_get_routed(h)
    ep.moe_ep_route(h, None, 4, 2, torch.tensor([[0, 1]] * 4, dtype=torch.int32, device=DEV))
    assert ep.moe_ep_get_routed(h) == (4, 2)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    f32 = lambda *s: torch.zeros(s, device=DEV)  # noqa: E731
    for dout, w, dw in ((bf(3, 64), f32(4, 2), f32(4, 2)), (bf(4, 64), f32(3, 2), f32(3, 2)),
                        (bf(4, 64), f32(4, 1), f32(4, 1)), (bf(4, 64), f32(4, 3), f32(4, 3))):
        with pytest.raises(ValueError, match="routed"):
            ep.moe_ep_combine_backward(h, dout, bf(8, 64), w, bf(8, 64), dw)
    ep.moe_ep_combine_backward(h, bf(5, 64), bf(8, 64), f32(6, 2), bf(8, 64), f32(6, 2))  # longer ones serve
    torch.cuda.synchronize()
    ep.moe_ep_destroy_handle(h)
    ep.moe_ep_destroy_group(g)
