"""The experts' feed-forward over the receive rows, its backward pass and the
combine's, against 64-bit values: ragged and empty experts, one row, odd
widths, padded blocks and slots whose other rows hold NaN."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from block64 import BF, D, U, close, down_bwd64, gate_up64, product64
from combine_layout_gb300 import synth

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
HT, LL = synth.MODE_HT, synth.MODE_LL


def _ep():
    import combine_layout_gb300.moe_ep as ep
    return ep


class Block:
    """One routed handle with random rows; rows the layout does not define hold NaN."""

    def __init__(self, mode, counts, H, F, k=1, S=None, align=1, seed=0, T=None):
        # counts: rows of each expert; tokens are dealt k experts each (-1: masked)
        ep = _ep()
        self.gen = torch.Generator().manual_seed(seed)
        E = len(counts)
        T = T or max(max(counts), -(-sum(counts) // k), 1)
        idx = np.full((T, k), -1, np.int32)
        # pair i goes to token i % T: an expert's rows are distinct tokens
        for i, e in enumerate(np.repeat(np.arange(E), counts)):
            idx[i % T, i // T] = e
        self.E, self.H, self.F, self.T, self.k, self.mode = E, H, F, T, k, mode
        S = S or T
        self.group = ep.moe_ep_create_group(mode, E, 1, S, H)
        self.handle = ep.moe_ep_create_handle(self.group, k)
        if align != 1:
            ep.moe_ep_set_row_align(self.handle, align)
        self.idx = torch.from_numpy(idx).to(DEV)
        ep.moe_ep_route(self.handle, None, T, k, self.idx)
        pad = lambda c: -(-c // align) * align  # noqa: E731
        starts = np.cumsum([0] + [pad(c) for c in counts]) if mode == HT else np.arange(E + 1) * S
        self.rows = E * S if mode == LL else T * k + E * (align - 1)
        self.of = [torch.arange(int(starts[e]), int(starts[e]) + counts[e]) for e in range(E)]
        self.defined = torch.cat(self.of)

    def row_tensor(self, width, fill=float("nan")):
        t = torch.full((self.rows, width), fill, dtype=torch.bfloat16)
        t[self.defined] = torch.randn((len(self.defined), width), generator=self.gen).to(torch.bfloat16)
        return t

    def weights(self, m, n):
        return (torch.randn((self.E, m, n), generator=self.gen) * n ** -0.5).to(torch.bfloat16)

    def untouched(self, t, value):
        mask = torch.ones(self.rows, dtype=torch.bool)
        mask[self.defined] = False
        rest = t.cpu()[mask].float()
        assert bool((rest == value).all()), "rows the layout does not define were written"

    def close(self):
        torch.cuda.synchronize()
        assert _ep().moe_ep_get_device_errors(self.group) == 0
        _ep().moe_ep_destroy_handle(self.handle)
        _ep().moe_ep_destroy_group(self.group)


SHAPES = {
    "one_row": dict(mode=HT, counts=[0, 1, 0, 0], H=64, F=64),
    "least_width": dict(mode=HT, counts=[3, 0, 5], H=8, F=8),
    "odd_width": dict(mode=HT, counts=[17, 1, 0, 40], H=264, F=200, k=2),
    "tile_edges": dict(mode=HT, counts=[255, 256, 257, 16, 15, 33], H=136, F=72, k=3),
    "many_tiles": dict(mode=HT, counts=[2400, 0, 130], H=128, F=328, k=2),
    "padded": dict(mode=HT, counts=[5, 0, 64, 100], H=128, F=136, k=2, align=64),
    "slots": dict(mode=LL, counts=[4, 0, 31, 1, 16], H=256, F=136, k=2, S=40),
    "slots_late": dict(mode=LL, counts=[300, 0, 9], H=64, F=24, k=1, S=320),
    "masked": dict(mode=HT, counts=[0, 0, 0], H=64, F=64),
    "many_experts": dict(mode=HT, counts=[(7 * e) % 5 for e in range(512)], H=64, F=16, k=4),
}


def _block(name, seed=0):
    return Block(seed=seed, **SHAPES[name])


def _act(ep, kind):
    return ep.MOE_EP_ACT_SILU if kind == "silu" else ep.MOE_EP_ACT_GELU


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("name", SHAPES)
def test_forward(name, kind):
    ep, b = _ep(), _block(name)
    x, w = b.row_tensor(b.H), b.weights(2 * b.F, b.H)
    hid = torch.full((b.rows, b.F), 7.0, dtype=torch.bfloat16, device=DEV)
    gu = torch.full((b.rows, 2 * b.F), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.moe_ep_ffn_gate_up(b.handle, x.to(DEV), w.to(DEV), hid, gu, _act(ep, kind))
    alone = torch.full_like(hid, 7.0)
    ep.moe_ep_ffn_gate_up(b.handle, x.to(DEV), w.to(DEV), alone, None, _act(ep, kind))
    for e, r in enumerate(b.of):
        want, tol, wgu, tgu = gate_up64(x[r], w[e], kind)
        close(hid[r.to(DEV)], want, tol, f"hid of expert {e}")
        close(gu[r.to(DEV)], wgu, tgu, f"gate_up of expert {e}")
    assert torch.equal(hid, alone)
    b.untouched(hid, 7.0)
    b.untouched(gu, 7.0)
    h, wd = b.row_tensor(b.F), b.weights(b.H, b.F)
    y = torch.full((b.rows, b.H), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.moe_ep_ffn_down(b.handle, h.to(DEV), wd.to(DEV), y)
    for e, r in enumerate(b.of):
        want, err = product64(h[r], wd[e])
        close(y[r.to(DEV)], want, BF * want.abs() * 1.01 + err, f"y of expert {e}")
    b.untouched(y, 7.0)
    b.close()


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("name", SHAPES)
def test_backward_of_rows(name, kind):
    ep, b = _ep(), _block(name, seed=1)
    dy, wd, gu = b.row_tensor(b.H), b.weights(b.H, b.F), b.row_tensor(2 * b.F)
    dgu = torch.full((b.rows, 2 * b.F), 7.0, dtype=torch.bfloat16, device=DEV)
    hid = torch.full((b.rows, b.F), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.moe_ep_ffn_down_backward(b.handle, dy.to(DEV), wd.to(DEV), gu.to(DEV), dgu, hid, _act(ep, kind))
    alone = torch.full_like(dgu, 7.0)
    ep.moe_ep_ffn_down_backward(b.handle, dy.to(DEV), wd.to(DEV), gu.to(DEV), alone, None, _act(ep, kind))
    for e, r in enumerate(b.of):
        want, tol, wh, th = down_bwd64(dy[r], wd[e], gu[r], kind)
        close(dgu[r.to(DEV)], want, tol, f"d_gate_up of expert {e}")
        close(hid[r.to(DEV)], wh, th, f"hid of expert {e}")
    assert torch.equal(dgu, alone)
    b.untouched(dgu, 7.0)
    b.untouched(hid, 7.0)
    g, w = b.row_tensor(2 * b.F), b.weights(2 * b.F, b.H)
    dx = torch.full((b.rows, b.H), 7.0, dtype=torch.bfloat16, device=DEV)
    ep.moe_ep_ffn_gate_up_backward(b.handle, g.to(DEV), w.to(DEV), dx)
    for e, r in enumerate(b.of):
        want, err = product64(g[r], w[e].T)
        close(dx[r.to(DEV)], want, BF * want.abs() * 1.01 + err, f"dx of expert {e}")
    b.untouched(dx, 7.0)
    b.close()


@pytest.mark.parametrize("form", ["bf16", "fp32", "accumulate"])
@pytest.mark.parametrize("name", SHAPES)
def test_weight_gradients(name, form):
    ep, b = _ep(), _block(name, seed=2)
    a, x = b.row_tensor(b.F), b.row_tensor(b.H)
    dt = torch.bfloat16 if form == "bf16" else torch.float32
    before = torch.randn((b.E, b.F, b.H), generator=b.gen).to(dt) if form == "accumulate" else \
        torch.full((b.E, b.F, b.H), float("nan"), dtype=dt)
    dw = before.to(DEV)
    ep.moe_ep_ffn_weight_grad(b.handle, a.to(DEV), x.to(DEV), dw, accumulate=form == "accumulate")
    for e, r in enumerate(b.of):
        want, err = product64(a[r].T.contiguous(), x[r].T.contiguous())
        if form == "accumulate":
            want = want + before[e].to(D)
        half = torch.finfo(dt).eps / 2
        close(dw[e], want, half * want.abs() * 1.01 + err, f"dw of expert {e}")
    b.close()


def test_a_nan_row_stays_in_its_row_and_its_experts_gradient():
    ep, b = _ep(), Block(HT, [5, 20, 3], 64, 64, k=1)
    x, a, w = b.row_tensor(64), b.row_tensor(64), b.weights(128, 64)
    bad = int(b.of[1][7])
    x[bad] = float("nan")
    hid = torch.zeros((b.rows, 64), dtype=torch.bfloat16, device=DEV)
    ep.moe_ep_ffn_gate_up(b.handle, x.to(DEV), w.to(DEV), hid)
    rows = torch.isnan(hid.float()).any(1).cpu()
    assert rows.nonzero().view(-1).tolist() == [bad]
    dw = torch.zeros((3, 64, 64), device=DEV)
    ep.moe_ep_ffn_weight_grad(b.handle, a.to(DEV), x.to(DEV), dw)
    assert torch.isnan(dw).flatten(1).any(1).tolist() == [False, True, False]
    b.close()


def test_backward_against_differences():
    """A directional derivative of sum(y * c) through gate_up and down."""
    ep, b = _ep(), Block(HT, [9, 0, 30], 64, 48, k=1)
    x, w, wd, c = b.row_tensor(64), b.weights(96, 64), b.weights(64, 48), b.row_tensor(64)
    z = lambda n: torch.zeros((b.rows, n), dtype=torch.bfloat16, device=DEV)  # noqa: E731
    hid, gu, dgu, dx = z(48), z(96), z(96), z(64)
    dev = [t.to(DEV) for t in (x, w, wd, c)]
    ep.moe_ep_ffn_gate_up(b.handle, dev[0], dev[1], hid, gu)
    ep.moe_ep_ffn_down_backward(b.handle, dev[3], dev[2], gu, dgu, hid)
    ep.moe_ep_ffn_gate_up_backward(b.handle, dgu, dev[1], dx)
    dw = torch.zeros((3, 96, 64), device=DEV)
    dwd = torch.zeros((3, 64, 48), device=DEV)
    ep.moe_ep_ffn_weight_grad(b.handle, dgu, dev[0], dw)
    ep.moe_ep_ffn_weight_grad(b.handle, dev[3], hid, dwd)

    def loss(x, w, wd):
        s = 0.0
        for e, r in enumerate(b.of):
            g, u = (x[r] @ w[e].T).chunk(2, 1)
            s = s + ((g * torch.sigmoid(g) * u) @ wd[e].T * c[r].to(D)).sum()
        return float(s)

    base = [torch.nan_to_num(t.to(D)) for t in (x, w, wd)]
    got = [torch.nan_to_num(dx.to(D).cpu()), dw.to(D).cpu(), dwd.to(D).cpu()]
    for i in range(3):
        v = torch.randn(base[i].shape, generator=b.gen, dtype=D)
        step = 1e-5
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + step * v, base[i] - step * v
        want = (loss(*up) - loss(*down)) / (2 * step)
        # the gradients carry three bf16 roundings at most, each at random: 3 h of their norm
        scale = float((got[i].abs() * v.abs()).pow(2).sum().sqrt())
        assert abs(float((got[i] * v).sum()) - want) <= 3 * BF * scale * 4
    b.close()


@pytest.mark.parametrize("mode,T,E,k,H", [(HT, 1, 8, 2, 64), (HT, 300, 16, 4, 264), (LL, 33, 8, 3, 1032),
                                         (HT, 40, 32, 20, 128), (HT, 513, 64, 8, 512), (HT, 7, 4, 1, 8)])
def test_combine_backward(mode, T, E, k, H):
    ep = _ep()
    gen = torch.Generator().manual_seed(T)
    idx = torch.rand((T, E), generator=gen).topk(k, 1).indices.to(torch.int32)
    idx[torch.rand((T, k), generator=gen) < 0.2] = -1
    idx[T // 2] = -1
    g = ep.moe_ep_create_group(mode, E, 1, T, H)
    h = ep.moe_ep_create_handle(g, k)
    ep.moe_ep_route(h, None, T, k, idx.to(DEV))
    rows = E * T if mode == LL else T * k
    row = torch.empty((T, k), dtype=torch.int32, device=DEV)
    ep.moe_ep_copy_layout(h, row=row)
    row = row.cpu().long()
    dout = torch.randn((T, H), generator=gen).to(torch.bfloat16)
    y = torch.full((rows, H), float("nan"), dtype=torch.bfloat16)
    at = row[row >= 0]
    y[at] = torch.randn((len(at), H), generator=gen).to(torch.bfloat16)
    w = torch.rand((T, k), generator=gen)
    dy = torch.full((rows, H), 7.0, dtype=torch.bfloat16, device=DEV)
    dw = torch.full((T, k), 7.0, device=DEV)
    ep.moe_ep_combine_backward(h, dout.to(DEV), y.to(DEV), w.to(DEV), dy, dw)
    torch.cuda.synchronize()
    want_dy = torch.full((rows, H), 7.0, dtype=D)
    want_dw, tol_dw = torch.zeros((T, k), dtype=D), torch.zeros((T, k), dtype=D)
    for t in range(T):
        for j in range(k):
            r = int(row[t, j])
            assert (r < 0) == (int(idx[t, j]) < 0)
            if r >= 0:
                want_dy[r] = w[t, j].to(D) * dout[t].to(D)
                p = dout[t].to(D) * y[r].to(D)
                want_dw[t, j], tol_dw[t, j] = p.sum(), H * U * p.abs().sum()
    # the product's fp32 rounding and the one to bf16
    close(dy, want_dy, (BF * 1.01 + U) * want_dy.abs(), "dy")
    close(dw, want_dw, tol_dw, "dw")
    ep.moe_ep_destroy_handle(h)
    ep.moe_ep_destroy_group(g)


def test_empty_batch():
    ep = _ep()
    g = ep.moe_ep_create_group(HT, 4, 1, 16, 64)
    h = ep.moe_ep_create_handle(g, 2)
    ep.moe_ep_route(h, None, 0, 2, None)
    z = lambda *s: torch.full(s, 7.0, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    x, hid, gu, w, wd = z(1, 64), z(1, 32), z(1, 64), z(4, 64, 64), z(4, 64, 32)
    ep.moe_ep_ffn_gate_up(h, x, w, hid, gu)
    ep.moe_ep_ffn_down(h, hid, wd, x)
    dw = z(4, 32, 64)
    ep.moe_ep_ffn_weight_grad(h, hid, x, dw)
    acc = torch.full((4, 32, 64), 3.0, device=DEV)
    ep.moe_ep_ffn_weight_grad(h, hid, x, acc, accumulate=True)
    torch.cuda.synchronize()
    assert bool((hid == 7).all()) and bool((x == 7).all()) and bool((gu == 7).all())
    assert bool((dw == 0).all()) and bool((acc == 3).all())
    ep.moe_ep_destroy_handle(h)
    ep.moe_ep_destroy_group(g)


def test_another_stream_and_a_captured_step():
    """A decoding step on a side stream, then captured and replayed on new tokens."""
    ep, b = _ep(), Block(LL, [4, 0, 3, 1], 128, 64, k=2, S=16)
    w, wd = b.weights(128, 128).to(DEV), b.weights(128, 64).to(DEV)
    x = b.row_tensor(128).to(DEV)
    hid = torch.zeros((b.rows, 64), dtype=torch.bfloat16, device=DEV)
    y = torch.zeros((b.rows, 128), dtype=torch.bfloat16, device=DEV)

    def step(s):
        ep.moe_ep_ffn_gate_up(b.handle, x, w, hid, stream=s)
        ep.moe_ep_ffn_down(b.handle, hid, wd, y, stream=s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    first = y.clone()
    at = b.defined.to(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(torch.cuda.current_stream())
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y[at], first[at])
    x[at] = -x[at]
    graph.replay()
    torch.cuda.synchronize()
    again = y.clone()
    step(None)
    torch.cuda.synchronize()
    assert torch.equal(again[at], y[at]) and not torch.equal(again[at], first[at])
    b.close()


def test_refusals():
    ep, b = _ep(), Block(HT, [4, 3], 64, 32, k=1)
    bf = dict(dtype=torch.bfloat16, device=DEV)
    x, w, hid, gu = torch.zeros(b.rows, 64, **bf), torch.zeros(2, 64, 64, **bf), torch.zeros(b.rows, 32, **bf), torch.zeros(b.rows, 64, **bf)
    wd = torch.zeros(2, 64, 32, **bf)
    dw = torch.zeros(2, 32, 64, **bf)
    bad = [
        lambda: ep.moe_ep_ffn_gate_up(b.handle, x, w, hid, act=2),
        lambda: ep.moe_ep_ffn_gate_up(b.handle, x[:3], w, hid),                       # rows
        lambda: ep.moe_ep_ffn_gate_up(b.handle, x, w, hid, x),                        # overlap
        lambda: ep.moe_ep_ffn_down(b.handle, torch.zeros(b.rows, 28, **bf), torch.zeros(2, 64, 28, **bf), x),  # F % 8
        lambda: ep.moe_ep_ffn_weight_grad(b.handle, hid, x, dw, accumulate=True),     # bf16 accumulate
        lambda: ep.moe_ep_combine_backward(b.handle, x[: b.T], x, torch.zeros(b.T, 1, device=DEV), x, torch.zeros(b.T, 1, device=DEV)),
    ]
    for f in bad:
        with pytest.raises(ep.MoeEpError) as err:
            f()
        assert err.value.status == ep.MOE_EP_ERR_INVALID
    shapes = [
        lambda: ep.moe_ep_ffn_gate_up(b.handle, x, w[:1], hid),
        lambda: ep.moe_ep_ffn_gate_up(b.handle, x.float(), w, hid),
        lambda: ep.moe_ep_ffn_gate_up(b.handle, x, w.transpose(1, 2), hid),
        lambda: ep.moe_ep_ffn_down(b.handle, hid, wd[:, :32], x),
        lambda: ep.moe_ep_ffn_weight_grad(b.handle, hid, x, dw[:, :16]),
    ]
    for f in shapes:
        with pytest.raises(ValueError):
            f()
    h2 = ep.moe_ep_create_handle(b.group, 1)
    with pytest.raises(ep.MoeEpError):                                                # no route yet
        ep.moe_ep_ffn_down(h2, hid, wd, x)
    ep.moe_ep_destroy_handle(h2)
    b.close()
