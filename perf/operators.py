"""The expert block's operators next to dispatch and combine, as measured cases.

ffn          the experts' gated feed-forward over the receive rows: gate and up projections,
             activation and product, then the down projection (optionally keeping the gate and up
             values a training step needs)
ffn_bwd      its backward pass: gradients of the rows and of both weight tensors
combine_bwd  the backward pass of the weighted combine: the experts' row gradients and the gate
             weights' gradients
norm         the norms after and before a block, fused with the block's gate and residual scale
norm_bwd     its backward pass

Every case runs in a plain form (torch, 32 bits, rounded once) or, with `own` set, through the
framework's entry points.
"""
import math

import torch

own = False

BF16 = torch.bfloat16
EPS = 1e-6


def listed():
    return [
        # one token through a serving step's norms
        dict(name="norm_token", op="norm", T=1, H=7168, post=True, gate="none", scale=1.0),
        # a long prompt's hidden states between two blocks, channel gate and scaled residual
        dict(name="norm_prefill", op="norm", T=16384, H=7168, post=True, gate="channel", scale=0.75),
        # a training batch's norms, backward
        dict(name="norm_bwd_batch", op="norm_bwd", T=4096, H=7168, post=True, gate="channel", scale=1.0),
        # a ragged batch of an odd width with a gate per token and no norm after the block
        dict(name="norm_bwd_ragged", op="norm_bwd", T=333, H=4104, post=False, gate="token", scale=0.5),
        # one token in a decoding step: eight experts' weights are read
        dict(name="ffn_token", op="ffn", mode="LL", T=1, S=128, E=64, k=8, H=7168, F=2048, act="silu", skew=0.0, save=False),
        # a decoding batch over every expert: about four rows each, bound by the weights
        dict(name="ffn_decode", op="ffn", mode="LL", T=128, S=128, E=256, k=8, H=7168, F=2048, act="silu", skew=0.0, save=False),
        # a training or prefill batch, 512 rows an expert, gate and up kept for the backward pass
        dict(name="ffn_prefill", op="ffn", mode="HT", T=4096, S=0, E=64, k=8, H=7168, F=2048, act="silu", skew=0.0, save=True),
        # odd sizes and a few hot experts
        dict(name="ffn_ragged", op="ffn", mode="HT", T=1001, S=0, E=16, k=2, H=4104, F=1368, act="gelu", skew=0.5, save=False),
        # the backward pass of a training batch
        dict(name="ffn_bwd_batch", op="ffn_bwd", mode="HT", T=4096, S=0, E=64, k=8, H=4096, F=2048, act="silu", skew=0.0, save=False),
        # a small, ragged backward pass, some experts with hardly a row
        dict(name="ffn_bwd_small", op="ffn_bwd", mode="HT", T=100, S=0, E=16, k=2, H=256, F=520, act="gelu", skew=0.5, save=False),
        # the combine's backward pass of a training batch
        dict(name="combine_bwd_batch", op="combine_bwd", mode="HT", T=4096, S=0, E=256, k=8, H=7168, skew=0.0),
        # ... and of a small slotted one
        dict(name="combine_bwd_slots", op="combine_bwd", mode="LL", T=77, S=128, E=16, k=2, H=1032, skew=0.0),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    v = max(lo, min(hi, int(round(v / step)) * step))
    return v + step if v == 3072 else v


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "ffn", "ffn", "ffn_bwd", "combine_bwd"])
    H = rng.choice([256, 512, 1024, 2048, 4096, 7168, _log(rng, 256, 7168, 8)])
    if op.startswith("norm"):
        return dict(op=op, T=_log(rng, 1, 16384 if op == "norm" else 8192), H=H, post=rng.random() < 0.7,
                    gate=rng.choice(["none", "channel", "token"]), scale=rng.choice([1.0, 0.5, 0.75]))
    mode = rng.choice(["HT", "HT", "LL"])
    E = rng.choice([8, 16, 32, 64])
    k = rng.choice([1, 2, 4, 6, 8])
    S = 128 if mode == "LL" else 0
    skew = rng.choice([0.0, 0.0, 0.5])
    if op == "combine_bwd":
        return dict(op=op, mode=mode, T=_log(rng, 1, 128 if mode == "LL" else 4096), S=S, E=E, k=k, H=H, skew=skew)
    F = rng.choice([256, 512, 1024, 2048, _log(rng, 256, 2048, 8)])
    T = _log(rng, 1, 128 if mode == "LL" else 4096)
    while 6.0 * T * k * H * F * (3 if op == "ffn_bwd" else 1) > 1.5e12:
        T = max(1, T // 2)
    return dict(op=op, mode=mode, T=T, S=S, E=E, k=k, H=H, F=F, act=rng.choice(["silu", "gelu"]), skew=skew,
                save=op == "ffn" and mode == "HT" and rng.random() < 0.5)


# ---------------------------------------------------------------------------- inputs
def _routing(case, gen):
    """Each token's experts, and where its rows are in the receive layout (stable, expert-major)."""
    T, E, k, S = case["T"], case["E"], case["k"], case["S"]
    scores = torch.rand((T, E), device="cuda", generator=gen)
    if case["skew"]:
        scores += case["skew"] * (torch.arange(E, device="cuda") + 1.0) ** -1.2
    idx = scores.topk(k, 1).indices
    flat = idx.reshape(-1)
    cnt = torch.bincount(flat, minlength=E)
    off = torch.cat([cnt.new_zeros(1), cnt.cumsum(0)])
    order = flat.argsort(stable=True)                 # pairs in (expert, token) order
    e_of = flat[order]
    at = torch.arange(T * k, device="cuda") - off[e_of]
    start = torch.arange(E, device="cuda") * S if case["mode"] == "LL" else off[:-1]
    row = torch.empty(T * k, dtype=torch.int64, device="cuda")
    row[order] = start[e_of] + at
    return dict(idx=idx.to(torch.int32), cnt=cnt, start=start, row=row.view(T, k), rows=E * S if case["mode"] == "LL" else T * k,
                defined=row[order], e_of=e_of, at=at)


def _plan(r):
    """The experts that have rows, and their rows as a padded [experts][most rows] table."""
    cnt = r["cnt"]
    live = cnt.nonzero().view(-1)
    most = int(cnt.max())
    slot = torch.arange(most, device="cuda")
    mask = slot < cnt[live, None]
    pad = torch.where(mask, r["start"][live, None] + slot, r["start"][live, None])
    return dict(live=None if live.numel() == cnt.numel() else live, pad=pad, mask=mask, rows=pad[mask])


def _handle(case, idx):
    from combine_layout_gb300 import moe_ep as ep
    g = ep.moe_ep_create_group(ep.MOE_EP_LL if case["mode"] == "LL" else ep.MOE_EP_HT, case["E"], case["E"],
                               case["S"] or case["T"], case["H"])
    h = ep.moe_ep_create_handle(g, case["k"])
    ep.moe_ep_route(h, None, case["T"], case["k"], idx)
    return _Owner(g, h)


class _Owner:
    """Frees the group and handle with the state that holds them."""

    def __init__(self, group, handle=None):
        self.group, self.handle = group, handle

    def __del__(self):
        from combine_layout_gb300 import moe_ep as ep
        if self.handle:
            ep.moe_ep_destroy_handle(self.handle)
        ep.moe_ep_destroy_group(self.group)


def _rows(r, width, gen, scale=1.0):
    """Random bf16 rows where the layout defines them, zeros in unused slots."""
    n = r["rows"]
    if n == r["defined"].numel():
        return torch.randn((n, width), device="cuda", dtype=BF16, generator=gen).mul_(scale)
    t = torch.zeros((n, width), device="cuda", dtype=BF16)
    t[r["defined"]] = torch.randn((r["defined"].numel(), width), device="cuda", dtype=BF16, generator=gen).mul_(scale)
    return t


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s, dtype=torch.float32: torch.randn(s, device="cuda", dtype=dtype, generator=gen)  # noqa: E731
    H = case["H"]
    if case["op"].startswith("norm"):
        T = case["T"]
        s = dict(o=rand(T, H, dtype=BF16), res=rand(T, H, dtype=BF16).mul_(2.0), w_pre=1.0 + 0.2 * rand(H),
                 w_post=1.0 + 0.2 * rand(H) if case["post"] else None, gate=None)
        if case["gate"] != "none":
            s["gate"] = 0.5 + 0.3 * rand(T if case["gate"] == "token" else H)
        if case["op"] == "norm_bwd":
            s.update(dr=rand(T, H, dtype=BF16), dy=rand(T, H, dtype=BF16))
        return s
    r = _routing(case, gen)
    s = dict(routing=r)
    if case["op"] == "combine_bwd":
        w = torch.rand((case["T"], case["k"]), device="cuda", generator=gen) + 0.1
        s.update(topk_w=w / w.sum(1, keepdim=True), dout=rand(case["T"], H, dtype=BF16), y=_rows(r, H, gen))
        return s
    E, F = case["E"], case["F"]
    s["w_gate_up"] = rand(E, 2 * F, H, dtype=BF16).mul_(H ** -0.5)
    s["w_down"] = rand(E, H, F, dtype=BF16).mul_(F ** -0.5)
    s["x"] = _rows(r, H, gen)
    if case["op"] == "ffn_bwd":
        s["gate_up"] = _rows(r, 2 * F, gen)
        s["dy"] = _rows(r, H, gen)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    H = case["H"]
    buf = lambda *shape, dtype=BF16: torch.empty(shape, device="cuda", dtype=dtype)  # noqa: E731
    if case["op"].startswith("norm"):
        T = case["T"]
        if case["op"] == "norm":
            s.update(res_out=buf(T, H), y=buf(T, H))
        else:
            s.update(do=buf(T, H), dres=buf(T, H), dw_pre=buf(H, dtype=torch.float32),
                     dw_post=buf(H, dtype=torch.float32) if case["post"] else None,
                     dgate=buf(*s["gate"].shape, dtype=torch.float32) if s["gate"] is not None else None)
        if own:
            from combine_layout_gb300 import moe_ep as ep
            s["ep"] = _Owner(ep.moe_ep_create_group(ep.MOE_EP_HT, 1, 1, max(T, 1), H))
            if case["op"] == "norm_bwd":
                s["work"] = buf(ep.moe_ep_norm_work_floats(s["ep"].group), dtype=torch.float32)
        return s
    r = s["routing"]
    n = r["rows"]
    zero = lambda w: torch.zeros((n, w), device="cuda", dtype=BF16)  # noqa: E731
    if case["op"] == "combine_bwd":
        s.update(dy=zero(H), dw=buf(case["T"], case["k"], dtype=torch.float32))
    else:
        s["plan"] = _plan(r)
        F = case["F"]
        s["hid"] = buf(n, F)
        if case["op"] == "ffn":
            s["y"] = zero(H)
            s["gate_up"] = zero(2 * F) if case["save"] else None
        else:
            s.update(d_gate_up=buf(n, 2 * F), dx=zero(H), dw_gate_up=torch.empty_like(s["w_gate_up"]), dw_down=torch.empty_like(s["w_down"]))
    if own:
        s["ep"] = _handle(case, r["idx"])
    return s


# ---------------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _act(g, kind):
    """act(g) and act'(g)."""
    if kind == "silu":
        sg = 1.0 / (1.0 + torch.exp(-g))
        return g * sg, sg * (1.0 + g * (1.0 - sg))
    cdf = 0.5 * (1.0 + torch.erf(g * 0.5 ** 0.5))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (2.0 * math.pi) ** -0.5


def _of_live(t, plan):
    return (t if plan["live"] is None else t[plan["live"]]).float()


def _padded(t, plan):
    """The experts' rows as [experts][most rows][width], zeros where an expert has fewer."""
    return t[plan["pad"]].float().masked_fill_(~plan["mask"][..., None], 0.0)


def _put(out, v, plan):
    out[plan["rows"]] = v[plan["mask"]].to(out.dtype)
    return out


def _whole(v, like, plan):
    """Per-expert gradients of every expert, zeros for those without rows."""
    if plan["live"] is None:
        return v.to(like.dtype)
    out = torch.zeros_like(like)
    out[plan["live"]] = v.to(like.dtype)
    return out


def _ffn_plain(s):
    p, c = s["plan"], s["case"]
    gu = torch.bmm(_padded(s["x"], p), _of_live(s["w_gate_up"], p).transpose(1, 2))
    g, u = gu.chunk(2, -1)
    a, _ = _act(g, c["act"])
    y = _put(s["y"], torch.bmm(a * u, _of_live(s["w_down"], p).transpose(1, 2)), p)
    return dict(y=y, gate_up=_put(s["gate_up"], gu, p)) if c["save"] else dict(y=y)


def _ffn_bwd_plain(s):
    p, c = s["plan"], s["case"]
    x, dy = _padded(s["x"], p), _padded(s["dy"], p)
    g, u = _padded(s["gate_up"], p).chunk(2, -1)
    a, da = _act(g, c["act"])
    dh = torch.bmm(dy, _of_live(s["w_down"], p))
    dgu = torch.cat([dh * u * da, dh * a], -1)
    dx = torch.bmm(dgu, _of_live(s["w_gate_up"], p))
    return dict(dx=_put(s["dx"], dx, p), dw_gate_up=_whole(torch.bmm(dgu.transpose(1, 2), x), s["w_gate_up"], p),
                dw_down=_whole(torch.bmm(dy.transpose(1, 2), a * u), s["w_down"], p))


def _combine_bwd_plain(s):
    row, dout = s["routing"]["row"], s["dout"].float()
    s["dy"][row] = (s["topk_w"][..., None] * dout[:, None, :]).to(BF16)
    return dict(dy=s["dy"], dw=(dout[:, None, :] * s["y"][row].float()).sum(-1))


def _gate(s):
    g = s["gate"]
    return 1.0 if g is None else g[:, None] if s["case"]["gate"] == "token" else g


def _rstd(t):
    return torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS)


def _norm_plain(s):
    o = s["o"].float()
    u = o if s["w_post"] is None else s["w_post"] * (o * _rstd(o))
    r = s["case"]["scale"] * s["res"].float() + _gate(s) * u
    return dict(res_out=r.to(BF16), y=(s["w_pre"] * (r * _rstd(r))).to(BF16))


def _norm_bwd_plain(s):
    c, o, dy = s["case"], s["o"].float(), s["dy"].float()
    p = _rstd(o)
    u = o if s["w_post"] is None else s["w_post"] * (o * p)
    r = c["scale"] * s["res"].float() + _gate(s) * u
    q = _rstd(r)
    n = r * q
    v = dy * s["w_pre"]
    d = s["dr"].float() + q * (v - n * (v * n).mean(-1, keepdim=True))
    out = dict(dres=(c["scale"] * d).to(BF16), dw_pre=(dy * n).sum(0))
    if s["gate"] is not None:
        out["dgate"] = (d * u).sum(-1 if c["gate"] == "token" else 0)
    du = _gate(s) * d
    if s["w_post"] is None:
        out["do"] = du.to(BF16)
    else:
        m, v = o * p, du * s["w_post"]
        out["dw_post"] = (du * m).sum(0)
        out["do"] = (p * (v - m * (v * m).mean(-1, keepdim=True))).to(BF16)
    return out


_run_plain = dict(ffn=_ffn_plain, ffn_bwd=_ffn_bwd_plain, combine_bwd=_combine_bwd_plain, norm=_norm_plain, norm_bwd=_norm_bwd_plain)


def _act_id(ep, s):
    return ep.MOE_EP_ACT_SILU if s["case"]["act"] == "silu" else ep.MOE_EP_ACT_GELU


def _ffn_own(s):
    from combine_layout_gb300 import moe_ep as ep
    h = s["ep"].handle
    ep.moe_ep_ffn_gate_up(h, s["x"], s["w_gate_up"], s["hid"], s["gate_up"], _act_id(ep, s))
    ep.moe_ep_ffn_down(h, s["hid"], s["w_down"], s["y"])
    return dict(y=s["y"], gate_up=s["gate_up"]) if s["case"]["save"] else dict(y=s["y"])


def _ffn_bwd_own(s):
    from combine_layout_gb300 import moe_ep as ep
    h = s["ep"].handle
    ep.moe_ep_ffn_down_backward(h, s["dy"], s["w_down"], s["gate_up"], s["d_gate_up"], s["hid"], _act_id(ep, s))
    ep.moe_ep_ffn_gate_up_backward(h, s["d_gate_up"], s["w_gate_up"], s["dx"])
    ep.moe_ep_ffn_weight_grad(h, s["d_gate_up"], s["x"], s["dw_gate_up"])
    ep.moe_ep_ffn_weight_grad(h, s["dy"], s["hid"], s["dw_down"])
    return dict(dx=s["dx"], dw_gate_up=s["dw_gate_up"], dw_down=s["dw_down"])


def _combine_bwd_own(s):
    from combine_layout_gb300 import moe_ep as ep
    ep.moe_ep_combine_backward(s["ep"].handle, s["dout"], s["y"], s["topk_w"], s["dy"], s["dw"])
    return dict(dy=s["dy"], dw=s["dw"])


def _norm_own(s):
    from combine_layout_gb300 import moe_ep as ep
    ep.moe_ep_norm_residual(s["ep"].group, s["o"], s["res"], s["w_post"], s["gate"], s["w_pre"], s["res_out"], s["y"],
                            res_scale=s["case"]["scale"], gate_per_token=s["case"]["gate"] == "token", eps=EPS)
    return dict(res_out=s["res_out"], y=s["y"])


def _norm_bwd_own(s):
    from combine_layout_gb300 import moe_ep as ep
    ep.moe_ep_norm_residual_backward(s["ep"].group, s["o"], s["res"], s["w_post"], s["gate"], s["w_pre"], s["dr"], s["dy"],
                                     s["do"], s["dres"], s["dw_post"], s["dgate"], s["dw_pre"], s["work"],
                                     res_scale=s["case"]["scale"], gate_per_token=s["case"]["gate"] == "token", eps=EPS)
    out = dict(do=s["do"], dres=s["dres"], dw_pre=s["dw_pre"])
    out.update({n: s[n] for n in ("dw_post", "dgate") if s[n] is not None})
    return out


_run_own = dict(ffn=_ffn_own, ffn_bwd=_ffn_bwd_own, combine_bwd=_combine_bwd_own, norm=_norm_own, norm_bwd=_norm_bwd_own)


# ---------------------------------------------------------------------------- what a pass needs
def work(case):
    T, H = case["T"], case["H"]
    if case["op"] == "norm":
        return dict(bytes=8.0 * T * H + 12.0 * H, flops=14.0 * T * H)
    if case["op"] == "norm_bwd":
        return dict(bytes=12.0 * T * H + 24.0 * H, flops=40.0 * T * H)
    k, E = case["k"], case["E"]
    n = T * k
    if case["op"] == "combine_bwd":
        return dict(bytes=2.0 * T * H + 4.0 * n * H + 12.0 * n, flops=3.0 * n * H)
    F = case["F"]
    live = E * (1.0 - (1.0 - k / E) ** T)             # experts with rows, evenly routed
    w = 6.0 * F * H
    if case["op"] == "ffn":
        return dict(bytes=live * w + 4.0 * n * H + (4.0 * n * F if case["save"] else 0.0), flops=6.0 * n * F * H)
    return dict(bytes=live * w + E * w + n * (6.0 * H + 4.0 * F), flops=12.0 * n * F * H)


# ---------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    return _norm64(case, s) if case["op"].startswith("norm") else _rows64(case, s)


def _norm64(case, s):
    d = {n: (None if v is None else v.double()) for n, v in s.items()}
    H, T, tok = case["H"], case["T"], case["gate"] == "token"
    gate = torch.ones(1, 1, dtype=torch.float64, device="cuda") if d["gate"] is None else d["gate"].reshape((T, 1) if tok else (1, H))
    inv = lambda t: 1.0 / torch.sqrt(t.pow(2).sum(1, keepdim=True) / H + EPS)  # noqa: E731
    o_inv = inv(d["o"])
    on = d["o"] * o_inv
    u = on * d["w_post"] if case["post"] else d["o"]
    r = d["res"] * case["scale"] + u * gate
    r_inv = inv(r)
    rn = r * r_inv
    if case["op"] == "norm":
        return dict(res_out=r, y=rn * d["w_pre"])
    back = lambda grad, unit, i: i * (grad - unit * ((grad * unit).sum(1, keepdim=True) / H))  # noqa: E731
    dr = d["dr"] + back(d["dy"] * d["w_pre"], rn, r_inv)
    out = dict(dres=dr * case["scale"], dw_pre=torch.einsum("th,th->h", d["dy"], rn))
    if s["gate"] is not None:
        out["dgate"] = torch.einsum("th,th->t" if tok else "th,th->h", dr, u)
    du = dr * gate
    out["do"] = back(du * d["w_post"], on, o_inv) if case["post"] else du
    if case["post"]:
        out["dw_post"] = torch.einsum("th,th->h", du, on)
    return out


def _rows64(case, s):
    r, H = s["routing"], case["H"]
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    if case["op"] == "combine_bwd":
        dy, dw = new(r["rows"], H), new(case["T"], case["k"])
        for j in range(case["k"]):
            at = r["row"][:, j]
            dy[at] = s["dout"].double() * s["topk_w"][:, j, None].double()
            dw[:, j] = torch.einsum("th,th->t", s["dout"].double(), s["y"][at].double())
        return dict(dy=dy, dw=dw)
    F = case["F"]
    fwd = case["op"] == "ffn"
    if fwd:
        out = dict(y=new(r["rows"], H))
        if case["save"]:
            out["gate_up"] = new(r["rows"], 2 * F)
    else:
        out = dict(dx=new(r["rows"], H), dw_gate_up=new(case["E"], 2 * F, H), dw_down=new(case["E"], H, F))
    for e, (b, n) in enumerate(zip(r["start"].tolist(), r["cnt"].tolist())):
        if not n:
            continue
        rows = slice(b, b + n)
        x, wg, wu, wd = s["x"][rows].double(), s["w_gate_up"][e, :F].double(), s["w_gate_up"][e, F:].double(), s["w_down"][e].double()
        if fwd:
            g, u = x @ wg.T, x @ wu.T
            if case["save"]:
                out["gate_up"][rows, :F], out["gate_up"][rows, F:] = g, u
        else:
            g, u = s["gate_up"][rows, :F].double(), s["gate_up"][rows, F:].double()
        if case["act"] == "silu":
            sig = torch.sigmoid(g)
            a, slope = g * sig, sig + g * sig * (1.0 - sig)
        else:
            phi = torch.special.ndtr(g)
            a, slope = g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        hid = a * u
        if fwd:
            out["y"][rows] = hid @ wd.T
            continue
        dy = s["dy"][rows].double()
        dh = dy @ wd
        dg, du = dh * u * slope, dh * a
        out["dx"][rows] = dg @ wg + du @ wu
        out["dw_gate_up"][e, :F], out["dw_gate_up"][e, F:] = dg.T @ x, du.T @ x
        out["dw_down"][e] = dy.T @ hid
    return out
