"""Workloads of the selective state-space mixer and of the channels-last group norm.

Three operators, each over [B, N = H * W, channels] grids of 16-bit activations:

* ``conv``: the short causal convolution over the scan order (depthwise, width 2 to 4,
  bias, SiLU), forward and backward;
* ``scan``: the selective state-space scan h = exp(dt A) h + dt u B, y = (C h + D u) silu(z),
  forward, backward, and its form for a single token (a 1 x 1 grid with the carried state);
* ``norm``: group norm with an activation, forward and backward.

``run`` computes a case either in its plain form (elementary torch operations in 32 bits,
rounded once at the end) or, where ``own`` is true, through the package's entry points.
``exact`` computes the same from the definitions in 64 bits.
"""
import math

import torch

own = False

ACT_NONE, ACT_SILU = 0, 1
_DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the convolution ahead of the scan at the 640-pixel grid, one image, forward
        dict(name="conv_fwd_40x40_d1024", op="conv", grad=False, B=1, H=40, W=40, D=1024, K=4, dir=0,
             dtype="fp16", state=True),
        # the same in training at the 768-pixel batch, column scan
        dict(name="conv_bwd_b8_48x48_d2048", op="conv", grad=True, B=8, H=48, W=48, D=2048, K=4, dir=2,
             dtype="bf16", state=False),
        # one high-resolution image (or a prompt of 16384 tokens) carried on from an earlier state
        dict(name="scan_fwd_128x128_d1024", op="scan", grad=False, B=1, H=128, W=128, D=1024, S=16, dir=0,
             dtype="bf16", gate=True, state=True),
        # the 768-pixel batch, scanned down the columns
        dict(name="scan_fwd_b8_48x48_d2048", op="scan", grad=False, B=8, H=48, W=48, D=2048, S=16, dir=2,
             dtype="fp16", gate=True, state=False),
        # a training step at the 640-pixel grid, one image
        dict(name="scan_bwd_40x40_d1024", op="scan", grad=True, B=1, H=40, W=40, D=1024, S=16, dir=1,
             dtype="fp16", gate=True, state=False),
        # a training batch on a ragged grid, scanned bottom to top
        dict(name="scan_bwd_b4_37x53_d1536", op="scan", grad=True, B=4, H=37, W=53, D=1536, S=16, dir=3,
             dtype="bf16", gate=True, state=True),
        # one token of one stream: latency
        dict(name="scan_token_b1_d1024", op="scan", grad=False, B=1, H=1, W=1, D=1024, S=16, dir=0,
             dtype="bf16", gate=True, state=True),
        # one token of each of 256 streams: the states' traffic
        dict(name="scan_token_b256_d2048", op="scan", grad=False, B=256, H=1, W=1, D=2048, S=16, dir=0,
             dtype="fp16", gate=True, state=True),
        # the norm of the mixer's output by head (16 heads of 64 channels), 640-pixel grid, one image
        dict(name="norm_fwd_40x40_c1024", op="norm", grad=False, B=1, H=40, W=40, C=1024, G=16, act="none",
             affine=True, dtype="fp16"),
        # norm and SiLU at the high-resolution grid
        dict(name="norm_fwd_128x128_c1024", op="norm", grad=False, B=1, H=128, W=128, C=1024, G=32, act="silu",
             affine=True, dtype="bf16"),
        # training on a ragged grid, one image in four
        dict(name="norm_bwd_b4_37x53_c768", op="norm", grad=True, B=4, H=37, W=53, C=768, G=12, act="none",
             affine=True, dtype="bf16"),
        # training at the 768-pixel batch
        dict(name="norm_bwd_b8_48x48_c2048", op="norm", grad=True, B=8, H=48, W=48, C=2048, G=32, act="silu",
             affine=True, dtype="fp16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("conv", "scan", "scan", "norm"))
    dtype = rng.choice(("fp16", "bf16"))
    grad = rng.random() < 0.5
    while True:
        B = _log_int(rng, 1, 8)
        H, W = _log_int(rng, 1, 128), _log_int(rng, 1, 128)
        N = H * W
        if op == "scan":
            if rng.random() < 0.2:       # single tokens
                B, H, W, N, grad = _log_int(rng, 1, 256), 1, 1, 1, False
            D = _log_int(rng, 32, 2048)
            S = rng.choice((4, 8, 12, 16, 16, 16, 32))
            # no more than the largest listed case, and few enough steps for the plain form
            if B * N * D * S > (4 * 1961 * 1536 * 16 if grad else 8 * 2304 * 2048 * 16):
                continue
            return dict(op="scan", grad=grad, B=B, H=H, W=W, D=D, S=S, dir=rng.randrange(4), dtype=dtype,
                        gate=rng.random() < 0.7, state=True if N == 1 else rng.random() < 0.5)
        if op == "conv":
            D = _log_int(rng, 32, 2048)
            if B * N * D > 8 * 2304 * 2048:
                continue
            return dict(op="conv", grad=grad, B=B, H=H, W=W, D=D, K=rng.choice((2, 3, 4, 4)), dir=rng.randrange(4),
                        dtype=dtype, state=rng.random() < 0.5)
        G = rng.choice((1, 2, 4, 8, 12, 16, 32))
        C = G * max(1, _log_int(rng, 32, 2048) // G)
        if B * N * C > 8 * 2304 * 2048 or N * (C // G) < 8:
            continue
        return dict(op="norm", grad=grad, B=B, H=H, W=W, C=C, G=G, act=rng.choice(("none", "silu")),
                    affine=rng.random() < 0.8, dtype=dtype)


def _elements(case):
    return case["B"] * case["H"] * case["W"] * case.get("D", case.get("C"))


def work(case):
    e, B = _elements(case), case["B"]
    N = case["H"] * case["W"]
    if case["op"] == "conv":
        D, K = case["D"], case["K"]
        par = 4 * D * (K + 1)
        st = 2 * B * (K - 1) * D
        if not case["grad"]:
            return {"bytes": 4 * e + par + 2 * st, "flops": e * (2 * K + 5)}
        return {"bytes": 6 * e + 2 * par + st * (3 if case["state"] else 0), "flops": e * (6 * K + 12)}
    if case["op"] == "scan":
        D, S = case["D"], case["S"]
        par = 4 * D * (S + 2)
        st = 4 * B * D * S
        bc = 2 * 2 * B * N * S
        g = 1 if case["gate"] else 0
        # an item is one state element of one token: the decay's product and exponential, the
        # update's two products and sum, the readout's product and sum
        if not case["grad"]:
            return {"bytes": 2 * e * (3 + g) + bc + par + st * (2 if case["state"] else 1), "flops": e * S * 7}
        # reads u, dt, dy (z), B, C; writes du, ddt (dz), dB, dC
        return {"bytes": 2 * e * (5 + 2 * g) + 2 * bc + 2 * par + st * (3 if case["state"] else 0),
                "flops": e * S * 22}
    C, G = case["C"], case["G"]
    par = 8 * C if case["affine"] else 0
    if not case["grad"]:
        return {"bytes": 4 * e + par + 8 * B * G, "flops": e * 10}
    return {"bytes": 6 * e + 2 * par + 8 * B * G, "flops": e * 20}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    t = _DT[case["dtype"]]
    B, N = case["B"], case["H"] * case["W"]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device=dev) * std

    s = dict(case=case)
    if case["op"] == "conv":
        D, K = case["D"], case["K"]
        # the first half of the in-projection's output: rows 2 D apart
        s["x"] = normal(B, N, 2 * D).to(t)[..., :D]
        s["w"] = normal(D, K, std=K ** -0.5)
        s["bias"] = normal(D, std=0.1)
        s["init"] = normal(B, K - 1, D).to(t) if case["state"] else None
        if case["grad"]:
            s["dy"] = normal(B, N, D).to(t)
            s["dfinal"] = normal(B, K - 1, D).to(t) if case["state"] else None
        return s
    if case["op"] == "scan":
        D, S = case["D"], case["S"]
        u = normal(B, N, D)
        s["u"] = (u * torch.sigmoid(u)).to(t)                       # the convolution's output
        s["dt"] = normal(B, N, D, std=0.5).to(t)
        # time steps between 0.001 and 0.1 at a zero pre-activation, decay rates near 1 .. S
        step = torch.exp(torch.rand(D, generator=gen, device=dev) * math.log(100.0) + math.log(1e-3))
        s["dt_bias"] = torch.log(torch.expm1(step))
        s["A"] = -torch.exp(torch.log(torch.arange(1, S + 1, device=dev, dtype=torch.float32)) + normal(D, S, std=0.1))
        bc = normal(B, N, 2 * S).to(t)                              # one projection holds B and C
        s["Bm"], s["Cm"] = bc[..., :S], bc[..., S:]
        s["D"] = 1.0 + normal(D, std=0.1)
        # the second half of the in-projection's output
        s["z"] = normal(B, N, 2 * D).to(t)[..., D:] if case["gate"] else None
        s["init"] = normal(B, D, S, std=0.3) if case["state"] else None
        if case["grad"]:
            s["dy"] = normal(B, N, D).to(t)
            s["dfinal"] = normal(B, D, S) if case["state"] else None
        return s
    C, G = case["C"], case["G"]
    # group means and spreads differ, as the heads' do
    mean = normal(B, 1, G, 1).repeat_interleave(C // G, 3).reshape(B, 1, C)
    std = torch.exp(normal(B, 1, G, 1, std=0.5)).repeat_interleave(C // G, 3).reshape(B, 1, C)
    s["x"] = (normal(B, N, C) * std + mean).to(t)
    s["gamma"] = 1.0 + normal(C, std=0.2) if case["affine"] else None
    s["beta"] = normal(C, std=0.2) if case["affine"] else None
    if case["grad"]:
        s["dy"] = normal(B, N, C).to(t)
        # a training step has the forward's statistics in hand
        xg = s["x"].double().reshape(B, N, G, C // G)
        m = xg.mean((1, 3))
        v = ((xg - m[:, None, :, None]) ** 2).mean((1, 3))
        s["stats"] = torch.stack((m, torch.rsqrt(v + 1e-5)), -1).float()
    return s


# ------------------------------------------------------------------ plain forms
def _order(case, device):
    """Token index of each scan position: rows left to right (0) or right to left (1), columns
    top to bottom (2) or bottom to top (3)."""
    H, W = case["H"], case["W"]
    n = torch.arange(H * W, device=device).reshape(H, W)
    d = case["dir"]
    n = (n, n.flip(1), n.t(), n.flip(0).t())[d]
    return n.reshape(-1)


def _unorder(t, order):
    out = torch.empty_like(t)
    out[:, order] = t
    return out


def _conv_plain(s):
    c = s["case"]
    t, K = s["x"].dtype, c["K"]
    order = _order(c, s["x"].device)
    x = s["x"].float()[:, order]
    B, N, D = x.shape
    init = s["init"].float() if s["init"] is not None else x.new_zeros(B, K - 1, D)
    X = torch.cat((init, x), 1)
    pre = s["bias"] + sum(s["w"][:, j] * X[:, j:j + N] for j in range(K))
    sig = 1.0 / (1.0 + torch.exp(-pre))
    if not c["grad"]:
        return _unorder((pre * sig).to(t), order), X[:, N:].to(t)
    ds = s["dy"].float()[:, order] * sig * (1.0 + pre * (1.0 - sig))
    dX = torch.zeros_like(X)
    for j in range(K):
        dX[:, j:j + N] += s["w"][:, j] * ds
    if s["dfinal"] is not None:
        dX[:, N:] += s["dfinal"].float()
    dw = torch.stack([(ds * X[:, j:j + N]).sum((0, 1)) for j in range(K)], 1)
    dinit = dX[:, :K - 1].to(t) if s["init"] is not None else None
    return _unorder(dX[:, K - 1:].to(t), order), dw, ds.sum((0, 1)), dinit


_BLOCK = 64   # tokens whose decays are formed at once


def _scan_plain(s):
    c = s["case"]
    t = s["u"].dtype
    order = _order(c, s["u"].device)
    f = lambda name: s[name].float()[:, order]  # noqa: E731
    u, raw, Bm, Cm = f("u"), f("dt") + s["dt_bias"], f("Bm"), f("Cm")
    dt = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
    A = s["A"]
    B, N, D = u.shape
    S = A.shape[1]
    h = s["init"].clone() if s["init"] is not None else u.new_zeros(B, D, S)
    y = torch.empty_like(u)
    hs = u.new_empty(B, N + 1, D, S) if c["grad"] else None   # the states before each token, and the last
    if c["grad"]:
        hs[:, 0] = h
    for p0 in range(0, N, _BLOCK):
        p1 = min(N, p0 + _BLOCK)
        a = torch.exp(dt[:, p0:p1, :, None] * A)
        b = (dt * u)[:, p0:p1, :, None] * Bm[:, p0:p1, None]
        blk = hs[:, p0 + 1:p1 + 1] if c["grad"] else torch.empty_like(a)
        for i in range(p1 - p0):
            h = a[:, i] * h + b[:, i]
            blk[:, i] = h
        y[:, p0:p1] = (blk * Cm[:, p0:p1, None]).sum(-1)
    yv = y + s["D"] * u
    if s["z"] is not None:
        z = f("z")
        sig = 1.0 / (1.0 + torch.exp(-z))
    if not c["grad"]:
        out = yv * z * sig if s["z"] is not None else yv
        return _unorder(out.to(t), order), h
    dy = f("dy")
    dyv, dz = dy, None
    if s["z"] is not None:
        dyv = dy * z * sig
        dz = _unorder((dy * yv * sig * (1.0 + z * (1.0 - sig))).to(t), order)
    du, ddt = s["D"] * dyv, torch.zeros_like(u)
    dB, dC = torch.zeros_like(Bm), torch.zeros_like(Cm)
    dA = torch.zeros_like(A)
    g = s["dfinal"].clone() if s["dfinal"] is not None else u.new_zeros(B, D, S)
    for p0 in range((N - 1) // _BLOCK * _BLOCK, -1, -_BLOCK):
        p1 = min(N, p0 + _BLOCK)
        a = torch.exp(dt[:, p0:p1, :, None] * A)
        w = dyv[:, p0:p1, :, None] * Cm[:, p0:p1, None]
        gs = torch.empty_like(a)
        for i in range(p1 - p0 - 1, -1, -1):
            gs[:, i] = g + w[:, i]
            g = a[:, i] * gs[:, i]
        ga = gs * hs[:, p0:p1] * a
        gb = (gs * Bm[:, p0:p1, None]).sum(-1)
        du[:, p0:p1] += gb * dt[:, p0:p1]
        ddt[:, p0:p1] = (ga * A).sum(-1) + gb * u[:, p0:p1]
        dA += (ga * dt[:, p0:p1, :, None]).sum((0, 1))
        dB[:, p0:p1] = (gs * (dt * u)[:, p0:p1, :, None]).sum(2)
        dC[:, p0:p1] = (hs[:, p0 + 1:p1 + 1] * dyv[:, p0:p1, :, None]).sum(2)
    ddt = ddt / (1.0 + torch.exp(-raw))
    o = lambda v: _unorder(v.to(t), order)  # noqa: E731
    return (o(du), o(ddt), dA, o(dB), o(dC), (dyv * u).sum((0, 1)), dz, ddt.sum((0, 1)),
            g if s["init"] is not None else None)


def _norm_plain(s):
    c = s["case"]
    x = s["x"].float()
    B, N, C = x.shape
    G = c["G"]
    xg = x.reshape(B, N, G, C // G)
    if c["grad"]:
        mean, rstd = (s["stats"][..., i].reshape(B, 1, G, 1) for i in (0, 1))
    else:
        mean = xg.mean((1, 3), keepdim=True)
        rstd = torch.rsqrt(((xg - mean) ** 2).mean((1, 3), keepdim=True) + 1e-5)
    xh = ((xg - mean) * rstd).reshape(B, N, C)
    z = xh * s["gamma"] + s["beta"] if c["affine"] else xh
    sig = 1.0 / (1.0 + torch.exp(-z))
    if not c["grad"]:
        y = z * sig if c["act"] == "silu" else z
        return y.to(s["x"].dtype), torch.stack((mean.reshape(B, G), rstd.reshape(B, G)), -1)
    dz = s["dy"].float()
    if c["act"] == "silu":
        dz = dz * sig * (1.0 + z * (1.0 - sig))
    dg = (dz * s["gamma"] if c["affine"] else dz).reshape(B, N, G, C // G)
    xh4 = xh.reshape(B, N, G, C // G)
    dx = rstd * (dg - dg.mean((1, 3), keepdim=True) - xh4 * (dg * xh4).mean((1, 3), keepdim=True))
    dgamma = (dz * xh).sum((0, 1)) if c["affine"] else None
    return dx.reshape(B, N, C).to(s["x"].dtype), dgamma, dz.sum((0, 1)) if c["affine"] else None


# ------------------------------------------------------------------ the package's calls
def _conv_own(s):
    from recurrent_vision_backbone_b200 import ssm
    c = s["case"]
    if not c["grad"]:
        return ssm.gtr_causal_conv_fwd(s["x"], s["w"], c["H"], c["W"], c["dir"], bias=s["bias"],
                                       activation=ssm.ACT_SILU, init_state=s["init"], final_state=True)
    return ssm.gtr_causal_conv_bwd(s["x"], s["w"], s["dy"], c["H"], c["W"], c["dir"], bias=s["bias"],
                                   activation=ssm.ACT_SILU, init_state=s["init"], d_final_state=s["dfinal"],
                                   want_init_grad=s["init"] is not None)


def _scan_own(s):
    from recurrent_vision_backbone_b200 import ssm
    c = s["case"]
    if not c["grad"]:
        return ssm.gtr_ssm_scan_fwd(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], c["H"], c["W"], c["dir"], D=s["D"],
                                    z=s["z"], dt_bias=s["dt_bias"], dt_softplus=True, init_state=s["init"],
                                    final_state=True)
    return ssm.gtr_ssm_scan_bwd(s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dy"], c["H"], c["W"], c["dir"],
                                D=s["D"], z=s["z"], dt_bias=s["dt_bias"], dt_softplus=True, init_state=s["init"],
                                d_final_state=s["dfinal"], want_init_grad=s["init"] is not None)


def _norm_own(s):
    from recurrent_vision_backbone_b200 import norm
    c = s["case"]
    act = ACT_SILU if c["act"] == "silu" else ACT_NONE
    if not c["grad"]:
        return norm.gtr_group_norm_fwd(s["x"], c["G"], gamma=s["gamma"], beta=s["beta"], eps=1e-5, activation=act)
    return norm.gtr_group_norm_bwd(s["x"], s["dy"], s["stats"], c["G"], gamma=s["gamma"], beta=s["beta"],
                                   activation=act)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"conv": _conv_own, "scan": _scan_own, "norm": _norm_own}[op](state)
    return {"conv": _conv_plain, "scan": _scan_plain, "norm": _norm_plain}[op](state)


# ------------------------------------------------------------------ definitions in 64 bits
def _prefix(a, b):
    """All h_p = a_p h_{p-1} + b_p (h_{-1} = 0) along axis 1 by doubling: the pair (a, b) of a
    span composed with the pair of the span before it."""
    n, step = a.shape[1], 1
    while step < n:
        b = torch.cat((b[:, :step], a[:, step:] * b[:, :-step] + b[:, step:]), 1)
        a = torch.cat((a[:, :step], a[:, step:] * a[:, :-step]), 1)
        step *= 2
    return b


def _conv_exact(s):
    c = s["case"]
    K, N = c["K"], c["H"] * c["W"]
    order = _order(c, s["x"].device)
    x = s["x"].double().requires_grad_(c["grad"])
    B, _, D = x.shape
    init = s["init"].double() if s["init"] is not None else x.new_zeros(B, K - 1, D).detach()
    w, bias = s["w"].double(), s["bias"].double()
    if c["grad"]:
        init.requires_grad_(True), w.requires_grad_(True), bias.requires_grad_(True)
    X = torch.cat((init, x[:, order]), 1)
    pre = torch.einsum("bndk,dk->bnd", X.unfold(1, K, 1), w) + bias
    y = torch.empty_like(pre).index_copy(1, order, pre * torch.sigmoid(pre))
    if not c["grad"]:
        return y, X[:, N:]
    loss = (y * s["dy"].double()).sum()
    if s["dfinal"] is not None:
        loss = loss + (X[:, N:] * s["dfinal"].double()).sum()
    gx, gw, gb, gi = torch.autograd.grad(loss, (x, w, bias, init))
    return gx, gw, gb, gi if s["init"] is not None else None


def _scan_exact(s):
    c = s["case"]
    order = _order(c, s["u"].device)
    u, dt, Bm, Cm = (s[k].double()[:, order] for k in ("u", "dt", "Bm", "Cm"))
    raw = dt + s["dt_bias"].double()
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    z = s["z"].double()[:, order] if s["z"] is not None else None
    A, Dk = s["A"].double(), s["D"].double()
    B, N, D = u.shape
    S = A.shape[1]
    dy = s["dy"].double()[:, order] if c["grad"] else None
    gate = z * torch.sigmoid(z) if z is not None else 1.0
    dyv = dy * gate if c["grad"] else None
    yv, fin, dinit = torch.empty_like(u), u.new_empty(B, D, S), u.new_empty(B, D, S)
    if c["grad"]:
        du, ddt = torch.empty_like(u), torch.empty_like(u)
        dB, dC, dA = torch.zeros_like(Bm), torch.zeros_like(Cm), torch.zeros_like(A)
    width = max(1, min(D, 100_000_000 // (N * S)))   # channels at a time: under a GB for each array
    for b in range(B):
        for d0 in range(0, D, width):
            e = slice(d0, min(D, d0 + width))
            dtb, ub = dt[b, :, e, None], u[b, :, e, None]
            a = torch.exp(dtb * A[e])[None]
            bx = (dtb * ub * Bm[b, :, None])[None]
            h0 = s["init"][b, e].double() if s["init"] is not None else u.new_zeros(e.stop - e.start, S)
            bx[:, 0] += a[:, 0] * h0
            h = _prefix(a, bx)
            yv[b, :, e] = (h[0] * Cm[b, :, None]).sum(-1) + Dk[e] * u[b, :, e]
            fin[b, e] = h[0, -1]
            if not c["grad"]:
                continue
            src = (dyv[b, :, e, None] * Cm[b, :, None])[None]
            if s["dfinal"] is not None:
                src[:, -1] += s["dfinal"][b, e].double()
            # reversed in time, a step's decay is the one of the token after it
            back = torch.cat((torch.zeros_like(a[:, :1]), a.flip(1)[:, :-1]), 1)
            g = _prefix(back, src.flip(1)).flip(1)[0]
            before = torch.cat((h0[None], h[0, :-1]), 0)
            da = g * before * a[0]
            gB = (g * Bm[b, :, None]).sum(-1)
            du[b, :, e] = gB * dt[b, :, e] + Dk[e] * dyv[b, :, e]
            ddt[b, :, e] = (da * A[e]).sum(-1) + gB * u[b, :, e]
            dA[e] += (da * dtb).sum(0)
            dB[b] += (g * dtb * ub).sum(1)
            dC[b] += (h[0] * dyv[b, :, e, None]).sum(1)
            dinit[b, e] = a[0, 0] * g[0]
    back = torch.empty_like(order)
    back[order] = torch.arange(N, device=order.device)
    if not c["grad"]:
        return (yv * gate)[:, back], fin
    ddt = ddt * torch.sigmoid(raw)
    dz = None
    if z is not None:
        sg = torch.sigmoid(z)
        dz = (dy * yv * (sg + z * sg * (1 - sg)))[:, back]
    return (du[:, back], ddt[:, back], dA, dB[:, back], dC[:, back], (dyv * u).sum((0, 1)), dz, ddt.sum((0, 1)),
            dinit if s["init"] is not None else None)


def _norm_exact(s):
    c = s["case"]
    x = s["x"].double().requires_grad_(c["grad"])
    B, N, C = x.shape
    G = c["G"]
    xg = x.reshape(B, N, G, C // G)
    if c["grad"]:
        # the gradient at the statistics that the call is given: value theirs, derivative x's
        m, v = xg.mean((1, 3), keepdim=True), xg.var((1, 3), unbiased=False, keepdim=True)
        r = torch.rsqrt(v + 1e-5)
        st = s["stats"].double()
        mean = m + (st[..., 0].reshape(B, 1, G, 1) - m).detach()
        rstd = r + (st[..., 1].reshape(B, 1, G, 1) - r).detach()
    else:
        var, mean = torch.var_mean(xg, (1, 3), unbiased=False, keepdim=True)
        rstd = torch.rsqrt(var + 1e-5)
    y = ((xg - mean) * rstd).reshape(B, N, C)
    gamma, beta = s["gamma"], s["beta"]
    if c["affine"]:
        gamma, beta = gamma.double().requires_grad_(c["grad"]), beta.double().requires_grad_(c["grad"])
        y = y * gamma + beta
    if c["act"] == "silu":
        y = y * torch.sigmoid(y)
    if not c["grad"]:
        return y, torch.stack((mean.reshape(B, G), rstd.reshape(B, G)), -1)
    loss = (y * s["dy"].double()).sum()
    if not c["affine"]:
        return torch.autograd.grad(loss, x)[0], None, None
    return torch.autograd.grad(loss, (x, gamma, beta))


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _conv_exact, "scan": _scan_exact, "norm": _norm_exact}[case["op"]](s)
