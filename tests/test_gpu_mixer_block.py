"""The operators as a block uses them (GPU only): group norm, an in-projection cut into x and z,
the causal convolution, a projection cut into dt, B and C, the gated scan, group norm over heads, an
out-projection and the residual; forward, backward, and a prompt followed by single tokens.

Bound of the training pass, as ||got - want|| / ||want|| against the same block in 64 bits with
autograd: the block stores eleven fp16 tensors forward and about as many gradients backward, each
rounded to within 2^-11; the projections and norms keep magnitudes (their gains are near 1, the
recurrence's and the activations' below 4): 22 x 4 x 2^-11 = 0.043.
"""
import pytest
import torch

from recurrent_vision_backbone_b200 import gla, norm, ssm
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu

C, D, S, G, HEADS, K = 96, 192, 16, 4, 6, 4
BOUND = 22 * 4 * 2.0 ** -11


def make(B, N, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: torch.randn(s, generator=g) * std  # noqa: E731
    p = dict(gamma1=1 + r(C, std=0.1), beta1=r(C, std=0.1), win=r(C, 2 * D, std=C ** -0.5), wconv=r(D, K, std=K ** -0.5),
             bconv=r(D, std=0.1), wx=r(D, D + 2 * S, std=D ** -0.5), dt_bias=r(D, std=0.5) - 2,
             A=-torch.exp(r(D, S, std=0.5)), Dk=1 + r(D, std=0.1), gamma2=1 + r(D, std=0.1), beta2=r(D, std=0.1),
             wout=r(D, C, std=D ** -0.5))
    for n in ("win", "wx", "wout"):
        p[n] = p[n].half()
    return r(B, N, C).half(), p, r(B, N, C).half()


def block64(x, p, H, W, direction):
    """The block in 64 bits, differentiable."""
    order = ref.scan_order(H, W, direction)
    n1 = ref.norm_fwd(x, G, p["gamma1"], p["beta1"], 1e-5, False)[0]
    xz = n1 @ p["win"]
    u = ref.conv_fwd(xz[..., :D], p["wconv"], order, p["bconv"], True, None)[0]
    dbc = u @ p["wx"]
    y, _ = ref.scan_fwd(u, dbc[..., :D], p["A"], dbc[..., D:D + S], dbc[..., D + S:], order, p["Dk"], xz[..., D:],
                        p["dt_bias"], True, None)
    n2 = ref.norm_fwd(y, HEADS, p["gamma2"], p["beta2"], 1e-5, True)[0]
    return x + n2 @ p["wout"]


def forward(x, p, H, W, direction, states=None):
    s = states or (None, None)
    n1, st1 = norm.gtr_group_norm_fwd(x, G, p["gamma1"], p["beta1"])
    xz = n1 @ p["win"]
    u, cs = ssm.gtr_causal_conv_fwd(xz[..., :D], p["wconv"], H, W, direction, bias=p["bconv"], init_state=s[0],
                                    final_state=s[0] if s[0] is not None else True)
    dbc = u @ p["wx"]
    y, hs = ssm.gtr_ssm_scan_fwd(u, dbc[..., :D], p["A"], dbc[..., D:D + S], dbc[..., D + S:], H, W, direction, D=p["Dk"],
                                 z=xz[..., D:], dt_bias=p["dt_bias"], init_state=s[1],
                                 final_state=s[1] if s[1] is not None else True)
    n2, st2 = norm.gtr_group_norm_fwd(y, HEADS, p["gamma2"], p["beta2"], activation=norm.ACT_SILU)
    return x + n2 @ p["wout"], (n1, st1, xz, u, dbc, y, st2, n2), (cs, hs)


def backward(x, p, H, W, direction, kept, dout):
    n1, st1, xz, u, dbc, y, st2, n2 = kept
    flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
    g = {"wout": flat(n2).t() @ flat(dout)}
    dy, g["gamma2"], g["beta2"] = norm.gtr_group_norm_bwd(y, dout @ p["wout"].t(), st2, HEADS, p["gamma2"], p["beta2"],
                                                          norm.ACT_SILU)
    du, ddt, g["A"], dB, dC, g["Dk"], dz, g["dt_bias"], _ = ssm.gtr_ssm_scan_bwd(
        u, dbc[..., :D], p["A"], dbc[..., D:D + S], dbc[..., D + S:], dy, H, W, direction, D=p["Dk"], z=xz[..., D:],
        dt_bias=p["dt_bias"], want_init_grad=False)
    ddbc = torch.cat((ddt, dB, dC), -1)
    g["wx"] = flat(u).t() @ flat(ddbc)
    dxc, g["wconv"], g["bconv"], _ = ssm.gtr_causal_conv_bwd(xz[..., :D], p["wconv"], du + ddbc @ p["wx"].t(), H, W,
                                                             direction, bias=p["bconv"], want_init_grad=False)
    dxz = torch.cat((dxc, dz), -1)
    g["win"] = flat(n1).t() @ flat(dxz)
    dx, g["gamma1"], g["beta1"] = norm.gtr_group_norm_bwd(x, dxz @ p["win"].t(), st1, G, p["gamma1"], p["beta1"])
    g["x"] = dx + dout
    return g


@pytest.mark.parametrize("B,H,W,direction", [(2, 9, 13, 3), (1, 1, 150, 0), (1, 12, 12, 2)])
def test_training_pass(B, H, W, direction):
    x, p, dout = make(B, H * W, seed=H)
    x64 = x.double().requires_grad_(True)
    p64 = {k: v.double().requires_grad_(True) for k, v in p.items()}
    out64 = block64(x64, p64, H, W, direction)
    want = dict(zip(["x"] + list(p64), torch.autograd.grad((out64 * dout.double()).sum(), [x64] + list(p64.values()))))
    dev = torch.device("cuda", 0)
    xd, pd = x.to(dev), {k: v.to(dev) for k, v in p.items()}
    out, kept, _ = forward(xd, pd, H, W, direction)
    got = backward(xd, pd, H, W, direction, kept, dout.to(dev))
    assert gla.device_status() == gla.GTR_OK
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    assert rel(out, out64.detach()) <= BOUND
    for k, w in want.items():
        assert rel(got[k], w) <= BOUND, k


def test_tokens_after_a_prompt():
    """The convolution and the scan carried token by token (a norm over the tokens seen has no such
    form: each token is normalised by itself here) against the whole sequence through the same calls."""
    dev, N, tail = torch.device("cuda", 0), 40, 5
    x, p, _ = make(1, N, seed=7)
    xd, pd = x.to(dev), {k: v.to(dev) for k, v in p.items()}
    xz = xd @ pd["win"]

    def run(xz, states):
        n = xz.shape[1]
        u, cs = ssm.gtr_causal_conv_fwd(xz[..., :D], pd["wconv"], 1, n, 0, bias=pd["bconv"], init_state=states[0],
                                        final_state=states[0] if states[0] is not None else True)
        dbc = torch.cat([u[:, i:i + 1] @ pd["wx"] for i in range(n)], 1)   # one token's product at a time, as it is served
        y, hs = ssm.gtr_ssm_scan_fwd(u, dbc[..., :D], pd["A"], dbc[..., D:D + S], dbc[..., D + S:], 1, n, 0, D=pd["Dk"],
                                     z=xz[..., D:], dt_bias=pd["dt_bias"], init_state=states[1],
                                     final_state=states[1] if states[1] is not None else True)
        return y, (cs, hs)
    whole, (wc, wh) = run(xz, (None, None))
    y, st = run(xz[:, :N - tail], (None, None))
    ys = [y]
    for i in range(N - tail, N):
        y, st = run(xz[:, i:i + 1], st)
        ys.append(y)
    got = torch.cat(ys, 1).double()
    # both are the same sums in other orders: an output's two roundings to fp16, and float32's
    scale = float(whole.double().abs().max())
    assert float((got - whole.double()).abs().max()) <= 2 * 2.0 ** -11 * scale
    assert torch.equal(st[0], wc)
    assert float((st[1] - wh).abs().max()) <= 1e-5 * float(wh.abs().max())
