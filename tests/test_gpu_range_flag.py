"""Which fp16 outputs set GTR_ERR_RANGE (GPU only): those that are stored as an infinity or NaN.  A
value from 65504 up to 65520 is stored as 65504, the largest finite fp16, and sets nothing, whichever
of an operator's kernels computes it."""
import pytest
import torch

from recurrent_vision_backbone_b200 import gla, norm, ssm

pytestmark = pytest.mark.gpu

INSIDE, OUTSIDE = 65512.0, 65524.0
H = torch.float16


def full(*shape, v=1.0, t=torch.float32):
    return torch.full(shape, v, dtype=t, device="cuda")


def off_grid(t):
    return torch.cat((t.new_zeros(1), t.reshape(-1)))[1:].view(t.shape)


def expect(out, value):
    assert torch.equal(out.float(), full(*out.shape, v=65504.0 if value == INSIDE else float("inf")))
    assert gla.device_status() == (gla.GTR_OK if value == INSIDE else gla.GTR_ERR_RANGE)
    assert gla.device_status() == gla.GTR_OK


@pytest.mark.parametrize("value", [INSIDE, OUTSIDE])
@pytest.mark.parametrize("B,N,S", [(1, 1, 16), (1, 1, 12), (300, 1, 8), (1, 1, 4), (1, 90, 16), (2, 1, 32)])
def test_scan(value, B, N, S):
    """out = D u: the states take no part (u B = 0)."""
    D = 1024 if B > 1 else 32
    u, zero = full(B, N, D, t=H), full(B, N, D, v=0.0, t=H)
    bc = full(B, N, S, v=0.0, t=H)
    out, _ = ssm.gtr_ssm_scan_fwd(u, zero, -full(D, S), bc, bc, 1, N, 0, D=full(D, v=value))
    expect(out, value)


@pytest.mark.parametrize("value", [INSIDE, OUTSIDE])
def test_scan_sums_over_channels(value):
    """dC = sum over the channels of d_out h, two channels of one state."""
    B, N, D, S = 1, 1, 2, 1
    one = full(B, N, D, t=H)
    h = value / 2 / 128
    got = ssm.gtr_ssm_scan_bwd(0 * one, one, full(D, S, v=0.0), 0 * one[..., :1], 0 * one[..., :1], 128 * one, 1, 1, 0,
                               dt_softplus=False, init_state=full(B, D, S, v=h))
    expect(got[4], value)


@pytest.mark.parametrize("value", [INSIDE, OUTSIDE])
@pytest.mark.parametrize("B,N,D", [(1, 5, 64), (1, 5, 33), (40, 64, 2048)])
def test_convolution(value, B, N, D):
    """out = bias."""
    out, _ = ssm.gtr_causal_conv_fwd(full(B, N, D, v=0.0, t=H), full(D, 4), 1, N, 0, bias=full(D, v=value), activation=0)
    expect(out, value)


@pytest.mark.parametrize("value", [INSIDE, OUTSIDE])
@pytest.mark.parametrize("C,G,aligned", [(64, 4, True), (64, 4, False), (40, 4, True), (33, 3, True)])
def test_norm(value, C, G, aligned):
    """out = beta: x has no spread."""
    x = full(1, 20, C, t=H)
    out, _ = norm.gtr_group_norm_fwd(x if aligned else off_grid(x), G, None, full(C, v=value))
    expect(out, value)


@pytest.mark.parametrize("value", [INSIDE, OUTSIDE])
@pytest.mark.parametrize("C,G,aligned", [(64, 4, True), (64, 4, False), (40, 4, True), (33, 3, True)])
def test_norm_gradient(value, C, G, aligned):
    """Two tokens of opposite d_out and x = mean: grad_x = rstd d_out."""
    x = full(1, 2, C, v=0.0, t=H)
    dy = full(1, 2, C, v=128.0, t=H)
    dy[:, 1] = -128
    st = torch.stack((full(1, G, v=0.0), full(1, G, v=value / 128)), -1)
    f = (lambda t: t) if aligned else off_grid
    got = norm.gtr_group_norm_bwd(f(x), f(dy), st, G)[0]
    expect(got[:, :1], value)
