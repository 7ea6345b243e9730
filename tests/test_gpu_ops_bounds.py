"""The operators against the element bounds of tests/ops_bounds.py (GPU only): tight enough that the share
of one chunk of tokens missing from a sum, or a state or a gradient not carried over a chunk's end, is
seen (tests/test_ops_bounds.py), at every shape of the other tests and at lengths where the chunks are
folded in several batches."""
import pytest
import torch

from recurrent_vision_backbone_b200 import gla, norm, ssm
from tests import ops_bounds as bounds
from tests import ops_reference as ref
from tests.test_gpu_norm import NORM, inputs as norm_inputs
from tests.test_gpu_ssm import CONV, NO_VALUE, SCAN, TYPES, conv_inputs, run_scan, run_scan_bwd, scan_inputs

pytestmark = pytest.mark.gpu

# 157 chunks; 79; decays down to nothing over many chunks; many sequences of a few chunks
LONG = [(1, 50, 100, 12, 16, 1, "bf16", True, True, True, True, True, 0.05),
        (2, 42, 60, 33, 8, 2, "fp16", True, True, True, True, True, 0.05),
        (1, 43, 47, 40, 12, 3, "fp16", True, True, True, True, True, 20.0),
        (60, 8, 20, 70, 24, 0, "bf16", True, True, True, True, True, 0.3)]


@pytest.mark.parametrize("case", SCAN + LONG)
def test_scan(case):
    B, H, W, D, S, direction, ty, gate, skip, bias, softplus, state, decay = case
    dev, N = torch.device("cuda", 0), H * W
    c, d = scan_inputs(B, H, W, D, S, TYPES[ty], dev, seed=H + D + S, gate=gate, skip=skip, bias=bias, state=state, decay=decay)
    out, fin = run_scan(d, H, W, direction, dt_softplus=softplus, init_state=d["init"], final_state=True)
    g = run_scan_bwd(d, H, W, direction, dt_softplus=softplus)
    assert gla.device_status() == gla.GTR_OK
    want = bounds.scan(c["u"], c["dt"], c["A"], c["Bm"], c["Cm"], ref.scan_order(H, W, direction), c["D"], c["z"], c["dt_bias"],
                       softplus, c["init"], c["dy"], c["df"], bounds.chain_of_scan(B, N))
    if max(float(v.abs().max()) for _, v, _ in want if v is not None) > NO_VALUE:
        pytest.skip("states past float32")   # time steps of either sign
    for (name, v, e), got in zip(want, (out, fin) + g):
        if got is not None and not (name == "D" and not skip):
            bounds.check(got, v, e, name)


@pytest.mark.parametrize("B,H,W,D,K,direction,ty,bias,silu,state", CONV + [(1, 128, 128, 72, 4, 2, "fp16", True, True, False)])
def test_convolution(B, H, W, D, K, direction, ty, bias, silu, state):
    dev = torch.device("cuda", 0)
    c, d = conv_inputs(B, H, W, D, K, TYPES[ty], bias, state, dev, seed=H + D + K)
    got = ssm.gtr_causal_conv_bwd(d["x"], d["w"], d["dy"], H, W, direction, bias=d["b"], activation=int(silu),
                                  init_state=d["init"], d_final_state=d["df"])
    assert gla.device_status() == gla.GTR_OK
    want = bounds.conv_bwd(c["x"], c["w"], c["dy"], ref.scan_order(H, W, direction), c["b"], silu, c["init"], c["df"])
    for (name, v, e), g in zip(want, got):
        if g is not None:
            bounds.check(g, v, e, name)


WIDE = [(1, 50, 32768, 1, "fp16", True, True, 0.0),     # a group over 128 blocks, over more than a warp joins, over 17
        (2, 37, 33000, 1, "bf16", True, True, 0.0), (3, 70, 4112, 1, "fp16", False, True, 0.5)]


@pytest.mark.parametrize("B,N,C,G,ty,silu,affine,mean", NORM + WIDE)
def test_norm(B, N, C, G, ty, silu, affine, mean):
    t = TYPES[ty]
    x, gamma, beta, dy = norm_inputs(B, N, C, t, True, mean, seed=N + C + 1)
    stats = ref.norm_fwd(x, G, gamma, beta, 1e-5, silu)[1].float()
    got = norm.gtr_group_norm_bwd(x.cuda(), dy.cuda(), stats.cuda(), G, gamma.cuda(), beta.cuda(), int(silu))
    assert gla.device_status() == gla.GTR_OK
    for (name, v, e), g in zip(bounds.norm_bwd(x, dy, stats, G, gamma, beta, silu), got):
        bounds.check(g, v, e, name)


@pytest.mark.parametrize("B,C,G,ty", [(1500, 128, 4, "fp16"), (700, 60, 5, "bf16"), (300, 33, 1, "fp16"), (2100, 512, 8, "bf16")])
def test_norm_of_each_token(B, C, G, ty):
    """The tokens as batch entries of one row each: statistics of every token by itself."""
    t = TYPES[ty]
    x, gamma, beta, dy = norm_inputs(B, 1, C, t, True, 0.5, seed=C)
    out, st = norm.gtr_group_norm_fwd(x.cuda(), G, gamma.cuda(), beta.cuda(), activation=1)
    y, stats, z = ref.norm_fwd(x, G, gamma, beta, 1e-5, True)
    # the mean and the deviations are sums of C / G values, C / G / 8 + 5 in a chain: 64 roundings of what meets in z
    shift = float((stats[..., 0].abs() * stats[..., 1]).max())
    bounds.check(out, y, 64 * ref.EPS32 * (z.abs() + gamma.abs() * (1 + shift) + beta.abs()), "out")
    got = norm.gtr_group_norm_bwd(x.cuda(), dy.cuda(), st, G, gamma.cuda(), beta.cuda(), 1)
    assert gla.device_status() == gla.GTR_OK
    for (name, v, e), g in zip(bounds.norm_bwd(x, dy, st.cpu(), G, gamma, beta, True), got):
        bounds.check(g, v, e, name)
