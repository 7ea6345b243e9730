"""Infinite and NaN values in the convolution and the norm (GPU only): they show where the formulas send
them and nowhere else (the other channels, groups, batch entries and the rows outside the window stay as
they are)."""
import pytest
import torch

from recurrent_vision_backbone_b200 import gla, norm, ssm
from tests import ops_bounds as bounds
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def same(got, want, err, what):
    """Infinities and NaN in the same places, finite values within err (where it is finite too) and half a step."""
    t, exact = got.dtype, want
    got, want = got.double().cpu(), want.to(t).double()   # (a finite sum may round to an infinity of the type)
    for name, f in (("NaN", torch.isnan), ("inf", torch.isposinf), ("-inf", torch.isneginf)):
        assert torch.equal(f(got), f(want)), f"{what}: {name} in {int(f(got).sum())} places, not {int(f(want).sum())}"
    ok = torch.isfinite(want) & torch.isfinite(err)
    bad = bounds.outside(got, exact, err, t) & ok   # rounded once, so by half a step from the exact value
    assert not bad.any(), f"{what}: {int(bad.sum())} finite values are off"


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("B,N,D,silu", [(2, 50, 24, True), (2, 50, 33, False), (40, 64, 2048, False), (3, 2, 40, True)])
def test_convolution(value, B, N, D, silu):
    g, K = torch.Generator().manual_seed(N + D), 4
    pos = lambda *s: torch.rand(s, generator=g) + 0.5  # noqa: E731
    x, dy, init, df = pos(B, N, D).to(BF), pos(B, N, D).to(BF), pos(B, K - 1, D).to(BF), pos(B, K - 1, D).to(BF)
    w, b = pos(D, K), pos(D)
    order = ref.scan_order(1, N, 0)
    for t in (x, dy):
        keep = t[0, N // 2, D // 2].clone()
        t[0, N // 2, D // 2] = value
        out, fin = ssm.gtr_causal_conv_fwd(x.cuda(), w.cuda(), 1, N, 0, bias=b.cuda(), activation=int(silu), init_state=init.cuda(),
                                           final_state=True)
        y, f = ref.conv_fwd(x, w, order, b, silu, init)
        same(out, y, 2e-6 * ref.conv_fwd(x, w, order, b, silu, init, mag=True), "out")   # 2 (K + 8) roundings
        assert torch.equal(fin.double().cpu().nan_to_num(7, 8), f.nan_to_num(7, 8))
        got = ssm.gtr_causal_conv_bwd(x.cuda(), w.cuda(), dy.cuda(), 1, N, 0, bias=b.cuda(), activation=int(silu),
                                      init_state=init.cuda(), d_final_state=df.cuda())
        for (name, v, e), o in zip(bounds.conv_bwd(x, w, dy, order, b, silu, init, df), got):
            same(o, v, e, name)
        t[0, N // 2, D // 2] = keep
    assert gla.device_status() == gla.GTR_OK


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("B,N,C,G", [(2, 100, 64, 4), (2, 100, 60, 5), (1, 300, 1024, 2), (3, 1, 48, 3)])
def test_norm(value, B, N, C, G):
    g = torch.Generator().manual_seed(N + C)
    x, dy = torch.randn(B, N, C, generator=g).to(BF), torch.randn(B, N, C, generator=g).to(BF)
    gamma, beta = torch.rand(C, generator=g) + 0.5, torch.randn(C, generator=g)
    stats = ref.norm_fwd(x, G, gamma, beta, 1e-5, False)[1].float()
    keep, at = x.clone(), (0, N // 2, C // 2)
    x[at] = value
    out, st = norm.gtr_group_norm_fwd(x.cuda(), G, gamma.cuda(), beta.cuda())
    y, s, z = ref.norm_fwd(x, G, gamma, beta, 1e-5, False)
    same(out, y, 256 * ref.EPS32 * (z.abs() + gamma.abs() * 4 + beta.abs()), "out")   # |mean| / deviation is below 3
    assert torch.equal(torch.isfinite(st.cpu()).all(-1), torch.isfinite(s).all(-1))
    assert int((~torch.isfinite(s)).any(-1).sum()) == 1
    x, dy[at] = keep, value
    got = norm.gtr_group_norm_bwd(x.cuda(), dy.cuda(), stats.cuda(), G, gamma.cuda(), beta.cuda())
    for (name, v, e), o in zip(bounds.norm_bwd(x, dy, stats, G, gamma, beta, False), got):
        same(o, v, e, name)
    assert gla.device_status() == gla.GTR_OK
