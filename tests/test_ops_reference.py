"""The 64-bit forms the operators' GPU tests compare with, themselves checked on the CPU:
gradients against central differences and against float64 autograd, scan orders against the
definition, and carried states against one run over the whole sequence."""
import pytest
import torch

from tests import ops_reference as ref


def rnd(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def scan_case(B, H, W, C, S, seed=0):
    N = H * W
    return dict(u=rnd(B, N, C, seed=seed), dt=rnd(B, N, C, seed=seed + 1), A=-torch.exp(rnd(C, S, seed=seed + 2)),
                Bm=rnd(B, N, S, seed=seed + 3), Cm=rnd(B, N, S, seed=seed + 4), D=rnd(C, seed=seed + 5),
                z=rnd(B, N, C, seed=seed + 6), dt_bias=rnd(C, seed=seed + 7), init=rnd(B, C, S, seed=seed + 8))


def differences(f, t, eps=1e-6):
    g = torch.empty_like(t)
    flat = t.reshape(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + eps
        hi = f()
        flat[i] = keep - eps
        lo = f()
        flat[i] = keep
        g.reshape(-1)[i] = (hi - lo) / (2 * eps)
    return g


@pytest.mark.parametrize("direction", range(4))
def test_scan_order_visits_neighbours_as_named(direction):
    H, W = 3, 4
    o = ref.scan_order(H, W, direction).tolist()
    want = {0: [y * W + x for y in range(H) for x in range(W)],
            1: [y * W + W - 1 - x for y in range(H) for x in range(W)],
            2: [y * W + x for x in range(W) for y in range(H)],
            3: [(H - 1 - y) * W + x for x in range(W) for y in range(H)]}[direction]
    assert o == want


@pytest.mark.parametrize("direction,softplus", [(0, True), (1, False), (2, True), (3, True)])
def test_scan_gradients_against_differences(direction, softplus):
    c = scan_case(2, 2, 3, 2, 3, seed=20 + direction)
    order = ref.scan_order(2, 3, direction)
    dy, df = rnd(2, 6, 2, seed=1), rnd(2, 2, 3, seed=2)

    def loss():
        y, h = ref.scan_fwd(c["u"], c["dt"], c["A"], c["Bm"], c["Cm"], order, c["D"], c["z"], c["dt_bias"], softplus,
                            c["init"])
        return float((y * dy).sum() + (h * df).sum())

    got = ref.scan_bwd(c["u"], c["dt"], c["A"], c["Bm"], c["Cm"], dy, order, c["D"], c["z"], c["dt_bias"], softplus,
                       c["init"], df)
    for name, g in zip(("u", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "init"), got):
        want = differences(loss, c[name])
        assert (g - want).abs().max() <= 1e-6 * max(1.0, float(want.abs().max())), name


@pytest.mark.parametrize("K,N,silu", [(2, 5, True), (3, 1, True), (4, 6, False), (4, 2, True)])
def test_conv_gradients_against_differences(K, N, silu):
    x, w, b, init = rnd(2, N, 3, seed=1), rnd(3, K, seed=2), rnd(3, seed=3), rnd(2, K - 1, 3, seed=4)
    dy, df = rnd(2, N, 3, seed=5), rnd(2, K - 1, 3, seed=6)
    order = ref.scan_order(1, N, 1)

    def loss():
        y, f = ref.conv_fwd(x, w, order, b, silu, init)
        return float((y * dy).sum() + (f * df).sum())

    got = ref.conv_bwd(x, w, dy, order, b, silu, init, df)
    for name, g, t in zip(("x", "w", "bias", "init"), got, (x, w, b, init)):
        want = differences(loss, t)
        assert (g - want).abs().max() <= 1e-6 * max(1.0, float(want.abs().max())), name


@pytest.mark.parametrize("silu,affine", [(False, True), (True, True), (True, False)])
def test_norm_gradients_against_autograd(silu, affine):
    x = rnd(2, 5, 6, seed=1).requires_grad_(True)
    gamma = rnd(6, seed=2).requires_grad_(True) if affine else None
    beta = rnd(6, seed=3).requires_grad_(True) if affine else None
    dy = rnd(2, 5, 6, seed=4)
    y, stats, _ = ref.norm_fwd(x, 3, gamma, beta, 1e-5, silu)
    want = torch.autograd.grad((y * dy).sum(), (x, gamma, beta) if affine else (x,))
    got = ref.norm_bwd(x.detach(), dy, stats.detach(), 3, gamma, beta, silu)
    for g, w_ in zip(got, want):
        assert (g - w_).abs().max() <= 1e-10


def test_carried_states_equal_one_run():
    c = scan_case(1, 1, 9, 3, 4, seed=50)
    whole = ref.scan_fwd(c["u"], c["dt"], c["A"], c["Bm"], c["Cm"], ref.scan_order(1, 9, 0), c["D"], c["z"], c["dt_bias"],
                         True, c["init"])
    h, ys = c["init"], []
    for lo, hi in ((0, 4), (4, 5), (5, 9)):
        y, h = ref.scan_fwd(c["u"][:, lo:hi], c["dt"][:, lo:hi], c["A"], c["Bm"][:, lo:hi], c["Cm"][:, lo:hi],
                            ref.scan_order(1, hi - lo, 0), c["D"], c["z"][:, lo:hi], c["dt_bias"], True, h)
        ys.append(y)
    assert torch.allclose(torch.cat(ys, 1), whole[0], rtol=1e-12, atol=1e-12)
    assert torch.allclose(h, whole[1], rtol=1e-12, atol=1e-12)
