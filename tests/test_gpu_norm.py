"""Channels-last group norm against its 64-bit form (GPU only).

Bounds: half a step of the output's type, and float32 roundings (2^-24) of the magnitudes that
meet in the result: |x| and |mean| over the deviation (their difference may cancel), gamma,
beta.  Sums over a group run as chains of at most some 100 values that are then merged, and a
silu has a slope of at most 1.1: 256 roundings cover the statistics, the normalisation and the
activation; sums over all tokens (the parameters' gradients) add one for each of the values a
chain holds, bounded by their number.
"""
import pytest
import torch

from recurrent_vision_backbone_b200 import gla, norm
from tests import ops_reference as ref
from tests.test_gpu_ssm import TYPES, check, guarded, rnd

pytestmark = pytest.mark.gpu

K = 256
NORM = [
    # B, N, C, groups, type, silu, affine, mean
    (1, 1, 64, 8, "fp16", False, True, 0.0),         # one token
    (2, 3, 8, 1, "bf16", True, True, 0.0),
    (1, 7, 30, 10, "fp16", True, True, 0.0),         # three channels a group
    (3, 50, 33, 1, "bf16", False, True, 0.0),        # odd channels
    (1, 400, 256, 4, "fp16", True, True, 0.0),
    (2, 1600, 128, 2, "bf16", True, False, 0.0),     # 64 channels a group, no affine
    (1, 1961, 768, 12, "fp16", False, True, 3.0),
    (2, 333, 96, 12, "bf16", True, True, 0.0),       # 8 channels a group
    (1, 2304, 512, 1, "fp16", True, True, 1.0),      # one group over all channels
    (4, 129, 520, 65, "fp16", True, True, 0.0),      # 65 groups
    (1, 5000, 64, 64, "fp16", False, True, 0.0),     # one channel a group (instance norm)
    (1, 640, 64, 4, "fp16", False, True, 50.0),      # a mean far above the spread
    (1, 16384, 32, 1, "bf16", True, True, 0.0),
    (5, 70, 24, 3, "bf16", False, False, 0.0),
    (1, 300, 1344, 7, "fp16", True, True, 0.0),      # 192 channels a group
    (2, 9000, 64, 2, "bf16", True, True, 0.5),
]


def inputs(B, N, C, t, affine, mean, seed):
    g = torch.Generator().manual_seed(seed)
    x = (rnd(g, B, N, C) + mean + rnd(g, B, 1, C, std=0.3)).to(t)
    gamma, beta = (1 + rnd(g, C, std=0.2), rnd(g, C, std=0.3)) if affine else (None, None)
    return x, gamma, beta, rnd(g, B, N, C).to(t)


def dev_of(*ts):
    return tuple(None if t is None else t.to("cuda:0") for t in ts)


@pytest.mark.parametrize("B,N,C,G,ty,silu,affine,mean", NORM)
def test_forward(B, N, C, G, ty, silu, affine, mean):
    t = TYPES[ty]
    x, gamma, beta, _ = inputs(B, N, C, t, affine, mean, seed=N + C)
    dx, dg, db = dev_of(x, gamma, beta)
    out, ok_o = guarded((B, N, C), t, dx.device)
    st, ok_s = guarded((B, G, 2), torch.float32, dx.device)
    ws, ok_w = guarded((max(norm.group_norm_fwd_workspace_bytes(B, N, C, G) // 4, 1),), torch.float32, dx.device)
    norm.gtr_group_norm_fwd(dx, G, dg, db, 1e-5, int(silu), out=out, stats=st, workspace=ws)
    assert gla.device_status() == gla.GTR_OK
    y, stats, _ = ref.norm_fwd(x, G, gamma, beta, 1e-5, silu)
    a = x.double().abs().reshape(B, N, G, C // G)
    m, r = stats[..., 0].reshape(B, 1, G, 1), stats[..., 1].reshape(B, 1, G, 1)
    mag = ((a + m.abs()) * r).reshape(B, N, C)
    if affine:
        mag = mag * gamma.double().abs() + beta.double().abs()
    check(out, y, mag, K, "out")
    check(st[..., 0], stats[..., 0], a.mean((1, 3)) + m.reshape(B, G).abs(), K, "mean")
    # the variance is a sum of squares of differences of rounded values around the mean
    check(st[..., 1], stats[..., 1], stats[..., 1] * (1 + ((a + m.abs()) * r).amax((1, 3))), K, "rstd")
    assert ok_o() and ok_s() and ok_w()
    again, _ = norm.gtr_group_norm_fwd(dx, G, dg, db, 1e-5, int(silu), out=dx)   # in place
    assert torch.equal(again, out)


@pytest.mark.parametrize("B,N,C,G,ty,silu,affine,mean", NORM)
def test_backward(B, N, C, G, ty, silu, affine, mean):
    t = TYPES[ty]
    x, gamma, beta, dy = inputs(B, N, C, t, affine, mean, seed=N + C)
    stats = ref.norm_fwd(x, G, gamma, beta, 1e-5, silu)[1].float()
    dx, dg, db, ddy, dst = dev_of(x, gamma, beta, dy, stats)
    outs = [guarded((B, N, C), t, dx.device), guarded((C,), torch.float32, dx.device),
            guarded((C,), torch.float32, dx.device)]
    ws, ok_w = guarded((max(norm.group_norm_bwd_workspace_bytes(B, N, C, G) // 4, 1),), torch.float32, dx.device)
    got = norm.gtr_group_norm_bwd(dx, ddy, dst, G, dg, db, int(silu), workspace=ws, grads=tuple(o for o, _ in outs))
    assert gla.device_status() == gla.GTR_OK
    args = (x, dy, stats, G, gamma, beta, silu)
    want, mag = ref.norm_bwd(*args), ref.norm_bwd(*args, mag=True)
    for name, g, w, m, k in zip(("x", "gamma", "beta"), got, want, mag, (K, K + B * N, K + B * N)):
        check(g, w, m, k, name)
    assert all(ok() for _, ok in outs) and ok_w()


@pytest.mark.parametrize("C,G", [(64, 4), (72, 8), (768, 12)])
def test_unaligned_tensors_and_absent_gradients(C, G):
    """Tensors off the 16-byte grid give the same values; each parameter gradient may be left out."""
    B, N = 2, 217
    x, gamma, beta, dy = inputs(B, N, C, torch.float16, True, 0.0, seed=C)
    dx, dg, db, ddy = dev_of(x, gamma, beta, dy)
    off = lambda t: torch.cat((t.new_zeros(1), t.reshape(-1)))[1:].view(t.shape)  # noqa: E731
    y, st = norm.gtr_group_norm_fwd(dx, G, dg, db, activation=1)
    y1, st1 = norm.gtr_group_norm_fwd(off(dx), G, dg, db, activation=1)
    want, _, z = ref.norm_fwd(x, G, gamma, beta, 1e-5, True)
    for o in (y, y1):
        check(o, want, 8 + z.abs() * 4, K, "out")
    a = norm.gtr_group_norm_bwd(dx, ddy, st, G, dg, db, 1)
    b = norm.gtr_group_norm_bwd(off(dx), off(ddy), st, G, dg, db, 1)
    w, m = (ref.norm_bwd(x, dy, st.cpu(), G, gamma, beta, True, mag=f) for f in (False, True))
    for g in (a, b):
        for i, k in enumerate((K, K + B * N, K + B * N)):
            check(g[i], w[i], m[i], k, str(i))
    only = norm.gtr_group_norm_bwd(dx, ddy, st, G, dg, db, 1, grads=(torch.empty_like(dx), None, None))
    assert torch.equal(only[0], a[0])
    only = norm.gtr_group_norm_bwd(dx, ddy, st, G, dg, db, 1, grads=(torch.empty_like(dx), None, torch.empty_like(db)))
    assert torch.equal(only[2], a[2])


def test_constant_groups_and_large_values():
    """A group without spread: rstd = 1 / sqrt(eps), out = beta; values at fp16's edge keep their
    statistics (their squares pass fp16, not float32); equal calls give equal bits."""
    dev = torch.device("cuda", 0)
    x = torch.full((1, 100, 64), 3.5, dtype=torch.float16, device=dev)
    beta = torch.arange(64, dtype=torch.float32, device=dev)
    y, st = norm.gtr_group_norm_fwd(x, 4, None, beta, 1e-5)
    assert torch.equal(st[..., 0], torch.full_like(st[..., 0], 3.5))
    assert torch.allclose(st[..., 1], torch.full_like(st[..., 1], 1e-5 ** -0.5), rtol=1e-6)
    assert torch.equal(y, beta.half().expand_as(y))
    g = torch.Generator().manual_seed(3)
    big = (rnd(g, 1, 500, 64).sign() * 60000).half()
    y, st = norm.gtr_group_norm_fwd(big.to(dev), 2)
    y2, st2 = norm.gtr_group_norm_fwd(big.to(dev), 2)
    assert torch.equal(y, y2) and torch.equal(st, st2)
    want, ws, _ = ref.norm_fwd(big, 2, None, None, 1e-5, False)
    check(y, want, want.abs() + 1, K, "out")
    assert gla.device_status() == gla.GTR_OK


def test_overflow_empty_and_refusals():
    dev = torch.device("cuda", 0)
    x = torch.randn(1, 40, 32, device=dev).half()
    norm.gtr_group_norm_fwd(x, 4, torch.full((32,), 1e5, device=dev))
    assert gla.device_status() == gla.GTR_ERR_RANGE and gla.device_status() == gla.GTR_OK
    x[0, 3, 5] = float("nan")
    norm.gtr_group_norm_fwd(x, 4)
    assert gla.device_status() == gla.GTR_ERR_RANGE and gla.device_status() == gla.GTR_OK
    e = torch.empty(2, 0, 32, dtype=torch.float16, device=dev)
    norm.gtr_group_norm_fwd(e, 4)
    one = torch.ones(32, device=dev)
    g = norm.gtr_group_norm_bwd(e, e.clone(), torch.zeros(2, 4, 2, device=dev), 4, one, one)
    assert not g[1].any() and not g[2].any()
    x = torch.randn(1, 40, 32, device=dev).half()
    for bad in (lambda: norm.gtr_group_norm_fwd(x, 5), lambda: norm.gtr_group_norm_fwd(x.float(), 4),
                lambda: norm.gtr_group_norm_fwd(x[..., :16], 4), lambda: norm.gtr_group_norm_fwd(x.cpu(), 4),
                lambda: norm.gtr_group_norm_fwd(x, 4, one.half())):
        with pytest.raises(ValueError):
            bad()
    st = torch.zeros(1, 4, 2, device=dev)
    for bad in (lambda: norm.gtr_group_norm_fwd(x, 4, eps=-1.0), lambda: norm.gtr_group_norm_fwd(x, 4, activation=7),
                lambda: norm.gtr_group_norm_bwd(x, x.clone(), st, 4, grads=(x, None, None))):
        with pytest.raises(gla.GTRError) as err:
            bad()
        assert err.value.status == gla.GTR_ERR_INVALID_ARG
    assert gla.device_status() == gla.GTR_OK


def test_captured_and_on_another_stream():
    dev = torch.device("cuda", 0)
    x, gamma, beta, dy = inputs(2, 900, 256, torch.bfloat16, True, 0.0, seed=1)
    dx, dg, db, ddy = dev_of(x, gamma, beta, dy)

    def run(stream=None):
        y, st = norm.gtr_group_norm_fwd(dx, 8, dg, db, activation=1, stream=stream)
        return (y, st) + norm.gtr_group_norm_bwd(dx, ddy, st, 8, dg, db, 1, stream=stream)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    on = run(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(on, run()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    x2, _, _, dy2 = inputs(2, 900, 256, torch.bfloat16, True, 2.0, seed=2)
    dx.copy_(x2), ddy.copy_(dy2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, run()))
