"""The bounds that the operators' GPU tests compare with, themselves checked on the CPU: their values are
the 64-bit forms', results in float32 steps keep within them, and results of kernels that went wrong
(nothing computed, the share of one chunk of tokens lost, a state or a gradient not carried into the
next chunk) do not."""
import pytest
import torch

from tests import ops_bounds as bounds
from tests import ops_reference as ref
from tests.test_gpu_norm import inputs as norm_inputs
from tests.test_gpu_ssm import TYPES, conv_inputs, scan_inputs

CPU = torch.device("cpu")
SCANS = [
    # B, N, D, S, type, decay, the states outlive a chunk
    (1, 5000, 12, 16, "bf16", 0.05, True),
    (1, 323, 31, 7, "fp16", 1.0, True),
    (2, 300, 96, 16, "fp16", 40.0, False),
    (100, 100, 40, 16, "fp16", 1.0, True),
    (2, 300, 48, 20, "bf16", 1.0, True),
]


def refused(mutant, want, err, dtype):
    """The share of the entries that the comparison throws out, the mutant rounded to its type first."""
    return float(bounds.outside(mutant.to(dtype).double(), want, err, dtype).double().mean())


def cut(c, lo, hi, init, dfinal):
    n = c["u"].shape[1]
    s = {k: v[:, lo:hi] if v is not None and v.dim() == 3 and k not in ("init", "df") and v.shape[1] == n else v for k, v in c.items()}
    return (s["u"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dy"], ref.scan_order(1, hi - lo, 0), s["D"], s["z"], s["dt_bias"], True,
            init, dfinal)


def forward(a):
    return ref.scan_fwd(*a[:5], *a[6:-1])


@pytest.mark.parametrize("B,N,D,S,ty,decay,carried", SCANS)
def test_scan_bounds(B, N, D, S, ty, decay, carried):
    t, f = TYPES[ty], torch.float32
    c, _ = scan_inputs(B, 1, N, D, S, t, CPU, seed=N + D, decay=decay)
    whole = cut(c, 0, N, c["init"], c["df"])
    r = {n: (v, e) for n, v, e in bounds.scan(*whole[:5], *whole[6:-1], dy=c["dy"], dfinal=c["df"], chain=bounds.chain_of_scan(B, N))}
    names = ("u", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "init")
    (y, h), grads = forward(whole), dict(zip(names, ref.scan_bwd(*whole)))
    for n, w in dict(grads, **{"out": y, "final state": h}).items():
        assert torch.allclose(r[n][0], w, rtol=1e-9, atol=1e-12), n
    types = {n: f if n in ("A", "D", "dt_bias", "init", "final state") else t for n in r}
    for n, (v, e) in r.items():
        assert refused(v, v, e, types[n]) == 0, n
        assert refused(torch.zeros_like(v), v, e, types[n]) > 0.9, n
    # the tokens of one chunk missing from the sums over tokens
    lo = N // 2 // 32 * 32
    hi = lo + 32
    h_lo = forward(cut(c, 0, lo, c["init"], None))[1]
    g_hi = ref.scan_bwd(*cut(c, hi, N, forward(cut(c, 0, hi, c["init"], None))[1], c["df"]))[8]
    lost = dict(zip(names, ref.scan_bwd(*cut(c, lo, hi, h_lo, g_hi))))
    for n in ("A", "D", "dt_bias"):
        b0 = {k: v[:1] if v is not None and v.shape[0] == B and k not in ("A", "D", "dt_bias") else v for k, v in c.items()}
        one = lost if B == 1 else dict(zip(names, ref.scan_bwd(*cut(b0, lo, hi, h_lo[:1], g_hi[:1]))))   # of one sequence
        assert refused(r[n][0] - one[n], *r[n], f) > 0.5, n
    if not carried:
        return
    # a state that does not reach the next chunk, a gradient that does not reach the one before
    y2, h2 = forward(cut(c, lo, N, None, None))
    assert refused(y2[:, :32], y[:, lo:hi], r["out"][1][:, lo:hi], t) > 0.2
    back = dict(zip(names, ref.scan_bwd(*cut(c, 0, lo, c["init"], None))))
    for n in ("u", "dt", "Bm"):
        assert refused(back[n][:, -8:], grads[n][:, lo - 8:lo], r[n][1][:, lo - 8:lo], t) > 0.2, n


@pytest.mark.parametrize("B,H,W,D,K,ty,silu", [(4, 64, 96, 130, 3, "bf16", True), (2, 64, 64, 520, 4, "fp16", True),
                                               (3, 1, 4099, 515, 2, "fp16", False), (1, 20, 20, 256, 4, "bf16", True)])
def test_convolution_bounds(B, H, W, D, K, ty, silu):
    t, f, N = TYPES[ty], torch.float32, H * W
    c, _ = conv_inputs(B, H, W, D, K, t, True, True, CPU, seed=D)
    order = ref.scan_order(1, N, 0)
    a = (c["x"], c["w"], c["dy"], order, c["b"], silu, c["init"], c["df"])
    r = bounds.conv_bwd(*a)
    for (n, v, e), w in zip(r, ref.conv_bwd(*a)):
        assert torch.allclose(v, w, rtol=1e-9, atol=1e-12), n
        ty_ = f if n in ("w", "bias") else t
        assert refused(v, v, e, ty_) == 0, n
        assert refused(torch.zeros_like(v), v, e, ty_) > 0.9, n
    lo = N // 2
    one = ref.conv_bwd(c["x"][:1, lo:lo + 32], c["w"], c["dy"][:1, lo:lo + 32], ref.scan_order(1, 32, 0), c["b"], silu,
                       c["x"][:1, lo - (K - 1):lo], None)
    for (n, v, e), w in list(zip(r, one))[1:3]:
        assert refused(v - w, v, e, f) > 0.5, n


@pytest.mark.parametrize("B,N,C,G,ty,silu", [(2, 9000, 64, 2, "bf16", True), (1, 16384, 32, 1, "bf16", True),
                                             (1, 5000, 64, 64, "fp16", False), (3, 50, 33, 1, "bf16", False)])
def test_norm_bounds(B, N, C, G, ty, silu):
    t, f = TYPES[ty], torch.float32
    x, gamma, beta, dy = norm_inputs(B, N, C, t, True, 0.5, seed=N + C)
    stats = ref.norm_fwd(x, G, gamma, beta, 1e-5, silu)[1].float()
    r = bounds.norm_bwd(x, dy, stats, G, gamma, beta, silu)
    for (n, v, e), w in zip(r, ref.norm_bwd(x, dy, stats, G, gamma, beta, silu)):
        assert torch.allclose(v, w, rtol=1e-9, atol=1e-12), n
        ty_ = t if n == "x" else f
        assert refused(v, v, e, ty_) == 0, n
        assert refused(torch.zeros_like(v), v, e, ty_) > 0.9, n
    lo = N // 2
    one = ref.norm_bwd(x[:1, lo:lo + 32], dy[:1, lo:lo + 32], stats[:1], G, gamma, beta, silu)
    for (n, v, e), w in list(zip(r, one))[1:]:
        assert refused(v - w, v, e, f) > 0.9, n
