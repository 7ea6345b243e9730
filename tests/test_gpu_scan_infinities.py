"""Infinite values in the selective scan (GPU only): an infinity reaches exactly the outputs that the
formulas send it to, whatever the number of states and channels.  The kernels hold states in groups of
8, 16 or 32 and channels in blocks; the ones that are only there to fill a group must stay out of every
sum (their products with an infinity would be 0 times infinity, no number).

All values are positive, so that a sum meets infinities of one sign only and the 64-bit form is an
infinity, not NaN, wherever it is not finite in most of the outputs.  Finite values are compared with a
tolerance of one step of bfloat16 (2^-7 relative: the output's half step, and as much again), and float32
roundings of the terms that meet in a value: a state gathers at most 10 a step (the update 8, the exponent
8 |t A| <= 1), forward and back, so 2 x 10 x 158 x 2^-24 = 2e-4 < 2^-12 of the terms' magnitudes at 150
tokens.  (dt's gradient needs that: q u and the sum over w A, A < 0, are of opposite signs, and their
difference may be far below either.)
"""
import pytest
import torch

from recurrent_vision_backbone_b200 import gla, ssm
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
NAMES = ("u", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "init")


def inputs(B, N, D, S, seed):
    g = torch.Generator().manual_seed(seed)
    pos = lambda *s: torch.rand(s, generator=g) + 0.5  # noqa: E731
    return dict(u=pos(B, N, D).to(BF), dt=(pos(B, N, D) - 1).to(BF), A=-0.02 * pos(D, S), Bm=pos(B, N, S).to(BF),
                Cm=pos(B, N, S).to(BF), D=pos(D), z=pos(B, N, D).to(BF), dt_bias=pos(D) - 1, init=pos(B, D, S),
                dy=pos(B, N, D).to(BF), df=pos(B, D, S))


def same(got, want, mag, what):
    """Infinities and NaN in the same places, finite values within a step and mag's roundings."""
    got, want = got.double().cpu(), want.to(got.dtype).double()
    for name, f in (("NaN", torch.isnan), ("inf", torch.isposinf), ("-inf", torch.isneginf)):
        assert torch.equal(f(got), f(want)), f"{what}: {name} in {int(f(got).sum())} places, not {int(f(want).sum())}"
    fin = torch.isfinite(want)
    assert ((got - want).abs()[fin] <= 2.0 ** -7 * want.abs()[fin] + 2.0 ** -12 * mag[fin]).all(), what


def plant(c, what, p, d):
    inf = float("inf")
    if what == "u":
        c["u"][0, p, d] = inf
    elif what == "dt":
        c["dt"][0, p, d] = inf
    elif what == "product":              # each finite, their product past float32
        c["u"][0, p, d], c["dt"][0, p, d] = 1e30, 1e30
    elif what == "Bm":
        c["Bm"][0, p, -1] = inf
    elif what == "Cm":
        c["Cm"][0, p, -1] = inf
    elif what == "dy":
        c["dy"][0, p, d] = inf
    return c


# one walk with two lanes a channel and with one, chunks, a single token; states that fill their group and not
SHAPES = [(1, 37, 40, 5), (1, 37, 40, 16), (2, 150, 33, 12), (1, 40, 31, 20), (1, 9, 3, 1), (97, 5, 6, 11), (450, 3, 5, 5),
          (2, 1, 20, 11), (2, 1, 20, 16), (97, 9, 40, 12), (450, 5, 16, 24), (1, 70, 128, 4), (3, 50, 7, 8),
          (1, 150, 40, 3), (1, 90, 64, 1), (450, 3, 5, 2), (450, 4, 5, 4), (1, 200, 24, 13), (450, 3, 5, 30)]


@pytest.mark.parametrize("B,N,D,S", SHAPES)
@pytest.mark.parametrize("what", ["u", "dt", "product", "Bm", "Cm"])
def test_forward(B, N, D, S, what):
    c = plant(inputs(B, N, D, S, seed=N + S), what, N // 2, D // 2)
    d = {k: v.cuda() for k, v in c.items()}
    out, fin = ssm.gtr_ssm_scan_fwd(d["u"], d["dt"], d["A"], d["Bm"], d["Cm"], 1, N, 0, D=d["D"], z=d["z"],
                                    dt_bias=d["dt_bias"], init_state=d["init"], final_state=True)
    args = (c["u"], c["dt"], c["A"], c["Bm"], c["Cm"], ref.scan_order(1, N, 0), c["D"], c["z"], c["dt_bias"], True, c["init"])
    (y, h), (my, mh) = ref.scan_fwd(*args), ref.scan_fwd(*args, mag=True)
    same(out, y, my, "out")
    same(fin, h, mh, "final state")
    assert gla.device_status() == gla.GTR_OK   # bfloat16 carries it itself


@pytest.mark.parametrize("B,N,D,S", SHAPES)
@pytest.mark.parametrize("what", ["u", "dt", "Bm", "Cm", "dy"])
def test_backward(B, N, D, S, what):
    c = plant(inputs(B, N, D, S, seed=N + S), what, N // 2, D // 2)
    d = {k: v.cuda() for k, v in c.items()}
    got = ssm.gtr_ssm_scan_bwd(d["u"], d["dt"], d["A"], d["Bm"], d["Cm"], d["dy"], 1, N, 0, D=d["D"], z=d["z"],
                               dt_bias=d["dt_bias"], init_state=d["init"], d_final_state=d["df"])
    args = (c["u"], c["dt"], c["A"], c["Bm"], c["Cm"], c["dy"], ref.scan_order(1, N, 0), c["D"], c["z"], c["dt_bias"], True,
            c["init"], c["df"])
    for name, g, w, m in zip(NAMES, got, ref.scan_bwd(*args), ref.scan_bwd(*args, mag=True)):
        same(g, w, m, name)
