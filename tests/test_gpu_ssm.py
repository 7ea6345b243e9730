"""Short causal convolution and selective scan against their 64-bit forms (GPU only).

Bounds, from the arithmetic: an output rounded once to its type is off by at most half a step
(2^-11 fp16, 2^-8 bf16, relative; 2^-25 absolute below fp16's normal range), on top of the float32
error of what is rounded.  That error is counted in roundings of 2^-24 of the sum of the terms'
magnitudes (``mag``).  A step of the scan costs at most 8 (the update, the input's products, the
exponential's own 2 ulp) and, through the exponent t A, 8 for each unit of |t A| (t's softplus, the
product, its scaling), and a state gathers at most one such share a step.
"""
import pytest
import torch

from recurrent_vision_backbone_b200 import gla, ssm
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: ref.EPS32}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 1e-38, torch.float32: 1e-38}


def check(got, want, mag, k, what):
    """|got - want| within half a step of got's type and k float32 roundings of mag."""
    assert got.shape == want.shape, what
    h = HALF_STEP[got.dtype]
    slack = k * ref.EPS32 * mag
    bound = (want.abs() + slack) * h + TINY[got.dtype] + slack
    err = (got.double().cpu() - want).abs()
    bad = ~(err <= bound)
    if bad.any():
        i = int(torch.argmax(torch.nan_to_num(err - bound, nan=float("inf"))))
        raise AssertionError(f"{what}: {int(bad.sum())} of {err.numel()} outside; worst at {i}: got "
                             f"{got.reshape(-1)[i].item()!r}, want {want.reshape(-1)[i].item()!r}, bound "
                             f"{bound.reshape(-1)[i].item():.3e}")


def rnd(gen, *shape, std=1.0):
    return torch.randn(shape, generator=gen) * std


def strided(t, extra, at):
    """The same values as a slice of wider rows (as a projection's output is cut)."""
    B, N, C = t.shape
    wide = torch.full((B, N, C + extra), float("nan"), dtype=t.dtype, device=t.device)
    wide[..., at:at + C] = t
    return wide[..., at:at + C]


def guarded(shape, dtype, dev):
    """A tensor inside a larger buffer of a fixed pattern, and a check that the rest kept it."""
    n = 1
    for s in shape:
        n *= s
    pad = 1024
    buf = torch.full((n + 2 * pad,), 7.25, dtype=dtype, device=dev)
    t = buf[pad:pad + n].view(shape)
    t.fill_(float("nan"))

    def intact():
        return bool((buf[:pad] == 7.25).all()) and bool((buf[pad + n:] == 7.25).all())
    return t, intact


# ------------------------------------------------------------------ convolution
CONV = [
    # B, H, W, D, K, direction, type, bias, silu, state
    (1, 1, 1, 64, 4, 0, "fp16", True, True, True),      # a single token with its carried inputs
    (2, 1, 2, 40, 4, 1, "bf16", True, True, True),      # fewer tokens than the window
    (1, 1, 3, 8, 4, 0, "fp16", False, False, True),
    (3, 5, 7, 24, 3, 2, "fp16", True, True, False),
    (1, 20, 20, 256, 4, 3, "bf16", True, True, True),
    (2, 9, 31, 33, 4, 1, "fp16", True, True, True),     # odd channels
    (1, 40, 40, 1024, 4, 2, "fp16", True, True, False),
    (2, 37, 53, 70, 2, 3, "bf16", False, True, True),   # even channels, no whole 16 bytes
    (1, 1, 1000, 1, 3, 0, "bf16", True, False, False),  # one channel
    (1, 3, 67, 136, 2, 0, "fp16", True, True, True),
    (2, 64, 64, 520, 4, 1, "fp16", True, True, True),   # positions enough for the walk over chunks
    (4, 64, 96, 130, 3, 1, "bf16", True, True, True),   # the same by single elements
    (3, 1, 4099, 515, 2, 0, "fp16", False, False, True),
    (40, 5, 9, 384, 4, 3, "bf16", True, True, True),    # many short sequences
]


def conv_inputs(B, H, W, D, K, t, bias, state, dev, seed):
    g = torch.Generator().manual_seed(seed)
    N = H * W
    x, w = rnd(g, B, N, D).to(t), rnd(g, D, K, std=K ** -0.5)
    b = rnd(g, D, std=0.2) if bias else None
    init = rnd(g, B, K - 1, D).to(t) if state else None
    dy, df = rnd(g, B, N, D).to(t), rnd(g, B, K - 1, D).to(t) if state else None
    to = lambda v: None if v is None else v.to(dev)  # noqa: E731
    return dict(x=x, w=w, b=b, init=init, dy=dy, df=df), {k: to(v) for k, v in
                                                         dict(x=x, w=w, b=b, init=init, dy=dy, df=df).items()}


@pytest.mark.parametrize("B,H,W,D,K,direction,ty,bias,silu,state", CONV)
@pytest.mark.parametrize("extra", [0, 8, 3])
def test_conv_forward(B, H, W, D, K, direction, ty, bias, silu, state, extra):
    dev, t = torch.device("cuda", 0), TYPES[ty]
    c, d = conv_inputs(B, H, W, D, K, t, bias, state, dev, seed=H * 7 + D + K)
    order = ref.scan_order(H, W, direction)
    x = strided(d["x"], extra, 0 if extra == 8 else extra) if extra else d["x"]
    out, ok_o = guarded((B, H * W, D), t, dev)
    fin, ok_f = guarded((B, K - 1, D), t, dev)
    ssm.gtr_causal_conv_fwd(x, d["w"], H, W, direction, bias=d["b"], activation=int(silu), init_state=d["init"], out=out,
                            final_state=fin)
    assert gla.device_status() == gla.GTR_OK
    want, wf = ref.conv_fwd(c["x"], c["w"], order, c["b"], silu, c["init"])
    # K products and sums, and the activation's few roundings (its slope is at most 1.1)
    check(out, want, ref.conv_fwd(c["x"], c["w"], order, c["b"], silu, c["init"], mag=True), 2 * (K + 8), "out")
    assert torch.equal(fin.cpu().double(), wf)
    assert ok_o() and ok_f()


@pytest.mark.parametrize("B,H,W,D,K,direction,ty,bias,silu,state", CONV)
@pytest.mark.parametrize("extra", [0, 3])
def test_conv_backward(B, H, W, D, K, direction, ty, bias, silu, state, extra):
    dev, t = torch.device("cuda", 0), TYPES[ty]
    c, d = conv_inputs(B, H, W, D, K, t, bias, state, dev, seed=H * 5 + D + K)
    order = ref.scan_order(H, W, direction)
    x, dy = (strided(d["x"], extra, 1), strided(d["dy"], extra, 2)) if extra else (d["x"], d["dy"])
    shapes = [((B, H * W, D), t), ((D, K), torch.float32), ((D,), torch.float32), ((B, K - 1, D), t)]
    outs = [guarded(s, ty_, dev) for s, ty_ in shapes]
    ws, ok_w = guarded((max(ssm.causal_conv_bwd_workspace_bytes(B, H, W, D, K) // 4, 1),), torch.float32, dev)
    got = ssm.gtr_causal_conv_bwd(x, d["w"], dy, H, W, direction, bias=d["b"], activation=int(silu),
                                  init_state=d["init"], d_final_state=d["df"], workspace=ws,
                                  grads=tuple(o for o, _ in outs))
    assert gla.device_status() == gla.GTR_OK
    args = (c["x"], c["w"], c["dy"], order, c["b"], silu, c["init"], c["df"])
    want, mag = ref.conv_bwd(*args), ref.conv_bwd(*args, mag=True)
    n = B * H * W
    for name, g, w_, m, k in zip(("x", "w", "bias", "init"), got, want, mag,
                                 (4 * (K + 8), 4 * (K + 8) + n, 4 * (K + 8) + n, 4 * (K + 8))):
        check(g, w_, m, k, name)
    assert all(ok() for _, ok in outs) and ok_w()


def test_conv_carried_state_equals_one_run():
    """Token by token with the state carried in place, against one run over the sequence."""
    dev = torch.device("cuda", 0)
    _, d = conv_inputs(3, 1, 11, 48, 4, torch.bfloat16, True, True, dev, seed=3)
    whole, wf = ssm.gtr_causal_conv_fwd(d["x"], d["w"], 1, 11, 0, bias=d["b"], init_state=d["init"], final_state=True)
    st = d["init"].clone()
    for lo, hi in ((0, 1), (1, 2), (2, 7), (7, 8), (8, 11)):
        y, _ = ssm.gtr_causal_conv_fwd(d["x"][:, lo:hi].contiguous(), d["w"], 1, hi - lo, 0, bias=d["b"], init_state=st,
                                       final_state=st)
        assert torch.equal(y, whole[:, lo:hi])
    assert torch.equal(st, wf)


@pytest.mark.parametrize("B,N,D", [(3, 2, 48), (40, 64, 2048), (700, 2, 256), (400, 33, 257)])
def test_conv_state_carried_in_place(B, N, D):
    """final_state = init_state gives what two tensors give, bit for bit, directly and by chunks."""
    dev = torch.device("cuda", 0)
    _, d = conv_inputs(B, 1, N, D, 4, torch.float16, True, True, dev, seed=D)
    out, fin = ssm.gtr_causal_conv_fwd(d["x"], d["w"], 1, N, 0, bias=d["b"], init_state=d["init"], final_state=True)
    st = d["init"].clone()
    got, _ = ssm.gtr_causal_conv_fwd(d["x"], d["w"], 1, N, 0, bias=d["b"], init_state=st, final_state=st)
    assert torch.equal(got, out) and torch.equal(st, fin)
    assert torch.equal(fin, torch.cat((d["init"], d["x"]), 1)[:, N:])


# ------------------------------------------------------------------ selective scan
def scan_inputs(B, H, W, D, S, t, dev, seed, gate=True, skip=True, bias=True, state=True, decay=1.0):
    g = torch.Generator().manual_seed(seed)
    N = H * W
    c = dict(u=rnd(g, B, N, D).to(t), dt=rnd(g, B, N, D, std=0.5).to(t), A=-decay * torch.exp(rnd(g, D, S, std=0.4)),
             Bm=rnd(g, B, N, S).to(t), Cm=rnd(g, B, N, S).to(t), D=rnd(g, D) if skip else None,
             z=rnd(g, B, N, D).to(t) if gate else None, dt_bias=rnd(g, D) - 1 if bias else None,
             init=rnd(g, B, D, S) if state else None, dy=rnd(g, B, N, D).to(t), df=rnd(g, B, D, S) if state else None)
    return c, {k: None if v is None else v.to(dev) for k, v in c.items()}


def exponent(c, softplus=True):
    raw = c["dt"].double() + (0 if c["dt_bias"] is None else c["dt_bias"].double())
    t = torch.nn.functional.softplus(raw) if softplus else raw
    return float((t.abs().amax((0, 1))[:, None] * c["A"].double().abs()).max())


SCAN = [
    # B, H, W, D, S, direction, type, gate, skip, bias, softplus, state, decay
    (1, 1, 1, 64, 16, 0, "fp16", True, True, True, True, True, 1.0),      # single tokens
    (5, 1, 1, 37, 8, 2, "bf16", True, True, True, True, True, 1.0),
    (3, 1, 1, 40, 4, 0, "fp16", False, False, False, True, False, 1.0),
    (2, 1, 1, 33, 32, 1, "bf16", True, True, True, False, True, 1.0),
    (2, 1, 1, 20, 11, 0, "fp16", True, True, True, True, True, 1.0),      # states that fill no lane
    (1, 1, 2, 1, 1, 0, "fp16", True, True, True, True, True, 1.0),        # one channel, one state
    (2, 1, 9, 3, 5, 1, "bf16", True, False, True, True, True, 1.0),
    (1, 5, 13, 64, 16, 2, "fp16", True, True, True, True, False, 1.0),
    (2, 7, 11, 129, 16, 3, "bf16", False, True, True, True, True, 1.0),   # a channel more than a block
    (1, 1, 64, 128, 16, 0, "fp16", True, True, True, True, True, 1.0),
    (1, 1, 65, 128, 16, 0, "fp16", True, True, True, True, True, 1.0),    # a token more than a chunk
    (1, 16, 16, 70, 32, 1, "fp16", True, True, True, True, True, 1.0),
    (2, 12, 25, 48, 20, 3, "bf16", True, True, False, True, True, 1.0),
    (1, 20, 20, 40, 8, 2, "fp16", True, True, True, True, True, 1.0),
    (1, 17, 19, 31, 7, 0, "bf16", True, True, True, False, True, 0.3),    # time steps of either sign
    (2, 6, 50, 96, 16, 1, "fp16", True, True, True, True, True, 40.0),    # decays down to nothing
    (1, 17, 19, 31, 7, 0, "bf16", True, True, False, False, True, 0.02),  # of either sign, within float32
]
SCAN += [
    # channels enough for one walk over whole sequences, two lanes a channel, then one
    (100, 2, 9, 40, 16, 1, "fp16", True, True, True, True, True, 1.0),
    (49, 3, 11, 136, 8, 2, "bf16", True, True, True, True, True, 1.0),
    (97, 1, 20, 33, 32, 0, "fp16", False, True, True, True, True, 1.0),
    (450, 1, 5, 24, 16, 3, "bf16", True, True, True, True, True, 1.0),
    (446, 1, 17, 9, 5, 0, "fp16", True, False, True, True, False, 1.0),
    # chunks enough for the backward's longer ones
    (100, 10, 10, 200, 16, 2, "fp16", True, True, True, True, True, 1.0),
    # many single tokens: as many sequences a thread as lanes share a channel
    (301, 1, 1, 1027, 4, 0, "fp16", True, True, True, True, True, 1.0),
    (301, 1, 1, 1027, 8, 0, "bf16", True, True, True, True, True, 1.0),
    (301, 1, 1, 1027, 16, 0, "fp16", False, True, True, True, False, 1.0),
    (301, 1, 1, 1027, 32, 0, "fp16", True, True, True, True, True, 1.0),
]
# A state that grows past float32 has no float32 value, and neither has what follows from it (an
# infinity times a decay, or less another, is no number): from the first position of a channel
# whose terms pass this size there is nothing to compare with.  (The first case of either sign
# reaches 1e111 by its last tokens.)
NO_VALUE = 1e30


@pytest.mark.parametrize("case", SCAN)
@pytest.mark.parametrize("extra", [0, 5])
def test_scan_forward(case, extra):
    B, H, W, D, S, direction, ty, gate, skip, bias, softplus, state, decay = case
    dev, t = torch.device("cuda", 0), TYPES[ty]
    c, d = scan_inputs(B, H, W, D, S, t, dev, seed=H * 3 + D + S, gate=gate, skip=skip, bias=bias, state=state, decay=decay)
    order, N = ref.scan_order(H, W, direction), H * W
    if extra:
        for i, n in enumerate(("u", "dt", "Bm", "Cm", "z")):
            if d[n] is not None:
                d[n] = strided(d[n], extra, i)
    out, ok_o = guarded((B, N, D), t, dev)
    fin, ok_f = guarded((B, D, S), torch.float32, dev)
    need = ssm.ssm_scan_fwd_workspace_bytes(B, H, W, D, S)
    ws, ok_w = guarded((max(need // 4, 1),), torch.float32, dev)
    ssm.gtr_ssm_scan_fwd(d["u"], d["dt"], d["A"], d["Bm"], d["Cm"], H, W, direction, D=d["D"], z=d["z"],
                         dt_bias=d["dt_bias"], dt_softplus=softplus, init_state=d["init"], out=out, final_state=fin,
                         workspace=ws)
    assert gla.device_status() == gla.GTR_OK
    args = (c["u"], c["dt"], c["A"], c["Bm"], c["Cm"], order, c["D"], c["z"], c["dt_bias"], softplus, c["init"])
    (y, h), (my, mh) = ref.scan_fwd(*args), ref.scan_fwd(*args, mag=True)
    k = (8 + 8 * exponent(c, softplus)) * (N + 8) + S
    gone = ref.to_grid(my[:, order].cummax(1)[0] > NO_VALUE, order)
    keep = lambda v: v.masked_fill(gone, 0)  # noqa: E731
    check(keep(out.cpu()), keep(y), keep(my), k, "out")
    last = gone[:, order[-1]][..., None].expand_as(h)
    check(fin.cpu().masked_fill(last, 0), h.masked_fill(last, 0), mh.masked_fill(last, 0), k, "final state")
    assert ok_o() and ok_f() and ok_w()


@pytest.mark.parametrize("case", SCAN)
@pytest.mark.parametrize("extra", [0, 5])
def test_scan_backward(case, extra):
    B, H, W, D, S, direction, ty, gate, skip, bias, softplus, state, decay = case
    dev, t = torch.device("cuda", 0), TYPES[ty]
    c, d = scan_inputs(B, H, W, D, S, t, dev, seed=H * 3 + D + S, gate=gate, skip=skip, bias=bias, state=state, decay=decay)
    order, N = ref.scan_order(H, W, direction), H * W
    if extra:
        for i, n in enumerate(("u", "dt", "Bm", "Cm", "z", "dy")):
            if d[n] is not None:
                d[n] = strided(d[n], extra, i % 5)
    f = torch.float32
    shapes = [((B, N, D), t), ((B, N, D), t), ((D, S), f), ((B, N, S), t), ((B, N, S), t), ((D,), f),
              ((B, N, D), t) if gate else None, ((D,), f), ((B, D, S), f)]
    outs = [None if s is None else guarded(s[0], s[1], dev) for s in shapes]
    ws, ok_w = guarded((ssm.ssm_scan_bwd_workspace_bytes(B, H, W, D, S) // 4,), f, dev)
    got = ssm.gtr_ssm_scan_bwd(d["u"], d["dt"], d["A"], d["Bm"], d["Cm"], d["dy"], H, W, direction, D=d["D"], z=d["z"],
                               dt_bias=d["dt_bias"], dt_softplus=softplus, init_state=d["init"], d_final_state=d["df"],
                               workspace=ws, grads=tuple(None if o is None else o[0] for o in outs))
    assert gla.device_status() == gla.GTR_OK
    args = (c["u"], c["dt"], c["A"], c["Bm"], c["Cm"], c["dy"], order, c["D"], c["z"], c["dt_bias"], softplus, c["init"],
            c["df"])
    want, mag = ref.scan_bwd(*args), ref.scan_bwd(*args, mag=True)
    # a state and a gradient of a state, and the sums over tokens, states and channels
    k = 2 * (8 + 8 * exponent(c, softplus)) * (N + 8) + B * N + S + D
    grows = any(float(m.max()) > NO_VALUE for m in mag if m is not None)   # sums over channels and tokens share it
    for name, g, w_, m in zip(("u", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "init"), got, want, mag):
        if g is not None and not grows:
            check(g, w_, m, k, name)
    assert all(o is None or o[1]() for o in outs) and ok_w()


def run_scan(d, H, W, direction, **kw):
    return ssm.gtr_ssm_scan_fwd(d["u"], d["dt"], d["A"], d["Bm"], d["Cm"], H, W, direction, D=d["D"], z=d["z"],
                                dt_bias=d["dt_bias"], **kw)


def run_scan_bwd(d, H, W, direction, **kw):
    return ssm.gtr_ssm_scan_bwd(d["u"], d["dt"], d["A"], d["Bm"], d["Cm"], d["dy"], H, W, direction, D=d["D"], z=d["z"],
                                dt_bias=d["dt_bias"], init_state=d["init"], d_final_state=d["df"], **kw)


def test_scan_long_sequence_with_few_channels():
    """16384 tokens cut into many chunks, the state carried over all of them (A small), against the
    64-bit form on the GPU."""
    dev = torch.device("cuda", 0)
    c, d = scan_inputs(1, 128, 128, 40, 16, torch.float16, dev, seed=9, decay=0.02)
    assert ssm.ssm_scan_fwd_workspace_bytes(1, 128, 128, 40, 16) > 0
    out, fin = run_scan(d, 128, 128, 3, init_state=d["init"], final_state=True)
    assert gla.device_status() == gla.GTR_OK
    args = (d["u"], d["dt"], d["A"], d["Bm"], d["Cm"], ref.scan_order(128, 128, 3, dev), d["D"], d["z"], d["dt_bias"],
            True, d["init"])
    (y, h), (my, mh) = ref.scan_fwd(*args), ref.scan_fwd(*args, mag=True)
    # the decays forget: a state gathers the shares of the last 1 / (1 - a) steps or so, a < 1 - 0.0003 here
    k = (8 + 8 * exponent(c)) * 3500
    check(out, y.cpu(), my.cpu(), k, "out")
    check(fin, h.cpu(), mh.cpu(), k, "final state")


def test_scan_backward_of_a_long_sequence():
    """5000 tokens in 157 chunks: the folds run over several batches of them."""
    dev, N = torch.device("cuda", 0), 5000
    c, d = scan_inputs(1, 50, 100, 12, 16, torch.bfloat16, dev, seed=19, decay=0.05)
    got = run_scan_bwd(d, 50, 100, 1)
    assert gla.device_status() == gla.GTR_OK
    args = (d["u"], d["dt"], d["A"], d["Bm"], d["Cm"], d["dy"], ref.scan_order(50, 100, 1, dev), d["D"], d["z"],
            d["dt_bias"], True, d["init"], d["df"])
    want, mag = ref.scan_bwd(*args), ref.scan_bwd(*args, mag=True)
    k = 2 * (8 + 8 * exponent(c)) * (N + 8) + N + 28
    for name, g, w_, m in zip(("u", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "init"), got, want, mag):
        check(g, w_.cpu(), m.cpu(), k, name)


@pytest.mark.parametrize("B,N", [(2, 1), (2, 7), (2, 200), (110, 30), (460, 9), (310, 1)])
def test_scan_state_carried_in_place(B, N):
    """final_state = init_state gives what two tensors give, bit for bit."""
    dev = torch.device("cuda", 0)
    _, d = scan_inputs(B, 1, N, 96 if B < 300 else 1000 if N == 1 else 40, 16, torch.bfloat16, dev, seed=N)
    out, fin = run_scan(d, 1, N, 0, init_state=d["init"], final_state=True)
    st = d["init"].clone()
    out2, _ = run_scan(d, 1, N, 0, init_state=st, final_state=st)
    assert torch.equal(out, out2) and torch.equal(st, fin)


@pytest.mark.parametrize("S", [16, 12])
def test_scan_prompt_then_single_tokens(S):
    """A prompt, then tokens one by one with the carried state, against one run over them all."""
    dev, N, tail = torch.device("cuda", 0), 150, 6
    c, d = scan_inputs(2, 1, N, 72, S, torch.float16, dev, seed=4)
    args = (c["u"], c["dt"], c["A"], c["Bm"], c["Cm"], ref.scan_order(1, N, 0), c["D"], c["z"], c["dt_bias"], True, c["init"])
    (y, h), (my, mh) = ref.scan_fwd(*args), ref.scan_fwd(*args, mag=True)
    k = (8 + 8 * exponent(c)) * (N + 8) + S
    cut = lambda lo, hi: {n: v if v is None or v.dim() != 3 or v.shape[1] != N else v[:, lo:hi].contiguous()  # noqa: E731
                          for n, v in d.items()}
    out, st = run_scan(cut(0, N - tail), 1, N - tail, 0, init_state=d["init"], final_state=True)
    outs = [out]
    for p in range(N - tail, N):
        o, _ = run_scan(cut(p, p + 1), 1, 1, 0, init_state=st, final_state=st)
        outs.append(o)
    check(torch.cat(outs, 1), y, my, k, "out")
    check(st, h, mh, k, "final state")


def test_scan_directions_are_the_reordered_sequence():
    """A grid scan equals the L2R scan of the tokens put in scan order, bit for bit."""
    dev, H, W = torch.device("cuda", 0), 13, 22
    _, d = scan_inputs(2, H, W, 64, 16, torch.float16, dev, seed=8)
    for direction in range(4):
        o = ref.scan_order(H, W, direction, dev)
        seq = {n: v[:, o].contiguous() if v is not None and v.dim() == 3 and v.shape[1] == H * W else v
               for n, v in d.items()}
        y, h = run_scan(d, H, W, direction, final_state=True)
        ys, hs = run_scan(seq, 1, H * W, 0, final_state=True)
        assert torch.equal(y[:, o], ys) and torch.equal(h, hs)
        g, gs = run_scan_bwd(d, H, W, direction), run_scan_bwd(seq, 1, H * W, 0)
        for a, b in zip(g, gs):
            tok = a.dim() == 3 and a.shape[1] == H * W
            assert torch.equal(a[:, o] if tok else a, b)


def test_equal_calls_give_equal_bits():
    dev = torch.device("cuda", 0)
    _, d = scan_inputs(2, 20, 30, 200, 16, torch.bfloat16, dev, seed=6)
    a, b = run_scan_bwd(d, 20, 30, 1), run_scan_bwd(d, 20, 30, 1)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    _, e = conv_inputs(2, 20, 30, 200, 4, torch.bfloat16, True, True, dev, seed=6)
    f = lambda: ssm.gtr_causal_conv_bwd(e["x"], e["w"], e["dy"], 20, 30, 1, bias=e["b"], init_state=e["init"])  # noqa: E731
    assert all(torch.equal(x, y) for x, y in zip(f(), f()))


def test_decays_of_zero_and_infinite_rates():
    """A = -inf forgets at every step: out = (C . B t u + D u) silu(z); nothing turns into NaN, in
    whole chunks and in the last, ragged one."""
    dev, N = torch.device("cuda", 0), 83
    c, d = scan_inputs(1, 1, N, 40, 16, torch.float16, dev, seed=12)
    d["A"].fill_(float("-inf"))
    out, fin = run_scan(d, 1, N, 0, init_state=d["init"], final_state=True)
    raw = c["dt"].double() + c["dt_bias"].double()
    x = torch.nn.functional.softplus(raw, threshold=60) * c["u"].double()
    h = x[..., None] * c["Bm"].double()[:, :, None]
    z = c["z"].double()
    y = ((h * c["Cm"].double()[:, :, None]).sum(-1) + c["D"].double() * c["u"].double()) * z * torch.sigmoid(z)
    mag = ((h * c["Cm"].double()[:, :, None]).abs().sum(-1) + (c["D"].double() * c["u"].double()).abs()) * (z * torch.sigmoid(z)).abs()
    check(out, y, mag, 64, "out")
    check(fin, h[:, -1], h[:, -1].abs(), 32, "final state")


def test_fp16_overflow_is_reported():
    dev = torch.device("cuda", 0)
    _, d = scan_inputs(1, 1, 40, 16, 8, torch.float16, dev, seed=2)
    d["u"].fill_(1000.0), d["D"].fill_(1000.0), d["z"].fill_(10.0)
    run_scan(d, 1, 40, 0)
    assert gla.device_status() == gla.GTR_ERR_RANGE
    assert gla.device_status() == gla.GTR_OK
    one = {n: v[:, :1].contiguous() if v is not None and v.dim() == 3 and v.shape[1] == 40 else v for n, v in d.items()}
    run_scan(one, 1, 1, 0)
    assert gla.device_status() == gla.GTR_ERR_RANGE
    _, e = conv_inputs(1, 1, 9, 16, 4, torch.float16, True, False, dev, seed=2)
    e["x"].fill_(60000.0), e["w"].fill_(1.0)
    ssm.gtr_causal_conv_fwd(e["x"], e["w"], 1, 9, 0)
    assert gla.device_status() == gla.GTR_ERR_RANGE
    e["x"].fill_(float("nan"))
    ssm.gtr_causal_conv_fwd(e["x"], e["w"], 1, 9, 0)
    assert gla.device_status() == gla.GTR_ERR_RANGE
    assert gla.device_status() == gla.GTR_OK


def test_empty_grids():
    dev = torch.device("cuda", 0)
    _, d = scan_inputs(2, 0, 5, 24, 8, torch.float16, dev, seed=2)
    out, fin = run_scan(d, 0, 5, 0, init_state=d["init"], final_state=True)
    assert out.shape == (2, 0, 24) and torch.equal(fin, d["init"])
    _, fin = run_scan(d, 0, 5, 0, final_state=True)
    assert not fin.any()
    g = run_scan_bwd(d, 0, 5, 0)
    assert torch.equal(g[8], d["df"]) and not g[2].any() and not g[5].any() and not g[7].any()
    _, e = conv_inputs(2, 0, 5, 24, 4, torch.float16, True, True, dev, seed=2)
    _, fin = ssm.gtr_causal_conv_fwd(e["x"], e["w"], 0, 5, 0, bias=e["b"], init_state=e["init"], final_state=True)
    assert torch.equal(fin, e["init"])
    g = ssm.gtr_causal_conv_bwd(e["x"], e["w"], e["dy"], 0, 5, 0, bias=e["b"], init_state=e["init"], d_final_state=e["df"])
    assert not g[1].any() and not g[2].any() and torch.equal(g[3], e["df"])


def test_captured_calls_replay_on_new_inputs():
    """Convolution, scan and their gradients recorded once in a graph, replayed on other inputs, and
    two graphs that share nothing replayed on two streams at once."""
    dev, H, W, D, S = torch.device("cuda", 0), 9, 33, 136, 16
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs, states, outs = [], [], []
    for i in range(2):
        _, d = scan_inputs(1, H, W, D, S, torch.float16, dev, seed=30 + i)
        _, e = conv_inputs(1, H, W, D, 4, torch.float16, True, False, dev, seed=40 + i)

        def run(d=d, e=e):
            u, _ = ssm.gtr_causal_conv_fwd(e["x"], e["w"], H, W, 2, bias=e["b"])
            dd = dict(d, u=u)
            y, h = run_scan(dd, H, W, 2, init_state=d["init"], final_state=True)
            g = run_scan_bwd(dd, H, W, 2)
            gc = ssm.gtr_causal_conv_bwd(e["x"], e["w"], g[0], H, W, 2, bias=e["b"])
            return (u, y, h) + g + gc[:3]
        with torch.cuda.stream(side[i]):
            run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side[i]):
            o = run()
        graphs.append(graph), states.append((d, e, run)), outs.append(o)
    for seed in (60, 61):
        for i, (d, e, _) in enumerate(states):
            _, nd = scan_inputs(1, H, W, D, S, torch.float16, dev, seed=seed + 10 * i)
            _, ne = conv_inputs(1, H, W, D, 4, torch.float16, True, False, dev, seed=seed + 20 * i)
            for old, new in ((d, nd), (e, ne)):
                for n, v in old.items():
                    if v is not None:
                        v.copy_(new[n])
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(side[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for (d, e, run), o in zip(states, outs):
            for a, b in zip(run(), o):
                assert (a is None and b is None) or torch.equal(a, b)
    assert gla.device_status() == gla.GTR_OK


def test_another_stream_than_the_current_one():
    """The stream argument: outputs and workspaces allocated by the call are safe on it."""
    dev = torch.device("cuda", 0)
    _, d = scan_inputs(1, 20, 40, 128, 16, torch.float16, dev, seed=5)
    want = run_scan(d, 20, 40, 0)[0]
    gw = run_scan_bwd(d, 20, 40, 0)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    junk = [torch.full((1 << 20,), float("nan"), device=dev) for _ in range(4)]
    del junk
    got = run_scan(d, 20, 40, 0, stream=s)[0]
    gg = run_scan_bwd(d, 20, 40, 0, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(gg, gw))


def off_grid(t):
    """The same values two bytes further on than the allocator's boundaries."""
    return torch.cat((t.new_zeros(1), t.reshape(-1)))[1:].view(t.shape)


@pytest.mark.parametrize("N", [1, 90, 700])
def test_each_tensor_off_the_16_byte_grid(N):
    """Rows of whole 16-byte pieces whose tensors start two bytes off, one tensor at a time: the
    results are those of aligned tensors, bit for bit."""
    dev, D = torch.device("cuda", 0), 128
    _, d = scan_inputs(2, 1, N, D, 16, torch.float16, dev, seed=N)
    want, wf = run_scan(d, 1, N, 0, init_state=d["init"], final_state=True)
    wg = run_scan_bwd(d, 1, N, 0)
    for name in ("u", "dt", "Bm", "Cm", "z", "dy", "out"):
        o = dict(d, **{name: off_grid(d[name])}) if name != "out" else d
        out = off_grid(torch.empty_like(want)) if name == "out" else None
        got, gf = run_scan(o, 1, N, 0, init_state=d["init"], final_state=True, out=out)
        assert torch.equal(got, want) and torch.equal(gf, wf), name
        grads = tuple(off_grid(torch.empty_like(g)) if name == "out" and g.dtype == torch.float16 else torch.empty_like(g)
                      for g in wg)
        for a, b in zip(run_scan_bwd(o, 1, N, 0, grads=grads), wg):
            assert torch.equal(a, b), name
    _, e = conv_inputs(2, 1, N, D, 4, torch.float16, True, True, dev, seed=N)
    conv = lambda e, **kw: ssm.gtr_causal_conv_fwd(e["x"], e["w"], 1, N, 0, bias=e["b"], init_state=e["init"], **kw)  # noqa: E731
    back = lambda e, **kw: ssm.gtr_causal_conv_bwd(e["x"], e["w"], e["dy"], 1, N, 0, bias=e["b"], init_state=e["init"],  # noqa: E731
                                                   d_final_state=e["df"], **kw)
    want, wf = conv(e, final_state=True)
    wg = back(e)
    for name in ("x", "init", "dy", "df", "out", "fin"):
        o = dict(e, **{name: off_grid(e[name])}) if name in e else e
        got, gf = conv(o, out=off_grid(torch.empty_like(want)) if name == "out" else None,
                       final_state=off_grid(torch.empty_like(wf)) if name == "fin" else True)
        assert torch.equal(got, want) and torch.equal(gf, wf), name
        grads = tuple(off_grid(torch.empty_like(g)) if name == "out" and g.dtype == torch.float16 else torch.empty_like(g)
                      for g in wg)
        for a, b in zip(back(o, grads=grads), wg):
            assert torch.equal(a, b), name
    assert gla.device_status() == gla.GTR_OK


def test_calls_at_the_same_time_on_two_streams():
    dev = torch.device("cuda", 0)
    ds = [scan_inputs(1, 20, 50, 96, 16, torch.bfloat16, dev, seed=s)[1] for s in (1, 2)]
    want = [(run_scan(d, 20, 50, 2), run_scan_bwd(d, 20, 50, 2)) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        for d, s in zip(ds, streams):
            with torch.cuda.stream(s):
                got.append((run_scan(d, 20, 50, 2), run_scan_bwd(d, 20, 50, 2)))
    torch.cuda.synchronize()
    for i, (f, g) in enumerate(got):
        wf, wg = want[i % 2]
        assert torch.equal(f[0], wf[0]) and all(torch.equal(a, b) for a, b in zip(g, wg))


def test_channels_past_32_bit_offsets():
    """Rows more than 2^31 elements into a tensor (a slice of very wide rows)."""
    dev, N, D = torch.device("cuda", 0), 40, 64
    ld = (1 << 31) // (N - 4)
    _, d = scan_inputs(1, 1, N, D, 16, torch.float16, dev, seed=7)
    want, wf = run_scan(d, 1, N, 0, init_state=d["init"], final_state=True)
    wide = torch.empty(N * ld, dtype=torch.float16, device=dev)
    u = wide.as_strided((1, N, D), (N * ld, ld, 1))
    u.copy_(d["u"])
    got, gf = run_scan(dict(d, u=u), 1, N, 0, init_state=d["init"], final_state=True)
    assert torch.equal(got, want) and torch.equal(gf, wf)
    _, e = conv_inputs(1, 1, N, D, 4, torch.float16, True, False, dev, seed=7)
    cw, _ = ssm.gtr_causal_conv_fwd(e["x"], e["w"], 1, N, 0)
    u.copy_(e["x"])
    cg, _ = ssm.gtr_causal_conv_fwd(u, e["w"], 1, N, 0)
    assert torch.equal(cg, cw)


def test_binding_refusals():
    dev = torch.device("cuda", 0)
    _, d = scan_inputs(1, 4, 4, 16, 8, torch.float16, dev, seed=1)
    a = (d["u"], d["dt"], d["A"], d["Bm"], d["Cm"])
    for bad in ((d["u"].float(),) + a[1:], (d["u"].bfloat16(),) + a[1:], a[:2] + (d["A"].half(),) + a[3:],
                a[:3] + (d["Bm"][..., :7],) + a[4:], (d["u"].transpose(1, 2).contiguous().transpose(1, 2),) + a[1:],
                (d["u"][:, :8],) + a[1:]):
        with pytest.raises(ValueError):
            ssm.gtr_ssm_scan_fwd(*bad, 4, 4, 0)
    with pytest.raises(ValueError):
        ssm.gtr_ssm_scan_fwd(*a, 4, 5, 0)
    for kw in (dict(out=d["u"]), dict(out=d["dt"])):
        with pytest.raises(gla.GTRError) as err:
            ssm.gtr_ssm_scan_fwd(*a, 4, 4, 0, **kw)
        assert err.value.status == gla.GTR_ERR_INVALID_ARG
    with pytest.raises(gla.GTRError) as err:
        ssm.gtr_ssm_scan_fwd(d["u"], d["dt"], torch.zeros(16, 33, device=dev), torch.zeros(1, 16, 33, device=dev).half(),
                             torch.zeros(1, 16, 33, device=dev).half(), 4, 4, 0)
    assert err.value.status == gla.GTR_ERR_UNSUPPORTED
    with pytest.raises(gla.GTRError) as err:
        ssm.gtr_causal_conv_fwd(d["u"], torch.zeros(16, 5, device=dev), 4, 4, 0)
    assert err.value.status == gla.GTR_ERR_UNSUPPORTED
    with pytest.raises(gla.GTRError) as err:
        ssm.gtr_causal_conv_fwd(d["u"], torch.zeros(16, 4, device=dev), 4, 4, 0, out=d["u"])
    assert err.value.status == gla.GTR_ERR_INVALID_ARG
    assert gla.device_status() == gla.GTR_OK
