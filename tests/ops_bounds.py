"""How far float32 arithmetic may take the operators' results from their 64-bit forms, element by element.

Each function returns the 64-bit results with a bound for each, by a forward error analysis along the
formulas: every rounding of a product or a sum is at most EPS32 = 2^-24 of its result, an exponential's
is 2 ulp (4 EPS32), a reciprocal's 1 ulp (2 EPS32), the exponent of 2^(t A log2 e) is off by 3 EPS32
relative (log2 e, A log2 e, the product) besides t's own error, and a sum's error grows with the length
of its longest chain, not with the number of its terms.  An error of a state passes on to the next
with the state, so it is forgotten as the state is.  The whole is doubled for what is formed twice or
joined otherwise than step by step: states by chunks (the exponent of a chunk's summed time steps),
decays multiplied up.

`check` makes the comparison, `outside` says where it fails.
"""
import torch

from tests.ops_reference import EPS32 as U
from tests.ops_reference import conv_rows, silu_grad, to_grid

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: U, torch.float64: U}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 1e-38, torch.float32: 1e-37, torch.float64: 1e-37}


def outside(got, want, err, dtype=None):
    """Where got is further from want than err and the rounding to its type (half a step)."""
    t = dtype or got.dtype
    return ~((got.double().cpu() - want).abs() <= err + (want.abs() + err) * HALF_STEP[t] + TINY[t])


def check(got, want, err, what):
    bad = outside(got, want, err)
    if bad.any():
        far = (got.double().cpu() - want).abs() - err
        i = int(torch.argmax(torch.nan_to_num(far, nan=float("inf"))))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst at {i}: got "
                             f"{got.reshape(-1)[i].item()!r}, want {want.reshape(-1)[i].item()!r}, err {err.reshape(-1)[i].item():.3e}")


def sigmoid(z):
    """sigmoid and its error (exponential and reciprocal; relative accuracy on both sides)."""
    s = torch.sigmoid(z)
    return s, U * s * ((1 - s) * (2 * z.abs() + 4) + 3)


def silu(z):
    s, es = sigmoid(z)
    return z * s, z.abs() * es + U * (z * s).abs()


def silu_slope(z):
    """silu'(z) = s (1 + z (1 - s)) and its error: s's, 1 - s's times z, four roundings."""
    s, es = sigmoid(z)
    one = 1 + z * (1 - s)
    return s * one, es * one.abs() + s * (z.abs() * (es + U) + 2 * U * (1 + z.abs())) + 2 * U * (s * one).abs()


# ------------------------------------------------------------------ selective scan
def _time_step(dt, dt_bias, softplus):
    """raw, its error, t, t's error, dt/draw and that one's error."""
    raw = dt.double() + (0 if dt_bias is None else dt_bias.double())
    er = U * raw.abs()
    if not softplus:
        return raw, raw, er, torch.ones_like(raw), torch.zeros_like(raw)
    t, e, s = torch.logaddexp(raw, torch.zeros_like(raw)), torch.exp(-raw.abs()), torch.sigmoid(raw)
    et = s * er + U * e * (2 * raw.abs() + 4) + 4 * U * t       # the polynomial, its product, the sum
    es = s * U * ((2 * raw.abs() + 4) * torch.where(raw < 0, torch.ones_like(s), 1 - s) + raw.abs() * (1 - s) + 4)
    return raw, t, et, s, es


def scan(u, dt, A, Bm, Cm, order, D=None, z=None, dt_bias=None, softplus=True, init=None, dy=None, dfinal=None, chain=None):
    """[(name, value, error)]: out and final state, and with dy the gradients in their order.  chain: the
    longest chain of a sum over tokens (see chain_of_scan)."""
    u, Bm, Cm = (v.double()[:, order] for v in (u, Bm, Cm))
    raw, t, et, sg, esg = _time_step(dt[:, order], dt_bias, softplus)
    A = A.double()
    B, N, C = u.shape
    S = A.shape[1]
    h = u.new_zeros(B, C, S) if init is None else init.double()
    eh = torch.zeros_like(h)
    Dk = u.new_zeros(C) if D is None else D.double()
    gate, egate = (torch.ones_like(u), torch.zeros_like(u)) if z is None else silu(z.double()[:, order])
    x, ex = t * u, u.abs() * et + U * (t * u).abs()

    def decay(p):
        m = t[:, p, :, None] * A
        a = torch.exp(m)
        return a, a * (et[:, p, :, None] * A.abs() + U * (3 * m.abs() + 4)) + 2.0 ** -125
    hs, ehs, ys, eys = [h], [eh], [], []
    for p in range(N):
        a, ea = decay(p)
        xb = x[:, p, :, None] * Bm[:, p, None]
        eh = a * eh + h.abs() * ea + ex[:, p, :, None] * Bm[:, p, None].abs() + U * xb.abs()
        h = a * h + xb
        eh = eh + U * h.abs()
        hs.append(h), ehs.append(eh)
        ch = h * Cm[:, p, None]
        ys.append(ch.sum(-1) + Dk * u[:, p])
        eys.append((Cm[:, p, None].abs() * eh).sum(-1) + (S + 3) * U * (ch.abs().sum(-1) + (Dk * u[:, p]).abs()))
    y, ey = torch.stack(ys, 1), torch.stack(eys, 1)
    o = lambda v: to_grid(v, order)  # noqa: E731
    out = [("out", o(y * gate), 2 * o(gate.abs() * ey + y.abs() * egate + U * (y * gate).abs())), ("final state", h, 2 * eh)]
    if dy is None:
        return out
    dy = dy.double()[:, order]
    e, ee = dy * gate, dy.abs() * egate + 2 * U * (dy * gate).abs()
    g = u.new_zeros(B, C, S) if dfinal is None else dfinal.double()
    eg = torch.zeros_like(g)
    du, edu, ddt, eddt = (torch.empty_like(u) for _ in range(4))
    dB, edB, dC, edC = (torch.empty_like(Bm) for _ in range(4))
    dA, edA, mA = (torch.zeros_like(A) for _ in range(3))
    over_c = 10 + C / 32                       # a lane's pair, the warp, four warps, the blocks along the channels
    for p in reversed(range(N)):
        a, ea = decay(p)
        up, tp, Bp, Cp, xp, ep = u[:, p], t[:, p], Bm[:, p, None], Cm[:, p, None], x[:, p, :, None], e[:, p, :, None]
        G = g + ep * Cp
        eG = eg + Cp.abs() * ee[:, p, :, None] + U * (ep * Cp).abs() + U * G.abs()
        Ga = G * a
        eGa = a * eG + G.abs() * ea + U * Ga.abs()
        w = Ga * hs[p]
        ew = hs[p].abs() * eGa + Ga.abs() * ehs[p] + U * w.abs()
        q, eq = (G * Bp).sum(-1), (Bp.abs() * eG).sum(-1) + (S + 3) * U * (G * Bp).abs().sum(-1)
        r, er = (w * A).sum(-1), (A.abs() * ew).sum(-1) + (S + 6) * U * (w * A).abs().sum(-1)
        du[:, p] = q * tp + Dk * e[:, p]
        edu[:, p] = tp.abs() * eq + q.abs() * et[:, p] + Dk.abs() * ee[:, p] + 2 * U * ((q * tp).abs() + (Dk * e[:, p]).abs())
        ddt[:, p] = (q * up + r) * sg[:, p]
        eddt[:, p] = sg[:, p] * (up.abs() * eq + er + 2 * U * ((q * up).abs() + r.abs())) + (q * up + r).abs() * esg[:, p] + \
            U * ddt[:, p].abs()
        wt = w * tp[..., None]
        dA += wt.sum(0)
        edA += (tp[..., None].abs() * ew + w.abs() * et[:, p, :, None] + U * wt.abs()).sum(0)
        mA += wt.abs().sum(0)
        dB[:, p] = (G * xp).sum(1)
        edB[:, p] = (xp.abs() * eG + G.abs() * ex[:, p, :, None] + U * (G * xp).abs()).sum(1) + over_c * U * (G * xp).abs().sum(1)
        eh1 = ep.abs() * hs[p + 1].abs()
        dC[:, p] = (ep * hs[p + 1]).sum(1)
        edC[:, p] = (ep.abs() * ehs[p + 1] + hs[p + 1].abs() * ee[:, p, :, None] + U * eh1).sum(1) + over_c * U * eh1.sum(1)
        g, eg = Ga, eGa
    eu = e * u
    dD, edD = eu.sum((0, 1)), (u.abs() * ee + U * eu.abs()).sum((0, 1)) + chain * U * eu.abs().sum((0, 1))
    dt_b, edt_b = ddt.sum((0, 1)), eddt.sum((0, 1)) + chain * U * ddt.abs().sum((0, 1))
    out += [("u", o(du), 2 * o(edu)), ("dt", o(ddt), 2 * o(eddt)), ("A", dA, 2 * (edA + chain * U * mA)),
            ("Bm", o(dB), 2 * o(edB)), ("Cm", o(dC), 2 * o(edC)), ("D", dD, 2 * edD)]
    if z is None:
        out.append(("z", None, None))
    else:
        s1, es1 = silu_slope(z.double()[:, order])
        dz = dy * y * s1
        out.append(("z", o(dz), 2 * o(dy.abs() * (s1.abs() * ey + y.abs() * es1) + 3 * U * dz.abs())))
    return out + [("dt_bias", dt_b, 2 * edt_b), ("init", g, 2 * eg)]


def chain_of_scan(B, N):
    """Tokens of a chunk in one lane (48), a warp's sums (5), the chunks by eighths (chunks hold 32 tokens or
    more), the eighths."""
    return 48 + 5 + -(-B * -(-N // 32) // 8) + 8


# ------------------------------------------------------------------ convolution
def conv_bwd(x, w, dy, order, bias, act, init, dfinal):
    """[(name, value, error)] of the gradients."""
    x, w, dy = x.double(), w.double(), dy.double()[:, order]
    (D, K), (B, N) = w.shape, x.shape[:2]
    X = conv_rows(x, init, order, K)
    b = w.new_zeros(D) if bias is None else bias.double()
    s = b + sum(w[:, j] * X[:, j:j + N] for j in range(K))
    es = (K + 1) * U * (b.abs() + sum((w[:, j] * X[:, j:j + N]).abs() for j in range(K)))
    if act:
        s1, es1 = silu_slope(s)
        ds, eds = dy * s1, dy.abs() * (es1 + 0.5 * es) + 2 * U * (dy * s1).abs()   # |silu''| <= 1/2
    else:
        ds, eds = dy, torch.zeros_like(dy)
    dX, edX, mX = (torch.zeros_like(X) for _ in range(3))
    for j in range(K):
        dX[:, j:j + N] += w[:, j] * ds
        edX[:, j:j + N] += w[:, j].abs() * eds
        mX[:, j:j + N] += (w[:, j] * ds).abs()
    if dfinal is not None:
        dX[:, N:] += dfinal.double()
        mX[:, N:] += dfinal.double().abs()
    edX += (K + 1) * U * mX
    # a block's positions in one thread: 148 x 8 blocks of 128 channels share them, 32 at least; its rows
    # by eighths
    groups = -(-D // 128)
    tile = max(32, -(-N // max(1, 148 * 8 // (groups * B))))
    chain = tile + -(-B * -(-N // tile) // 8) + 8
    dw, edw = [], []
    for j in range(K):
        p = ds * X[:, j:j + N]
        dw.append(p.sum((0, 1)))
        edw.append((X[:, j:j + N].abs() * eds + U * p.abs()).sum((0, 1)) + chain * U * p.abs().sum((0, 1)))
    db, edb = ds.sum((0, 1)), eds.sum((0, 1)) + chain * U * ds.abs().sum((0, 1))
    o = lambda v: to_grid(v[:, K - 1:], order)  # noqa: E731
    return [("x", o(dX), 2 * o(edX)), ("w", torch.stack(dw, 1), 2 * torch.stack(edw, 1)), ("bias", db, 2 * edb),
            ("init", dX[:, :K - 1], 2 * edX[:, :K - 1])]


# ------------------------------------------------------------------ group norm
def norm_bwd(x, dy, stats, G, gamma, beta, act):
    """[(name, value, error)] of the gradients at given statistics."""
    x, dy, st = x.double(), dy.double(), stats.double()
    B, N, C = x.shape
    mean, rstd = (st[..., i].reshape(B, 1, G, 1).expand(B, 1, G, C // G).reshape(B, 1, C) for i in (0, 1))
    xh = (x - mean) * rstd
    exh = 2 * U * xh.abs()
    gam = x.new_ones(C) if gamma is None else gamma.double()
    bet = x.new_zeros(C) if beta is None else beta.double()
    z = xh * gam + bet
    ez = gam.abs() * exh + U * ((xh * gam).abs() + z.abs())
    if act:
        s1, es1 = silu_slope(z)
        dz, edz = dy * s1, dy.abs() * (es1 + 0.5 * ez) + 2 * U * (dy * s1).abs()
    else:
        dz, edz = dy, torch.zeros_like(dy)
    # every eighth token of a range in one thread, the eighths; the ranges by eighths, the eighths.  The ranges
    # make three blocks an SM or more with the blocks along the channels (of 32 channels or more), of 64
    # tokens at least, 128 at most where a warp joins a group's figures (of 256 channels each)
    rows = -(-N // max(1, min(148 * 3 // (B * -(-C // 32)), -(-N // 64), 128 // -(-C // G // 256))))
    chain = rows / 8 + 8 + B * -(-N // min(rows, 32)) / 8 + 8
    p, ep = dz * xh, xh.abs() * edz + dz.abs() * exh + U * (dz * xh).abs()
    tok = lambda v: v.sum((0, 1))  # noqa: E731
    gg, egg = tok(p), tok(ep) + chain * U * tok(p.abs())
    gb, egb = tok(dz), tok(edz) + chain * U * tok(dz.abs())
    M = N * C // G
    grp = lambda v: v.reshape(B, N, G, C // G).sum((1, 3), keepdim=True).expand(B, 1, G, C // G).reshape(B, 1, C) / M  # noqa: E731
    gchain = rows / 8 + 8 + C / G + N / 32 + 160
    m1, em1 = grp(gam * dz), grp(gam.abs() * edz) + gchain * U * grp((gam * dz).abs())
    m2, em2 = grp(gam * p), grp(gam.abs() * ep) + gchain * U * grp((gam * p).abs())
    dx = rstd * (gam * dz - m1 - xh * m2)
    edx = rstd * (gam.abs() * edz + em1 + xh.abs() * em2 + exh * m2.abs() + 3 * U * ((gam * dz).abs() + m1.abs() + (xh * m2).abs()))
    return [("x", dx, 2 * edx), ("gamma", gg, 2 * egg), ("beta", gb, 2 * egb)]
