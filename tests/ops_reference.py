"""Plain 64-bit forms of the convolution, the selective scan and the group norm for the tests,
written from their formulas, token by token where the operator is a recurrence.

Each returns its results and, with ``mag=True``, the same sums over the magnitudes of their
terms: the scale that float32 roundings of those sums go by.
"""
import torch

EPS32 = 2.0 ** -24      # half a step of float32, relative


def scan_order(H, W, direction, device="cpu"):
    n = torch.arange(H * W, device=device).reshape(H, W)
    n = (n, n.flip(1), n.t(), n.flip(0).t())[direction]
    return n.reshape(-1)


def to_grid(t, order):
    out = torch.empty_like(t)
    out[:, order] = t
    return out


def silu_grad(z):
    s = torch.sigmoid(z)
    return s * (1 + z * (1 - s))


# ------------------------------------------------------------------ convolution
def conv_rows(x, init, order, K):
    B, _, D = x.shape
    first = x.new_zeros(B, K - 1, D) if init is None else init.double()
    return torch.cat((first, x[:, order]), 1)


def conv_fwd(x, w, order, bias, silu, init, mag=False):
    """(out, final rows), or (bound of the pre-activation's terms, same shape as out)."""
    x, w = x.double(), w.double()
    K, N = w.shape[1], x.shape[1]
    X = conv_rows(x, init, order, K)
    b = w.new_zeros(w.shape[0]) if bias is None else bias.double()
    if mag:
        return to_grid(b.abs() + sum(w[:, j].abs() * X[:, j:j + N].abs() for j in range(K)), order)
    s = b + sum(w[:, j] * X[:, j:j + N] for j in range(K))
    return to_grid(s * torch.sigmoid(s) if silu else s, order), X[:, N:]


def conv_bwd(x, w, dy, order, bias, silu, init, dfinal, mag=False):
    """(dx, dw, dbias, dinit), or the sums of their terms' magnitudes."""
    x, w, dy = x.double(), w.double(), dy.double()[:, order]
    K, N = w.shape[1], x.shape[1]
    X = conv_rows(x, init, order, K)
    b = 0 if bias is None else bias.double()
    s = b + sum(w[:, j] * X[:, j:j + N] for j in range(K))
    ds = dy * silu_grad(s) if silu else dy
    if mag:
        # a rounding of s by its terms' size moves silu' by at most half of that
        ds = dy.abs() * (1.1 + 0.5 * (b if bias is None else b.abs()) +
                         0.5 * sum(w[:, j].abs() * X[:, j:j + N].abs() for j in range(K)))
        w, X = w.abs(), X.abs()
    dX = torch.zeros_like(X)
    for j in range(K):
        dX[:, j:j + N] += w[:, j] * ds
    if dfinal is not None:
        dX[:, N:] += dfinal.double().abs() if mag else dfinal.double()
    dw = torch.stack([(ds * X[:, j:j + N]).sum((0, 1)) for j in range(K)], 1)
    return to_grid(dX[:, K - 1:], order), dw, ds.sum((0, 1)), dX[:, :K - 1]


# ------------------------------------------------------------------ selective scan
def _scan_inputs(u, dt, A, Bm, Cm, order, z, dt_bias, softplus):
    u, Bm, Cm = (t.double()[:, order] for t in (u, Bm, Cm))
    raw = dt.double()[:, order]
    if dt_bias is not None:
        raw = raw + dt_bias.double()
    t = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    gate = None if z is None else z.double()[:, order]
    return u, t, raw, A.double(), Bm, Cm, gate


def scan_fwd(u, dt, A, Bm, Cm, order, D=None, z=None, dt_bias=None, softplus=True, init=None, mag=False):
    """(out, final state), or the sums of their terms' magnitudes (the decays kept)."""
    u, t, raw, A, Bm, Cm, z = _scan_inputs(u, dt, A, Bm, Cm, order, z, dt_bias, softplus)
    B, N, C = u.shape
    h = u.new_zeros(B, C, A.shape[1]) if init is None else init.double()
    Dk = u.new_zeros(C) if D is None else D.double()
    if mag:
        u, Bm, Cm, h, Dk, t_in = u.abs(), Bm.abs(), Cm.abs(), h.abs(), Dk.abs(), t.abs()
    else:
        t_in = t
    ys = []
    for p in range(N):
        h = torch.exp(t[:, p, :, None] * A) * h + (t_in[:, p] * u[:, p])[..., None] * Bm[:, p, None]
        ys.append((h * Cm[:, p, None]).sum(-1) + Dk * u[:, p])
    y = torch.stack(ys, 1)
    if z is not None:
        g = z * torch.sigmoid(z)
        y = y * (g.abs() if mag else g)
    return to_grid(y, order), h


def scan_bwd(u, dt, A, Bm, Cm, dy, order, D=None, z=None, dt_bias=None, softplus=True, init=None, dfinal=None, mag=False):
    """(du, ddt, dA, dB, dC, dD, dz, ddt_bias, dinit), or the sums of their terms' magnitudes."""
    u, t, raw, A, Bm, Cm, z = _scan_inputs(u, dt, A, Bm, Cm, order, z, dt_bias, softplus)
    dy = dy.double()[:, order]
    B, N, C = u.shape
    S = A.shape[1]
    h = u.new_zeros(B, C, S) if init is None else init.double()
    g = u.new_zeros(B, C, S) if dfinal is None else dfinal.double()
    Dk = u.new_zeros(C) if D is None else D.double()
    decay, t_in, Aq = A, t, A
    gz = None if z is None else z * torch.sigmoid(z)
    if mag:
        u, Bm, Cm, dy, h, g, Dk, t_in, Aq = (v.abs() for v in (u, Bm, Cm, dy, h, g, Dk, t, A))
        gz = None if z is None else gz.abs()
    e = dy if z is None else dy * gz
    before, after = [], []
    for p in range(N):
        before.append(h)
        h = torch.exp(t[:, p, :, None] * decay) * h + (t_in[:, p] * u[:, p])[..., None] * Bm[:, p, None]
        after.append(h)
    du, ddt, dz = torch.empty_like(u), torch.empty_like(u), torch.empty_like(u)
    dA, dB, dC = torch.zeros_like(A), torch.empty_like(Bm), torch.empty_like(Cm)
    for p in reversed(range(N)):
        a = torch.exp(t[:, p, :, None] * decay)
        G = g + e[:, p, :, None] * Cm[:, p, None]
        w = G * a * before[p]
        q = (G * Bm[:, p, None]).sum(-1)
        du[:, p] = q * t_in[:, p] + Dk * e[:, p]
        ddt[:, p] = (w * Aq).sum(-1) + q * u[:, p]
        dA += (w * t_in[:, p, :, None]).sum(0)
        dB[:, p] = (G * (t_in[:, p] * u[:, p])[..., None]).sum(1)
        dC[:, p] = (after[p] * e[:, p, :, None]).sum(1)
        y = (after[p] * Cm[:, p, None]).sum(-1) + Dk * u[:, p]
        if z is not None:
            sg = silu_grad(z[:, p])
            dz[:, p] = dy[:, p] * y * (sg.abs() + 0.5 if mag else sg)
        g = a * G
    if softplus:
        ddt = ddt * torch.sigmoid(raw)
    o = lambda v: to_grid(v, order)  # noqa: E731
    return (o(du), o(ddt), dA, o(dB), o(dC), (e * u).sum((0, 1)), None if z is None else o(dz), ddt.sum((0, 1)), g)


# ------------------------------------------------------------------ group norm
def norm_fwd(x, G, gamma, beta, eps, silu):
    """(out, stats, z) with x [B, N, C]."""
    x = x.double()
    B, N, C = x.shape
    xg = x.reshape(B, N, G, C // G)
    mean = xg.mean((1, 3), keepdim=True)
    rstd = 1 / torch.sqrt(((xg - mean) ** 2).mean((1, 3), keepdim=True) + eps)
    z = ((xg - mean) * rstd).reshape(B, N, C)
    if gamma is not None:
        z = z * gamma.double()
    if beta is not None:
        z = z + beta.double()
    return (z * torch.sigmoid(z) if silu else z), torch.stack((mean.reshape(B, G), rstd.reshape(B, G)), -1), z


def norm_bwd(x, dy, stats, G, gamma, beta, silu, mag=False):
    """(dx, dgamma, dbeta) for given statistics, or the sums of their terms' magnitudes."""
    x, dy, st = x.double(), dy.double(), stats.double()
    B, N, C = x.shape
    mean, rstd = (st[..., i].reshape(B, 1, G, 1) for i in (0, 1))
    xh = ((x.reshape(B, N, G, C // G) - mean) * rstd)
    gam = x.new_ones(C) if gamma is None else gamma.double()
    bet = x.new_zeros(C) if beta is None else beta.double()
    z = xh.reshape(B, N, C) * gam + bet
    dz = dy * silu_grad(z) if silu else dy
    if mag:
        # x - mean may cancel: its terms are |x| and |mean|, and a rounding of z moves silu' by half of that
        xh = (x.abs().reshape(B, N, G, C // G) + mean.abs()) * rstd
        gam = gam.abs()
        dz = dy.abs() * (1.1 + 0.5 * (xh.reshape(B, N, C) * gam + bet.abs()) if silu else 1.0)
    dzg = (dz * gam).reshape(B, N, G, C // G)
    m1, m2 = dzg.mean((1, 3), keepdim=True), (dzg * xh).mean((1, 3), keepdim=True)
    dx = rstd * (dzg + m1 + xh * m2) if mag else rstd * (dzg - m1 - xh * m2)
    return dx.reshape(B, N, C), (dz * xh.reshape(B, N, C)).sum((0, 1)), dz.sum((0, 1))
