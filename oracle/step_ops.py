"""float64 definitions of the operators next to retention: head norms with the
position rotation, the gated recurrence, gradient clipping, each with its
gradients and with the bounds of an fp32 computation's error (u: the rounding
of fp32).  numpy only; shares no code with the library."""
import numpy as np

U = 2.0 ** -24


# ---- head norms with the rotation --------------------------------------------
def default_theta(dk):
    return (10000.0 ** (-2.0 * np.arange(dk // 2) / dk)).astype(np.float32)


def _turn(x, pos, theta, sign):
    """Rows [B, T, H, dk] at positions pos [B, T], turned by sign * pos * theta."""
    a = np.asarray(pos, np.float64)[:, :, None, None] * np.asarray(theta, np.float64)
    c, s = np.cos(a), sign * np.sin(a)
    y = np.empty_like(x)
    y[..., 0::2] = x[..., 0::2] * c - x[..., 1::2] * s
    y[..., 1::2] = x[..., 1::2] * c + x[..., 0::2] * s
    return y


def _pairs(x):
    """|x0| + |x1| of each pair, at both of its places."""
    m = np.abs(x[..., 0::2]) + np.abs(x[..., 1::2])
    return np.repeat(m, 2, -1)


def qk_norm(x, w, pos, theta, eps, s, rotate=True):
    """(y, size): size bounds what a relative error of the norm or of cos and sin scales."""
    x = np.asarray(x, np.float64)
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        n = n * np.asarray(w, np.float64)
    return s * (_turn(n, pos, theta, 1) if rotate else n), abs(s) * _pairs(n)


def qk_norm_backward(x, w, dy, pos, theta, eps, s, rotate=True):
    """(dx, dw, size of dx, size of dw)."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    u = s * (_turn(dy, pos, theta, -1) if rotate else dy)
    um = abs(s) * _pairs(dy)
    wd = 1.0 if w is None else np.asarray(w, np.float64)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g, gm = wd * u, np.abs(wd) * um
    dx = r * (g - x * r * r * (g * x).mean(-1, keepdims=True))
    mx = r * (gm + np.abs(x) * r * r * (gm * np.abs(x)).mean(-1, keepdims=True))
    ax = tuple(range(x.ndim - 1))
    return dx, (u * x * r).sum(ax), mx, (um * np.abs(x) * r).sum(ax)


# ---- gated recurrence ----------------------------------------------------------
def _parts(g, rate, normalize):
    s = 1.0 / (1.0 + np.exp(-np.asarray(g, np.float64)))
    q = np.asarray(rate, np.float64) * s
    a = np.exp(-q)
    m = np.sqrt(-np.expm1(-2 * q)) if normalize else np.ones_like(a)
    # an fp32 sigmoid and 1 - s are off by their argument's rounding, g u, and a few u of themselves; q follows it
    es = (8 + 2 * np.abs(np.asarray(g, np.float64))) * U
    return s, q, a, m, es


def _run(a, u, start):
    out = np.empty_like(u)
    h = start
    for t in range(u.shape[1]):
        h = a[:, t] * h + u[:, t]
        out[:, t] = h
    return out


def _bound(q, es, a, m, x, start):
    """Magnitudes of the recurrence, and what its fp32 form is off by at most: each step's decay is off by q times the
    relative error of q, relative to itself, m x by the error of m, and h by a few roundings."""
    size = _run(a, m * np.abs(x), np.abs(start))
    before = np.concatenate([np.abs(start)[:, None], size[:, :-1]], 1)
    step = (es + 16 * U) * q * a * before + (es + 8 * U) * m * np.abs(x) + 8 * U * size
    return size, _run(a, step, np.zeros_like(start))


def gate(x, g, rate, state, normalize=True):
    """(h, bound of its fp32 error), [B, T, D]; state [B, D] or None."""
    x = np.asarray(x, np.float64)
    s, q, a, m, es = _parts(g, rate, normalize)
    start = np.zeros((x.shape[0], x.shape[2])) if state is None else np.asarray(state, np.float64)
    return _run(a, m * x, start), _bound(q, es, a, m, x, start)[1]


def gate_backward(x, g, rate, state, dh, dstate, normalize=True):
    """((dx, dg, drate, dstate_in), the bounds of their fp32 errors)."""
    x, dh, rate = np.asarray(x, np.float64), np.asarray(dh, np.float64), np.asarray(rate, np.float64)
    s, q, a, m, es = _parts(g, rate, normalize)
    B, T, D = x.shape
    zero = np.zeros((B, D))
    start = zero if state is None else np.asarray(state, np.float64)
    last = zero if dstate is None else np.asarray(dstate, np.float64)
    before = lambda h, h0: np.concatenate([h0[:, None], h[:, :-1]], 1)
    h = _run(a, m * x, start)
    hm, hb = _bound(q, es, a, m, x, start)
    hp, hpm, hpb = before(h, start), before(hm, np.abs(start)), before(hb, zero)
    # mu_t = a_t (dh_t + mu_{t+1}), from the last token to the first
    rev = lambda z: z[:, ::-1]
    mu = rev(_run(rev(a), rev(a * dh), last))
    mum = rev(_run(rev(a), rev(a * np.abs(dh)), np.abs(last)))
    after = lambda z, z0: np.concatenate([z[:, 1:], z0[:, None]], 1)
    lam, lamm = dh + after(mu, last), np.abs(dh) + after(mum, np.abs(last))
    ea = (es + 16 * U) * q + 8 * U  # of a, relative to it
    mub = rev(_run(rev(a), rev(ea * a * lamm), zero))
    lamb = after(mub, zero) + U * lamm
    dx = m * lam
    dxb = m * lamb + (es + 8 * U) * m * lamm
    dl, dlm = mu * hp, mum * hpm
    dlb = mub * hpm + mum * hpb + 4 * U * dlm
    if normalize:
        ratio = np.divide(a, m, out=np.zeros_like(a), where=m > 0)
        dl = dl - mu * x * ratio
        t = mum * np.abs(x) * ratio
        dlm = dlm + t
        dlb = dlb + mub * np.abs(x) * ratio + (ea + es + 12 * U) * t
    k = rate * s / (1 + np.exp(np.asarray(g, np.float64)))  # 1 - s without its cancellation
    dg = -k * dl
    dgb = k * dlb + (2 * es + 16 * U) * k * dlm
    drate = -(s * dl).sum((0, 1))
    chain = 64 + B * T / 2048  # additions in a row: a slice, its tile's slices, a 64th of the tiles, six more
    drb = (s * dlb).sum((0, 1)) + ((es + (chain + 8) * U) * s * dlm).sum((0, 1))
    first = mu[:, 0] if T else last
    firstb = mub[:, 0] if T else zero
    return (dx, dg, drate, first), (dxb, dgb, drb, firstb)


# ---- gradients -------------------------------------------------------------------
def clip(grads, max_norm):
    """([g f], norm) of float64 arrays; a norm beyond fp32 leaves them as they are."""
    norm = np.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads))
    with np.errstate(over="ignore"):  # infinite as fp32
        finite = np.isfinite(np.float32(norm))
    f = max_norm / norm if max_norm < norm and finite else 1.0
    return [np.asarray(g, np.float64) * f for g in grads], norm
