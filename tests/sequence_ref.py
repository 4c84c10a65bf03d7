"""64-bit plain implementations of the operators over sequences (gated linear
recurrence, normed and rotated heads, token log probabilities, clipped policy
loss, and their gradients) on the host, in NumPy, with the error bounds of a
computation in fp32.  Bounds leave out the rounding to the output's type, which
`close` adds."""
import numpy as np
import torch

U = 2.0 ** -24      # unit roundoff of fp32


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, want, err, dtype):
    """got (a tensor) is want but for err and one rounding to its type."""
    assert got.dtype == dtype and tuple(got.shape) == np.shape(want), (got.dtype, got.shape, np.shape(want))
    g = f64(got)
    half = torch.finfo(dtype).eps / 2
    room = err * (1 + half) + half * np.abs(want) + 2.0 ** -133     # subnormal bf16: half a step
    bad = ~(np.abs(g - want) <= room)
    assert not bad.any(), (int(bad.sum()), bad.size, np.argwhere(bad)[:3].tolist(), g[bad][:3],
                           np.asarray(want)[bad][:3], np.broadcast_to(room, g.shape)[bad][:3])


# ---------------------------------------------------------------- recurrence

def _sigmoid(g):
    e = np.exp(-np.abs(g))
    return np.where(g >= 0, 1, e) / (1 + e), np.where(g >= 0, e, 1) / (1 + e)


def _gate_error(g):
    """Relative error of the smaller of a and 1 - a: t = exp(-|g|) with its
    argument rounded twice on the way to a power of two (2 |g| U, 1.5 for the
    change of base) and 4 ulp for the power, 1 + t, one division."""
    return (3 * np.abs(g) + 12) * U


def scan(gate, x, state, starts, mask, mix):
    """(h, last, error of h, error of last) of [batch, length, dim].

    Every step costs a relative error of the smaller share (of what it
    multiplies) and a few roundings of the terms; in whatever order partial
    recurrences are joined, the terms are bounded by the recurrence of their
    absolute values."""
    b, t, d = x.shape
    p = np.zeros((b, d)) if state is None else state.copy()
    size, err = np.abs(p), np.zeros((b, d))
    h, eh = np.zeros(x.shape), np.zeros(x.shape)
    for i in range(t):
        a, u = _sigmoid(gate[:, i])
        w = u if mix else np.ones_like(u)
        live = np.ones(b, bool) if mask is None else mask[:, i].astype(bool)
        cut = np.zeros(b, bool) if starts is None else starts[:, i].astype(bool)
        q = np.where(cut[:, None], 0, p)
        qs = np.where(cut[:, None], 0, size)
        e = np.minimum(a, u) * _gate_error(gate[:, i])
        new = a * q + w * x[:, i]
        ns = a * qs + w * np.abs(x[:, i])
        ne = a * np.where(cut[:, None], 0, err) + e * (qs + mix * np.abs(x[:, i])) + \
            6 * U * (qs + np.abs(x[:, i]))
        p, size, err = (np.where(live[:, None], n, o) for n, o in ((new, p), (ns, size), (ne, err)))
        h[:, i], eh[:, i] = p, err
    return h, p, eh, err


def scan_grad(dh, gate, x, h, state, dlast, starts, mask, mix):
    """((dgate, dx, dstate), their errors)."""
    b, t, d = dh.shape
    l = np.zeros((b, d)) if dlast is None else dlast.copy()
    size, err = np.abs(l), np.zeros((b, d))
    out = [np.zeros(dh.shape) for _ in range(4)]
    for i in reversed(range(t)):
        l, size = l + dh[:, i], size + np.abs(dh[:, i])
        err = err + 2 * U * size
        a, u = _sigmoid(gate[:, i])
        eg = _gate_error(gate[:, i])
        live = (np.ones(b, bool) if mask is None else mask[:, i].astype(bool))[:, None]
        cut = (np.zeros(b, bool) if starts is None else starts[:, i].astype(bool))[:, None]
        before = h[:, i - 1] if i else np.zeros((b, d)) if state is None else state
        q = np.where(cut, 0, before)
        v = q - x[:, i] if mix else q
        w = u if mix else np.ones_like(u)
        vals = (a * u * l * v, w * l,
                a * u * (err * np.abs(v) + (2 * eg + 8 * U) * size * (np.abs(q) + mix * np.abs(x[:, i]))),
                w * (err + (mix * eg + 4 * U) * size))
        for o, val in zip(out, vals):
            o[:, i] = np.where(live, val, 0)
        keep = np.where(cut, 0, a)
        e = np.minimum(a, u) * eg + 6 * U
        l, size, err = (np.where(live, n, o) for n, o in
                        ((keep * l, l), (keep * size, size),
                         (keep * err + np.where(cut, 0, e) * size, err)))
    return (out[0], out[1], l), (out[2], out[3], err)


# ---------------------------------------------------------------- heads

def _pairs(dim, rotary, neighbours):
    m = np.arange(rotary // 2)
    return (2 * m, 2 * m + 1) if neighbours else (m, m + rotary // 2)


def _turn(n, cos, sin, i, j):
    y = n.copy()
    y[..., i], y[..., j] = n[..., i] * cos - n[..., j] * sin, n[..., j] * cos + n[..., i] * sin
    return y


def _reach(n, cos, sin, i, j):
    """Sum of the magnitudes of _turn's terms."""
    n, c, s = np.abs(n), np.abs(cos), np.abs(sin)
    y = n.copy()
    y[..., i], y[..., j] = n[..., i] * c + n[..., j] * s, n[..., j] * c + n[..., i] * s
    return y


def _angles(cos, sin, pos):
    """Table rows of the tokens and which of them are tokens."""
    if cos is None:
        return np.ones((len(pos), 1, 0)), np.zeros((len(pos), 1, 0)), np.ones(len(pos), bool)
    ok = (pos >= 0) & (pos < len(cos))
    at = np.where(ok, pos, 0)
    if len(cos) == 0:
        z = np.zeros((len(pos), 1, cos.shape[1]))
        return z, z, ok
    return cos[at][:, None], sin[at][:, None], ok


def heads(x, w, cos, sin, pos, eps, neighbours):
    """(y, error) of [tokens, heads, dim].  A sum of dim <= 1024 squares goes
    through at most 64 additions in a row; half of its error and a few
    roundings reach the scale; a turned element has three more roundings."""
    d = x.shape[-1]
    c, s, ok = _angles(cos, sin, pos)
    i, j = _pairs(d, 2 * c.shape[-1], neighbours)
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1 if w is None else w)
    y = _turn(n, c, s, i, j)
    err = (32 + 10) * U * _reach(n, c, s, i, j)
    return np.where(ok[:, None, None], y, 0), np.where(ok[:, None, None], err, 0)


def heads_grad(dy, x, w, cos, sin, pos, eps, neighbours):
    """((dx, dw), errors).  Row sums as in `heads`; a weight's sum goes through
    at most 1024 additions in a row."""
    d = x.shape[-1]
    c, s, ok = _angles(cos, sin, pos)
    i, j = _pairs(d, 2 * c.shape[-1], neighbours)
    rstd = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    h = x * rstd
    g = _turn(dy, c, -s, i, j)
    reach = _reach(dy, c, s, i, j)
    live = ok[:, None, None]
    g, reach = np.where(live, g, 0), np.where(live, reach, 0)
    k = 64 + 20
    aw = 1 if w is None else np.abs(w)
    gw = g * (1 if w is None else w)
    dx = rstd * (gw - h * (gw * h).mean(-1, keepdims=True))
    ex = rstd * k * U * (reach * aw + np.abs(h) * (reach * aw * np.abs(h)).mean(-1, keepdims=True))
    dw = np.where(live, g * h, 0).sum((0, 1))
    ew = (1024 + k) * U * np.where(live, reach * np.abs(h), 0).sum((0, 1))
    return (np.where(live, dx, 0), dw), (np.where(live, ex, 0), ew)


# ---------------------------------------------------------------- log probabilities

def log_probs(l, y, scale):
    """(log_probs, lse, errors) of [tokens, vocab].  A term exp((l - top)
    scale) has three roundings of its argument and 4 ulp; the sum at most 1024
    additions in a row."""
    v = l.shape[1]
    ok = (y >= 0) & (y < v)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        top = l.max(1)
        arg = (l - top[:, None]) * scale
        e = np.exp(arg)
        s = e.sum(1)
        far = np.where(e > 0, np.abs(arg) * e, 0).sum(1) / s
        rest = np.log(s)
        rel = 4 * U * far + (1024 + 8) * U
        lp = arg[np.arange(len(y)), np.where(ok, y, 0)] - rest
        lse = top * scale + rest
    elp = rel + 4 * U * (np.abs(lp) + 2 * np.abs(rest))
    else_ = rel + 4 * U * (np.abs(top * scale) + np.abs(rest))
    z = np.zeros(len(y))
    return np.where(ok, lp, z), np.where(ok, lse, z), np.where(ok, elp, z), np.where(ok, else_, z)


def log_probs_grad(d, l, y, lse, scale):
    """(dlogits, error) from the rounded lse: the argument scale * l - lse has
    a rounding of each term and its own."""
    v = l.shape[1]
    live = (y >= 0) & (y < v) & (d != 0)
    with np.errstate(invalid="ignore", over="ignore"):
        arg = scale * l - lse[:, None]
        p = np.exp(arg)
        rel = np.where(p > 0, 4 * U * (np.abs(scale * l) + np.abs(lse[:, None])) + 8 * U, 0)
    hot = np.zeros(l.shape)
    hot[np.arange(len(y))[live], y[live]] = 1
    f = (scale * d)[:, None]
    g, err = f * (hot - p), np.abs(f) * (4 * U * hot + p * rel + 4 * U * p)
    return np.where(live[:, None], g, 0), np.where(live[:, None], err, 0)


# ---------------------------------------------------------------- policy loss

def _policy(lp, old, adv, ref, mask, low, high):
    m = np.ones(lp.shape, bool) if mask is None else mask.astype(bool)
    lp, old = np.where(m, lp, 0), np.where(m, old, 0)
    adv = np.broadcast_to(adv[:, None] if adv.ndim == 1 else adv, lp.shape)
    d = lp - old
    cut = m & np.where(adv >= 0, d > np.log1p(high), d < np.log1p(-low))
    e = np.zeros(lp.shape) if ref is None else np.where(m, ref, 0) - lp
    return m, d, cut, np.where(m, adv, 0), e


def policy(lp, old, adv, ref, mask, low, high, kl, by_sequence):
    """((loss, kl, clipped, weights), errors): a ratio has the rounding of its
    argument and 4 ulp, k 16 roundings or those of its three terms; a sum at
    most 64 additions in a row."""
    m, d, cut, adv, e = _policy(lp, old, adv, ref, mask, low, high)
    r = np.where(cut, np.where(adv >= 0, 1 + high, 1 - low), np.exp(d))
    k = np.where(np.abs(e) < 1e-3, e * e * (0.5 + e / 6 + e * e / 24), np.expm1(e) - e)
    k = np.where(m, k, 0)
    each = np.where(m, -r * adv + kl * k, 0)
    ek = U * (16 * k + np.where(np.abs(e) > 1, 4 * (np.exp(e) + 1 + np.abs(e)), 0) +
              2 * np.abs(e) * np.abs(np.expm1(e)))
    ee = U * (np.abs(d) + 8) * np.abs(r * adv) + abs(kl) * (ek + 2 * U * k)
    n = m.sum(1)
    if by_sequence:
        w = np.where(n > 0, 1 / (np.maximum(n, 1) * max((n > 0).sum(), 1)), 0)
    else:
        w = np.where(n > 0, 1 / max(n.sum(), 1), 0)
    mean = lambda z: float((w * (z * m).sum(1)).sum())  # noqa: E731
    return ((mean(each), mean(k), mean(cut), w),
            (mean(ee) + 64 * U * mean(np.abs(r * adv) + abs(kl) * k), mean(ek) + 64 * U * mean(k),
             64 * U * mean(cut), 2 * U * w))


def policy_grad(lp, old, adv, ref, mask, low, high, kl, w, dloss):
    m, d, cut, adv, e = _policy(lp, old, adv, ref, mask, low, high)
    pull = np.where(cut, 0, np.exp(d) * adv)
    f = dloss * w[:, None]
    g = f * (-pull - kl * np.expm1(e))
    err = np.abs(f) * U * ((np.abs(d) + 10) * np.abs(pull) +
                           abs(kl) * (12 * np.abs(np.expm1(e)) + 2 * np.abs(e) * np.exp(e)))
    return np.where(m, g, 0), np.where(m, err, 0)
