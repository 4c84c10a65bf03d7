"""64-bit plain implementations of the training operators (layer norm behind
dropout and the residual add, dropout, the expert router with its balance
loss, and their gradients) on the host, in NumPy, for the tests."""
import numpy as np
import torch

U = 2.0 ** -24      # unit roundoff of fp32
UB = 2.0 ** -8      # twice that of bf16: one rounding, and a tie seen from either side


def f64(t):
    return t.detach().double().cpu().numpy()


def out_ulp(dtype):
    """Relative error of the one rounding to the output's type."""
    return UB if dtype == torch.bfloat16 else U


def philox(c, k):
    """Philox4x32-10 block of counter words c[0..3] and key words k[0..1]
    (Python integers)."""
    c, k = list(c), list(k)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def factors(n, p, seed, offset, start=0):
    """0 or the kept elements' factor, for elements start .. start + n - 1."""
    if p == 0:
        return np.ones(n)
    t = int(np.floor(np.float64(np.float32(p)) * 65536 + 0.5))
    scale = 65536.0 / (65536 - t) if t < 65536 else 0.0
    first = start // 8
    blocks = (start + n + 7) // 8 - first
    ctr = (np.arange(first, first + blocks, dtype=np.uint64) + np.uint64(offset))
    m = np.uint64(0xFFFFFFFF)
    sh = np.uint64(32)
    c = [ctr & m, ctr >> sh, np.zeros(blocks, np.uint64), np.zeros(blocks, np.uint64)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> sh) ^ c[1] ^ np.uint64(k0), b & m, (a >> sh) ^ c[3] ^ np.uint64(k1), a & m]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    h = np.stack([c[0] & np.uint64(0xFFFF), c[0] >> np.uint64(16), c[1] & np.uint64(0xFFFF),
                  c[1] >> np.uint64(16), c[2] & np.uint64(0xFFFF), c[2] >> np.uint64(16),
                  c[3] & np.uint64(0xFFFF), c[3] >> np.uint64(16)], 1).reshape(-1)
    return np.where(h[start - 8 * first:start - 8 * first + n] >= t, scale, 0.0)


def dropped(x, f):
    """x times its factors; a dropped element is 0 whatever it holds."""
    with np.errstate(invalid="ignore"):
        return np.where(f == 0, 0.0, x * f)


def norm(x, r, w, b, eps, f):
    """(y, s, mean, rstd) of 2-D x."""
    s = dropped(x, f) + (0.0 if r is None else r)
    mean = s.mean(1)
    rstd = 1.0 / np.sqrt(((s - mean[:, None]) ** 2).mean(1) + eps)
    h = (s - mean[:, None]) * rstd[:, None]
    return h * (1.0 if w is None else w) + (0.0 if b is None else b), s, mean, rstd


def norm_bounds(x, r, w, b, eps, f):
    """Error bounds of (s, mean, rstd, y) before the rounding to the output's
    type.  A sum over a row of at most a few tens of thousand elements goes
    through at most K = 128 additions in a row (a thread's own, then a tree):
    error <= K U of the mean magnitude.  s costs two roundings; the variance
    two per term, and the mean's error squared."""
    K = 128 * U
    y, s, mean, rstd = norm(x, r, w, b, eps, f)
    ds = 2 * U * (np.abs(dropped(x, f)) + (0.0 if r is None else np.abs(r)))
    dm = K * np.abs(s).mean(1) + ds.mean(1)
    rel = K + 4 * U + (dm * rstd) ** 2 + (ds * rstd[:, None]).max(1)
    h = (s - mean[:, None]) * rstd[:, None]
    dh = rstd[:, None] * (dm[:, None] + ds) + np.abs(h) * (rel[:, None] + 3 * U)
    aw = 1.0 if w is None else np.abs(w)
    dy = aw * dh + 4 * U * (aw * np.abs(h) + (0.0 if b is None else np.abs(b)))
    return ds, dm, rel * rstd, dy


def norm_grad(dy, s, mean, rstd, w, ds, f):
    """(dx, dresidual, dweight, dbias) and their error bounds before the
    rounding to the output's type (row sums as in norm_bounds; a column sum
    goes through at most 512 additions in a row)."""
    K, KC = 128 * U, 512 * U
    h = (s - mean[:, None]) * rstd[:, None]
    g = dy * (1.0 if w is None else w)
    mg, mh = g.mean(1)[:, None], (g * h).mean(1)[:, None]
    r = rstd[:, None]
    d = r * (g - mg - h * mh)
    ag, agh = np.abs(g).mean(1)[:, None], np.abs(g * h).mean(1)[:, None]
    err = r * K * (np.abs(g) + ag + np.abs(h) * agh)
    if ds is not None:
        d = d + ds
        err = err + 2 * U * np.abs(ds)
    dw, db = (dy * h).sum(0), dy.sum(0)
    scale = float(np.max(f)) if np.size(f) else 1.0
    return ((dropped(d, f), d, dw, db),
            (err * max(scale, 1.0) + 2 * U * np.abs(d) * scale, err,
             KC * np.abs(dy * h).sum(0), KC * np.abs(dy).sum(0)))


def route(l, k, mask, normalize):
    """dict of weights, index, counts, mean_prob, loss, p, routed, and
    `reach`: how far each logit is below its row's largest."""
    T, E = l.shape
    routed = np.zeros(T, bool)
    p = np.zeros((T, E))
    index = np.full((T, k), -1, np.int64)
    weights = np.zeros((T, k))
    for t in range(T):
        row = l[t]
        if (mask is not None and not mask[t]) or not (np.isnan(row).any() or (row > -np.inf).any()):
            continue
        routed[t] = True
        order = sorted(range(E), key=lambda e: ((0, 0.0) if np.isnan(row[e]) else (1, -row[e]), e))
        picks = [e for e in order[:k] if not row[e] == -np.inf]
        index[t, :len(picks)] = picks
        with np.errstate(invalid="ignore"):
            x = np.exp(row - row[order[0]])
        p[t] = x / x.sum()
        weights[t, :len(picks)] = x[picks] / x[picks].sum() if normalize else p[t, picks]
    n = int(routed.sum())
    counts = np.bincount(index[index >= 0], minlength=E)
    mean_prob = p.sum(0) / max(n, 1)
    loss = E * (counts / (k * max(n, 1)) * mean_prob).sum()
    return dict(weights=weights, index=index, counts=np.append(counts, n), mean_prob=mean_prob,
                loss=loss, p=p, routed=routed)


def route_grad(l, index, counts, dw, dloss, mask, normalize):
    """dlogits, by the chain rule through p and the weights, row by row with
    the softmax's Jacobian written out."""
    T, E = l.shape
    k = index.shape[1]
    n = max(int(counts[E]), 1)
    out = np.zeros((T, E))
    for t in range(T):
        row = l[t]
        if (mask is not None and not mask[t]) or not (np.isnan(row).any() or (row > -np.inf).any()):
            continue
        with np.errstate(invalid="ignore"):
            x = np.exp(row - np.max(row))
        p = x / x.sum()
        g = dloss * E * counts[:E] / (k * n) / n
        picks = [(j, e) for j, e in enumerate(index[t]) if 0 <= e < E]
        es = [e for _, e in picks]
        d = np.array([dw[t, j] for j, _ in picks])
        if normalize and picks:
            w = x[es] / x[es].sum()
            out[t, es] += (np.diag(w) - np.outer(w, w)) @ d
        elif picks:
            g = g.copy()
            g[es] += d
        out[t] += (np.diag(p) - np.outer(p, p)) @ g
    return out
