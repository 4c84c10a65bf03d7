"""Measured cases of the training operators around the optimizer step: layer
norm (alone, and behind dropout and the residual add), dropout from a
counter-based generator, and the expert router with its balance loss, each
forward and backward.

`run` computes a case either in elementary torch operations in 32 bits
(`own` false) or through newton_schulz_05_gb300.layers (`own` true).

Sizes: 2048, 4096, 10240, 11008 and 1408 are the widths of the parameter sets in
synth/, 16 and 64 the expert counts of its stacks; 1023 and 1409 are ragged
neighbours of common widths.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # one token's hidden state: the call's own latency
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 2048, "dtype": "bf16",
         "wdtype": "bf16", "p": 0.0, "wide": False},
        # the norm in front of a dense layer, four sequences of 4096 tokens
        {"name": "norm_dense", "op": "norm", "rows": 16384, "cols": 4096, "dtype": "bf16",
         "wdtype": "f32", "p": 0.0, "wide": False},
        # fp32 activations of a ragged width, rows cut out of a wider buffer
        {"name": "norm_ragged", "op": "norm", "rows": 4099, "cols": 1409, "dtype": "f32",
         "wdtype": "f32", "p": 0.0, "wide": True},
        # sublayer output dropped out, added to the residual stream and normed
        {"name": "add_norm", "op": "norm", "rows": 8192, "cols": 10240, "dtype": "bf16",
         "wdtype": "bf16", "p": 0.1, "wide": False},
        # gradient of the norm in front of a dense layer
        {"name": "norm_grad_dense", "op": "norm_grad", "rows": 16384, "cols": 4096,
         "dtype": "bf16", "wdtype": "f32", "p": 0.0, "wide": False},
        # the same for a small microbatch of a ragged width
        {"name": "norm_grad_ragged", "op": "norm_grad", "rows": 517, "cols": 1023,
         "dtype": "f32", "wdtype": "f32", "p": 0.0, "wide": False},
        # gradient through norm, residual add and dropout
        {"name": "add_norm_grad", "op": "norm_grad", "rows": 8192, "cols": 4096,
         "dtype": "bf16", "wdtype": "bf16", "p": 0.1, "wide": False},
        # dropout of a small fp32 tensor of odd size, added to a residual
        {"name": "dropout_small", "op": "dropout", "n": 245761, "dtype": "f32", "p": 0.2,
         "residual": True},
        # dropout of a whole batch's feed-forward activations
        {"name": "dropout_large", "op": "dropout", "n": 16384 * 11008, "dtype": "bf16", "p": 0.1,
         "residual": False},
        # a short microbatch over 16 experts
        {"name": "route_small", "op": "route", "tokens": 96, "experts": 16, "k": 2,
         "dtype": "f32", "normalize": True, "masked": False},
        # 128 Ki tokens over 64 experts, padded tokens among them
        {"name": "route_large", "op": "route", "tokens": 131072, "experts": 64, "k": 6,
         "dtype": "bf16", "normalize": True, "masked": True},
        # gradient of a router over many experts, weights left unnormalised
        {"name": "route_grad", "op": "route_grad", "tokens": 65537, "experts": 160, "k": 8,
         "dtype": "f32", "normalize": False, "masked": True},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "norm_grad", "dropout", "route", "route_grad"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "dropout":
        return {"op": op, "n": _spread(rng, 1, 1 << 27 if dtype == "bf16" else 1 << 25),
                "dtype": dtype, "p": rng.choice([0.05, 0.1, 0.2, 0.5]),
                "residual": rng.random() < 0.5}
    if op in ("norm", "norm_grad"):
        cols = _spread(rng, 24, 16384)
        if rng.random() < 0.5 and cols > 64:
            cols -= cols % 64
        top = (1 << 26 if dtype == "bf16" else 1 << 24) // cols
        return {"op": op, "rows": _spread(rng, 1, min(top, 1 << 18)), "cols": cols, "dtype": dtype,
                "wdtype": rng.choice([dtype, "f32"]), "p": rng.choice([0.0, 0.0, 0.1, 0.25]),
                "wide": rng.random() < 0.2}
    experts = _spread(rng, 4, 512)
    if rng.random() < 0.5 and experts > 8:
        experts -= experts % 8
    return {"op": op, "tokens": _spread(rng, 1, min((1 << 24) // experts, 1 << 18)),
            "experts": experts, "k": rng.randint(1, min(8, experts)), "dtype": dtype,
            "normalize": rng.random() < 0.5, "masked": rng.random() < 0.5}


def work(case):
    if case["op"] == "dropout":
        es = DT[case["dtype"]].itemsize
        return {"bytes": case["n"] * es * (3 if case["residual"] else 2), "flops": 2 * case["n"]}
    if case["op"] in ("norm", "norm_grad"):
        es, ws = DT[case["dtype"]].itemsize, DT[case["wdtype"]].itemsize
        elems = case["rows"] * case["cols"]
        drop = case["p"] > 0
        if case["op"] == "norm":   # x -> y, or x and residual -> sum and y
            return {"bytes": elems * es * (4 if drop else 2) + 8 * case["rows"] + 2 * case["cols"] * ws,
                    "flops": 8 * elems}
        # dy, sum -> dx, or dy, sum and dsum -> dresidual and dx; weight -> dweight, dbias
        return {"bytes": elems * es * (5 if drop else 3) + 8 * case["rows"] + 3 * case["cols"] * ws,
                "flops": 14 * elems}
    es = DT[case["dtype"]].itemsize
    t, e, k = case["tokens"], case["experts"], case["k"]
    mask = t if case["masked"] else 0
    if case["op"] == "route":
        return {"bytes": t * e * es + 8 * t * k + mask + 8 * e, "flops": 5 * t * e}
    return {"bytes": 2 * t * e * es + 8 * t * k + mask + 4 * e, "flops": 8 * t * e}


# ---------------------------------------------------------------- inputs

def _rows(gen, rows, cols, dtype, wide, std=1.0):
    """Activations: normal values with a few loud channels, rows `cols` long;
    where `wide`, cut out of rows 8 elements longer."""
    ld = cols + 8 if wide else cols
    x = torch.randn(rows, ld, generator=gen, device="cuda") * std
    x[:, :: max(1, ld // 5)] *= 8.0
    x += 0.25 * std
    return x.to(dtype)[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DT[case["dtype"]]
    s = dict(case, seed=(seed * 0x9E3779B97F4A7C15 + 12345) % (1 << 63), offset=7 + seed % 1000)
    if case["op"] == "dropout":
        s["x"] = torch.randn(case["n"], generator=gen, device="cuda").to(dt)
        s["r"] = torch.randn(case["n"], generator=gen, device="cuda").to(dt) if case["residual"] else None
    elif case["op"] in ("norm", "norm_grad"):
        rows, cols, wdt = case["rows"], case["cols"], DT[case["wdtype"]]
        s["w"] = (1.0 + 0.2 * torch.randn(cols, generator=gen, device="cuda")).to(wdt)
        s["b"] = (0.1 * torch.randn(cols, generator=gen, device="cuda")).to(wdt)
        s["x"] = _rows(gen, rows, cols, dt, case["wide"])
        s["r"] = _rows(gen, rows, cols, dt, case["wide"], 2.0) if case["p"] > 0 else None
        if case["op"] == "norm_grad":
            f = _norm(s)   # what the forward pass left
            s["sum"] = f.get("sum", s["x"])
            s["mean"], s["rstd"] = f["mean"], f["rstd"]
            s["dy"] = (1e-2 * torch.randn(rows, cols, generator=gen, device="cuda")).to(dt)
            s["ds"] = (1e-2 * torch.randn(rows, cols, generator=gen, device="cuda")).to(dt) \
                if case["p"] > 0 else None
            del s["x"], s["r"]
    else:
        t, e = case["tokens"], case["experts"]
        lean = 0.7 * torch.randn(e, generator=gen, device="cuda")
        s["logits"] = (1.2 * torch.randn(t, e, generator=gen, device="cuda") + lean).to(dt)
        s["mask"] = None
        if case["masked"]:   # padded tokens hold whatever was there before
            s["mask"] = torch.rand(t, generator=gen, device="cuda") > 0.04
            s["logits"][~s["mask"]] = float("nan")
            s["logits"][torch.rand(t, generator=gen, device="cuda") < 0.01] = float("-inf")
            s["logits"][:, e // 2] = float("-inf")   # an expert taken out of service
        if case["op"] == "route_grad":
            f = _route(s)
            s["index"], s["counts"] = f["index"], f["counts"]
            s["dw"] = 1e-2 * torch.randn(t, case["k"], generator=gen, device="cuda")
            s["dloss"] = torch.rand((), generator=gen, device="cuda") + 0.5
    return s


# ---------------------------------------------------------------- plain forms

def _keep(n, p, seed, offset):
    """Keep flags of n elements and the factor of the kept ones: element i has
    half i % 8 of the Philox4x32-10 block numbered offset + i // 8."""
    low = 0xFFFFFFFF
    c = torch.arange(offset, offset + (n + 7) // 8, device="cuda", dtype=torch.int64)
    c0, c1, c2, c3 = c & low, (c >> 32) & low, torch.zeros_like(c), torch.zeros_like(c)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack((c0, c1, c2, c3), 1)
    halves = torch.stack((words & 0xFFFF, words >> 16), 2).reshape(-1)[:n]
    t = math.floor(p * 65536 + 0.5)
    return halves >= t, (65536.0 / (65536 - t) if t < 65536 else 0.0)


def _dropped(x, p, seed, offset):
    if p == 0:
        return x
    keep, scale = _keep(x.numel(), p, seed, offset)
    return torch.where(keep.view(x.shape), x * scale, 0.0)


def _dropout(s):
    y = _dropped(s["x"].float(), s["p"], s["seed"], s["offset"])
    return {"y": (y if s["r"] is None else s["r"].float() + y).to(s["x"].dtype)}


def _norm(s):
    dt = s["x"].dtype
    h = _dropped(s["x"].float(), s["p"], s["seed"], s["offset"])
    if s["r"] is not None:
        h = s["r"].float() + h
    mean = h.mean(1)
    d = h - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + EPS)
    out = {"y": (d * rstd[:, None] * s["w"].float() + s["b"].float()).to(dt), "mean": mean, "rstd": rstd}
    if s["r"] is not None:
        out["sum"] = h.to(dt)
    return out


def _norm_grad(s):
    dt, wdt = s["dy"].dtype, s["w"].dtype
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (s["sum"].float() - s["mean"][:, None]) * rstd
    g = dy * s["w"].float()
    d = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * rstd
    out = {"dweight": (dy * xh).sum(0).to(wdt), "dbias": dy.sum(0).to(wdt)}
    if s["ds"] is not None:
        d = d + s["ds"].float()
        out["dresidual"] = d.to(dt)
    out["dx"] = _dropped(d, s["p"], s["seed"], s["offset"]).to(dt)
    return out


def _softmax(s):
    """Probabilities of the routed tokens (zeros for the others), who is
    routed, and the logits with the others' rows set to zero."""
    l = s["logits"].float()
    valid = (l > float("-inf")).any(1)
    if s["mask"] is not None:
        valid = valid & s["mask"]
    l = torch.where(valid[:, None], l, 0.0)
    e = torch.exp(l - l.amax(1, keepdim=True))
    return torch.where(valid[:, None], e / e.sum(1, keepdim=True), 0.0), valid, l


def _route(s):
    p, valid, l = _softmax(s)
    e, k = s["experts"], s["k"]
    top, index = torch.sort(l, dim=1, descending=True, stable=True)
    top, index = top[:, :k], index[:, :k]
    ok = valid[:, None] & (top > float("-inf"))
    if s["normalize"]:
        w = torch.exp(top - top[:, :1])
        w = w / w.sum(1, keepdim=True)
    else:
        w = p.gather(1, index)
    counts = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    counts.scatter_add_(0, torch.where(ok, index, e).view(-1),
                        torch.ones(index.numel(), dtype=torch.int32, device="cuda"))
    n = valid.sum()
    counts[e] = n
    n = n.clamp(min=1).float()
    mean_prob = p.sum(0) / n
    loss = e * (counts[:e].float() / (k * n) * mean_prob).sum()
    return {"weights": torch.where(ok, w, 0.0), "index": torch.where(ok, index, -1).to(torch.int32),
            "counts": counts, "mean_prob": mean_prob, "loss": loss}


def _route_grad(s):
    p, valid, l = _softmax(s)
    e, k = s["experts"], s["k"]
    n = s["counts"][e].clamp(min=1).float()
    b = s["dloss"] * e * s["counts"][:e].float() / (k * n * n)
    ok = s["index"] >= 0
    at = torch.where(ok, s["index"], e).long()
    wide = torch.zeros(l.shape[0], e + 1, device="cuda")
    dw = torch.where(ok, s["dw"], 0.0)
    if s["normalize"]:
        w = torch.exp(l.gather(1, at.clamp(max=e - 1)) - l.amax(1, keepdim=True))
        w = torch.where(ok, w, 0.0)
        w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
        picked = wide.scatter(1, at, w * (dw - (w * dw).sum(1, keepdim=True)))[:, :e]
        g = p * (b - (p * b).sum(1, keepdim=True)) + picked
    else:
        b = b + wide.scatter(1, at, dw)[:, :e]
        g = p * (b - (p * b).sum(1, keepdim=True))
    return {"dlogits": torch.where(valid[:, None], g, 0.0).to(s["logits"].dtype)}


PLAIN = {"dropout": _dropout, "norm": _norm, "norm_grad": _norm_grad, "route": _route,
         "route_grad": _route_grad}


def run(s):
    if not own:
        return PLAIN[s["op"]](s)
    from newton_schulz_05_gb300 import layers
    drop = dict(p=s.get("p", 0.0), seed=s["seed"], offset=s["offset"])
    if s["op"] == "dropout":
        return {"y": layers.dropout_forward(s["x"], residual=s["r"], **drop)}
    if s["op"] == "norm":
        o = layers.layer_norm_forward(s["x"], s["w"], s["b"], eps=EPS, residual=s["r"], **drop)
        out = {"y": o.y, "mean": o.mean, "rstd": o.rstd}
        if s["r"] is not None:
            out["sum"] = o.sum
        return out
    if s["op"] == "norm_grad":
        o = layers.layer_norm_backward(s["dy"], s["sum"], s["mean"], s["rstd"], s["w"],
                                       dsum=s["ds"], **drop)
        out = {"dweight": o.dweight, "dbias": o.dbias, "dx": o.dx}
        if s["ds"] is not None:
            out["dresidual"] = o.dresidual
        return out
    if s["op"] == "route":
        o = layers.route_forward(s["logits"], s["k"], token_mask=s["mask"], normalize=s["normalize"])
        return {"weights": o.weights, "index": o.index, "counts": o.counts,
                "mean_prob": o.mean_prob, "loss": o.loss}
    return {"dlogits": layers.route_backward(s["logits"], s["index"], s["counts"], dweights=s["dw"],
                                             dloss=s["dloss"], token_mask=s["mask"],
                                             normalize=s["normalize"])}


# ---------------------------------------------------------------- 64 bits

def _factors64(n, p, seed, offset):
    """0 or the kept elements' factor, for n elements, on the host's integers."""
    u = np.uint64
    ctr = u(offset) + np.arange(-(-n // 8), dtype=np.uint64)
    x = [ctr & u(0xFFFFFFFF), ctr >> u(32), np.zeros_like(ctr), np.zeros_like(ctr)]
    key = [seed % 2 ** 32, seed // 2 ** 32]
    for r in range(10):
        lo, hi = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
        x = [(hi >> u(32)) ^ x[1] ^ u((key[0] + r * 0x9E3779B9) % 2 ** 32), hi & u(0xFFFFFFFF),
             (lo >> u(32)) ^ x[3] ^ u((key[1] + r * 0xBB67AE85) % 2 ** 32), lo & u(0xFFFFFFFF)]
    u16 = np.empty((ctr.size, 8), np.uint16)
    for j in range(4):
        u16[:, 2 * j], u16[:, 2 * j + 1] = x[j] & u(0xFFFF), x[j] >> u(16)
    t = int(math.floor(p * 2 ** 16 + 0.5))
    keep = torch.from_numpy(u16.reshape(-1)[:n] >= t).cuda()
    return keep.double() * (2 ** 16 / (2 ** 16 - t))


def exact(case, seed):
    s = prepare(case, seed)
    f64 = lambda t: t.to(torch.float64)  # noqa: E731
    if case["op"] == "dropout":
        y = _factors64(case["n"], case["p"], s["seed"], s["offset"]) * f64(s["x"])
        return {"y": y if s["r"] is None else y.add_(f64(s["r"]))}
    if case["op"] in ("norm", "norm_grad"):
        rows, cols, p = case["rows"], case["cols"], case["p"]
        drop = _factors64(rows * cols, p, s["seed"], s["offset"]).view(rows, cols) if p > 0 else None
        if case["op"] == "norm":
            h = f64(s["x"])
            if drop is not None:
                h = f64(s["r"]) + drop * h
            var, mean = torch.var_mean(h, dim=1, correction=0, keepdim=True)
            y = torch.addcmul(f64(s["b"]), (h - mean) / (var + EPS).sqrt(), f64(s["w"]))
            out = {"y": y, "mean": mean[:, 0], "rstd": (var[:, 0] + EPS) ** -0.5}
            return out if drop is None else dict(out, sum=h)
        # project g = dy w off the constant and off the normed row, then scale
        norm = (f64(s["sum"]) - f64(s["mean"])[:, None]) * f64(s["rstd"])[:, None]
        dy = f64(s["dy"])
        g = dy * f64(s["w"])
        one = g.new_ones(cols, 1)
        dx = g - (g @ one) / cols - norm * (torch.einsum("rc,rc->r", g, norm)[:, None] / cols)
        dx = dx * f64(s["rstd"])[:, None]
        out = {"dweight": torch.einsum("rc,rc->c", dy, norm), "dbias": dy.sum(0)}
        if drop is None:
            return dict(out, dx=dx)
        dx = dx + f64(s["ds"])
        return dict(out, dresidual=dx, dx=dx * drop)
    # the router: by automatic differentiation of the definition
    e, k = case["experts"], case["k"]
    live = torch.ones(case["tokens"], dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    live = live & ~torch.isneginf(s["logits"]).all(1)
    l = torch.where(live[:, None], f64(s["logits"]), 0.0).requires_grad_()
    p = torch.softmax(l, 1) * live[:, None]
    n = max(1, int(live.sum()))
    index = s["index"].long() if case["op"] == "route_grad" else \
        torch.argsort(l.detach(), dim=1, descending=True, stable=True)[:, :k]
    ok = live[:, None] & (index >= 0)
    at = index.clamp(min=0)
    ok = ok & ~torch.isneginf(l.detach().gather(1, at))
    picked = l.gather(1, at)
    if case["normalize"]:
        w = torch.softmax(torch.where(ok, picked, -1e300), 1) * ok
    else:
        w = p.gather(1, at) * ok
    counts = f64(torch.bincount(at[ok], minlength=e))
    mean_prob = p.sum(0) / n
    loss = e * torch.dot(counts / (k * n), mean_prob)
    if case["op"] == "route":
        return {"weights": w.detach(), "index": None, "counts": None, "mean_prob": mean_prob.detach(),
                "loss": loss.detach()}
    ((w * f64(s["dw"])).sum() + loss * f64(s["dloss"])).backward()
    return {"dlogits": l.grad}
