"""Measured cases of the training operators for sequences: the gated linear
recurrence, norms of query and key heads with the rotation of positions, log
probabilities of given tokens over a vocabulary, and the clipped policy loss on
them, each forward and backward.

`run` computes a case either in elementary torch operations in 32 bits
(`own` false) or through newton_schulz_05_gb300.layers (`own` true).

Sizes: 2048, 4096 and 1409 are the widths (and a ragged neighbour of one) of the
parameter sets in synth/; heads of 128 and 80 elements, vocabularies of 2^17 and
50021 and the lengths are generic.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
CLIP_LOW, CLIP_HIGH, KL = 0.2, 0.28, 0.04
SCALE = 0.8


def listed():
    return [
        # one new token of 48 sequences that are being generated: the state steps once
        {"name": "scan_token", "op": "scan", "batch": 48, "length": 1, "dim": 2048, "dtype": "bf16",
         "mix": True, "state": True, "starts": False, "masked": False, "wide": True},
        # one very long document, few channels
        {"name": "scan_long", "op": "scan", "batch": 1, "length": 65536, "dim": 2048, "dtype": "bf16",
         "mix": True, "state": False, "starts": False, "masked": False, "wide": True},
        # packed documents and padding, fp32, a ragged width
        {"name": "scan_packed", "op": "scan", "batch": 3, "length": 2047, "dim": 1409, "dtype": "f32",
         "mix": False, "state": True, "starts": True, "masked": True, "wide": False},
        # gradient over a training batch of packed documents
        {"name": "scan_grad", "op": "scan_grad", "batch": 8, "length": 4096, "dim": 4096, "dtype": "bf16",
         "mix": True, "state": False, "starts": True, "masked": False, "wide": False},
        # queries and keys of one new token of 32 sequences, at far positions
        {"name": "heads_token", "op": "heads", "tokens": 32, "q_heads": 32, "k_heads": 8, "dim": 128,
         "rotary": 128, "dtype": "bf16", "wdtype": "bf16", "neighbours": False, "table": 131072},
        # a training batch, queries and keys inside the projections' joint output
        {"name": "heads_batch", "op": "heads", "tokens": 32768, "q_heads": 32, "k_heads": 8, "dim": 128,
         "rotary": 128, "dtype": "bf16", "wdtype": "f32", "neighbours": False, "table": 8192},
        # gradient in fp32: as many keys as queries, half of each head rotated, neighbours paired
        {"name": "heads_grad", "op": "heads_grad", "tokens": 8191, "q_heads": 12, "k_heads": 12, "dim": 80,
         "rotary": 40, "dtype": "f32", "wdtype": "f32", "neighbours": True, "table": 4096},
        # a small batch, fp32 logits over a vocabulary of odd size, some tokens ignored
        {"name": "log_probs_odd", "op": "log_probs", "tokens": 509, "vocab": 50021, "dtype": "f32",
         "ignored": True},
        # a training batch over a large vocabulary
        {"name": "log_probs_batch", "op": "log_probs", "tokens": 8192, "vocab": 131072, "dtype": "bf16",
         "ignored": False},
        # its gradient; prompt tokens have none
        {"name": "log_probs_grad", "op": "log_probs_grad", "tokens": 8192, "vocab": 131072, "dtype": "bf16",
         "ignored": False},
        # loss of a small batch of answers, one advantage an answer, mean over each answer
        {"name": "policy_small", "op": "policy", "batch": 64, "length": 513, "each_token": False,
         "ref": True, "masked": True, "by_sequence": True},
        # gradient over a large batch with an advantage for each token
        {"name": "policy_grad", "op": "policy_grad", "batch": 2048, "length": 8192, "each_token": True,
         "ref": True, "masked": True, "by_sequence": False},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_grad", "scan_grad", "heads", "heads_grad", "log_probs",
                     "log_probs_grad", "policy", "policy_grad"])
    dtype = rng.choice(["bf16", "f32"])
    if op in ("scan", "scan_grad"):
        dim = _spread(rng, 64, 8192)
        if rng.random() < 0.6:
            dim = max(64, dim - dim % 64)
        top = (1 << 26 if dtype == "bf16" else 1 << 25) // dim
        length = 1 if op == "scan" and rng.random() < 0.2 else _spread(rng, 2, min(top, 65536))
        return {"op": op, "batch": _spread(rng, 1, max(1, min(256, top // length))), "length": length,
                "dim": dim, "dtype": dtype, "mix": rng.random() < 0.6, "state": rng.random() < 0.5,
                "starts": rng.random() < 0.4, "masked": rng.random() < 0.3, "wide": rng.random() < 0.3}
    if op in ("heads", "heads_grad"):
        dim = rng.choice([32, 64, 64, 80, 96, 128, 128, 128, 192, 256])
        k = rng.choice([1, 2, 4, 8, 16])
        q = k * rng.choice([1, 2, 4, 8]) if k < 16 else k
        top = (1 << 26 if dtype == "bf16" else 1 << 25) // (dim * (q + k))
        return {"op": op, "tokens": _spread(rng, 1, min(top, 65536)), "q_heads": q, "k_heads": k, "dim": dim,
                "rotary": rng.choice([dim, dim, dim // 2]), "dtype": dtype,
                "wdtype": rng.choice([dtype, "f32"]), "neighbours": rng.random() < 0.3,
                "table": rng.choice([2048, 8192, 131072])}
    if op in ("log_probs", "log_probs_grad"):
        vocab = _spread(rng, 256, 1 << 18)
        if rng.random() < 0.6:
            vocab -= vocab % 64
        top = (1 << 28 if dtype == "bf16" else 1 << 27) // vocab
        return {"op": op, "tokens": _spread(rng, 1, min(top, 65536)), "vocab": vocab, "dtype": dtype,
                "ignored": rng.random() < 0.3}
    batch = _spread(rng, 1, 4096)
    return {"op": op, "batch": batch, "length": _spread(rng, 1, min(32768, (1 << 24) // batch)),
            "each_token": rng.random() < 0.5, "ref": rng.random() < 0.6, "masked": rng.random() < 0.8,
            "by_sequence": rng.random() < 0.5}


def work(case):
    op = case["op"]
    if op in ("scan", "scan_grad"):
        rows, es = case["batch"] * case["length"], DT[case["dtype"]].itemsize
        n = rows * case["dim"]
        flags = rows * (case["starts"] + case["masked"])
        state = 4 * case["batch"] * case["dim"]     # the last state, and the first where there is one
        if op == "scan":
            return {"bytes": 3 * n * es + flags + state * (1 + case["state"]), "flops": 10 * n}
        return {"bytes": 6 * n * es + flags + state * (1 + 2 * case["state"]), "flops": 18 * n}
    if op in ("heads", "heads_grad"):
        es, ws = DT[case["dtype"]].itemsize, DT[case["wdtype"]].itemsize
        n = case["tokens"] * (case["q_heads"] + case["k_heads"]) * case["dim"]
        turns = min(case["tokens"], case["table"]) * case["rotary"] * 4 + 8 * case["tokens"]
        if op == "heads":
            return {"bytes": 2 * n * es + turns + 2 * case["dim"] * ws, "flops": 7 * n}
        return {"bytes": 3 * n * es + turns + 4 * case["dim"] * ws, "flops": 14 * n}
    if op in ("log_probs", "log_probs_grad"):
        t, es = case["tokens"], DT[case["dtype"]].itemsize
        live = t * 0.75 if case["ignored"] else t
        if op == "log_probs":
            return {"bytes": int(live * case["vocab"]) * es + 16 * t, "flops": int(4 * live * case["vocab"])}
        # the gradient of a token without one is written but nothing of it read
        live = t * (0.5625 if case["ignored"] else 0.75)
        return {"bytes": int((live + t) * case["vocab"]) * es + 16 * t,
                "flops": int(4 * live * case["vocab"])}
    n, b = case["batch"] * case["length"], case["batch"]
    read = n * (8 + 4 * case["ref"] + case["masked"]) + 4 * (n if case["each_token"] else b)
    if op == "policy":
        return {"bytes": read + 4 * b + 12, "flops": 12 * n}
    return {"bytes": read + 4 * n + 4 * b, "flops": 10 * n}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def chance(p, *shape):
        return torch.rand(*shape, generator=gen, device="cuda") < p

    op = case["op"]
    if op in ("scan", "scan_grad"):
        b, t, d, dt = case["batch"], case["length"], case["dim"], DT[case["dtype"]]
        # gates lean towards keeping, channels differ; where `wide`, gate and x are
        # the two halves of one projection's output
        gate = 1.5 * normal(b, t, d) + (1.0 + 1.5 * normal(d))
        x = normal(b, t, d)
        if case["wide"]:
            both = torch.cat((gate, x), 2).to(dt)
            s["gate"], s["x"] = both[..., :d], both[..., d:]
        else:
            s["gate"], s["x"] = gate.to(dt), x.to(dt)
        s["h0"] = normal(b, d) if case["state"] else None
        s["first"] = chance(1 / 300, b, t) if case["starts"] else None
        s["mask"] = None
        if case["masked"]:      # padding holds whatever was there before
            s["mask"] = ~chance(0.06, b, t)
            s["gate"][~s["mask"]] = float("nan")
            s["x"][~s["mask"]] = float("nan")
        if op == "scan_grad":
            s["h"] = _scan(s)["h"]
            s["dh"] = (1e-2 * normal(b, t, d)).to(dt)
            s["dstate"] = 1e-2 * normal(b, d)
    elif op in ("heads", "heads_grad"):
        t, q, k, d, dt = case["tokens"], case["q_heads"], case["k_heads"], case["dim"], DT[case["dtype"]]
        joint = normal(t, q + 2 * k, d)     # queries, keys and values of one projection
        joint[..., :: max(1, d // 3)] *= 6.0
        joint = joint.to(dt)
        s["q"], s["k"] = joint[:, :q], joint[:, q:q + k]
        s["wq"], s["wk"] = ((1.0 + 0.2 * normal(d)).to(DT[case["wdtype"]]) for _ in range(2))
        rate = 10000.0 ** (-torch.arange(0, case["rotary"], 2, device="cuda", dtype=torch.float64)
                           / case["rotary"])
        angle = torch.arange(case["table"], device="cuda", dtype=torch.float64)[:, None] * rate
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        start = torch.randint(0, case["table"], (1,), generator=gen, device="cuda")
        s["pos"] = (start + torch.arange(t, device="cuda")) % case["table"]
        if t <= 64:
            s["pos"] = torch.randint(0, case["table"], (t,), generator=gen, device="cuda")
        if op == "heads_grad":
            s["dq"], s["dk"] = ((1e-2 * normal(t, h, d)).to(dt) for h in (q, k))
    elif op in ("log_probs", "log_probs_grad"):
        t, v = case["tokens"], case["vocab"]
        logits = 2.0 * normal(t, v)
        s["tokens"] = torch.randint(0, v, (t,), generator=gen, device="cuda")
        # a sampled token is a likely one: raised above the others
        logits[torch.arange(t, device="cuda"), s["tokens"]] += 12.0 * torch.rand(t, generator=gen, device="cuda")
        logits[:, v // 3] = float("-inf")      # a symbol that is never allowed
        s["logits"] = logits.to(DT[case["dtype"]])
        del logits
        s["tokens"] = torch.where(s["tokens"] == v // 3, 0, s["tokens"])
        if case["ignored"]:
            s["tokens"][chance(0.25, t)] = -100
        if op == "log_probs_grad":
            s["lse"] = _log_probs(s)["lse"]
            s["dlp"] = torch.where(chance(0.25, t), 0.0, 1e-2 * normal(t))
    else:
        b, t = case["batch"], case["length"]
        s["lp"] = -3.0 * torch.rand(b, t, generator=gen, device="cuda") ** 2
        s["old"] = s["lp"] + 0.15 * normal(b, t)
        s["ref"] = s["lp"] + 0.3 * normal(b, t) if case["ref"] else None
        s["adv"] = normal(b, t) if case["each_token"] else normal(b)
        s["mask"] = None
        if case["masked"]:      # answers of different lengths, some of them empty
            ends = torch.randint(0, t + 1, (b,), generator=gen, device="cuda")
            s["mask"] = torch.arange(t, device="cuda") < ends[:, None]
            s["lp"][~s["mask"]] = float("nan")
            s["old"][~s["mask"]] = float("inf")
        if op == "policy_grad":
            s["weights"] = _policy(s)["weights"]
            s["dloss"] = torch.rand((), generator=gen, device="cuda") + 0.5
    return s


# ---------------------------------------------------------------- plain forms

def _gates(s):
    """Shares of the state before and of the input, as the tokens' flags have them,
    and the inputs without what masked tokens hold."""
    g, x = s["gate"].float(), s["x"].float()
    if s["mask"] is not None:
        m = s["mask"][..., None]
        g, x = torch.where(m, g, 0.0), torch.where(m, x, 0.0)
    keep = 1.0 / (1.0 + torch.exp(-g))
    take = 1.0 / (1.0 + torch.exp(g)) if s["mix"] else torch.ones_like(g)
    carried = keep
    if s["first"] is not None:
        carried = torch.where(s["first"][..., None], 0.0, carried)
    if s["mask"] is not None:
        carried = torch.where(m, carried, 1.0)
        take = torch.where(m, take, 0.0)
    return g, x, carried, take


def _recur(a, b):
    """All y_t = a_t y_{t-1} + b_t along dimension 1, by doubling."""
    step = 1
    while step < a.shape[1]:
        b = torch.cat((b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]), 1)
        a = torch.cat((a[:, :step], a[:, step:] * a[:, :-step]), 1)
        step *= 2
    return b


def _scan(s):
    _, x, a, u = _gates(s)
    b = u * x
    if s["h0"] is not None:
        b[:, 0] += a[:, 0] * s["h0"]
    h = _recur(a, b)
    return {"h": h.to(s["x"].dtype), "state": h[:, -1].clone()}


def _scan_grad(s):
    dt = s["x"].dtype
    g, x, a, u = _gates(s)
    dh = s["dh"].float()
    dh[:, -1] += s["dstate"]
    later = torch.cat((a[:, 1:], torch.zeros_like(a[:, :1])), 1)
    l = _recur(later.flip(1), dh.flip(1)).flip(1)
    h0 = torch.zeros_like(s["dstate"]) if s["h0"] is None else s["h0"]
    before = torch.cat((h0[:, None], s["h"][:, :-1].float()), 1)
    if s["first"] is not None:
        before = torch.where(s["first"][..., None], 0.0, before)
    slope = 1.0 / ((1.0 + torch.exp(-g)) * (1.0 + torch.exp(g)))
    dgate = slope * l * (before - x if s["mix"] else before)
    if s["mask"] is not None:
        dgate = torch.where(s["mask"][..., None], dgate, 0.0)
    out = {"dgate": dgate.to(dt), "dx": (u * l).to(dt)}
    if s["h0"] is not None:
        out["dstate"] = a[:, 0] * l[:, 0]
    return out


def _turn(s, n, back):
    """Heads [tokens, heads, dim] turned by their positions' angles, or back."""
    r = s["rotary"]
    c, i = s["cos"][s["pos"]][:, None], s["sin"][s["pos"]][:, None]
    if back:
        i = -i
    if s["neighbours"]:
        u, v = n[..., 0:r:2], n[..., 1:r:2]
        turned = torch.stack((u * c - v * i, v * c + u * i), -1).flatten(-2)
    else:
        u, v = n[..., :r // 2], n[..., r // 2:r]
        turned = torch.cat((u * c - v * i, v * c + u * i), -1)
    return torch.cat((turned, n[..., r:]), -1)


def _heads(s):
    def one(x, w):
        y = x.float()
        y = y * (1.0 / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS)) * w.float()
        return _turn(s, y, False).to(x.dtype)

    return {"q": one(s["q"], s["wq"]), "k": one(s["k"], s["wk"])}


def _heads_grad(s):
    def one(dy, x, w):
        y = x.float()
        rstd = 1.0 / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS)
        y = y * rstd
        g = _turn(s, dy.float(), True)
        dw = (g * y).sum((0, 1)).to(w.dtype)
        g = g * w.float()
        return ((g - y * (g * y).mean(-1, keepdim=True)) * rstd).to(x.dtype), dw

    (dq, dwq), (dk, dwk) = one(s["dq"], s["q"], s["wq"]), one(s["dk"], s["k"], s["wk"])
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def _log_probs(s):
    l, y = s["logits"].float() * SCALE, s["tokens"]
    live = (y >= 0) & (y < s["vocab"])
    top = l.amax(1)
    rest = torch.log(torch.exp(l - top[:, None]).sum(1))
    at = l.gather(1, torch.where(live, y, 0)[:, None])[:, 0]
    return {"log_probs": torch.where(live, at - top - rest, 0.0),
            "lse": torch.where(live, top + rest, 0.0)}


def _log_probs_grad(s):
    l, y = s["logits"].float() * SCALE, s["tokens"]
    live = (y >= 0) & (y < s["vocab"])
    g = torch.where(live, s["dlp"], 0.0)
    p = torch.exp(l - s["lse"][:, None])
    p = torch.where((g != 0)[:, None], p, 0.0)
    p.scatter_add_(1, torch.where(live, y, 0)[:, None], torch.full_like(g, -1.0)[:, None])
    return {"dlogits": (p * (-SCALE * g)[:, None]).to(s["logits"].dtype)}


def _policy_terms(s):
    """Ratios, whether each is cut off, advantages, how far the reference is, and
    the mask; masked tokens count as unchanged ones."""
    lp, old, mask = s["lp"], s["old"], s["mask"]
    ref = lp if s["ref"] is None else s["ref"]
    adv = s["adv"] if s["adv"].dim() == 2 else s["adv"][:, None].expand_as(lp)
    if mask is None:
        mask = torch.ones_like(lp, dtype=torch.bool)
    lp, old, ref = (torch.where(mask, v, 0.0) for v in (lp, old, ref))
    d = lp.double() - old.double()      # next to a border the last bit decides
    cut = torch.where(adv >= 0, d > math.log1p(CLIP_HIGH), d < math.log1p(-CLIP_LOW))
    return torch.exp(d.float()), cut & mask, adv, (ref.double() - lp.double()), mask


def _policy(s):
    r, cut, adv, x, mask = _policy_terms(s)
    bound = torch.where(adv >= 0, 1.0 + CLIP_HIGH, 1.0 - CLIP_LOW)
    kl = (torch.expm1(x) - x).float()      # the difference of near numbers, taken in 64 bits
    each = KL * kl - torch.where(cut, bound, r) * adv
    each, kl = torch.where(mask, each, 0.0), torch.where(mask, kl, 0.0)
    n = mask.sum(1)
    if s["by_sequence"]:
        w = torch.where(n > 0, 1.0 / (n.clamp(min=1).float() * (n > 0).sum().clamp(min=1).float()), 0.0)
    else:
        w = torch.where(n > 0, 1.0 / n.sum().clamp(min=1).float(), 0.0)
    return {"loss": (w * each.sum(1)).sum(), "kl": (w * kl.sum(1)).sum(),
            "clipped": (w * cut.sum(1).float()).sum(), "weights": w}


def _policy_grad(s):
    r, cut, adv, x, mask = _policy_terms(s)
    g = torch.where(cut, 0.0, -r * adv) - KL * torch.expm1(x).float()
    return {"dlog_probs": torch.where(mask, s["dloss"] * s["weights"][:, None] * g, 0.0)}


PLAIN = {"scan": _scan, "scan_grad": _scan_grad, "heads": _heads, "heads_grad": _heads_grad,
         "log_probs": _log_probs, "log_probs_grad": _log_probs_grad, "policy": _policy,
         "policy_grad": _policy_grad}


def run(s):
    if not own:
        return PLAIN[s["op"]](s)
    from newton_schulz_05_gb300 import layers
    op = s["op"]
    if op == "scan":
        o = layers.gated_scan_forward(s["gate"], s["x"], state=s["h0"], starts=s["first"],
                                      token_mask=s["mask"], mix=s["mix"])
        return {"h": o.h, "state": o.state}
    if op == "scan_grad":
        o = layers.gated_scan_backward(s["dh"], s["gate"], s["x"], s["h"], state=s["h0"],
                                       dstate=s["dstate"], starts=s["first"], token_mask=s["mask"],
                                       mix=s["mix"])
        out = {"dgate": o.dgate, "dx": o.dx}
        if s["h0"] is not None:
            out["dstate"] = o.dstate
        return out
    turn = dict(cos=s.get("cos"), sin=s.get("sin"), positions=s.get("pos"), eps=EPS,
                neighbours=s.get("neighbours"))
    if op == "heads":
        o = layers.norm_rotate_heads_forward(s["q"], s["k"], s["wq"], s["wk"], **turn)
        return {"q": o.q, "k": o.k}
    if op == "heads_grad":
        o = layers.norm_rotate_heads_backward(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], **turn)
        return {"dq": o.dq, "dk": o.dk, "dwq": o.dq_weight, "dwk": o.dk_weight}
    if op == "log_probs":
        o = layers.token_log_probs_forward(s["logits"], s["tokens"], scale=SCALE)
        return {"log_probs": o.log_probs, "lse": o.lse}
    if op == "log_probs_grad":
        return {"dlogits": layers.token_log_probs_backward(s["dlp"], s["logits"], s["tokens"], s["lse"],
                                                           scale=SCALE)}
    loss = dict(ref_log_probs=s["ref"], token_mask=s["mask"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl=KL)
    if op == "policy":
        o = layers.policy_loss_forward(s["lp"], s["old"], s["adv"], by_sequence=s["by_sequence"], **loss)
        return {"loss": o.loss, "kl": o.kl, "clipped": o.clipped, "weights": o.weights}
    return {"dlog_probs": layers.policy_loss_backward(s["lp"], s["old"], s["adv"], s["weights"],
                                                      dloss=s["dloss"], **loss)}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f64 = lambda t: t.to(torch.float64)  # noqa: E731
    op = case["op"]
    if op in ("scan", "scan_grad"):     # one token after the other
        b, t, d = case["batch"], case["length"], case["dim"]
        live = torch.ones(b, t, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
        cut = torch.zeros_like(live) if s["first"] is None else s["first"]
        state = torch.zeros(b, d, dtype=torch.float64, device="cuda") if s["h0"] is None else f64(s["h0"])
        if op == "scan":
            h = torch.empty(b, t, d, dtype=torch.float64, device="cuda")
            for i in range(t):
                a = torch.sigmoid(f64(s["gate"][:, i]))
                new = a * torch.where(cut[:, i, None], 0.0, state)
                new = new + ((1 - a) if case["mix"] else 1.0) * f64(s["x"][:, i])
                state = torch.where(live[:, i, None], new, state)
                h[:, i] = state
            return {"h": h, "state": state}
        later = f64(s["dstate"])            # what reaches the state behind token i
        dgate = torch.zeros(b, t, d, dtype=torch.float64, device="cuda")
        dx = torch.zeros_like(dgate)
        for i in reversed(range(t)):
            a = torch.sigmoid(f64(s["gate"][:, i]))
            total = later + f64(s["dh"][:, i])
            x, here, begin = f64(s["x"][:, i]), live[:, i, None], cut[:, i, None]
            prev = torch.where(begin, 0.0, f64(s["h"][:, i - 1]) if i else state)
            dgate[:, i] = torch.where(here, a * (1 - a) * total * (prev - x if case["mix"] else prev), 0.0)
            dx[:, i] = torch.where(here, total * (1 - a) if case["mix"] else total, 0.0)
            later = torch.where(here, torch.where(begin, 0.0, a * total), total)
        out = {"dgate": dgate, "dx": dx}
        return dict(out, dstate=later) if case["state"] else out
    if op in ("heads", "heads_grad"):
        # pairs as complex numbers
        r = case["rotary"]
        unit = torch.complex(f64(s["cos"]), f64(s["sin"]))[s["pos"]][:, None]

        def forward(x, w):
            y = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w
            if case["neighbours"]:
                z = torch.view_as_complex(y[..., :r].unflatten(-1, (r // 2, 2)).contiguous()) * unit
                z = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(y[..., :r // 2], y[..., r // 2:r]) * unit
                z = torch.cat((z.real, z.imag), -1)
            return torch.cat((z, y[..., r:]), -1)

        if op == "heads":
            return {n: forward(f64(s[n]), f64(s["w" + n])) for n in ("q", "k")}
        out = {}
        for n in ("q", "k"):
            x, w = f64(s[n]).requires_grad_(), f64(s["w" + n]).requires_grad_()
            out["d" + n], out["dw" + n] = torch.autograd.grad(forward(x, w), (x, w), f64(s["d" + n]))
        return out
    if op in ("log_probs", "log_probs_grad"):
        v, y = case["vocab"], s["tokens"]
        live = (y >= 0) & (y < v)
        lp, lse = torch.zeros(len(y), dtype=torch.float64, device="cuda"), None
        lse = torch.zeros_like(lp)
        grad = op == "log_probs_grad"
        out = torch.empty(len(y), v, dtype=torch.float64, device="cuda") if grad else None
        rows = max(1, (1 << 27) // v)
        for i in range(0, len(y), rows):
            l = f64(s["logits"][i:i + rows]) * SCALE
            at = y[i:i + rows].clamp(0, v - 1)[:, None]
            if not grad:
                lse[i:i + rows] = torch.logsumexp(l, 1)
                lp[i:i + rows] = l.gather(1, at)[:, 0] - lse[i:i + rows]
                continue
            p = torch.exp(l - f64(s["lse"][i:i + rows])[:, None])
            g = SCALE * torch.where(live[i:i + rows], f64(s["dlp"][i:i + rows]), 0.0)[:, None]
            p = torch.where(g == 0, 0.0, p * -g)
            out[i:i + rows] = p.scatter_add(1, at, g)
        if grad:
            return {"dlogits": out}
        return {"log_probs": torch.where(live, lp, 0.0), "lse": torch.where(live, lse, 0.0)}
    mask = torch.ones_like(s["lp"], dtype=torch.bool) if s["mask"] is None else s["mask"]
    lp = torch.where(mask, f64(s["lp"]), 0.0).requires_grad_()
    old = torch.where(mask, f64(s["old"]), 0.0)
    adv = f64(s["adv"]).reshape(case["batch"], -1)
    r = (lp - old).exp()
    # min(r A, clip(r) A); past the border nothing depends on r
    cut = torch.where(adv >= 0, r.detach().log() > math.log1p(CLIP_HIGH),
                      r.detach().log() < math.log1p(-CLIP_LOW)) & mask
    each = -torch.where(cut, r.detach().clamp(1 - CLIP_LOW, 1 + CLIP_HIGH), r) * adv
    kl = torch.zeros_like(each)
    if s["ref"] is not None:
        x = torch.where(mask, f64(s["ref"]), 0.0) - lp
        kl = x.expm1() - x
    each = (each + KL * kl) * mask
    n = f64(mask.sum(1))
    if op == "policy":
        w = 1 / (n * (n > 0).sum()) if case["by_sequence"] else torch.ones_like(n) / n.sum()
        w = torch.where(n > 0, w, 0.0)
        mean = lambda z: (z * mask).sum(1).mul(w).sum().detach()  # noqa: E731
        return {"loss": mean(each), "kl": mean(kl), "clipped": mean(f64(cut)), "weights": w}
    total = (each.sum(1) * f64(s["weights"])).sum() * f64(s["dloss"])
    return {"dlog_probs": torch.autograd.grad(total, lp)[0] * mask}
