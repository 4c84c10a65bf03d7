"""Norms of query and key heads with the rotation of positions, and the
gradient, against 64-bit formulas."""
import numpy as np
import pytest
import torch

import sequence_ref as ref
from helpers import muon

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module")
def layers():
    muon()
    from newton_schulz_05_gb300 import layers
    return layers


def inputs(layers, t, qh, kh, d, rotary, dtype, wdtype=F32, table=50, seed=0, layout="joint", weights=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    if layout == "joint":          # queries, keys and values of one projection
        joint = (n(t, qh + 2 * kh, d) * (1 + 3 * torch.rand(t, 1, 1, generator=gen, device="cuda"))).to(dtype)
        q, k = joint[:, :qh], joint[:, qh:qh + kh]
    elif layout == "odd":          # at an odd address, heads and tokens apart
        wide = n(t, qh + kh, d + 3).to(dtype)
        q, k = wide[:, :qh, 1:d + 1], wide[:, qh:, 2:d + 2]
    elif layout == "heads first":  # [heads, tokens, dim] seen as tokens
        q, k = (n(h, t, d).to(dtype).transpose(0, 1) for h in (qh, kh))
    else:
        q, k = n(t, qh, d).to(dtype), n(t, kh, d).to(dtype)
    wq, wk = ((1 + 0.3 * n(d)).to(wdtype) if weights else None for _ in range(2))
    cos = sin = None
    if rotary:
        cos, sin = layers.rotation_table(table, rotary, base=100.0)
    pos = torch.randint(0, table, (t,), generator=gen, device="cuda")
    return q, k, wq, wk, dict(cos=cos, sin=sin, positions=pos), n


def want(q, k, wq, wk, how, neighbours, dq=None, dk=None):
    c = {n: None if how[n] is None else ref.f64(how[n]) for n in ("cos", "sin")}
    pos = how["positions"].cpu().numpy()
    f = lambda t: None if t is None else ref.f64(t)  # noqa: E731
    if dq is None:
        return [ref.heads(f(x), f(w), c["cos"], c["sin"], pos, EPS, neighbours) for x, w in ((q, wq), (k, wk))]
    return [ref.heads_grad(f(g), f(x), f(w), c["cos"], c["sin"], pos, EPS, neighbours)
            for g, x, w in ((dq, q, wq), (dk, k, wk))]


def check(layers, q, k, wq, wk, how, n, neighbours, dtype, wdtype):
    o = layers.norm_rotate_heads_forward(q, k, wq, wk, eps=EPS, neighbours=neighbours, **how)
    for got, (y, err) in zip(o, want(q, k, wq, wk, how, neighbours)):
        ref.close(got, y, err, dtype)
    dq, dk = n(*q.shape).to(dtype), n(*k.shape).to(dtype)
    g = layers.norm_rotate_heads_backward(dq, dk, q, k, wq, wk, eps=EPS, neighbours=neighbours, **how)
    for dx, dw, ((ex, ew), (rx, rw)) in zip(g[:2], g[2:], want(q, k, wq, wk, how, neighbours, dq, dk)):
        ref.close(dx, ex, rx, dtype)
        ref.close(dw, ew, rw, wdtype)


@pytest.mark.parametrize("dtype,wdtype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("t,qh,kh,d,rotary", [
    (1, 1, 1, 128, 128), (1, 32, 8, 128, 128), (7, 4, 2, 64, 64), (33, 8, 1, 64, 32), (5, 3, 3, 80, 40),
    (9, 6, 2, 96, 96), (3, 16, 16, 256, 256), (4, 2, 1, 192, 64), (6, 2, 2, 16, 16), (5, 1, 2, 32, 16),
    (11, 2, 1, 8, 8), (3, 2, 1, 512, 512), (2, 1, 1, 1024, 1024), (2, 2, 1, 1000, 500), (700, 4, 2, 128, 128),
    (3, 40, 40, 64, 64)])
def test_heads_and_gradient(layers, t, qh, kh, d, rotary, neighbours, dtype, wdtype):
    q, k, wq, wk, how, n = inputs(layers, t, qh, kh, d, rotary, dtype, wdtype)
    check(layers, q, k, wq, wk, how, n, neighbours, dtype, wdtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["dense", "odd", "heads first"])
@pytest.mark.parametrize("d,rotary", [(128, 128), (64, 0), (1, 0), (2, 2), (7, 6), (34, 34), (65, 10), (100, 4),
                                      (72, 36), (104, 24), (1023, 1022), (24, 24)])
def test_odd_widths_and_strides(layers, d, rotary, layout, dtype):
    for neighbours in (False, True):
        q, k, wq, wk, how, n = inputs(layers, 21, 3, 2, d, rotary, dtype, layout=layout, seed=d)
        check(layers, q, k, wq, wk, how, n, neighbours, dtype, F32)


@pytest.mark.parametrize("d,rotary", [(128, 128), (33, 8)])
def test_positions_outside_of_the_table_are_no_tokens(layers, d, rotary):
    q, k, wq, wk, how, n = inputs(layers, 12, 3, 2, d, rotary, F32, table=9)
    bad = torch.tensor([0, 5, 6, 11], device="cuda")
    how["positions"][bad] = torch.tensor([-1, 9, -2 ** 62, 2 ** 62], device="cuda")
    q[bad] = float("nan")
    k[bad] = float("inf")
    o = layers.norm_rotate_heads_forward(q, k, wq, wk, eps=EPS, **how)
    assert not o.q[bad].any() and not o.k[bad].any() and bool(o.q.isfinite().all())
    dq, dk = n(*q.shape), n(*k.shape)
    dq[bad] = float("nan")
    g = layers.norm_rotate_heads_backward(dq, dk, q, k, wq, wk, eps=EPS, **how)
    assert not g.dq[bad].any() and not g.dk[bad].any()
    keep = torch.ones(12, dtype=torch.bool, device="cuda")
    keep[bad] = False
    how2 = dict(how, positions=how["positions"][keep])
    for dx, dw, ((ex, ew), (rx, rw)) in zip(g[:2], g[2:], want(q[keep], k[keep], wq, wk, how2, False, dq[keep],
                                                               dk[keep])):
        ref.close(dx[keep], ex, rx, F32)
        ref.close(dw, ew, rw, F32)
    # an empty table: nothing is a token; a table is not needed where nothing is turned
    none = dict(cos=how["cos"][:0], sin=how["sin"][:0], positions=how["positions"])
    assert not layers.norm_rotate_heads_forward(q, k, **none).q.any()


def test_without_weights_keys_or_positions(layers):
    q, k, _, _, how, n = inputs(layers, 24, 4, 2, 64, 64, F32, weights=False, layout="dense")
    check(layers, q, k, None, None, how, n, False, F32, F32)
    one = layers.norm_rotate_heads_forward(q, eps=EPS, **how)
    both = layers.norm_rotate_heads_forward(q, k, eps=EPS, **how)
    assert one.k is None and torch.equal(one.q, both.q)
    g = layers.norm_rotate_heads_backward(q, None, q, eps=EPS, need_k_weight=False, **how)
    assert g.dk is None and g.dk_weight is None
    # the position of a token is its place in the last dimension of the tokens
    table = dict(cos=how["cos"], sin=how["sin"])
    a = layers.norm_rotate_heads_forward(q.view(3, 8, 4, 64), k.view(3, 8, 2, 64), eps=EPS, **table)
    pos = torch.arange(8, device="cuda").repeat(3)
    b = layers.norm_rotate_heads_forward(q, k, eps=EPS, **table, positions=pos)
    assert a.q.shape == (3, 8, 4, 64) and torch.equal(a.q.view(24, 4, 64), b.q) and torch.equal(a.k.view(24, 2, 64), b.k)


def test_extreme_values(layers):
    q = torch.zeros(4, 2, 64, device="cuda")
    q[1] = 1e-30
    q[2] = 1e15
    q[3, 0] = float("nan")
    how = dict(zip(("cos", "sin"), layers.rotation_table(4, 64)))
    y = layers.norm_rotate_heads_forward(q, eps=EPS, **how).q
    assert not y[0].any() and float(y[1].abs().max()) < 1e-25
    assert abs(float(y[2].square().mean()) - 1) < 1e-5
    assert bool(y[3, 0].isnan().all()) and not y[3, 1].any()


def test_without_eps(layers):
    # three heads of a warp's four, and a token that is none: no 0 / 0 from what is not there
    q, k, wq, wk, how, n = inputs(layers, 9, 3, 1, 128, 128, F32, table=5)
    how["positions"][4] = 7
    o = layers.norm_rotate_heads_forward(q, k, wq, wk, eps=0.0, **how)
    assert bool(o.q.isfinite().all()) and not o.q[4].any()
    g = layers.norm_rotate_heads_backward(n(*q.shape), n(*k.shape), q, k, wq, wk, eps=0.0, **how)
    assert all(bool(t.isfinite().all()) for t in g) and not g.dq[4].any()


def test_no_tokens_and_no_heads(layers):
    how = dict(zip(("cos", "sin"), layers.rotation_table(4, 8)))
    w = torch.ones(8, device="cuda")
    for shape in ((0, 2, 8), (3, 0, 8)):
        q = torch.empty(shape, device="cuda")
        assert layers.norm_rotate_heads_forward(q, q, w, w, **how).q.shape == shape
        g = layers.norm_rotate_heads_backward(q, q, q, q, w, w, **how)
        assert g.dq.shape == shape and not g.dq_weight.any() and not g.dk_weight.any()
    q, k = torch.randn(3, 0, 8, device="cuda"), torch.randn(3, 2, 8, device="cuda")
    assert torch.equal(layers.norm_rotate_heads_forward(q, k, w, w, **how).k,
                       layers.norm_rotate_heads_forward(k, None, w, **how).q)


def test_refusals(layers):
    q, k, wq, wk, how, _ = inputs(layers, 6, 4, 2, 64, 64, F32, layout="dense")
    f = layers.norm_rotate_heads_forward
    for bad in (dict(cos=how["cos"]), dict(cos=how["cos"], sin=how["sin"][:3]),
                dict(cos=torch.zeros(5, 33, device="cuda"), sin=torch.zeros(5, 33, device="cuda")),
                dict(how, positions=how["positions"][:5]), dict(how, positions=how["positions"].view(2, 3))):
        with pytest.raises(ValueError):
            f(q, k, wq, wk, **bad)
    with pytest.raises(TypeError):
        f(q, k, wq, wk, **dict(how, positions=how["positions"].int()))
    with pytest.raises(TypeError):
        f(q, k.bfloat16(), wq, wk, **how)
    with pytest.raises(TypeError):
        f(q, k, wq, wk.bfloat16(), **how)
    for a in ((q, k[:5], wq, wk), (q, k[..., :32], wq, wk), (q, k, wq[:63], wk), (q.transpose(1, 2), k, wq, wk),
              (q[0, 0],)):
        with pytest.raises(ValueError):
            f(*a, **how)
    with pytest.raises(ValueError):
        layers.norm_rotate_heads_backward(q, None, q, k, wq, wk, **how)
    with pytest.raises(ValueError):
        layers.norm_rotate_heads_backward(q[:, :2], k, q, k, wq, wk, **how)


@pytest.mark.parametrize("neighbours", [False, True])
def test_differentiable(layers, neighbours):
    q, k, wq, wk, how, n = inputs(layers, 10, 4, 2, 64, 32, F32, layout="dense")
    leaves = [t.clone().requires_grad_() for t in (q, k, wq, wk)]
    a = leaves[0].view(2, 5, 4, 64).transpose(0, 1)       # not tokens at one stride
    pos = how["positions"].view(2, 5)
    o = layers.norm_rotate_heads(a, leaves[1].view(2, 5, 2, 64).transpose(0, 1), *leaves[2:], cos=how["cos"],
                                 sin=how["sin"], positions=pos.t(), eps=EPS, neighbours=neighbours)
    cq, ck = n(10, 4, 64), n(10, 2, 64)
    total = (o.q.transpose(0, 1) * cq.view(2, 5, 4, 64)).sum() + (o.k.transpose(0, 1) * ck.view(2, 5, 2, 64)).sum()
    got = torch.autograd.grad(total, leaves)
    side = want(q, k, wq, wk, how, neighbours, cq, ck)
    for g, (e, r) in zip(got, [(s[0][0], s[1][0]) for s in side] + [(s[0][1], s[1][1]) for s in side]):
        ref.close(g, e, r, F32)
    # keys alone reach the loss; broadcast gradients
    o = layers.norm_rotate_heads(leaves[0], leaves[1], cos=how["cos"], sin=how["sin"])
    gq, gk = torch.autograd.grad(o.k.sum(), leaves[:2])
    assert not gq.any() and bool(gk.any())


def test_equal_bits_each_time(layers):
    q, k, wq, wk, how, n = inputs(layers, 3000, 8, 2, 128, 128, BF16)
    dq, dk = n(*q.shape).bfloat16(), n(*k.shape).bfloat16()
    first = layers.norm_rotate_heads_backward(dq, dk, q, k, wq, wk, **how)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, layers.norm_rotate_heads_backward(
            dq, dk, q, k, wq, wk, **how)))
