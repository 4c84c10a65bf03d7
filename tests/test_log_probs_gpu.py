"""Log probabilities of given tokens over a vocabulary, and their gradient,
against 64-bit formulas."""
import numpy as np
import pytest
import torch

import sequence_ref as ref
from helpers import muon

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def layers():
    muon()
    from newton_schulz_05_gb300 import layers
    return layers


def inputs(t, v, dtype, layout="dense", seed=0, ignored=0.2):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pad = {"dense": 0, "columns": 24, "odd": 5}[layout]
    at = {"dense": 0, "columns": 8, "odd": 3}[layout]
    wide = (3 * torch.randn(t, v + pad, generator=gen, device="cuda")).to(dtype)
    l = wide[:, at:at + v]
    y = torch.randint(0, v, (t,), generator=gen, device="cuda")
    y[torch.rand(t, generator=gen, device="cuda") < ignored] = -100
    d = torch.randn(t, generator=gen, device="cuda")
    d[torch.rand(t, generator=gen, device="cuda") < 0.2] = 0
    return l, y, d


def check(layers, l, y, d, scale, dtype):
    o = layers.token_log_probs_forward(l, y, scale=scale)
    l64, y64 = ref.f64(l), y.cpu().numpy()
    lp, lse, ep, es = ref.log_probs(l64, y64, scale)
    ref.close(o.log_probs, lp, ep, F32)
    ref.close(o.lse, lse, es, F32)
    g = layers.token_log_probs_backward(d, l, y, o.lse, scale=scale)
    e, r = ref.log_probs_grad(ref.f64(d), l64, y64, ref.f64(o.lse), scale)
    ref.close(g, e, r, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("t,v", [(1, 1), (1, 2), (3, 7), (2, 8), (5, 31), (4, 32), (7, 64), (300, 100), (2, 255),
                                 (3, 256), (5, 1000), (1, 1024), (2, 4096), (1, 8192), (9, 8191), (3, 16385),
                                 (1, 50021), (160, 5003), (1, 131072), (2, 262144), (700, 512), (400, 33)])
def test_log_probs_and_gradient(layers, t, v, dtype):
    for layout in ("dense", "columns", "odd"):
        l, y, d = inputs(t, v, dtype, layout, seed=v)
        check(layers, l, y, d, 0.7, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("v", [40, 5000, 70001])
def test_masked_symbols_and_extremes(layers, v, dtype):
    l, y, d = inputs(6, v, dtype, seed=1, ignored=0)
    y[:] = v // 2
    d[:] = 1.0
    l[0, ::2] = float("-inf")
    l[0, v // 2] = 1.0
    l[1] = float("-inf")                  # one symbol left
    l[1, v // 2] = -5.0
    l[2] = torch.finfo(dtype).min         # masked by the lowest value
    l[2, v // 2:] = 0.5
    l[3] = 30000.0                        # far from zero, all alike
    l[4, 0] = -30000.0
    l[5] = -80.0                          # one far above the others
    l[5, v - 1] = 100.0
    check(layers, l, y, d, 1.0, dtype)
    # the masked symbol is asked for
    o = layers.token_log_probs_forward(l[:2], torch.tensor([0, 0], device="cuda"))
    assert bool((o.log_probs == float("-inf")).all()) and bool(o.lse.isfinite().all())


@pytest.mark.parametrize("v", [40, 70000])
def test_rows_without_meaning_stay_alone(layers, v):
    l, y, d = inputs(8, v, F32, seed=2, ignored=0)
    d[:] = 1.0
    want = layers.token_log_probs_forward(l, y)
    gw = layers.token_log_probs_backward(d, l, y, want.lse)
    m = l.clone()
    m[1, v - 1] = float("nan")
    m[3, 0] = float("inf")
    m[5] = float("-inf")
    m[6] = float("nan")
    y2 = y.clone()
    y2[6] = v                              # ignored, as its row is garbage
    m[7] = float("inf")
    d2 = d.clone()
    d2[7] = 0.0                            # no gradient reaches it
    got = layers.token_log_probs_forward(m, y2)
    g = layers.token_log_probs_backward(d2, m, y2, got.lse)
    for i in (0, 2, 4):
        assert got.log_probs[i] == want.log_probs[i] and torch.equal(g[i], gw[i])
    assert bool(got.log_probs[[1, 3, 5]].isnan().all())
    assert got.log_probs[6] == 0 and got.lse[6] == 0 and not g[6].any() and not g[7].any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradient_in_place(layers, dtype):
    for t, v in ((5, 1000), (3, 4099), (2, 65536)):
        l, y, d = inputs(t, v, dtype, seed=3)
        l = l.clone()
        lse = layers.token_log_probs_forward(l, y).lse
        want = layers.token_log_probs_backward(d, l, y, lse)
        version = l._version
        assert layers.token_log_probs_backward(d, l, y, lse, out=l) is l
        assert torch.equal(l, want) and l._version > version
    leaf = torch.zeros(3, 7, device="cuda", requires_grad=True)
    y, d = torch.zeros(3, dtype=torch.int64, device="cuda"), torch.ones(3, device="cuda")
    with pytest.raises(RuntimeError, match="grad"):
        layers.token_log_probs_backward(d, leaf, y, d, out=leaf)
    wide = torch.zeros(3, 9, device="cuda")
    with pytest.raises(ValueError):
        layers.token_log_probs_backward(d, wide[:, :7], y, d, out=wide[:, :7])


def test_differentiable_is_the_cross_entropy(layers):
    gen = torch.Generator(device="cuda").manual_seed(4)
    l = torch.randn(3, 5, 100, generator=gen, device="cuda", requires_grad=True)
    y = torch.randint(0, 100, (3, 5), generator=gen, device="cuda")
    y[0, 0] = -100
    loss = -layers.token_log_probs(l, y).sum() / 14
    (g,) = torch.autograd.grad(loss, l)
    p = l.detach().double().requires_grad_()
    want = torch.nn.functional.cross_entropy(p.view(15, 100), y.view(15), ignore_index=-100)
    (e,) = torch.autograd.grad(want, p)
    assert abs(float(loss.detach()) - float(want.detach())) < 1e-6 and float((g.double() - e).norm()) < 1e-6 * float(e.norm())
    # logits that are no rows, a broadcast gradient
    (g2,) = torch.autograd.grad(layers.token_log_probs(l.transpose(0, 1), y.t()).sum(), l)
    assert float((g2.double() + 14 * e).norm()) < 1e-5 * float(g2.norm())


def test_refusals_and_empty(layers):
    l = torch.zeros(2, 3, 8, device="cuda")
    y = torch.zeros(2, 3, dtype=torch.int64, device="cuda")
    f = layers.token_log_probs_forward
    with pytest.raises(TypeError):
        f(l, y.int())
    for bad in (y.view(3, 2), y[:1]):
        with pytest.raises(ValueError):
            f(l, bad)
    with pytest.raises(ValueError):
        f(l.transpose(1, 2), y)
    with pytest.raises(muon().MuonError):
        f(l, y, scale=0.0)
    o = f(l, y.view(-1))
    assert o.log_probs.shape == (2, 3)
    with pytest.raises(ValueError):
        layers.token_log_probs_backward(o.lse.view(3, 2), l, y, o.lse)
    empty = torch.empty(0, 8, device="cuda")
    assert f(empty, y[:0, 0]).lse.shape == (0,)
    assert layers.token_log_probs_backward(o.lse[:0, 0], empty, y[:0, 0], o.lse[:0, 0]).shape == (0, 8)


def test_more_than_2_32_elements(layers):
    t, v = 33000, 131072
    l = torch.zeros(t, v, dtype=BF16, device="cuda")
    y = torch.full((t,), 5, dtype=torch.int64, device="cuda")
    l[-1, 5] = 10.0
    o = layers.token_log_probs_forward(l, y)
    assert abs(float(o.log_probs[0]) + np.log(v)) < 1e-5
    e = 10 - np.log(np.exp(10.0) + v - 1)
    assert abs(float(o.log_probs[-1]) - e) < 1e-5
    g = layers.token_log_probs_backward(torch.ones(t, device="cuda"), l, y, o.lse, out=l)
    assert abs(float(g[-1, 5]) - (1 - np.exp(e))) < 4e-3 and abs(float(g[-1, -1]) * (np.exp(10.0) + v - 1) + 1) < 4e-3
    assert abs(float(g[0, 5]) - 1) < 4e-3


@pytest.mark.parametrize("t,v", [(40, 32768), (2, 262144), (500, 1003)])
def test_equal_bits_each_time(layers, t, v):
    l, y, d = inputs(t, v, BF16, seed=5)
    o = layers.token_log_probs_forward(l, y)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(o, layers.token_log_probs_forward(l, y)))
