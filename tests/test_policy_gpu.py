"""Clipped policy loss with a KL term, and its gradient, against 64-bit
formulas."""
import numpy as np
import pytest
import torch

import sequence_ref as ref
from helpers import muon

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.fixture(scope="module")
def layers():
    muon()
    from newton_schulz_05_gb300 import layers
    return layers


def inputs(b, t, each=True, with_ref=True, masked=True, layout="dense", seed=0, spread=0.3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731

    def rows(v):
        if layout == "dense":
            return v
        wide = torch.full((b, t + 5), float("nan"), device="cuda")
        wide[:, 3:t + 3] = v
        return wide[:, 3:t + 3]

    lp = -4 * torch.rand(b, t, generator=gen, device="cuda") ** 2
    old, r = lp + spread * n(b, t), lp + spread * n(b, t)
    mask = None
    if masked:
        mask = torch.arange(t, device="cuda") < torch.randint(0, t + 1, (b, 1), generator=gen, device="cuda")
        lp[~mask], old[~mask], r[~mask] = float("nan"), float("inf"), float("-inf")
    adv = rows(n(b, t)) if each else n(b)
    return dict(lp=rows(lp), old=rows(old), adv=adv, r=rows(r) if with_ref else None, mask=mask)


def check(layers, v, low=0.2, high=0.28, kl=0.05, by_sequence=False):
    how = dict(ref_log_probs=v["r"], token_mask=v["mask"], clip_low=low, clip_high=high, kl=kl)
    o = layers.policy_loss_forward(v["lp"], v["old"], v["adv"], by_sequence=by_sequence, **how)
    w = {k: None if t is None else ref.f64(t) for k, t in v.items()}
    val, err = ref.policy(w["lp"], w["old"], w["adv"], w["r"], w["mask"], low, high, kl, by_sequence)
    for got, e, r in zip(o, val, err):
        ref.close(got, np.asarray(e), r, F32)
    dloss = torch.tensor(0.7, device="cuda")
    g = layers.policy_loss_backward(v["lp"], v["old"], v["adv"], o.weights, dloss=dloss, **how)
    e, r = ref.policy_grad(w["lp"], w["old"], w["adv"], w["r"], w["mask"], low, high, kl, ref.f64(o.weights),
                           float(dloss))
    ref.close(g, e, r, F32)


@pytest.mark.parametrize("by_sequence", [False, True])
@pytest.mark.parametrize("each,with_ref,masked", [(True, True, True), (False, True, True), (True, False, False),
                                                  (False, False, True), (False, True, False)])
@pytest.mark.parametrize("b,t,layout", [(1, 1, "dense"), (1, 2, "odd"), (3, 7, "dense"), (2, 31, "odd"), (40, 4, "dense"),
                                        (5, 32, "dense"), (4, 100, "odd"), (2, 1000, "dense"), (3, 4095, "dense"),
                                        (2, 4096, "dense"), (1, 4097, "odd"), (2, 9001, "dense"), (700, 33, "dense"),
                                        (1, 40000, "dense"), (5000, 1, "dense"), (64, 513, "dense")])
def test_policy_loss_and_gradient(layers, b, t, layout, each, with_ref, masked, by_sequence):
    check(layers, inputs(b, t, each, with_ref, masked, layout, seed=t), by_sequence=by_sequence)


@pytest.mark.parametrize("spread", [1e-4, 1.0, 4.0])
def test_near_and_far_policies(layers, spread):
    # k of near policies is a difference of near numbers; ratios of far ones span many powers
    check(layers, inputs(4, 3000, spread=spread))


@pytest.mark.parametrize("low,high,kl", [(0.0, 0.0, 0.1), (0.99, 10.0, 0.0), (0.2, 0.2, -0.3)])
def test_other_bounds(layers, low, high, kl):
    check(layers, inputs(4, 600, seed=2), low, high, kl)


def test_the_border_is_decided_on_the_exact_difference(layers):
    # differences a fraction of an fp32 step from log(1 + high) and log(1 - low), on both sides
    high, low = 0.2, 0.2
    lp, old = [], []
    rng = np.random.default_rng(0)
    for bound in (np.log1p(high), np.log1p(-low)):
        for a in -np.abs(rng.normal(size=200)) * 3:
            a = np.float32(a)
            b = np.float32(np.float64(a) - bound)
            for o in (np.nextafter(b, np.float32(-9)), b, np.nextafter(b, np.float32(9))):
                lp.append(a)
                old.append(o)
    lp, old = (torch.tensor(np.array(v, np.float32), device="cuda")[None] for v in (lp, old))
    for adv in (1.0, -1.0):
        v = dict(lp=lp, old=old, adv=torch.full((1,), adv, device="cuda"), r=None, mask=None)
        o = layers.policy_loss_forward(lp, old, v["adv"], clip_low=low, clip_high=high)
        d = lp.double() - old.double()
        cut = (d > np.log1p(high)) if adv > 0 else (d < np.log1p(-low))
        assert 0 < int(cut.sum()) < cut.numel()
        assert abs(float(o.clipped) - float(cut.double().mean())) < 1e-6
        g = layers.policy_loss_backward(lp, old, v["adv"], o.weights, clip_low=low, clip_high=high)
        assert torch.equal(g != 0, ~cut)


def test_nothing_that_counts(layers):
    v = inputs(3, 50)
    mask = torch.zeros(3, 50, dtype=torch.bool, device="cuda")
    for by_sequence in (False, True):
        o = layers.policy_loss_forward(v["lp"], v["old"], v["adv"], token_mask=mask, by_sequence=by_sequence)
        assert float(o.loss) == float(o.kl) == float(o.clipped) == 0 and not o.weights.any()
    assert not layers.policy_loss_backward(v["lp"], v["old"], v["adv"], o.weights, token_mask=mask).any()
    for shape in ((0, 5), (3, 0)):
        e = torch.empty(shape, device="cuda")
        o = layers.policy_loss_forward(e, e, e)
        assert float(o.loss) == 0 and o.weights.shape == shape[:1] and not o.weights.any()
        assert layers.policy_loss_backward(e, e, e, o.weights).shape == shape


def test_what_is_not_finite(layers):
    v = inputs(2, 8, masked=False, with_ref=False)
    v["adv"][:] = 1.0
    v["old"][0, 0] = float("-inf")         # an infinite ratio is cut off
    o = layers.policy_loss_forward(v["lp"], v["old"], v["adv"])
    assert bool(o.loss.isfinite())
    g = layers.policy_loss_backward(v["lp"], v["old"], v["adv"], o.weights)
    assert g[0, 0] == 0 and bool(g.isfinite().all())
    v["lp"][1, 3] = float("nan")
    assert bool(layers.policy_loss_forward(v["lp"], v["old"], v["adv"]).loss.isnan())
    g = layers.policy_loss_backward(v["lp"], v["old"], v["adv"], o.weights)
    assert bool(g[1, 3].isnan()) and int(g.isnan().sum()) == 1


def test_a_reference_without_weight_counts_for_nothing(layers):
    v = inputs(3, 40, masked=False)
    v["r"][1, 5] = float("-inf")
    how = dict(kl=0.0)
    a = layers.policy_loss_forward(v["lp"], v["old"], v["adv"], ref_log_probs=v["r"], **how)
    b = layers.policy_loss_forward(v["lp"], v["old"], v["adv"], **how)
    assert a.loss == b.loss and a.clipped == b.clipped and bool(a.kl.isinf())
    g = layers.policy_loss_backward(v["lp"], v["old"], v["adv"], a.weights, ref_log_probs=v["r"], **how)
    assert torch.equal(g, layers.policy_loss_backward(v["lp"], v["old"], v["adv"], b.weights, **how))


def test_gradient_in_place_through_the_c_abi(layers):
    lib = muon().load()
    v = inputs(3, 700, masked=False)
    o = layers.policy_loss_forward(v["lp"], v["old"], v["adv"], ref_log_probs=v["r"], kl=0.1)
    want = layers.policy_loss_backward(v["lp"], v["old"], v["adv"], o.weights, ref_log_probs=v["r"], kl=0.1)
    for name in ("lp", "old", "r"):
        c = {k: None if t is None else t.clone() for k, t in v.items()}
        assert lib.muon_policy_loss_backward(3, 700, c["lp"].data_ptr(), 700, c["old"].data_ptr(), 700,
                                             c["adv"].data_ptr(), 700, c["r"].data_ptr(), 700, None, 0.2, 0.2, 0.1,
                                             o.weights.data_ptr(), None, c[name].data_ptr(), None) == 0
        torch.cuda.synchronize()
        assert torch.equal(c[name], want)


def test_differentiable_and_shapes(layers):
    v = inputs(6, 40, each=False, seed=3)
    lp = torch.where(v["mask"], v["lp"], 0).requires_grad_()
    o = layers.policy_loss(lp.view(2, 3, 40), v["old"].view(2, 3, 40), v["adv"].view(2, 3),
                           ref_log_probs=v["r"].view(2, 3, 40), token_mask=v["mask"].view(2, 3, 40), kl=0.1,
                           by_sequence=True)
    assert o.weights.shape == (2, 3)
    (g,) = torch.autograd.grad(3 * o.loss, lp)
    w = {k: None if t is None else ref.f64(t) for k, t in v.items()}
    e, r = ref.policy_grad(w["lp"], w["old"], w["adv"], w["r"], w["mask"], 0.2, 0.2, 0.1, ref.f64(o.weights).reshape(-1), 3.0)
    ref.close(g, e, r, F32)
    # rows that are not rows: transposed
    a = layers.policy_loss(lp.t(), v["old"].t(), v["adv"][:, None].expand(6, 40).t(), token_mask=v["mask"].t())
    b = layers.policy_loss(lp, v["old"], v["adv"], token_mask=v["mask"])
    assert abs(float(a.loss.detach()) - float(b.loss.detach())) < 1e-6
    one = layers.policy_loss_forward(lp[0].detach(), v["old"][0], v["adv"][0], token_mask=v["mask"][0])
    assert one.weights.shape == ()
    f = layers.policy_loss_forward
    x = lp.detach()
    for bad in ((x, v["old"][:5], v["adv"]), (x, v["old"], v["adv"][:5]), (x, v["old"], v["adv"].view(2, 3)),
                (x.t(), v["old"].t(), v["adv"])):
        with pytest.raises(ValueError):
            f(*bad)
    with pytest.raises(ValueError):
        f(x, v["old"], v["adv"], token_mask=v["mask"].view(40, 6))
    with pytest.raises(TypeError):
        f(x, v["old"].double(), v["adv"])
    with pytest.raises(muon().MuonError):
        f(x, v["old"], v["adv"], clip_low=1.0)


def test_equal_bits_each_time(layers):
    v = inputs(50, 3000)
    o = layers.policy_loss_forward(v["lp"], v["old"], v["adv"], token_mask=v["mask"])
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(o, layers.policy_loss_forward(v["lp"], v["old"], v["adv"],
                                                                                 token_mask=v["mask"])))
