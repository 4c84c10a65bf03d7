"""Gradient of the policy loss's KL term where the reference all but forbids a token,
or forbids it."""
import numpy as np
import pytest
import torch

import sequence_ref as ref
from helpers import muon

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layers():
    muon()
    from newton_schulz_05_gb300 import layers
    return layers


@pytest.mark.parametrize("t", [1, 7, 64, 601])
@pytest.mark.parametrize("each", [True, False])
def test_far_references(layers, t, each):
    gen = torch.Generator(device="cuda").manual_seed(t)
    lp = -2 * torch.rand(3, t, generator=gen, device="cuda")
    old = lp + 0.1 * torch.randn(3, t, generator=gen, device="cuda")
    adv = torch.randn((3, t) if each else (3,), generator=gen, device="cuda")
    far = torch.tensor([float("-inf"), torch.finfo(torch.float32).min, -1e9, -3e7, -2e7, -100.0, -20.0, -3.0, -1.5, 12.0],
                       device="cuda")
    r = far[torch.randint(0, len(far), (3, t), generator=gen, device="cuda")]
    r[0, 0], r[2, t - 1] = far[0], far[2]
    kl, low, high = 0.05, 0.2, 0.28
    w = torch.tensor([0.5, 1.0, 0.25], device="cuda")
    got = layers.policy_loss_backward(lp, old, adv, w, ref_log_probs=r, clip_low=low, clip_high=high, kl=kl)
    l, o, e = ref.f64(lp), ref.f64(old), ref.f64(r) - ref.f64(lp)
    a = np.broadcast_to(ref.f64(adv).reshape(3, -1), (3, t))
    d = l - o
    pull = np.where(np.where(a >= 0, d > np.log1p(high), d < np.log1p(-low)), 0, np.exp(d) * a)
    change, size = np.expm1(e), np.abs(np.where(np.isinf(e), 0, e))
    f = ref.f64(w)[:, None]
    # as for other references: the rounded e's error, 4 ulp of an exponential, a few products
    room = f * ref.U * ((np.abs(d) + 10) * np.abs(pull) + kl * (12 * np.abs(change) + 2 * size * np.exp(e)))
    ref.close(got, f * (-pull - kl * change), room, torch.float32)


def test_a_forbidden_token_through_the_differentiable_loss(layers):
    lp = torch.full((1, 4), -1.0, device="cuda", requires_grad=True)
    r = torch.tensor([[-1.0, -1e9, float("-inf"), -1.0]], device="cuda")
    o = layers.policy_loss(lp, lp.detach(), torch.zeros(1, device="cuda"), ref_log_probs=r, kl=0.2)
    (g,) = torch.autograd.grad(o.loss, lp)
    # d kl / d log_probs = 1 - exp(-inf), a quarter of it each; the step of 0.05 in fp32 is 2^-28
    assert float((g - torch.tensor([[0.0, 0.05, 0.05, 0.0]], device="cuda")).abs().max()) <= 2.0 ** -26
