"""The example model, whose block runs the recurrence, the heads and the log
probabilities one after the other, and the policy loss on them, against the same
model in plain 64-bit torch."""
import importlib.util
import os
import sys

import pytest
import torch

from helpers import muon

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    muon()
    spec = importlib.util.spec_from_file_location("sequence_block", os.path.join(ROOT, "examples", "sequence_block.py"))
    module = importlib.util.module_from_spec(spec)
    sys.modules["sequence_block"] = module
    spec.loader.exec_module(module)
    return module


def _plain(model, params, tokens, starts):
    embed, into, back, heads, join, out = params[:6]
    norms = [(params[6 + 2 * i], params[7 + 2 * i]) for i in range(3)]
    qw, kw = params[12:]
    b, t = tokens.shape

    def norm(s, w, bias):
        m = s.mean(-1, keepdim=True)
        return (s - m) / (((s - m) ** 2).mean(-1, keepdim=True) + 1e-5).sqrt() * w + bias

    s = embed[tokens]
    gate, x = (norm(s, *norms[0]) @ into).chunk(2, dim=-1)
    a = torch.sigmoid(gate)
    h, state = [], torch.zeros_like(x[:, 0])
    for i in range(t):
        state = a[:, i] * torch.where(starts[:, i, None], 0.0, state) + (1 - a[:, i]) * x[:, i]
        h.append(state)
    s = s + torch.stack(h, 1) @ back
    joint = (norm(s, *norms[1]) @ heads).view(b, t, -1, model.dim)
    q, k, v = joint.split([model.q_heads, model.k_heads, model.k_heads], dim=2)
    half = model.dim // 2
    angle = torch.arange(t, dtype=torch.float64)[:, None] * 100.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    c, n = angle.cos()[:, None], angle.sin()[:, None]

    def turned(z, w):
        z = z / ((z * z).mean(-1, keepdim=True) + 1e-6).sqrt() * w
        u, y = z[..., :half], z[..., half:]
        return torch.cat((u * c - y * n, y * c + u * n), -1)

    q, k = turned(q, qw), turned(k, kw)
    share = model.q_heads // model.k_heads
    k, v = (z.repeat_interleave(share, dim=2) for z in (k, v))
    score = torch.einsum("bihd,bjhd->bhij", q, k) / model.dim ** 0.5
    score = torch.softmax(score.masked_fill(torch.ones(t, t, dtype=torch.bool).triu(1), float("-inf")), -1)
    s = s + torch.einsum("bhij,bjhd->bihd", score, v).flatten(2) @ join
    logits = norm(s, *norms[2]) @ out
    lp = torch.log_softmax(logits[:, :-1], -1).gather(2, tokens[:, 1:, None])[..., 0]
    return torch.where(starts[:, 1:], 0.0, lp)


@pytest.mark.parametrize("policy", [False, True])
def test_model_equals_plain_64_bit_operations(example, policy):
    model = example.Model()
    params = model.parameters()
    tokens, starts = example.text(0)
    lp = model.log_probs(tokens, starts)
    p64 = [p.detach().double().cpu().requires_grad_() for p in params]
    want = _plain(model, p64, tokens.cpu(), starts.cpu())
    assert float((lp.detach().double().cpu() - want.detach()).abs().max()) <= 1e-4
    mask = ~starts[:, 1:]
    if policy:
        gen = torch.Generator(device="cuda").manual_seed(1)
        old = (lp + 0.2 * torch.randn(lp.shape, generator=gen, device="cuda")).detach()
        ref = (lp + 0.2 * torch.randn(lp.shape, generator=gen, device="cuda")).detach()
        adv = torch.randn(lp.shape, generator=gen, device="cuda")
        loss = example.layers.policy_loss(lp, old, adv, ref_log_probs=ref, token_mask=mask, kl=0.1).loss
        d, e = want - old.double().cpu(), ref.double().cpu() - want
        a, r = adv.double().cpu(), d.exp()
        each = -torch.minimum(r * a, r.clamp(0.8, 1.2) * a) + 0.1 * (e.exp() - e - 1)
        loss64 = (each * mask.cpu()).sum() / mask.sum().cpu()
    else:
        loss, loss64 = -lp.sum() / mask.sum(), -want.sum() / mask.sum().cpu()
    grads = torch.autograd.grad(loss, params)
    g64 = torch.autograd.grad(loss64, p64)
    # fp32 products of a few hundred terms through a dozen layers: 1e-4 of the norm
    assert abs(float(loss.detach()) - float(loss64.detach())) <= 1e-4 * max(1.0, abs(float(loss64.detach())))
    for g, w in zip(grads, g64):
        assert float((g.double().cpu() - w).norm()) <= 2e-4 * float(w.norm())


def test_training_runs(example):
    losses = example.train(steps=8)
    assert len(losses) == 8 + 2 * 2 and all(x == x and abs(x) < 1e3 for x in losses)
