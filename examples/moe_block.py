"""Train a small mixture-of-experts block on one GPU: every operator of
newton_schulz_05_gb300.layers between the matrix products, every parameter
stepped by MuonWithAdamW.

    python examples/moe_block.py --steps 100

The model reads a sequence of symbols and predicts, at each position, the
symbol seen `lag` positions earlier plus a fixed permutation: a mixing matrix
over positions finds the symbol, the experts learn the permutation.  Matrices
and the [E, M, N] expert stacks take the Muon step, norm scales and biases take
AdamW.  Data and weights are synthetic and seeded.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import newton_schulz_05_gb300 as muon  # noqa: E402
from newton_schulz_05_gb300 import layers  # noqa: E402


class Block:
    """Embedding, norm, mixing over positions, dropout + residual + norm,
    routed experts, dropout + residual + norm, output matrix."""

    def __init__(self, symbols=48, length=32, width=64, hidden=96, experts=8, k=2, p=0.05,
                 seed=0, device="cuda"):
        g = torch.Generator(device="cpu").manual_seed(seed)

        def matrix(*shape, std):
            return (torch.randn(shape, generator=g) * std).to(device).requires_grad_()

        def vector(n, value):
            return torch.full((n,), value, device=device).requires_grad_()

        self.k, self.p, self.experts = k, p, experts
        self.random = layers.RandomCounter(seed)
        self.embed = matrix(symbols, width, std=0.5)
        self.mix = matrix(length, length, std=0.2)
        self.router = matrix(width, experts, std=0.1)
        self.up = matrix(experts, width, hidden, std=0.1)
        self.down = matrix(experts, hidden, width, std=0.1)
        self.out = matrix(width, symbols, std=0.1)
        self.norms = [(vector(width, 1.0), vector(width, 0.0)) for _ in range(3)]

    def parameters(self):
        return [self.embed, self.mix, self.router, self.up, self.down, self.out] + \
               [t for pair in self.norms for t in pair]

    def _drop(self, numel):
        return dict(p=self.p, seed=self.random.seed, offset=self.random.take(numel))

    def __call__(self, tokens, mask=None):
        """(logits, balance loss, counts) of tokens [batch, length]; mask:
        which tokens are routed."""
        s = self.embed[tokens]
        y = layers.layer_norm(s, *self.norms[0])
        x = torch.einsum("ij,bjc->bic", self.mix, y)
        y, s = layers.dropout_add_layer_norm(x, s, *self.norms[1], **self._drop(x.numel()))
        r = layers.route(y @ self.router, self.k, token_mask=mask)
        # every expert on every token, weighted by the router: enough for a few small experts
        h = torch.einsum("bic,ech->beih", y, self.up)
        h = torch.einsum("beih,ehc->biec", h * torch.sigmoid(h), self.down)
        at = torch.where(r.index < 0, 0, r.index).long()
        share = torch.zeros(*y.shape[:2], self.experts, device=y.device)
        x = torch.einsum("bie,biec->bic", share.scatter_add(2, at, r.weights), h)
        y, s = layers.dropout_add_layer_norm(x, s, *self.norms[2], **self._drop(x.numel()))
        return y @ self.out, r.loss, r.counts


def batch(step, size=64, symbols=48, length=32, lag=3, device="cuda"):
    g = torch.Generator(device="cpu").manual_seed(1000 + step)
    tokens = torch.randint(0, symbols, (size, length), generator=g)
    permutation = torch.randperm(symbols, generator=torch.Generator().manual_seed(7))
    target = permutation[torch.roll(tokens, lag, dims=1)]
    return tokens.to(device), target.to(device)


def train(steps=100, lr=0.05, balance=0.01, report=None):
    """Loss of every step, and the last step's expert counts and balance loss."""
    model = Block()
    params = model.parameters()
    opt = muon.MuonWithAdamW(params, lr=lr, wd=0.01, adamw_lr=3e-3)
    losses = []
    for step in range(steps):
        tokens, target = batch(step)
        logits, even, counts = model(tokens)
        loss = torch.nn.functional.cross_entropy(logits.flatten(0, 1), target.flatten())
        grads = torch.autograd.grad(loss + balance * even, params)
        with torch.no_grad():
            opt.step([g.contiguous() for g in grads])
        losses.append(loss.detach())
        even = even.detach()
        if report and (step % report == 0 or step == steps - 1):
            print("step %4d  loss %.4f  balance %.3f  tokens an expert %s"
                  % (step, losses[-1], even, counts[:-1].tolist()))
    return [float(x) for x in losses], counts.tolist(), float(even)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=100)
    a = ap.parse_args()
    train(a.steps, report=10)
