"""Train a small language model on one GPU whose block mixes positions in two
ways, a gated recurrence and attention with normed and rotated heads, first on
given text and then on rewarded answers of its own:

    python examples/sequence_block.py --steps 60

Matrices take the Muon step, norm scales and biases AdamW (MuonWithAdamW).  The
text repeats a short random pattern, with a separator in front of each document;
documents are packed into sequences, and the recurrence starts over at each.
Data and weights are synthetic and seeded.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import newton_schulz_05_gb300 as muon  # noqa: E402
from newton_schulz_05_gb300 import layers  # noqa: E402


class Model:
    """Embedding; norm, gated recurrence, residual; norm, attention, residual;
    norm, output matrix."""

    def __init__(self, symbols=53, width=64, q_heads=4, k_heads=2, dim=32, length=96, seed=0, device="cuda"):
        g = torch.Generator(device="cpu").manual_seed(seed)

        def matrix(*shape, std):
            return (torch.randn(shape, generator=g) * std).to(device).requires_grad_()

        def vector(n, value):
            return torch.full((n,), value, device=device).requires_grad_()

        self.q_heads, self.k_heads, self.dim = q_heads, k_heads, dim
        self.embed = matrix(symbols, width, std=0.5)
        self.into = matrix(width, 2 * width, std=0.2)          # gate and input of the recurrence
        self.back = matrix(width, width, std=0.1)
        self.heads = matrix(width, (q_heads + 2 * k_heads) * dim, std=0.15)
        self.join = matrix(q_heads * dim, width, std=0.1)
        self.out = matrix(width, symbols, std=0.1)
        self.norms = [(vector(width, 1.0), vector(width, 0.0)) for _ in range(3)]
        self.head_norms = [vector(dim, 1.0), vector(dim, 1.0)]
        self.cos, self.sin = layers.rotation_table(length, dim, base=100.0, device=device)

    def parameters(self):
        return [self.embed, self.into, self.back, self.heads, self.join, self.out] + \
               [t for pair in self.norms for t in pair] + self.head_norms

    def __call__(self, tokens, starts=None, token_mask=None):
        """Logits of tokens [batch, length]; starts: first tokens of documents."""
        b, t = tokens.shape
        s = self.embed[tokens]
        y = layers.layer_norm(s, *self.norms[0])
        gate, x = (y @ self.into).chunk(2, dim=-1)
        h = layers.gated_scan(gate, x, starts=starts, token_mask=token_mask).h
        s = s + h @ self.back
        y = layers.layer_norm(s, *self.norms[1])
        joint = (y @ self.heads).view(b, t, -1, self.dim)
        q, k, v = joint.split([self.q_heads, self.k_heads, self.k_heads], dim=2)
        q, k = layers.norm_rotate_heads(q, k, *self.head_norms, cos=self.cos, sin=self.sin)
        share = self.q_heads // self.k_heads
        k, v = (z.repeat_interleave(share, dim=2) for z in (k, v))
        score = torch.einsum("bihd,bjhd->bhij", q, k) / self.dim ** 0.5
        later = torch.ones(t, t, dtype=torch.bool, device=tokens.device).triu(1)
        score = torch.softmax(score.masked_fill(later, float("-inf")), -1)
        a = torch.einsum("bhij,bjhd->bihd", score, v).flatten(2)
        s = s + a @ self.join
        return layers.layer_norm(s, *self.norms[2]) @ self.out

    def log_probs(self, tokens, starts=None, scale=1.0):
        """Of each token after the ones in front of it, [batch, length - 1]; 0 where it starts
        a document, which nothing predicts."""
        given = tokens[:, 1:]
        if starts is not None:
            given = torch.where(starts[:, 1:], -100, given)
        return layers.token_log_probs(self(tokens, starts)[:, :-1], given, scale=scale)


def text(step, batch=16, length=96, symbols=53, device="cuda"):
    """Packed documents, each a pattern of a few symbols over and over, and their first tokens."""
    g = torch.Generator(device="cpu").manual_seed(1000 + step)
    tokens = torch.zeros(batch, length, dtype=torch.int64)
    starts = torch.zeros(batch, length, dtype=torch.bool)
    for row in range(batch):
        at = 0
        while at < length:
            n = int(torch.randint(12, 60, (1,), generator=g))
            pattern = torch.randint(1, symbols, (int(torch.randint(2, 6, (1,), generator=g)),), generator=g)
            body = pattern.repeat(n)[:n]
            body[0] = 0
            end = min(length, at + n)
            tokens[row, at:end] = body[:end - at]
            starts[row, at] = True
            at = end
    return tokens.to(device), starts.to(device)


def train(steps=60, lr=0.03, report=None):
    """Losses of the given text, then of the rewarded answers."""
    model = Model()
    params = model.parameters()
    opt = muon.MuonWithAdamW(params, lr=lr, wd=0.01, adamw_lr=3e-3)
    losses = []

    def step(loss):
        grads = torch.autograd.grad(loss, params)
        with torch.no_grad():
            opt.step([g.contiguous() for g in grads])
        losses.append(loss.detach())
        if report and (len(losses) % report == 0):
            print("step %4d  loss %.4f" % (len(losses), losses[-1]))

    for i in range(steps):
        tokens, starts = text(i)
        counted = ~starts[:, 1:]
        step(-model.log_probs(tokens, starts).sum() / counted.sum())
    # answers the model would have given, rewarded for every token that is even
    for i in range(steps // 4):
        tokens, starts = text(steps + i)
        with torch.no_grad():
            old = model.log_probs(tokens, starts)
            reward = (tokens[:, 1:] % 2 == 0).float()
            advantage = (reward - reward.mean()) / reward.std()
        for _ in range(2):
            o = layers.policy_loss(model.log_probs(tokens, starts), old, advantage, ref_log_probs=old,
                                   token_mask=~starts[:, 1:], clip_high=0.28, kl=0.02)
            step(o.loss)
    return [float(x) for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    train(a.steps, report=10)
