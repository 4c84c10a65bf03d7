"""examples/moe_block.py: the training operators and the optimizer together.
Its forward pass and gradients against the same model in plain 64-bit torch
operations, and training that lowers the loss and keeps the experts in use."""
import importlib.util
import os

import pytest
import torch

import layers_ref as ref
from helpers import muon

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    muon()
    spec = importlib.util.spec_from_file_location("moe_block", os.path.join(ROOT, "examples", "moe_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _plain(model, params, tokens, index):
    """The block in 64 bits, with the picks given (a discrete choice)."""
    embed, mix, router, up, down, out = params[:6]
    norms = [(params[6 + 2 * i], params[7 + 2 * i]) for i in range(3)]
    offset = 0

    def norm(s, w, b):
        m = s.mean(-1, keepdim=True)
        return (s - m) / (((s - m) ** 2).mean(-1, keepdim=True) + 1e-5).sqrt() * w + b

    def drop(x):
        nonlocal offset
        f = torch.from_numpy(ref.factors(x.numel(), model.p, model.random.seed, offset))
        offset += (x.numel() + 7) // 8
        return x * f.view(x.shape)

    s = embed[tokens]
    y = norm(s, *norms[0])
    s = s + drop(torch.einsum("ij,bjc->bic", mix, y))
    y = norm(s, *norms[1])
    l = y @ router
    p = torch.softmax(l, -1)
    w = torch.softmax(l.gather(-1, index), -1)
    h = torch.einsum("bic,ech->beih", y, up)
    h = torch.einsum("beih,ehc->biec", h * torch.sigmoid(h), down)
    x = (h.gather(2, index[..., None].expand(*index.shape, h.shape[-1])) * w[..., None]).sum(2)
    y = norm(s + drop(x), *norms[2])
    e = l.shape[-1]
    c = torch.bincount(index.reshape(-1), minlength=e).double() / index.numel()
    return y @ out, e * (c * p.mean((0, 1))).sum()


def test_block_equals_plain_64_bit_operations(example):
    model = example.Block(p=0.2)
    params = model.parameters()
    tokens, target = example.batch(0)
    logits, even, counts = model(tokens)
    loss = torch.nn.functional.cross_entropy(logits.flatten(0, 1), target.flatten()) + 0.1 * even
    grads = torch.autograd.grad(loss, params)
    # the picks the GPU made, from the logits it saw
    m2 = example.Block(p=0.2)
    with torch.no_grad():
        s = m2.embed[tokens]
        y = example.layers.layer_norm(s, *m2.norms[0])
        x = torch.einsum("ij,bjc->bic", m2.mix, y)
        y, _ = example.layers.dropout_add_layer_norm(x, s, *m2.norms[1], **m2._drop(x.numel()))
        index = example.layers.route(y @ m2.router, m2.k).index.long().cpu()
    p64 = [p.detach().double().cpu().requires_grad_() for p in params]
    want, even64 = _plain(model, p64, tokens.cpu(), index)
    loss64 = torch.nn.functional.cross_entropy(want.flatten(0, 1), target.cpu().flatten()) + 0.1 * even64
    g64 = torch.autograd.grad(loss64, p64)
    # fp32 products of a few hundred terms through four layers: 1e-4 of the norm
    assert abs(float(loss) - float(loss64)) <= 1e-5 * float(loss64)
    for g, e in zip(grads, g64):
        assert float((g.double().cpu() - e).norm()) <= 1e-4 * float(e.norm())
    assert int(counts[:-1].sum()) == 2 * tokens.numel() and int(counts[-1]) == tokens.numel()


def test_training_lowers_the_loss_and_uses_every_expert(example):
    losses, counts, even = example.train(steps=60)
    first, last = sum(losses[:5]) / 5, sum(losses[-5:]) / 5
    assert last < 0.5 * first, (first, last)
    assert min(counts[:-1]) > 0 and 0.9 < even < 2.0
