"""The differentiable operators take weights and tables of any strides, as they take
activations."""
import pytest
import torch

from helpers import muon

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layers():
    muon()
    from newton_schulz_05_gb300 import layers
    return layers


def test_weights_and_tables_that_are_no_dense_vectors(layers):
    gen = torch.Generator(device="cuda").manual_seed(0)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, k, both = n(6, 3, 64), n(6, 2, 64), n(64, 2)
    cos, sin = layers.rotation_table(6, 64)
    wide = torch.stack((cos, sin), -1)      # [table, pairs, 2]

    def run(split, table):
        leaf = both.clone().requires_grad_()
        o = layers.norm_rotate_heads(q, k, *split(leaf), cos=table(wide[..., 0]), sin=table(wide[..., 1]))
        (g,) = torch.autograd.grad((o.q * q).sum() + (o.k.square() * k).sum(), leaf)
        return o.q, o.k, g

    got = run(lambda w: w.unbind(1), lambda t: t)
    want = run(lambda w: [c.contiguous() for c in w.unbind(1)], lambda t: t.contiguous())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x, leaf = n(5, 64), both.clone().requires_grad_()
    y = layers.layer_norm(x, *leaf.unbind(1))
    assert torch.equal(y, layers.layer_norm(x, *(c.contiguous() for c in leaf.unbind(1))))
    y, _ = layers.dropout_add_layer_norm(x, x, *leaf.unbind(1), p=0.1, seed=3)
    (g,) = torch.autograd.grad(y.sum(), leaf)
    assert g.shape == both.shape
