"""What a call of the training operators may do to tensors, threads and memory
around it."""
import pytest
import torch

from helpers import muon

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layers():
    muon()
    from newton_schulz_05_gb300 import layers
    return layers


def test_writing_into_a_saved_tensor_is_noticed(layers):
    a = torch.randn(64, device="cuda", requires_grad=True)
    x = a * 2
    y = (x * x).sum()                               # saves x
    with torch.no_grad():
        layers.dropout_forward(x, 0.5, seed=1, out=x)
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()
    # a view of what was saved counts too
    x = a * 2
    y = (x * x).sum()
    layers.dropout_forward(torch.ones(8, device="cuda"), 0.5, seed=1, out=x.detach()[8:16])
    with pytest.raises(RuntimeError, match="inplace"):
        y.backward()


def test_out_that_requires_grad_is_refused_while_grads_are_recorded(layers):
    x = torch.randn(64, device="cuda")
    leaf = torch.zeros(64, device="cuda", requires_grad=True)
    for out in (leaf, leaf * 2):
        with pytest.raises(RuntimeError, match="grad"):
            layers.dropout_forward(x, 0.5, seed=1, out=out)
        with torch.no_grad():
            assert layers.dropout_forward(x, 0.5, seed=1, out=out) is out
