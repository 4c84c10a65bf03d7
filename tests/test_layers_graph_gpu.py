"""The training operators inside a captured CUDA graph, back to back on one
stream, and their refusal to be differentiated twice."""
import pytest
import torch

from helpers import muon

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layers():
    muon()
    from newton_schulz_05_gb300 import layers
    return layers


def _chain(layers, x, r, w, router):
    o = layers.layer_norm_forward(x, w, w, residual=r, p=0.1, seed=5, offset=3)
    t = layers.route_forward(o.y @ router, 2)
    dl = layers.route_backward(o.y @ router, t.index, t.counts, dweights=t.weights, dloss=t.loss)
    dy = layers.dropout_forward((dl @ router.t()).contiguous(), 0.2, seed=6)
    g = layers.layer_norm_backward(dy, o.sum, o.mean, o.rstd, w, dsum=r, p=0.1, seed=5, offset=3)
    return list(o) + list(t) + [dl, dy] + list(g)


@pytest.mark.parametrize("rows,cols", [(37, 200), (3000, 1023), (517, 4096)])
def test_replayed_graph_gives_the_same_bits(layers, rows, cols):
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, r = (torch.randn(rows, cols, generator=gen, device="cuda") for _ in range(2))
    w = torch.randn(cols, generator=gen, device="cuda")
    router = torch.randn(cols, 16, generator=gen, device="cuda")
    want = [t.clone() for t in _chain(layers, x, r, w, router)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _chain(layers, x, r, w, router)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _chain(layers, x, r, w, router)
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_second_derivatives_are_refused(layers):
    x = torch.randn(4, 16, device="cuda", requires_grad=True)
    for y in (layers.layer_norm(x), layers.dropout(x, 0.1, seed=1), layers.route(x, 2).weights):
        (g,) = torch.autograd.grad((y * y).sum(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            g.sum().backward()
