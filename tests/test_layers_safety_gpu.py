"""What a call of the training operators may do to tensors, threads and memory
around it."""
import ctypes
import threading
import time

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


def test_shapes_that_only_count_alike_are_refused(layers):
    b, t, e = 3, 8, 16
    l = torch.randn(b, t, e, device="cuda")
    mask = torch.rand(b, t, device="cuda") > 0.3
    o = layers.route_forward(l, 2, token_mask=mask)
    flat = layers.route_forward(l, 2, token_mask=mask.view(-1))
    assert torch.equal(o.index, flat.index)
    with pytest.raises(ValueError):
        layers.route_forward(l, 2, token_mask=mask.view(t, b))
    with pytest.raises(ValueError):
        layers.route(l, 2, token_mask=mask.t())
    dw = torch.randn(b, t, 2, device="cuda")
    args = (l, o.index, o.counts)
    g = layers.route_backward(*args, dweights=dw, token_mask=mask)
    assert torch.equal(g, layers.route_backward(*args, dweights=dw.view(-1, 2), token_mask=mask))
    for bad in (dw.view(t, b, 2), dw.view(2, -1)):
        with pytest.raises(ValueError):
            layers.route_backward(*args, dweights=bad, token_mask=mask)
    with pytest.raises(ValueError):
        layers.route_backward(*args, dweights=dw, token_mask=mask.view(t, b))
    n = layers.layer_norm_forward(l)
    g = layers.layer_norm_backward(l, l, n.mean, n.rstd)
    for mean, rstd in ((n.mean.view(-1), n.rstd.view(-1)), (n.mean[..., None], n.rstd[None])):
        assert torch.equal(g.dx, layers.layer_norm_backward(l, l, mean, rstd).dx)
    for mean, rstd in ((n.mean.view(t, b), n.rstd), (n.mean, n.rstd.view(t, b)), (n.mean.view(2, -1), n.rstd)):
        with pytest.raises(ValueError):
            layers.layer_norm_backward(l, l, mean, rstd)


def test_every_result_has_memory_of_its_own(layers):
    x = torch.randn(40, 24, device="cuda")
    w = torch.ones(24, device="cuda")
    o = layers.layer_norm_forward(x, w, w, residual=x, p=0.1)
    g = layers.layer_norm_backward(x, o.sum, o.mean, o.rstd, w, p=0.1)
    r = layers.route_forward(x, 2)
    for out in (o, g, r):
        storages = [t.untyped_storage() for t in out]
        assert len({s.data_ptr() for s in storages}) == len(out)
        for t, s in zip(out, storages):
            assert s.nbytes() == t.numel() * t.element_size() and t.storage_offset() == 0


def test_other_threads_run_while_a_call_is_in_the_library(layers):
    # the library's entry point replaced by the C library's usleep, which takes the
    # number of elements for microseconds and returns 0 (no error)
    binding = layers._b()
    lib = muon().load()
    names = ("muon_layer_norm", "muon_layer_norm_backward", "muon_layer_norm_workspace_bytes",
             "muon_dropout", "muon_route", "muon_route_workspace_bytes", "muon_route_backward")
    real = {n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names}
    sleep = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p).value
    x = torch.zeros(500000, device="cuda")
    out = torch.empty_like(x)
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.005)

    thread = threading.Thread(target=tick)
    binding.bind(dict(real, muon_dropout=sleep))
    try:
        thread.start()
        begin = time.perf_counter()
        layers.dropout_forward(x, 0.5, seed=1, out=out)
        end = time.perf_counter()
    finally:
        stop.set()
        thread.join()
        binding.bind(real)
    assert end - begin >= 0.4                       # the call did wait ...
    assert sum(begin + 0.05 < t < end - 0.05 for t in ticks) >= 10      # ... and the thread ran
