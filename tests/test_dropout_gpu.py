"""Dropout on the GPU against the 64-bit host reference: which elements are
kept must agree exactly, values within one fp32 rounding per operation and one
to the output's type."""
import numpy as np
import pytest
import torch

import layers_ref as ref
from helpers import muon

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def layers():
    muon()
    from newton_schulz_05_gb300 import layers
    return layers


def draw(n, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, generator=g)
    return torch.where(x == 0, 1.0, x).to(dtype).cuda()


def check(y, x, r, p, seed, offset, start=0):
    f = ref.factors(x.numel(), p, seed, offset, start)
    a = ref.f64(x).reshape(-1) * f
    want = a if r is None else a + ref.f64(r).reshape(-1)
    got = ref.f64(y).reshape(-1)
    bound = 2 * ref.U * (np.abs(a) + np.abs(want)) + ref.out_ulp(x.dtype) * np.abs(want)
    assert np.all(np.abs(got - want) <= bound)
    if r is None:
        assert np.array_equal(got == 0, f == 0)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 64, 1000, 4099, 65536, 100003, 1 << 20])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("p", [0.1, 0.5])
def test_dropout(layers, n, dtype, p):
    x, r = draw(n, dtype, 1), draw(n, dtype, 2)
    for seed, offset in ((0, 0), (0xFEDCBA9876543210, (1 << 32) - 3), (7, (1 << 63) + 5)):
        check(layers.dropout_forward(x, p, seed=seed, offset=offset), x, None, p, seed, offset)
        check(layers.dropout_forward(x, p, seed=seed, offset=offset, residual=r), x, r, p, seed, offset)


@pytest.mark.parametrize("leads", [(1, 1, 1), (3, 0, 0), (0, 5, 0), (0, 0, 2), (4, 4, 4), (8, 8, 8)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_odd_addresses(layers, dtype, leads):
    n = 5003
    x, r = draw(n + 8, dtype, 1)[leads[0]:leads[0] + n], draw(n + 8, dtype, 2)[leads[1]:leads[1] + n]
    buf = torch.full((n + 16,), 9.0, device="cuda", dtype=dtype)
    y = buf[leads[2]:leads[2] + n]
    check(layers.dropout_forward(x, 0.3, seed=4, offset=6, residual=r, out=y), x, r, 0.3, 4, 6)
    assert bool((buf[:leads[2]] == 9).all()) and bool((buf[leads[2] + n:] == 9).all())


def test_edges_of_p_and_in_place(layers):
    x, r = draw(1003, F32, 1), draw(1003, F32, 2)
    assert torch.equal(layers.dropout_forward(x, 0.0, seed=1), x)
    assert not layers.dropout_forward(x, 1.0, seed=1).any()
    assert torch.equal(layers.dropout_forward(x, 1.0, seed=1, residual=r), r)
    want = layers.dropout_forward(x, 0.4, seed=1, residual=r)
    for out in (x.clone(), r.clone()):
        a = dict(x=x, residual=r)
        a["x" if torch.equal(out, x) else "residual"] = out
        got = layers.dropout_forward(a["x"], 0.4, seed=1, residual=a["residual"], out=out)
        assert got is out and torch.equal(out, want)


def test_dropped_infinities_are_zeros(layers):
    f = ref.factors(4000, 0.5, 3, 0)
    x = draw(4000, BF, 1)
    bad = torch.where(torch.from_numpy(f == 0).cuda(), torch.tensor(float("nan"), dtype=BF, device="cuda"), x)
    bad[np.flatnonzero(f == 0)[::2].tolist()] = float("inf")
    assert torch.equal(layers.dropout_forward(bad, 0.5, seed=3), layers.dropout_forward(x, 0.5, seed=3))


def test_nothing_to_do_and_another_stream(layers):
    assert layers.dropout_forward(torch.empty(0, device="cuda"), 0.1, seed=1).numel() == 0
    x = draw(70001, BF, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = layers.dropout_forward(x, 0.1, seed=1, stream=side)
    b = layers.dropout_forward(x, 0.1, seed=1)
    side.synchronize()
    assert torch.equal(a, b)


def test_more_than_32_bits_of_elements(layers):
    n = (1 << 32) + 4099
    x = torch.ones(n, device="cuda", dtype=BF)
    y = layers.dropout_forward(x, 0.3, seed=5, offset=2)
    for start in (0, (1 << 31) - 100, (1 << 32) - 100, n - 2001):
        check(y[start:start + 2001], x[start:start + 2001], None, 0.3, 5, 2, start)


def test_autograd(layers):
    x, r = (draw(999, F32, i).view(27, 37).requires_grad_() for i in (1, 2))
    c = draw(999, F32, 3).view(27, 37)
    y = layers.dropout(x, 0.3, seed=6, offset=1, residual=r)
    (y * c).sum().backward()
    f = ref.factors(999, 0.3, 6, 1).reshape(27, 37)
    want = ref.f64(c) * f
    assert np.all(np.abs(ref.f64(x.grad) - want) <= 2 * ref.U * np.abs(want))
    assert torch.equal(r.grad, c)
    x.grad = None
    layers.dropout(x.t(), 0.3, seed=6).sum().backward()      # strided input, expanded gradient
    f = ref.factors(999, 0.3, 6, 0).reshape(37, 27).T
    assert np.all(np.abs(ref.f64(x.grad) - f) <= 2 * ref.U * f)


def test_refusals(layers):
    x = torch.zeros((4, 8), device="cuda")
    with pytest.raises(ValueError):
        layers.dropout_forward(x.t(), 0.1, seed=0)
    with pytest.raises(ValueError):
        layers.dropout_forward(x, 0.1, seed=0, residual=x[:2])
    with pytest.raises(TypeError):
        layers.dropout_forward(x, 0.1, seed=0, out=x.bfloat16())
    with pytest.raises(muon().MuonError):
        layers.dropout_forward(x, -0.1, seed=0)
