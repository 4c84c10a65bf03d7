"""Gated linear recurrence at gates near 1, where what a token takes in and what
the state loses are far below the state: against the 64-bit recurrence, with room for
their own relative error and not for one of the size of the state's."""
import numpy as np
import pytest
import torch

import sequence_ref as ref
from helpers import muon

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U = ref.U


@pytest.fixture(scope="module")
def layers():
    muon()
    from newton_schulz_05_gb300 import layers
    return layers


def recurrence(gate, x, state, mix):
    """(h, error).  With u = 1 - a and size the recurrence of absolute values, a token has
    the relative error of the smaller of a and u (three roundings of t = exp(-|g|)'s argument, 4 U of the
    power, 1 + t, 2 U of the reciprocal, their product: (3 |g| + 12) U) of what it
    multiplies, three roundings of its input, and six of the carried state: a's own 3 U and
    a product in the tokens that one thread takes, and the joins."""
    p = np.zeros(x[:, 0].shape) if state is None else state.copy()
    size, err = np.abs(p), np.zeros(p.shape)
    h, eh = np.zeros(x.shape), np.zeros(x.shape)
    for i in range(x.shape[1]):
        g, v = gate[:, i], x[:, i]
        e = np.exp(-np.abs(g))
        a, u = np.where(g >= 0, 1, e) / (1 + e), np.where(g >= 0, e, 1) / (1 + e)
        share = (3 * np.abs(g) + 12) * U
        w = u if mix else 1.0
        err = a * err + np.minimum(a, u) * share * size + 6 * U * a * size + w * np.abs(v) * (share * mix + 3 * U)
        p, size = a * p + w * v, a * size + w * np.abs(v)
        h[:, i], eh[:, i] = p, err
    return h, eh


def inputs(b, t, d, dtype, seed):
    """Gates of 6 to 20, one a channel; inputs of either sign."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    gate = torch.linspace(6, 20, d, device="cuda").to(dtype).expand(b, t, d).contiguous()
    return gate, torch.randn(b, t, d, generator=gen, device="cuda").to(dtype), gen


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("mix", [True, False])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("b,t,d", [(2, 1, 64), (2, 3, 72), (3, 16, 33), (400, 20, 512), (2, 40, 64), (1, 300, 130),
                                   (2, 300, 64), (20, 70, 1024)])
def test_gates_near_one(layers, b, t, d, state, mix, dtype):
    gate, x, gen = inputs(b, t, d, dtype, t)
    # far below what comes in, so that it does not hide it
    s = 1e-3 * torch.randn(b, d, generator=gen, device="cuda") if state else None
    o = layers.gated_scan_forward(gate, x, state=s, mix=mix)
    h, err = recurrence(ref.f64(gate), ref.f64(x), None if s is None else ref.f64(s), mix)
    ref.close(o.h, h, err, dtype)
    ref.close(o.state, h[:, -1], err[:, -1], F32)
    dh, ds = torch.randn(x.shape, generator=gen, device="cuda").to(dtype), torch.randn(b, d, generator=gen, device="cuda")
    g = layers.gated_scan_backward(dh, gate, x, o.h, state=s, dstate=ds, mix=mix)
    want, room = ref.scan_grad(ref.f64(dh), ref.f64(gate), ref.f64(x), ref.f64(o.h), None if s is None else ref.f64(s),
                               ref.f64(ds), None, None, mix)
    for got, e, r, kind in zip(g, want, room, (dtype, dtype, F32)):
        ref.close(got, e, r, kind)


@pytest.mark.parametrize("mix", [True, False])
def test_gates_near_one_a_token_at_a_time(layers, mix):
    gate, x, _ = inputs(2, 50, 64, F32, 5)
    h, err = recurrence(ref.f64(gate), ref.f64(x), None, mix)
    state = torch.zeros(2, 64, device="cuda")
    for t in range(50):
        o = layers.gated_scan_forward(gate[:, t:t + 1], x[:, t:t + 1], state=state, mix=mix)
        ref.close(o.h[:, 0], h[:, t], err[:, t], F32)
        state = o.state


def test_constant_input_stays_a_token_at_a_time(layers):
    # 2000 tokens of gate 8 come back to the state by half of its rounding each at most where
    # they are added as take * (x - p), and that difference is 0 here
    gate, x = torch.full((1, 1, 64), 8.0, device="cuda"), torch.full((1, 1, 64), 0.7, device="cuda")
    state = x[:, 0].clone()
    for _ in range(2000):
        state = layers.gated_scan_forward(gate, x, state=state).state
    assert float((state - 0.7).abs().max()) < 1e-6


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_state_decays_over_a_long_document(layers, dtype):
    """Nothing comes in, and each token takes less than fp32's step at 1 from the state: a segment of
    at least 8 tokens rounds it once, besides the error of what the tokens lose."""
    t = 65536
    gate = torch.linspace(16, 18.5, 64, device="cuda").to(dtype)
    x = torch.zeros(1, t, 64, device="cuda", dtype=dtype)
    lose = 1 / (1 + np.exp(ref.f64(gate)))
    want = np.exp(t * np.log1p(-lose))
    room = want * (t / 8 * U + t * lose * (3 * ref.f64(gate) + 12) * U + 64 * U)
    for mix in (True, False):
        o = layers.gated_scan_forward(gate.expand(1, t, 64).contiguous(), x, state=torch.ones(1, 64, device="cuda"), mix=mix)
        ref.close(o.state[0], want, room, F32)
