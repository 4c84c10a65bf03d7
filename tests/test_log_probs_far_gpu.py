"""Gradient of token log probabilities for rows far from zero: nothing but the type's
lowest or highest value, and logits whose log sum has no digits left for the rest."""
import numpy as np
import pytest
import torch

import sequence_ref as ref
from helpers import muon

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def layers():
    muon()
    from newton_schulz_05_gb300 import layers
    return layers


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [0.5, 1.0, 2.0])
@pytest.mark.parametrize("v", [5, 40, 1000, 5000, 70001])
def test_rows_far_from_zero(layers, v, scale, dtype):
    ends = torch.finfo(dtype)
    gen = torch.Generator(device="cuda").manual_seed(v)
    l = torch.randn(7, v, generator=gen, device="cuda")
    l[0], l[1], l[2], l[3] = ends.min, ends.max, -1e9, 1e9
    l[4] = l[4] * 100 - 1e6
    l[5, 1:] = ends.min           # one symbol left
    l = l.to(dtype)
    y = torch.tensor([0, 1, 2, 3, 4, 0, 1], device="cuda")
    o = layers.token_log_probs_forward(l, y, scale=scale)
    # equal logits: the sum of v ones and its logarithm, at most 1024 additions in a row
    assert float((o.log_probs[:4] + np.log(v)).abs().max()) <= (1024 + 8 + 4 * np.log(v)) * ref.U
    d = torch.tensor([1.0, -2.0, 0.5, 1.0, 1.0, 1.0, 1.0], device="cuda")
    got = layers.token_log_probs_backward(d, l, y, o.lse, scale=scale)
    with np.errstate(over="ignore"):
        arg = np.minimum(scale * ref.f64(l) - ref.f64(o.lse)[:, None], 0)
    p = np.exp(arg)
    hot = np.zeros(p.shape)
    hot[np.arange(7), y.cpu().numpy()] = 1
    f = scale * ref.f64(d)[:, None]
    # the argument is rounded twice more and its base changed, 4 U of the power, the products
    rel = np.where(p > 0, (4 * np.abs(np.where(p > 0, arg, 0)) + 12) * ref.U, 0)
    # a power under the smallest normal number, 2^-126, is 0: off by less than that, times |f|
    ref.close(got, f * (hot - p), np.abs(f) * (p * rel + 4 * ref.U * hot + 2.0 ** -126), dtype)


def test_rows_without_meaning_are_not_hidden(layers):
    l = torch.zeros(4, 40, device="cuda")
    l[0, 3], l[1, 3], l[2] = float("nan"), float("inf"), float("-inf")
    y, d = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.ones(4, device="cuda")
    o = layers.token_log_probs_forward(l, y)
    g = layers.token_log_probs_backward(d, l, y, o.lse)
    assert bool(o.log_probs[:3].isnan().all()) and bool(g[:3].isnan().all()) and bool(g[3].isfinite().all())
