"""The router with several token groups a warp, and its gradient against
differences that are sure to be taken, against torch in 64 bits (bounds as in
test_route_gpu)."""
import numpy as np
import pytest
import torch

import layers_ref as ref
from test_route_gpu import BF, F32, draw, layers  # noqa: F401

pytestmark = pytest.mark.gpu


# more tokens than the blocks take at once, in the form that shares a token among
# lanes (few enough tokens, or ragged rows): regular and ragged counts of experts
@pytest.mark.parametrize("tokens,experts,k", [(40000, 16, 2), (30011, 48, 5), (30011, 100, 6),
                                              (60000, 100, 3), (20000, 200, 9), (9000, 300, 4),
                                              (7000, 1000, 12), (70001, 64, 10)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("normalize", [True, False])
def test_many_tokens_a_warp(layers, tokens, experts, k, dtype, normalize):  # noqa: F811
    l = draw(tokens, experts, dtype, 21)
    g = torch.Generator().manual_seed(22)
    mask = (torch.rand(tokens, generator=g) > 0.1).cuda()
    l[~mask] = float("nan")
    l[:, experts // 2] = float("-inf")
    l[5:9] = float("-inf")
    mask[5:9] = True
    o = layers.route_forward(l, k, token_mask=mask, normalize=normalize)
    l64 = l.double()
    routed = mask & (l64 > float("-inf")).any(1)
    safe = torch.where(routed[:, None], l64, 0.0)
    p = torch.softmax(safe, 1) * routed[:, None]
    top, idx = torch.sort(safe, dim=1, descending=True, stable=True)
    below = (top[:, :1] - safe).clamp(max=1e6)
    top, idx = top[:, :k], idx[:, :k]
    ok = routed[:, None] & (top > float("-inf"))
    assert torch.equal(o.index.long(), torch.where(ok, idx, -1))
    w = torch.softmax(torch.where(ok, top, -1e300), 1) if normalize else p.gather(1, idx)
    w = torch.where(ok, w, 0.0)
    at = torch.where(ok, below.gather(1, idx), 0.0)
    assert bool(((o.weights.double() - w).abs() <= (at + 150) * ref.U * w + 1e-37).all())
    n = int(routed.sum())
    counts = torch.bincount(idx[ok], minlength=experts)
    assert torch.equal(o.counts.long(), torch.cat((counts, routed.sum()[None])))
    mp = p.sum(0) / n
    assert bool(((o.mean_prob.double() - mp).abs() <= 720 * ref.U * mp + 1e-37).all())
    loss = experts * float((counts.double() / (k * n) * mp).sum())
    assert abs(float(o.loss) - loss) <= 800 * ref.U * loss
    # gradient: (reach + 600) U of the terms' magnitude, one rounding to the type
    dw = torch.randn(tokens, k, generator=g).cuda()
    dl = torch.tensor(0.7, device="cuda")
    got = layers.route_backward(l, o.index, o.counts, dweights=dw, dloss=dl, token_mask=mask,
                                normalize=normalize).double()
    d = torch.where(ok, dw.double(), 0.0)
    b = (0.7 * experts / (k * n) / n * counts.double()).expand(tokens, experts)
    zero = torch.zeros_like(safe)
    if normalize:
        wd = (w * d).sum(1, keepdim=True)
        add = zero.scatter_add(1, idx, w * (d - wd))
        mag_add = zero.scatter_add(1, idx, w * (d.abs() + (w * d.abs()).sum(1, keepdim=True)))
        mag_b = b
    else:
        add, mag_add = zero, zero
        mag_b = b + zero.scatter_add(1, idx, d.abs())
        b = b + zero.scatter_add(1, idx, d)
    want = (p * (b - (p * b).sum(1, keepdim=True)) + add) * routed[:, None]
    mag = p * (mag_b + (p * mag_b).sum(1, keepdim=True)) + mag_add
    bound = (below + 600) * ref.U * mag + ref.out_ulp(dtype) * want.abs() + 1e-37
    assert bool(((got - want).abs() <= bound).all())


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("experts,k", [(12, 4), (64, 6), (100, 3)])
def test_gradient_against_differences_with_the_picks_held(layers, experts, k, normalize):  # noqa: F811
    # logits 0.05 apart in shuffled order: a step of h = 1e-3 along a direction of
    # entries below 5 cannot swap two of them.  Truncation O(h^2), rounding 1e-6 / h
    t, h = 25, 1e-3
    g = torch.Generator().manual_seed(31)
    order = torch.stack([torch.randperm(experts, generator=g) for _ in range(t)])
    l = (order.float() * 0.05).cuda()
    v = torch.randn(t, experts, generator=g).clamp(-5, 5).cuda()
    cw = torch.randn(t, k, generator=g).cuda()
    mask = torch.ones(t, dtype=torch.bool, device="cuda")
    mask[3] = False
    o = layers.route_forward(l, k, token_mask=mask, normalize=normalize)
    one = torch.tensor(0.3, device="cuda")
    grad = ref.f64(layers.route_backward(l, o.index, o.counts, dweights=cw, dloss=one, token_mask=mask,
                                         normalize=normalize))

    def total(z):
        q = layers.route_forward(z, k, token_mask=mask, normalize=normalize)
        assert torch.equal(q.index, o.index)
        return float((q.weights.double() * cw.double()).sum() + 0.3 * q.loss.double())

    fd = (total(l + h * v) - total(l - h * v)) / (2 * h)
    assert abs(fd - (grad * ref.f64(v)).sum()) <= 5e-3 * np.linalg.norm(grad) * float(v.norm())
