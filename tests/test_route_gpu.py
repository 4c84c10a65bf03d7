"""Expert router on the GPU against the 64-bit host reference.  Picks and
counts must agree exactly.  A probability costs one rounding of v - max (a
relative error of U per unit of it after exp), exp itself and a sum over the
experts: relative error <= (reach + 150) U, where reach is how far the logit
is below its row's largest.  Sums over tokens add at most 512 U."""
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


def draw(t, e, dtype, seed, std=1.5):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(t, e, generator=g) * std + torch.randn(e, generator=g)
    return l.to(dtype).cuda()


def reach(l):
    """How far each logit of a routed row is below its row's largest."""
    top = np.max(np.where(np.isnan(l), -np.inf, l), axis=1, initial=-np.inf, keepdims=True)
    with np.errstate(invalid="ignore", over="ignore"):
        d = top - l
    return np.where(np.isfinite(d), d, 0.0)


def check_forward(layers, l, k, mask, normalize):
    o = layers.route_forward(l, k, token_mask=mask, normalize=normalize)
    torch.cuda.synchronize()
    a, m = ref.f64(l), None if mask is None else mask.cpu().numpy().astype(bool)
    want = ref.route(a, k, m, normalize)
    assert o.index.dtype == o.counts.dtype == torch.int32
    assert np.array_equal(o.index.cpu().numpy(), want["index"])
    assert np.array_equal(o.counts.cpu().numpy(), want["counts"])
    d = reach(a)
    at = np.take_along_axis(d, np.maximum(want["index"], 0), 1)
    w = want["weights"]
    assert np.all(np.abs(ref.f64(o.weights) - w) <= (at + 150) * ref.U * w + 1e-37)
    n = max(1, int(want["counts"][-1]))
    mp = (want["p"] * (np.minimum(d, 1e6) + 700)).sum(0) * ref.U / n
    assert np.all(np.abs(ref.f64(o.mean_prob) - want["mean_prob"]) <= mp + 1e-37)
    bound = (want["counts"][:-1] / (k * n) * mp).sum() * l.shape[1] + 64 * ref.U * want["loss"]
    assert abs(float(o.loss) - want["loss"]) <= bound + 1e-37
    return o


def check_backward(layers, l, o, dw, dloss, mask, normalize):
    got = layers.route_backward(l, o.index, o.counts, dweights=dw, dloss=dloss, token_mask=mask,
                                normalize=normalize)
    torch.cuda.synchronize()
    a, m = ref.f64(l), None if mask is None else mask.cpu().numpy().astype(bool)
    index, counts = o.index.cpu().numpy(), o.counts.cpu().numpy()
    d64 = np.zeros(index.shape) if dw is None else ref.f64(dw)
    l64 = 0.0 if dloss is None else float(dloss)
    want = ref.route_grad(a, index, counts, d64, l64, m, normalize)
    q = ref.route(a, index.shape[1], m, normalize)
    e, k, n = a.shape[1], index.shape[1], max(1, int(counts[-1]))
    ab = np.broadcast_to(abs(l64) * e * counts[:e] / (k * n) / n, a.shape).copy()
    picked = np.zeros(a.shape)
    for t in range(a.shape[0]):
        for j, x in enumerate(index[t]):
            if x >= 0:
                if normalize:
                    picked[t, x] = q["weights"][t, j] * (abs(d64[t, j]) + (q["weights"][t] * np.abs(d64[t])).sum())
                else:
                    ab[t, x] += abs(d64[t, j])
    mag = q["p"] * (ab + (q["p"] * ab).sum(1, keepdims=True)) + picked
    bound = (np.minimum(reach(a), 1e6) + 600) * ref.U * mag + ref.out_ulp(l.dtype) * np.abs(want) + 1e-37
    g = ref.f64(got)
    assert np.all(np.abs(g - want) <= bound), np.max(np.abs(g - want) / bound)
    return got


def check_both(layers, l, k, mask=None, seed=0):
    g = torch.Generator().manual_seed(100 + seed)
    for normalize in (True, False):
        o = check_forward(layers, l, k, mask, normalize)
        dw = torch.randn(l.shape[0], k, generator=g).cuda()
        dl = torch.randn((), generator=g).cuda()
        check_backward(layers, l, o, dw, dl, mask, normalize)
        check_backward(layers, l, o, None, dl, mask, normalize)
        check_backward(layers, l, o, dw, None, mask, normalize)


SIZES = [(1, 1, 1), (1, 16, 2), (3, 2, 2), (65, 4, 1), (40, 7, 3), (33, 8, 8), (100, 9, 2),
         (96, 16, 2), (31, 17, 5), (64, 32, 4), (50, 33, 6), (257, 64, 6), (20, 65, 8),
         (40, 100, 3), (45, 128, 8), (30, 129, 7), (33, 160, 8), (20, 255, 10), (64, 256, 8),
         (10, 257, 4), (12, 300, 32), (9, 512, 8), (6, 513, 5), (5, 1000, 16), (6, 1024, 32),
         (12, 32, 32), (5000, 16, 2)]


@pytest.mark.parametrize("tokens,experts,k", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_route_and_gradient(layers, tokens, experts, k, dtype):
    check_both(layers, draw(tokens, experts, dtype, 1), k)


@pytest.mark.parametrize("experts,k", [(3, 2), (8, 4), (16, 2), (64, 6), (160, 8), (300, 3), (600, 9)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_masks_and_experts_out_of_service(layers, experts, k, dtype):
    t = 83
    l = draw(t, experts, dtype, 2)
    g = torch.Generator().manual_seed(3)
    mask = (torch.rand(t, generator=g) > 0.3).cuda()
    l[~mask] = float("nan")                               # padded tokens hold anything
    l[5:9] = float("-inf")                                # a row that leaves nothing
    l[10, 1:] = float("-inf")                             # fewer than k experts left
    l[11] = torch.finfo(dtype).min                        # the type's lowest value is a number
    l[12, ::2] = torch.finfo(dtype).min
    l[13, 0] = torch.finfo(dtype).max
    l[:, experts // 2] = float("-inf")                    # an expert that serves nobody
    check_both(layers, l, k, mask)
    check_both(layers, torch.where(mask[:, None], l, 0.0), k, mask.to(torch.uint8) * 200)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("experts,k", [(8, 3), (64, 8), (200, 32), (1024, 5)])
def test_ties_go_to_the_lowest_index(layers, dtype, experts, k):
    g = torch.Generator().manual_seed(4)
    l = torch.randint(-2, 3, (70, experts), generator=g).to(dtype).cuda()
    l[3] = 0.0
    l[4, ::3] = -0.0                                       # equal to +0
    l[4, 1::3] = 0.0
    check_both(layers, l, k)


@pytest.mark.parametrize("experts", [5, 16, 64, 100, 520])
@pytest.mark.parametrize("pad,lead", [(8, 0), (3, 0), (0, 1), (5, 7)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_row_strides_and_odd_addresses(layers, experts, pad, lead, dtype):
    t = 50
    buf = torch.full((t * (experts + pad) + lead,), 99.0, device="cuda", dtype=dtype)
    v = buf[lead:].view(t, experts + pad)[:, :experts]
    v.copy_(draw(t, experts, dtype, 5))
    check_both(layers, v, 2)


def test_all_masked_and_no_tokens(layers):
    l = draw(40, 16, F32, 6)
    mask = torch.zeros(40, dtype=torch.bool, device="cuda")
    check_both(layers, l, 2, mask)
    o = layers.route_forward(torch.empty((0, 16), device="cuda"), 2)
    assert o.weights.shape == (0, 2) and float(o.loss) == 0 and not o.counts.any() and not o.mean_prob.any()
    g = layers.route_backward(torch.empty((0, 16), device="cuda"), o.index, o.counts)
    assert g.shape == (0, 16)


def test_nan_and_inf_of_a_routed_token(layers):
    for dtype in (BF, F32):
        l = draw(20, 24, dtype, 7)
        l[3, 5] = float("nan")
        l[4, 6] = float("inf")
        o = layers.route_forward(l, 3)
        idx = o.index.cpu().numpy()
        assert idx[3, 0] == 5 and idx[4, 0] == 6
        assert all(len(set(r)) == 3 and r.min() >= 0 and r.max() < 24 for r in idx)
        w = ref.f64(o.weights)
        assert np.isnan(w[3]).all() and np.isnan(w[4, 0]) and np.isfinite(np.delete(w, [3, 4], 0)).all()
        assert np.isnan(float(o.loss)) and int(o.counts[-1]) == 20
        g = ref.f64(layers.route_backward(l, o.index, o.counts, dweights=torch.ones_like(o.weights)))
        assert np.isfinite(np.delete(g, [3, 4], 0)).all() and np.isnan(g[3]).any() and np.isnan(g[4]).any()


def test_nan_of_either_sign_ranks_first(layers):
    for dtype in (BF, F32):
        l = draw(6, 100, dtype, 14)
        l[1, 70], l[2, 3] = float("nan"), -l.new_tensor(float("nan"))
        l[2, 50] = float("inf")
        idx = layers.route_forward(l, 2).index.cpu().numpy()
        assert idx[1, 0] == 70 and list(idx[2]) == [3, 50]


def test_indices_out_of_range_are_missing_picks(layers):
    l = draw(30, 16, F32, 8)
    o = layers.route_forward(l, 3)
    bad = o.index.clone()
    bad[4, 1], bad[5, 2], bad[6, 0] = -7, 16, 1 << 30
    fixed = torch.where((bad < 0) | (bad >= 16), -1, bad)
    dw = torch.randn(30, 3, device="cuda")
    for normalize in (True, False):
        a = layers.route_backward(l, bad, o.counts, dweights=dw, normalize=normalize)
        b = layers.route_backward(l, fixed, o.counts, dweights=dw, normalize=normalize)
        assert torch.equal(a, b)


def test_gradients_of_missing_picks_have_no_effect(layers):
    l = draw(40, 12, F32, 15)
    l[3:9, 2:] = float("-inf")                    # two experts left for four picks
    mask = torch.ones(40, dtype=torch.bool, device="cuda")
    mask[20:25] = False
    dw = torch.randn(40, 4, device="cuda")
    for normalize in (True, False):
        o = layers.route_forward(l, 4, token_mask=mask, normalize=normalize)
        bad = torch.where(o.index < 0, float("nan"), dw)
        a = layers.route_backward(l, o.index, o.counts, dweights=bad, dloss=o.loss, token_mask=mask,
                                  normalize=normalize)
        b = layers.route_backward(l, o.index, o.counts, dweights=dw, dloss=o.loss, token_mask=mask,
                                  normalize=normalize)
        assert int((o.index < 0).sum()) == 6 * 2 + 5 * 4 and torch.equal(a, b)


def test_same_bits_every_time_and_on_another_stream(layers):
    l = draw(30011, 48, BF, 9)
    dw = torch.randn(30011, 5, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    runs = []
    for stream in (None, None, side):
        o = layers.route_forward(l, 5, stream=stream)
        runs.append(list(o) + [layers.route_backward(l, o.index, o.counts, dweights=dw,
                                                     dloss=o.loss, stream=stream)])
    side.synchronize()
    torch.cuda.synchronize()
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_many_tokens(layers):
    # more tokens than the blocks take at once: counts and sums against torch in 64 bits
    for tokens, experts, k, dtype in ((200003, 24, 4, BF), (70001, 256, 8, F32)):
        l = draw(tokens, experts, dtype, 10)
        o = layers.route_forward(l, k, normalize=False)
        p = torch.softmax(l.double(), 1)
        idx = torch.sort(l.float(), dim=1, descending=True, stable=True)[1][:, :k]
        assert torch.equal(o.index.long(), idx)
        c = torch.bincount(idx.reshape(-1), minlength=experts)
        assert torch.equal(o.counts.long(), torch.cat((c, torch.tensor([tokens], device="cuda"))))
        mp = p.mean(0)
        assert bool(((o.mean_prob.double() - mp).abs() <= 720 * ref.U * mp).all())
        loss = experts * float((c.double() / (k * tokens) * mp).sum())
        assert abs(float(o.loss) - loss) <= 800 * ref.U * loss


@pytest.mark.parametrize("experts,k", [(8, 1), (16, 2), (24, 3), (40, 4), (64, 6), (72, 5), (160, 8),
                                       (256, 8), (512, 7)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("normalize", [True, False])
def test_large_batches(layers, experts, k, dtype, normalize):
    # batches of many tokens, with ties, padded tokens, rows that leave nothing
    # or fewer than k experts, and numbers at the type's ends, against torch in
    # 64 bits; the same tokens in small batches give the same picks
    tokens = 49152 + 77
    g = torch.Generator().manual_seed(16)
    l = (torch.randint(-12, 13, (tokens, experts), generator=g) / 4).to(dtype).cuda()
    l[::3] = draw(len(range(0, tokens, 3)), experts, dtype, 17)
    mask = (torch.rand(tokens, generator=g) > 0.1).cuda()
    mask[1000:1040] = mask[2000:2030] = mask[3000:3003] = True
    l[~mask] = float("nan")
    l[1000:1040] = float("-inf")
    l[2000:2030, min(2, experts - 1):] = float("-inf")
    l[3000] = torch.finfo(dtype).min
    l[3001, ::2] = torch.finfo(dtype).min
    l[3002, 0] = torch.finfo(dtype).max
    l[2000:2030, :2] = 1.0
    o = layers.route_forward(l, k, token_mask=mask, normalize=normalize)
    l64 = l.double()
    routed = mask & (l64 > float("-inf")).any(1)
    safe = torch.where(routed[:, None], l64, 0.0)
    p = torch.softmax(safe, 1) * routed[:, None]
    top, idx = torch.sort(safe, dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    ok = routed[:, None] & (top > float("-inf"))
    assert torch.equal(o.index.long(), torch.where(ok, idx, -1))
    w = torch.softmax(torch.where(ok, top, -1e300), 1) if normalize else p.gather(1, idx)
    w = torch.where(ok, w, 0.0)
    at = torch.where(ok, (top[:, :1] - top).clamp(max=1e6), 0.0)
    assert bool(((o.weights.double() - w).abs() <= (at + 150) * ref.U * w + 1e-37).all())
    n = int(routed.sum())
    assert torch.equal(o.counts.long(), torch.cat((torch.bincount(idx[ok], minlength=experts),
                                                   routed.sum()[None])))
    mp = p.sum(0) / n
    assert bool(((o.mean_prob.double() - mp).abs() <= 720 * ref.U * mp + 1e-37).all())
    part = layers.route_forward(l[900:3100], k, token_mask=mask[900:3100], normalize=normalize)
    assert torch.equal(part.index, o.index[900:3100])
    dw = torch.randn(tokens, k, device="cuda")
    a = layers.route_backward(l, o.index, o.counts, dweights=dw, dloss=o.loss, token_mask=mask,
                              normalize=normalize)
    b = layers.route_backward(l[900:3100], o.index[900:3100].contiguous(), o.counts,
                              dweights=dw[900:3100].contiguous(), dloss=o.loss,
                              token_mask=mask[900:3100], normalize=normalize)
    assert torch.equal(a[900:3100], b)


def test_more_than_32_bits_of_logits(layers):
    tokens, experts, k = (1 << 22) + 37, 520, 3
    l = torch.zeros((tokens, experts), device="cuda", dtype=BF)
    l[-20:] = draw(20, experts, BF, 11)
    o = layers.route_forward(l, k)
    tail = layers.route_forward(l[-20:].clone(), k)
    assert torch.equal(o.index[-20:], tail.index) and torch.equal(o.weights[-20:], tail.weights)
    assert torch.equal(o.index[:5].cpu(), torch.arange(3, dtype=torch.int32).expand(5, 3))
    dw = torch.zeros(tokens, k, device="cuda")
    dw[-20:] = torch.randn(20, k, device="cuda")
    g = layers.route_backward(l, o.index, o.counts, dweights=dw)
    h = layers.route_backward(l[-20:].clone(), tail.index, tail.counts, dweights=dw[-20:].clone())
    assert torch.equal(g[-20:], h) and not g[:-20].any()


@pytest.mark.parametrize("normalize", [True, False])
def test_autograd_and_differences(layers, normalize):
    l = draw(25, 12, F32, 12)
    cw = torch.randn(25, 4, device="cuda")
    mask = torch.ones(25, dtype=torch.bool, device="cuda")
    mask[3] = False
    x = l.clone().requires_grad_()
    o = layers.route(x, 4, token_mask=mask, normalize=normalize)
    ((o.weights * cw).sum() + 0.3 * o.loss).backward()
    want = ref.route_grad(ref.f64(l), o.index.cpu().numpy(), o.counts.cpu().numpy(), ref.f64(cw),
                          0.3, mask.cpu().numpy(), normalize)
    g = ref.f64(x.grad)
    assert np.linalg.norm(g - want) <= 1e-5 * np.linalg.norm(want)
    x.grad = None
    layers.route(x, 4, token_mask=mask, normalize=normalize).loss.backward()    # the loss alone
    assert np.linalg.norm(ref.f64(x.grad)) > 0 and not ref.f64(x.grad)[3].any()
    # central differences of the GPU's own forward pass (picks unchanged):
    # truncation O(h^2), rounding 1e-6 / h
    v = torch.randn(25, 12, device="cuda")
    h = 1e-3

    def total(z):
        q = layers.route_forward(z, 4, token_mask=mask, normalize=normalize)
        same = torch.equal(q.index, o.index)
        return float((q.weights.double() * cw.double()).sum() + 0.3 * q.loss.double()), same

    (a, sa), (b, sb) = total(l + h * v), total(l - h * v)
    if sa and sb:
        assert abs((a - b) / (2 * h) - (want * ref.f64(v)).sum()) <= 5e-3 * np.linalg.norm(want) * float(v.norm())


def test_leading_dimensions(layers):
    l = draw(24, 16, F32, 13)
    a = layers.route_forward(l.view(2, 3, 4, 16), 2)
    b = layers.route_forward(l, 2)
    assert a.weights.shape == (2, 3, 4, 2) and torch.equal(a.index.view(24, 2), b.index)


def test_refusals(layers):
    l = torch.zeros((4, 8), device="cuda")
    o = layers.route_forward(l, 2)
    with pytest.raises(muon().MuonError):
        layers.route_forward(l, 9)
    with pytest.raises(muon().MuonError):
        layers.route_forward(l, 0)
    with pytest.raises(ValueError):
        layers.route_forward(l.t(), 2)
    with pytest.raises(TypeError):
        layers.route_forward(l, 2, token_mask=torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        layers.route_forward(l, 2, token_mask=torch.ones(3, device="cuda", dtype=torch.bool))
    with pytest.raises(TypeError):
        layers.route_backward(l, o.index.long(), o.counts)
    with pytest.raises(ValueError):
        layers.route_backward(l, o.index, o.counts[:4])
    with pytest.raises(ValueError):
        layers.route_backward(l, o.index[:2], o.counts)
