"""Layer norm, alone and behind dropout and the residual add, and its gradient
on the GPU, against the 64-bit host reference.  Every output must lie within
the bound that layers_ref derives from fp32 sums of a row's (a column's)
length, plus one rounding to its own type."""
import numpy as np
import pytest
import torch

import layers_ref as ref
from helpers import muon

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


@pytest.fixture(scope="module")
def layers():
    muon()
    from newton_schulz_05_gb300 import layers
    return layers


def draw(shape, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(dtype).cuda()


def placed(t, pad, lead):
    """t's values as rows `pad` elements further apart, starting `lead`
    elements into their storage."""
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + lead,), 7.0, dtype=t.dtype, device=t.device)
    v = buf[lead:lead + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(t)
    return v


def near(got, want, bound, dtype):
    got = ref.f64(got).reshape(np.shape(want))
    tol = bound + ref.out_ulp(dtype) * np.abs(want) + 1e-37
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)


def check_forward(layers, x, r, w, b, p, seed=11, offset=5):
    o = layers.layer_norm_forward(x, w, b, eps=EPS, residual=r, p=p, seed=seed, offset=offset)
    torch.cuda.synchronize()
    rows, cols = x.shape
    f = ref.factors(rows * cols, p, seed, offset).reshape(rows, cols)
    a = [None if t is None else ref.f64(t) for t in (x, r, w, b)]
    eps = float(np.float32(EPS))
    y, s, mean, rstd = ref.norm(*a, eps, f)
    ds, dm, dr, dy = ref.norm_bounds(*a, eps, f)
    near(o.y, y, dy, x.dtype)
    near(o.mean, mean, dm, F32)
    near(o.rstd, rstd, dr, F32)
    if r is None and p == 0:
        assert o.sum is x
    else:
        near(o.sum, s, ds, x.dtype)
    return o


def check_backward(layers, dy, s, mean, rstd, w, ds, p, seed=11, offset=5):
    g = layers.layer_norm_backward(dy, s, mean, rstd, w, dsum=ds, p=p, seed=seed, offset=offset)
    torch.cuda.synchronize()
    rows, cols = dy.shape
    f = ref.factors(rows * cols, p, seed, offset).reshape(rows, cols)
    a = [None if t is None else ref.f64(t) for t in (dy, s, mean.view(-1), rstd.view(-1), w, ds)]
    want, bound = ref.norm_grad(*a, f)
    near(g.dx, want[0], bound[0], dy.dtype)
    near(g.dresidual, want[1], bound[1], dy.dtype)
    wdt = F32 if w is None else w.dtype
    assert g.dweight.dtype == g.dbias.dtype == wdt
    near(g.dweight, want[2], bound[2], wdt)
    near(g.dbias, want[3], bound[3], wdt)
    if p == 0:
        assert g.dresidual is g.dx
    else:   # a dropped element's gradient is an exact zero
        assert not ref.f64(g.dx)[f == 0].any()
    return g


# rows x cols: one element, one row, widths around every change of layout, odd
# widths, and rows longer than one block holds
SIZES = [(1, 1), (3, 2), (1, 2048), (5, 7), (64, 8), (33, 63), (9, 64), (17, 65), (300, 100),
         (41, 255), (40, 256), (7, 257), (1000, 24), (19, 511), (12, 512), (11, 1000), (6, 1023),
         (6, 1024), (5, 1025), (4, 1409), (9, 2047), (3, 2050), (700, 128), (5, 4096), (3, 4097),
         (2, 8191), (3, 8192), (2, 10240), (2, 11008), (3, 16383), (2, 16384), (2, 16392),
         (1, 20001)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype,wdtype", [(BF, F32), (BF, BF), (F32, F32), (F32, BF)])
def test_norm_and_gradient(layers, rows, cols, dtype, wdtype):
    x = draw((rows, cols), dtype, 1, 1.3, 0.4)
    w, b = draw(cols, wdtype, 2, 0.3, 1.0), draw(cols, wdtype, 3, 0.2)
    o = check_forward(layers, x, None, w, b, 0.0)
    check_backward(layers, draw((rows, cols), dtype, 4, 0.1), x, o.mean, o.rstd, w, None, 0.0)


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_dropout_add_norm_and_gradient(layers, rows, cols, dtype):
    x, r = draw((rows, cols), dtype, 1, 1.3), draw((rows, cols), dtype, 5, 2.0, -0.3)
    w, b = draw(cols, dtype, 2, 0.3, 1.0), draw(cols, dtype, 3, 0.2)
    o = check_forward(layers, x, r, w, b, 0.25)
    check_backward(layers, draw((rows, cols), dtype, 4, 0.1), o.sum, o.mean, o.rstd, w,
                   draw((rows, cols), dtype, 6, 0.1), 0.25)


@pytest.mark.parametrize("pads,leads", [((0, 0, 0), (1, 1, 1)), ((8, 8, 8), (0, 0, 0)),
                                        ((3, 3, 3), (0, 0, 0)), ((0, 8, 3), (0, 0, 0)),
                                        ((1, 0, 5), (3, 0, 2)), ((8, 0, 8), (4, 4, 4))])
@pytest.mark.parametrize("rows,cols", [(13, 96), (21, 1000), (10, 1023), (9, 4100)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_row_strides_and_odd_addresses(layers, rows, cols, dtype, pads, leads):
    # x, residual and dsum (dy and sum share x's and residual's placement)
    x, r = draw((rows, cols), dtype, 1), draw((rows, cols), dtype, 5)
    dy, ds = draw((rows, cols), dtype, 4, 0.1), draw((rows, cols), dtype, 6, 0.1)
    wbuf, bbuf = draw(cols + 3, dtype, 2, 0.3, 1.0), draw(cols + 1, dtype, 3)
    w, b = wbuf[3:], bbuf[1:]
    o = check_forward(layers, placed(x, pads[0], leads[0]), placed(r, pads[1], leads[1]), w, b, 0.1)
    for p in (0.0, 0.1):
        check_backward(layers, placed(dy, pads[0], leads[0]), placed(o.sum, pads[1], leads[1]),
                       o.mean, o.rstd, w, placed(ds, pads[2], leads[2]), p)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [40, 1024, 3000])
def test_without_weight_bias_or_parts_of_the_gradient(layers, dtype, cols):
    x, dy = draw((50, cols), dtype, 1), draw((50, cols), dtype, 4, 0.1)
    w, b = draw(cols, F32, 2, 0.3, 1.0), draw(cols, F32, 3)
    check_forward(layers, x, None, None, None, 0.0)
    check_forward(layers, x, None, None, b, 0.0)
    check_forward(layers, x, None, None, None, 0.5)      # dropout without a residual
    check_forward(layers, x, x, None, None, 0.0)         # a residual without dropout
    o = check_forward(layers, x, None, w, None, 0.0)
    full = check_backward(layers, dy, x, o.mean, o.rstd, w, None, 0.0)
    check_backward(layers, dy, x, o.mean, o.rstd, None, None, 0.0)
    for nw, nb in ((True, False), (False, True), (False, False)):
        g = layers.layer_norm_backward(dy, x, o.mean, o.rstd, w, need_weight=nw, need_bias=nb)
        assert (g.dweight is not None) == nw and (g.dbias is not None) == nb
        near(g.dx, ref.f64(full.dx), 1e-6 * np.abs(ref.f64(full.dx)), dtype)
        if nw:
            assert torch.equal(g.dweight, full.dweight)
        if nb:
            assert torch.equal(g.dbias, full.dbias)


@pytest.mark.parametrize("cols", [64, 999, 4096, 20000])
def test_loud_offset_rows_keep_their_variance(layers, cols):
    # a mean a thousand times the spread, and one channel a thousand times the rest
    x = draw((6, cols), F32, 1, 1.0, 1000.0)
    x[3:] -= 1000.0
    x[3:, 0] = 1000.0
    check_forward(layers, x, None, None, None, 0.0)


def test_constant_rows_and_infinities_stay_in_their_row(layers):
    x = draw((6, 300), F32, 1)
    x[1] = 3.0
    x[2, 7] = float("inf")
    x[3, 9] = float("nan")
    o = layers.layer_norm_forward(x)
    y = ref.f64(o.y)
    assert np.all(np.abs(y[1]) <= 300 * 3 * ref.U / np.sqrt(EPS))
    assert np.isnan(y[2]).any() and np.isnan(y[3]).all()
    want = ref.norm(ref.f64(x)[[0, 4, 5]], None, None, None, EPS, np.ones((3, 300)))[0]
    assert np.allclose(y[[0, 4, 5]], want, atol=1e-4)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_dropped_infinities_are_zeros(layers, dtype):
    rows, cols, p = 20, 777, 0.5
    f = ref.factors(rows * cols, p, 3, 0).reshape(rows, cols)
    x = draw((rows, cols), dtype, 1)
    r = draw((rows, cols), dtype, 2)
    bad = x.clone()
    bad[torch.from_numpy(f == 0).cuda()] = float("nan")
    a = layers.layer_norm_forward(x, residual=r, p=p, seed=3)
    b = layers.layer_norm_forward(bad, residual=r, p=p, seed=3)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


# a probability that rounds to nothing, the largest below one, and one, on both
# sides of every choice of how the random bits are drawn: NaN and infinities in
# dropped places leave no trace, forwards or backwards
@pytest.mark.parametrize("p", [1e-6, 0.3, 65535 / 65536, 1.0])
@pytest.mark.parametrize("dtype,cols", [(BF, 512), (BF, 4096), (BF, 5632), (BF, 16384), (BF, 1001),
                                        (BF, 16400), (F32, 256), (F32, 4096), (F32, 10240),
                                        (F32, 333)])
def test_extreme_dropout(layers, dtype, cols, p):
    rows = 7
    x, r = draw((rows, cols), dtype, 1), draw((rows, cols), dtype, 5)
    w, b = draw(cols, dtype, 2, 0.3, 1.0), draw(cols, dtype, 3, 0.2)
    o = check_forward(layers, x, r, w, b, p)
    check_backward(layers, draw((rows, cols), dtype, 4, 0.1), o.sum, o.mean, o.rstd, w, None, p)
    f = ref.factors(rows * cols, p, 11, 5).reshape(rows, cols)
    gone = torch.from_numpy(f == 0).cuda()
    bad = x.clone()
    bad[gone] = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda",
                             dtype=dtype).repeat(gone.sum() // 3 + 1)[:gone.sum()]
    again = layers.layer_norm_forward(bad, w, b, eps=EPS, residual=r, p=p, seed=11, offset=5)
    assert all(torch.equal(u, v) for u, v in zip(o, again))


@pytest.mark.parametrize("shape", [(0, 16), (2, 0, 16)])
def test_no_rows(layers, shape):
    x = torch.empty(shape, device="cuda", dtype=BF)
    w = torch.ones(16, device="cuda")
    o = layers.layer_norm_forward(x, w, w)
    assert o.y.shape == shape and o.mean.shape == shape[:-1]
    g = layers.layer_norm_backward(x, x, o.mean, o.rstd, w)
    assert g.dx.shape == shape and not g.dweight.any() and not g.dbias.any()


def test_same_bits_every_time_and_on_another_stream(layers):
    x, r, dy = (draw((3000, 1001), BF, i) for i in range(3))
    w = draw(1001, F32, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    runs = []
    for stream in (None, None, side):
        o = layers.layer_norm_forward(x, w, w, residual=r, p=0.1, seed=8, stream=stream)
        g = layers.layer_norm_backward(dy, o.sum, o.mean, o.rstd, w, dsum=r, p=0.1, seed=8,
                                       stream=stream)
        runs.append(list(o) + list(g))
    side.synchronize()
    torch.cuda.synchronize()
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_more_than_32_bits_of_elements(layers):
    rows, cols = 262200, 8200                  # 2.15e9 elements
    x = torch.zeros((rows, cols), device="cuda", dtype=BF)
    tail = draw((3, cols), BF, 1)
    x[-3:] = tail
    o = layers.layer_norm_forward(x, residual=x, p=0.5, seed=2, offset=3)
    f = ref.factors(3 * cols, 0.5, 2, 3, start=(rows - 3) * cols).reshape(3, cols)
    t = ref.f64(tail)
    y, s, mean, rstd = ref.norm(t, t, None, None, float(np.float32(EPS)), f)
    ds, dm, dr, dy = ref.norm_bounds(t, t, None, None, float(np.float32(EPS)), f)
    near(o.y[-3:], y, dy, BF)
    near(o.sum[-3:], s, ds, BF)
    g = layers.layer_norm_backward(x, o.sum, o.mean, o.rstd, p=0.5, seed=2, offset=3)
    want, bound = ref.norm_grad(t, ref.f64(o.sum[-3:]), ref.f64(o.mean[-3:]), ref.f64(o.rstd[-3:]),
                                None, None, f)
    near(g.dx[-3:], want[0], bound[0], BF)
    near(g.dresidual[-3:], want[1], bound[1], BF)
    near(g.dweight, want[2], bound[2], F32)      # the other rows' dy is zero
    near(g.dbias, want[3], bound[3], F32)


def test_autograd_equals_the_64_bit_graph(layers):
    # (y, s) of a sublayer end, s used again past the norm, the weight shared
    # by two norms, and an expanded gradient (sum): against torch in 64 bits
    rows, cols, p, seed, off = 37, 130, 0.2, 21, 9
    x, r = (draw((rows, cols), F32, i).requires_grad_() for i in (1, 2))
    w, b = (draw(cols, F32, i, 0.3, 1.0).requires_grad_() for i in (3, 4))
    c = draw((rows, cols), F32, 5)
    y, s = layers.dropout_add_layer_norm(x, r, w, b, p=p, seed=seed, offset=off)
    z = layers.layer_norm(y * c + s, w)
    (z * z * c).sum().backward()
    X, R, W, B = (t.detach().double().cpu().requires_grad_() for t in (x, r, w, b))
    C = c.double().cpu()
    f = torch.from_numpy(ref.factors(rows * cols, p, seed, off).reshape(rows, cols))

    def ln(v, scale, shift):
        m = v.mean(1, keepdim=True)
        q = ((v - m) ** 2).mean(1, keepdim=True)
        return (v - m) / (q + EPS).sqrt() * scale + shift

    S = R + f * X
    Z = ln(ln(S, W, B) * C + S, W, 0.0)
    (Z * Z * C).sum().backward()
    for got, want in ((x, X), (r, R), (w, W), (b, B)):
        g, e = ref.f64(got.grad), want.grad.numpy()
        assert np.linalg.norm(g - e) <= 1e-5 * np.linalg.norm(e)
    x.grad = None
    layers.layer_norm(x[:, :64].t()).sum().backward()     # strided input, expanded gradient
    assert x.grad.shape == x.shape and ref.f64(x.grad)[:, 64:].any() == False  # noqa: E712


def test_gradient_against_differences(layers):
    # central differences of a scalar of the GPU's own forward pass: the
    # truncation is O(h^2) = 1e-4, the forward's rounding 1e-6 / h
    x, r = draw((4, 50), F32, 1), draw((4, 50), F32, 2)
    w, b = draw(50, F32, 3, 0.3, 1.0), draw(50, F32, 4)
    cy, cs = draw((4, 50), F32, 5).double(), draw((4, 50), F32, 6).double()
    drop = dict(p=0.3, seed=4, offset=1)

    def total(x, r, w, b):
        o = layers.layer_norm_forward(x, w, b, residual=r, **drop)
        return float((cy * o.y.double()).sum() + (cs * o.sum.double()).sum())

    o = layers.layer_norm_forward(x, w, b, residual=r, **drop)
    g = layers.layer_norm_backward(cy.float(), o.sum, o.mean, o.rstd, w, dsum=cs.float(), **drop)
    args, h = [x, r, w, b], 1e-2
    for i, grad in enumerate((g.dx, g.dresidual, g.dweight, g.dbias)):
        v = draw(args[i].shape, F32, 30 + i)
        at = [[a + (sign * h * v if j == i else 0) for j, a in enumerate(args)] for sign in (1, -1)]
        fd = (total(*at[0]) - total(*at[1])) / (2 * h)
        an = float((grad.double() * v.double()).sum())
        assert abs(fd - an) <= 2e-3 * float(grad.double().norm() * v.double().norm())


def test_refusals(layers):
    x = torch.zeros((4, 8), device="cuda")
    w = torch.ones(8, device="cuda")
    with pytest.raises(ValueError):
        layers.layer_norm_forward(x.t())
    with pytest.raises(ValueError):
        layers.layer_norm_forward(x, w[:4])
    with pytest.raises(TypeError):
        layers.layer_norm_forward(x, w, w.bfloat16())
    with pytest.raises(TypeError):
        layers.layer_norm_forward(x, residual=x.bfloat16())
    with pytest.raises(ValueError):
        layers.layer_norm_forward(x, residual=x[:2])
    with pytest.raises(muon().MuonError):
        layers.layer_norm_forward(x, p=1.5)
    with pytest.raises(ValueError):
        layers.layer_norm_backward(x, x, w[:3], w[:4])
    with pytest.raises(TypeError):
        layers.layer_norm_backward(x, x, w[:4].bfloat16(), w[:4])
    with pytest.raises(ValueError):
        layers.layer_norm_forward(x, w.cpu())
