"""Layer norm and its gradient at numbers of rows and widths where the row
groups of a block differ: one and two rows just below the widths of each
layout, and many rows a group, against the 64-bit host reference with the
bounds of layers_ref."""
import ctypes

import pytest
import torch

import layers_ref as ref
from helpers import muon
from test_norm_gpu import (BF, EPS, F32, check_backward, check_forward, draw, layers,  # noqa: F401
                           near, placed)

pytestmark = pytest.mark.gpu


def loud(layers, cols, dtype):
    """A large gradient of the same width whose values stay behind in the
    multiprocessors' shared memory."""
    x = torch.full((2000, cols), 3e4, device="cuda", dtype=dtype)
    x[:, ::2] = -3e4
    one = torch.ones(2000, device="cuda")
    layers.layer_norm_backward(x, x, one, one, dsum=x)
    layers.layer_norm_backward(x, x, one, one)


# just below the widths at which a row takes more threads, elements a thread or
# row groups a block
WIDTHS = [63, 255, 511, 1023, 1533, 1535, 2045, 2047, 4093, 4094, 4095, 8191]


@pytest.mark.parametrize("rows", [1, 2])
@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_and_two_rows_of_ragged_widths(layers, rows, cols, dtype):  # noqa: F811
    x, r = draw((rows, cols), dtype, 1, 1.3, 0.4), draw((rows, cols), dtype, 5, 2.0)
    dy, ds = draw((rows, cols), dtype, 4, 0.1), draw((rows, cols), dtype, 6, 0.1)
    w, b = draw(cols, F32, 2, 0.3, 1.0), draw(cols, F32, 3, 0.2)
    for p, res, dsum in ((0.0, None, None), (0.0, r, ds), (0.25, r, ds)):
        o = check_forward(layers, x, res, w, b, p)
        loud(layers, cols, dtype)
        check_backward(layers, dy, o.sum, o.mean, o.rstd, w, dsum, p)


@pytest.mark.parametrize("ld", [1, 3, 7, 4097])
@pytest.mark.parametrize("dtype,cols", [(BF, 1529), (BF, 4089), (F32, 4094), (F32, 4096), (BF, 61)])
def test_one_row_of_any_stride(layers, dtype, cols, ld):  # noqa: F811
    # the stride of a single row has no meaning, whatever it is
    lib = muon().load()
    dt = 1 if dtype == F32 else 0
    dy, s = draw((1, cols), dtype, 4, 0.1), draw((1, cols), dtype, 1)
    w = draw(cols, F32, 2, 0.3, 1.0)
    o = layers.layer_norm_forward(s, w)
    want = layers.layer_norm_backward(dy, s, o.mean, o.rstd, w)
    loud(layers, cols, dtype)
    need = ctypes.c_size_t()
    assert lib.muon_layer_norm_workspace_bytes(1, cols, ctypes.byref(need)) == 0
    ws = torch.empty(need.value, dtype=torch.uint8, device="cuda")
    dx, (dw, db), y = torch.empty_like(dy), torch.empty(2, cols, device="cuda"), torch.empty_like(s)
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.muon_layer_norm_backward(
        1, cols, dt, 1, dy.data_ptr(), ld, s.data_ptr(), ld, o.mean.data_ptr(), o.rstd.data_ptr(),
        w.data_ptr(), None, 0, 0.0, 0, 0, dx.data_ptr(), None, dw.data_ptr(), db.data_ptr(),
        ws.data_ptr(), need.value, stream) == 0
    assert lib.muon_layer_norm(1, cols, dt, 1, s.data_ptr(), ld, None, 0, w.data_ptr(), None, EPS, 0.0,
                               0, 0, None, y.data_ptr(), None, None, stream) == 0
    torch.cuda.synchronize()
    for got, exact in ((dx, want.dx), (dw, want.dweight), (db, want.dbias), (y, o.y)):
        assert torch.equal(got, exact)


# several rows a row group: the ring wraps, the warps' slots are used again, and
# a thread adds up columns over its rows
@pytest.mark.parametrize("rows,cols", [(40000, 24), (20000, 61), (6000, 200), (6000, 397), (3000, 512),
                                       (6000, 1023), (3000, 1024), (3000, 1500), (1500, 2999),
                                       (1500, 4096), (1000, 6001), (700, 8192), (500, 11008),
                                       (400, 16384), (350, 16001), (700, 17000)])
@pytest.mark.parametrize("dtype,p", [(BF, 0.0), (F32, 0.0), (BF, 0.2), (F32, 0.2)])
def test_many_rows_a_group(layers, rows, cols, dtype, p):  # noqa: F811
    x, dy = draw((rows, cols), dtype, 1, 1.3, 0.4), draw((rows, cols), dtype, 4, 0.1)
    w, b = draw(cols, dtype, 2, 0.3, 1.0), draw(cols, F32, 3, 0.2).to(dtype)
    r, ds = (draw((rows, cols), dtype, i) if p else None for i in (5, 6))
    o = check_forward(layers, x, r, w, b, p)
    check_backward(layers, dy, o.sum, o.mean, o.rstd, w, ds, p)


@pytest.mark.parametrize("pads,leads", [((8, 8), (0, 0)), ((7, 7), (0, 0)), ((7, 0), (0, 0)), ((0, 0), (1, 3))])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_rows_of_other_strides(layers, dtype, pads, leads):  # noqa: F811
    rows, cols = 2500, 1409
    x, r = (placed(draw((rows, cols), dtype, i), pads[0], leads[0]) for i in (1, 5))
    dy = placed(draw((rows, cols), dtype, 4, 0.1), pads[1], leads[1])
    w, b = draw(cols, F32, 2, 0.3, 1.0), draw(cols, F32, 3)
    o = check_forward(layers, x, r, w, b, 0.0)
    check_backward(layers, dy, placed(o.sum, pads[0], leads[0]), o.mean, o.rstd, w, None, 0.0)


# h = (sum - mean) rstd is 0 in a constant row, however large mean * rstd is
@pytest.mark.parametrize("cols", [7, 56, 61, 333, 1000, 1023, 4093, 8190, 16401])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradient_of_large_constant_rows(layers, dtype, cols):  # noqa: F811
    rows = 5
    s = torch.full((rows, cols), 2.0 ** 120, device="cuda", dtype=dtype)
    s[::2] = draw((3, cols), dtype, 1)
    mean, rstd = (torch.full((rows,), v, device="cuda") for v in (2.0 ** 120, 512.0))
    mean[::2], rstd[::2] = 0.1, 1.1
    w = draw(cols, F32, 2, 0.3, 1.0)
    check_backward(layers, draw((rows, cols), dtype, 4, 0.1), s, mean, rstd, w, None, 0.0)
    check_backward(layers, draw((rows, cols), dtype, 4, 0.1), s, mean, rstd, w,
                   draw((rows, cols), dtype, 6, 0.1), 0.25)
    check_backward(layers, placed(draw((rows, cols), dtype, 4, 0.1), 3, 1), s, mean, rstd, w, None, 0.0)


# sums of these are exact in fp32, so the mean is the value itself and y the bias
@pytest.mark.parametrize("cols", [3, 49, 63, 333, 1000, 1023, 3001, 4099, 10240, 16383])
@pytest.mark.parametrize("value", [3.0, 1000.0, -640.0])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_constant_rows_give_the_bias(layers, dtype, value, cols):  # noqa: F811
    x = torch.full((5, cols), value, device="cuda", dtype=dtype)
    w, b = draw(cols, dtype, 2, 0.3, 1.0), draw(cols, dtype, 3)
    o = layers.layer_norm_forward(x, w, b, eps=EPS)
    assert bool((o.mean == value).all()) and torch.equal(o.y, b.expand(5, cols))
    near(o.rstd, ref.f64(torch.full((5,), EPS).double()) ** -0.5, 1e-3, F32)


@pytest.mark.parametrize("cols", [7, 64, 333, 1024, 4093, 16400])
def test_mean_of_rows_with_infinities(layers, cols):  # noqa: F811
    x = draw((4, cols), F32, 1)
    inf = float("inf")
    x[0, 3], x[1, 5], x[2, 2], x[2, 4] = inf, -inf, inf, -inf
    mean = layers.layer_norm_forward(x).mean.tolist()
    assert mean[0] == inf and mean[1] == -inf and mean[2] != mean[2] and abs(mean[3]) < 2
