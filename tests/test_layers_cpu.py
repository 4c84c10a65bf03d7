"""Training operators without a GPU: the host reference against published
values of the generator, its gradients against differences, and every refusal
of the library's entry points (arguments are checked before any device work)."""
import ctypes

import numpy as np
import pytest
import torch

import layers_ref as ref

OK, INVALID, SHAPE, DTYPE, ALIGN, CUDA, WORKSPACE = 0, -1, -2, -3, -4, -5, -7
A, B, C, D, E_, F = (0x100000 * i for i in range(1, 7))     # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from newton_schulz_05_gb300 import build
    build.build()
    import newton_schulz_05_gb300 as m
    return m.load()


def test_reference_generator_known_answers():
    # the known-answer vectors published with the generator
    f = 0xFFFFFFFF
    assert ref.philox([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ref.philox([f] * 4, [f] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert ref.philox([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344],
                      [0xA4093822, 0x299F31D0]) == [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


@pytest.mark.parametrize("start,n", [(0, 40), (3, 17), (8, 1), (13, 3)])
def test_reference_factors_follow_the_generator(start, n):
    seed, offset, p = 0x0123456789ABCDEF, (1 << 32) - 2, 0.3
    t = int(np.floor(float(np.float32(p)) * 65536 + 0.5))
    got = ref.factors(n, p, seed, offset, start)
    for i in range(n):
        c = offset + (start + i) // 8
        w = ref.philox([c & 0xFFFFFFFF, c >> 32, 0, 0], [seed & 0xFFFFFFFF, seed >> 32])
        j = (start + i) % 8
        h = (w[j // 2] >> (16 * (j % 2))) & 0xFFFF
        assert got[i] == (65536 / (65536 - t) if h >= t else 0.0)


def test_reference_keeps_the_promised_share():
    n = 1 << 16
    for p in (0.1, 0.5, 0.9):
        kept = (ref.factors(n, p, 5, 0) != 0).mean()
        assert abs(kept - (1 - p)) < 6 * np.sqrt(p * (1 - p) / n)
    assert not ref.factors(n, 1.0, 5, 0).any()


def _difference(f, x, v, h):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


def test_reference_norm_gradient_against_differences():
    rng = np.random.default_rng(0)
    x, r, w, b = rng.normal(size=(3, 11)), rng.normal(size=(3, 11)), rng.normal(size=11), rng.normal(size=11)
    cy, cs = rng.normal(size=(3, 11)), rng.normal(size=(3, 11))
    f = ref.factors(33, 0.3, 9, 4).reshape(3, 11)

    def total(x=x, r=r, w=w, b=b):
        y, s, _, _ = ref.norm(x, r, w, b, 1e-5, f)
        return (cy * y).sum() + (cs * s).sum()

    _, s, mean, rstd = ref.norm(x, r, w, b, 1e-5, f)
    (dx, dr, dw, db), _ = ref.norm_grad(cy, s, mean, rstd, w, cs, f)
    for name, val, grad in (("x", x, dx), ("r", r, dr), ("w", w, dw), ("b", b, db)):
        v = rng.normal(size=val.shape)
        fd = _difference(lambda z: total(**{name: z}), val, v, 1e-5)
        assert abs(fd - (grad * v).sum()) < 1e-6 * np.linalg.norm(grad) * np.linalg.norm(v)


@pytest.mark.parametrize("normalize", [True, False])
def test_reference_route_gradient_against_differences(normalize):
    rng = np.random.default_rng(1)
    l = rng.normal(size=(6, 7))
    l[2, 3] = -np.inf
    l[4] = -np.inf
    mask = np.array([1, 0, 1, 1, 1, 1], bool)
    o = ref.route(l, 3, mask, normalize)
    cw, cl = rng.normal(size=(6, 3)), 0.7

    def total(z):
        q = ref.route(z, 3, mask, normalize)
        assert np.array_equal(q["index"], o["index"])
        return (cw * q["weights"]).sum() + cl * q["loss"]

    g = ref.route_grad(l, o["index"], o["counts"], cw, cl, mask, normalize)
    v = rng.normal(size=l.shape)
    fd = _difference(total, l, v, 1e-6)
    assert abs(fd - (g * v).sum()) < 1e-6 * np.linalg.norm(g) * np.linalg.norm(v)
    assert not g[1].any() and not g[4].any() and g[2, 3] == 0


def _norm(lib, rows=4, cols=8, dt=0, wdt=1, x=A, ldx=8, r=None, ldr=8, w=B, b=C, eps=1e-5, p=0.0,
          s=None, y=D, mean=E_, rstd=F):
    return lib.muon_layer_norm(rows, cols, dt, wdt, x, ldx, r, ldr, w, b, eps, p, 1, 0, s, y, mean,
                               rstd, None)


def test_layer_norm_refusals(lib):
    assert _norm(lib, rows=-1) == INVALID
    assert _norm(lib, cols=0) == SHAPE and _norm(lib, cols=(1 << 30) + 1) == SHAPE
    assert _norm(lib, dt=2) == DTYPE and _norm(lib, wdt=-1) == DTYPE
    assert _norm(lib, x=None) == INVALID and _norm(lib, y=None) == INVALID
    assert _norm(lib, ldx=-8) == INVALID and _norm(lib, ldr=-1) == INVALID
    for eps in (-1e-5, float("nan"), float("inf")):
        assert _norm(lib, eps=eps) == INVALID
    for p in (-0.1, 1.1, float("nan")):
        assert _norm(lib, p=p) == INVALID
    assert _norm(lib, x=A + 1) == ALIGN and _norm(lib, w=B + 2) == ALIGN
    assert _norm(lib, y=D + 1) == ALIGN and _norm(lib, s=D + 1) == ALIGN
    assert _norm(lib, mean=E_ + 2) == ALIGN and _norm(lib, r=A + 1) == ALIGN
    assert _norm(lib, rows=0, x=None, y=None) == OK          # nothing to do


def _norm_bwd(lib, rows=4, cols=8, dt=0, wdt=1, dy=A, ld=8, s=B, lds=8, mean=C, rstd=C, w=D,
              ds=None, ldds=8, p=0.0, dx=E_, dr=None, dw=F, db=F, ws=0x700, nbytes=1 << 30):
    return lib.muon_layer_norm_backward(rows, cols, dt, wdt, dy, ld, s, lds, mean, rstd, w, ds,
                                        ldds, p, 1, 0, dx, dr, dw, db, ws, nbytes, None)


def test_layer_norm_backward_refusals(lib):
    assert _norm_bwd(lib, rows=-1) == INVALID and _norm_bwd(lib, cols=0) == SHAPE
    assert _norm_bwd(lib, dt=7) == DTYPE and _norm_bwd(lib, wdt=7) == DTYPE
    for a in ("dy", "s", "mean", "rstd"):
        assert _norm_bwd(lib, **{a: None}) == INVALID
    for a in ("ld", "lds", "ldds"):
        assert _norm_bwd(lib, **{a: -1}) == INVALID
    assert _norm_bwd(lib, p=2.0) == INVALID
    for a in ("dy", "s", "mean", "rstd", "w", "ds", "dx", "dr", "dw", "db"):
        assert _norm_bwd(lib, **{a: A + 1}) == ALIGN
    assert _norm_bwd(lib, ws=None) == INVALID and _norm_bwd(lib, ws=0x710) == ALIGN
    need = ctypes.c_size_t()
    assert lib.muon_layer_norm_workspace_bytes(4, 8, ctypes.byref(need)) == OK and need.value > 0
    assert _norm_bwd(lib, nbytes=need.value - 1) == WORKSPACE
    assert lib.muon_layer_norm_workspace_bytes(4, 8, None) == INVALID
    assert lib.muon_layer_norm_workspace_bytes(-1, 8, ctypes.byref(need)) == INVALID
    assert lib.muon_layer_norm_workspace_bytes(4, 0, ctypes.byref(need)) == SHAPE


def test_dropout_refusals(lib):
    def call(n=8, dt=0, x=A, r=None, p=0.1, y=B):
        return lib.muon_dropout(n, dt, x, r, p, 1, 0, y, None)
    assert call(n=-1) == INVALID and call(x=None) == INVALID and call(y=None) == INVALID
    assert call(dt=3) == DTYPE
    assert call(p=-1e-6) == INVALID and call(p=1.5) == INVALID and call(p=float("nan")) == INVALID
    assert call(x=A + 1) == ALIGN and call(r=A + 1) == ALIGN and call(y=B + 1) == ALIGN
    assert call(n=0, x=None, y=None) == OK


def _route(lib, tokens=4, experts=8, k=2, dt=1, l=A, ld=8, mask=None, w=B, i=C, c=D, mp=E_, loss=F,
           ws=0x700, nbytes=1 << 30):
    return lib.muon_route(tokens, experts, k, dt, l, ld, mask, 1, w, i, c, mp, loss, ws, nbytes, None)


def _route_bwd(lib, tokens=4, experts=8, k=2, dt=1, l=A, ld=8, mask=None, i=C, c=D, dw=E_, dl=F, o=B):
    return lib.muon_route_backward(tokens, experts, k, dt, l, ld, mask, 1, i, c, dw, dl, o, None)


def test_route_refusals(lib):
    for call in (_route, _route_bwd):
        assert call(lib, tokens=-1) == INVALID and call(lib, k=0) == INVALID
        assert call(lib, ld=-1) == INVALID and call(lib, l=None) == INVALID
        assert call(lib, experts=0, k=1) == SHAPE and call(lib, experts=1025) == SHAPE
        assert call(lib, k=9) == SHAPE and call(lib, experts=64, k=33) == SHAPE
        assert call(lib, tokens=1 << 31) == SHAPE and call(lib, tokens=1 << 30, k=2) == SHAPE
        assert call(lib, dt=2) == DTYPE and call(lib, l=A + 2) == ALIGN
        assert call(lib, i=None) == INVALID and call(lib, c=None) == INVALID
        assert call(lib, i=C + 2) == ALIGN and call(lib, c=C + 1) == ALIGN
    for a in ("w", "mp", "loss", "ws"):
        assert _route(lib, **{a: None}) == INVALID
        assert _route(lib, **{a: A + 2}) == ALIGN
    assert _route_bwd(lib, o=None) == INVALID and _route_bwd(lib, o=B + 2) == ALIGN
    assert _route_bwd(lib, dw=B + 2) == ALIGN and _route_bwd(lib, dl=B + 2) == ALIGN
    assert _route_bwd(lib, tokens=0, l=None, i=None, c=None, o=None) == OK
    need = ctypes.c_size_t()
    assert lib.muon_route_workspace_bytes(4, 8, ctypes.byref(need)) == OK and need.value > 0
    assert _route(lib, nbytes=need.value - 1) == WORKSPACE
    assert lib.muon_route_workspace_bytes(4, 8, None) == INVALID
    assert lib.muon_route_workspace_bytes(-1, 8, ctypes.byref(need)) == INVALID
    assert lib.muon_route_workspace_bytes(4, 2000, ctypes.byref(need)) == SHAPE


def test_fault_switch_fails_the_launch(lib, monkeypatch):
    monkeypatch.setenv("MUON_FAULT", "launch")
    assert _norm(lib) == CUDA and _norm_bwd(lib) == CUDA
    assert _route(lib) == CUDA and _route_bwd(lib) == CUDA
    assert lib.muon_dropout(8, 0, A, None, 0.1, 1, 0, B, None) == CUDA
    assert _norm(lib, cols=0) == SHAPE      # arguments are still checked first


def test_binding_refuses_host_tensors_and_wrong_types():
    from newton_schulz_05_gb300 import layers
    x = torch.zeros(2, 4)
    with pytest.raises(ValueError):
        layers.layer_norm_forward(x)
    with pytest.raises(TypeError):
        layers.layer_norm_forward(x.half())
    with pytest.raises(ValueError):
        layers.dropout_forward(x, 0.1, seed=0)
    with pytest.raises(TypeError):
        layers.dropout_forward(x.double(), 0.1, seed=0)
    with pytest.raises(ValueError):
        layers.route_forward(x, 2)
    with pytest.raises(ValueError):
        layers.layer_norm_forward(torch.zeros(()))


def test_random_counter_never_overlaps():
    from newton_schulz_05_gb300.layers import RandomCounter
    c = RandomCounter(3, 10)
    assert [c.take(n) for n in (1, 8, 9, 0, 16)] == [10, 11, 12, 14, 14] and c.offset == 16
