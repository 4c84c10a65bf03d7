"""Operators over sequences without a GPU: the host reference's gradients
against differences, and every refusal of the library's entry points
(arguments are checked before any device work)."""
import ctypes

import numpy as np
import pytest
import torch

import sequence_ref as ref

OK, INVALID, SHAPE, DTYPE, ALIGN, CUDA, WORKSPACE = 0, -1, -2, -3, -4, -5, -7
A, B, C, D, E, F, G = (0x100000 * i for i in range(1, 8))     # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from newton_schulz_05_gb300 import build
    build.build()
    import newton_schulz_05_gb300 as m
    return m.load()


def _agrees(f, args, grads, rng, tol=1e-6):
    """Differences of f along random directions against the gradients."""
    for i, g in enumerate(grads):
        if g is None:
            continue
        v = rng.normal(size=args[i].shape)
        at = lambda h: f(*[a + h * v if k == i else a for k, a in enumerate(args)])  # noqa: E731
        fd = (at(1e-5) - at(-1e-5)) / 2e-5
        assert abs(fd - (g * v).sum()) <= tol * (np.linalg.norm(g) * np.linalg.norm(v) + 1), i


@pytest.mark.parametrize("mix", [True, False])
def test_reference_scan_gradient_against_differences(mix):
    rng = np.random.default_rng(0)
    gate, x, ch = (rng.normal(size=(2, 9, 3)) for _ in range(3))
    state, cl = rng.normal(size=(2, 3)), rng.normal(size=(2, 3))
    starts, mask = rng.random((2, 9)) < 0.2, rng.random((2, 9)) < 0.8

    def total(gate, x, state):
        h, last, _, _ = ref.scan(gate, x, state, starts, mask, mix)
        return (ch * h).sum() + (cl * last).sum()

    h = ref.scan(gate, x, state, starts, mask, mix)[0]
    grads, _ = ref.scan_grad(ch, gate, x, h, state, cl, starts, mask, mix)
    _agrees(total, (gate, x, state), grads, rng)


def test_reference_scan_is_the_recurrence():
    rng = np.random.default_rng(1)
    gate, x = rng.normal(size=(1, 5, 1)), rng.normal(size=(1, 5, 1))
    p = 0.25
    for t in range(5):
        if t == 3:
            p = 0.0
        if t != 2:
            a = 1 / (1 + np.exp(-gate[0, t, 0]))
            p = a * p + (1 - a) * x[0, t, 0]
    starts, mask = np.array([[0, 0, 1, 1, 0]]), np.array([[1, 1, 0, 1, 1]])
    h, last, _, _ = ref.scan(gate, x, np.full((1, 1), 0.25), starts, mask, True)
    assert abs(last[0, 0] - p) < 1e-15 and h[0, 2, 0] == h[0, 1, 0]


@pytest.mark.parametrize("rotary,neighbours", [(0, False), (6, False), (6, True), (4, False), (4, True)])
def test_reference_heads_gradient_against_differences(rotary, neighbours):
    rng = np.random.default_rng(2)
    x, c = rng.normal(size=(5, 2, 6)), rng.normal(size=(5, 2, 6))
    w = rng.normal(size=6)
    angle = rng.normal(size=(4, rotary // 2))
    cos, sin = (np.cos(angle), np.sin(angle)) if rotary else (None, None)
    pos = np.array([3, 0, 4, -1, 1])

    def total(x, w):
        return (c * ref.heads(x, w, cos, sin, pos, 1e-6, neighbours)[0]).sum()

    grads, _ = ref.heads_grad(c, x, w, cos, sin, pos, 1e-6, neighbours)
    _agrees(total, (x, w), grads, rng)
    y = ref.heads(x, None, cos, sin, pos, 0.0, neighbours)[0]
    live = np.ones(5, bool) if not rotary else np.array([1, 1, 0, 0, 1], bool)
    assert np.allclose((y[live] ** 2).mean(-1), 1)      # a rotation keeps the norm
    assert not y[~live].any()


def test_reference_log_probs_gradient_against_differences():
    rng = np.random.default_rng(3)
    l, c = rng.normal(size=(4, 7)), rng.normal(size=4)
    y = np.array([0, 6, -100, 3])

    def total(l):
        return (c * ref.log_probs(l, y, 0.7)[0]).sum()

    lse = ref.log_probs(l, y, 0.7)[1]
    _agrees(total, (l,), [ref.log_probs_grad(c, l, y, lse, 0.7)[0]], rng)


@pytest.mark.parametrize("by_sequence", [True, False])
@pytest.mark.parametrize("each", [True, False])
def test_reference_policy_gradient_against_differences(by_sequence, each):
    rng = np.random.default_rng(4)
    lp, old, r = (-rng.random((3, 8)) for _ in range(3))
    adv = rng.normal(size=(3, 8) if each else 3)
    mask = rng.random((3, 8)) < 0.7
    mask[1] = False

    def total(lp):
        return ref.policy(lp, old, adv, r, mask, 0.2, 0.3, 0.1, by_sequence)[0][0]

    (_, kl, clipped, w), _ = ref.policy(lp, old, adv, r, mask, 0.2, 0.3, 0.1, by_sequence)
    assert kl > 0 and 0 < clipped < 1 and abs((w * mask.sum(1)).sum() - 1) < 1e-12
    _agrees(total, (lp,), [ref.policy_grad(lp, old, adv, r, mask, 0.2, 0.3, 0.1, w, 1.0)[0]], rng)


def _scan(lib, batch=2, length=4, dim=8, dt=0, g=A, ldg=8, x=B, ldx=8, s=None, st=None, m=None, h=C, last=D):
    return lib.muon_gated_scan(batch, length, dim, dt, g, ldg, x, ldx, s, st, m, 1, h, last, None)


def _scan_bwd(lib, batch=2, length=4, dim=8, dt=0, dh=A, lddh=8, g=B, ldg=8, x=C, ldx=8, h=D, ldh=8, s=None,
              dl=None, mix=1, dg=E, dx=F, ds=G):
    return lib.muon_gated_scan_backward(batch, length, dim, dt, dh, lddh, g, ldg, x, ldx, h, ldh, s, dl, None,
                                        None, mix, dg, dx, ds, None)


def test_scan_refusals(lib):
    for call in (_scan, _scan_bwd):
        assert call(lib, batch=-1) == INVALID and call(lib, length=-1) == INVALID
        assert call(lib, dim=0) == SHAPE and call(lib, dim=(1 << 20) + 1) == SHAPE
        assert call(lib, batch=1 << 31) == SHAPE and call(lib, length=1 << 31) == SHAPE
        assert call(lib, batch=1 << 20, dim=1 << 13) == SHAPE
        assert call(lib, dt=2) == DTYPE
        for a in ("g", "x", "h"):
            assert call(lib, **{a: None}) == INVALID and call(lib, **{a: A + 1}) == ALIGN
        assert call(lib, ldg=-1) == INVALID and call(lib, ldx=-8) == INVALID
        assert call(lib, ldg=1 << 32) == SHAPE and call(lib, ldx=1 << 32) == SHAPE
        assert call(lib, s=A + 2) == ALIGN
        assert call(lib, batch=0, g=None, x=None, h=None) == OK
    assert _scan(lib, last=A + 2) == ALIGN
    assert _scan_bwd(lib, dh=None) == INVALID and _scan_bwd(lib, dh=A + 1) == ALIGN
    assert _scan_bwd(lib, ldh=-1) == INVALID and _scan_bwd(lib, lddh=-1) == INVALID
    assert _scan_bwd(lib, ldh=1 << 32) == SHAPE and _scan_bwd(lib, lddh=1 << 32) == SHAPE
    for a in ("dg", "dx"):
        assert _scan_bwd(lib, **{a: A + 1}) == ALIGN
    assert _scan_bwd(lib, dl=A + 2) == ALIGN and _scan_bwd(lib, ds=A + 2) == ALIGN


def _heads(lib, tokens=4, qh=4, kh=2, dim=16, rotary=8, dt=0, wdt=1, q=A, ldq=64, qs=16, k=B, ldk=32, ks=16,
           qw=C, kw=C, eps=1e-6, cos=D, sin=D, table=9, pos=E, period=4, oq=F, ok=G):
    return lib.muon_norm_rotate_heads(tokens, qh, kh, dim, rotary, dt, wdt, q, ldq, qs, k, ldk, ks, qw, kw,
                                      eps, cos, sin, table, pos, period, 0, oq, ok, None)


def _heads_bwd(lib, tokens=4, qh=4, kh=2, dim=16, rotary=8, dt=0, wdt=1, dq=A, lddq=64, dqs=16, dk=B, lddk=32,
               dks=16, q=A, ldq=64, qs=16, k=B, ldk=32, ks=16, qw=C, kw=C, eps=1e-6, cos=D, sin=D, table=9,
               pos=E, period=4, gq=F, gk=G, gqw=F, gkw=G, ws=0x700, nbytes=1 << 30):
    return lib.muon_norm_rotate_heads_backward(
        tokens, qh, kh, dim, rotary, dt, wdt, dq, lddq, dqs, dk, lddk, dks, q, ldq, qs, k, ldk, ks, qw, kw,
        eps, cos, sin, table, pos, period, 0, gq, gk, gqw, gkw, ws, nbytes, None)


def test_heads_refusals(lib):
    for call in (_heads, _heads_bwd):
        assert call(lib, tokens=-1) == INVALID and call(lib, qh=-1) == INVALID and call(lib, kh=-1) == INVALID
        assert call(lib, tokens=1 << 31) == SHAPE and call(lib, qh=65537) == SHAPE
        assert call(lib, dim=0, rotary=0) == SHAPE and call(lib, dim=1025) == SHAPE
        assert call(lib, rotary=7) == SHAPE and call(lib, rotary=18) == SHAPE and call(lib, rotary=-2) == INVALID
        assert call(lib, dt=2) == DTYPE and call(lib, wdt=2) == DTYPE
        for eps in (-1e-6, float("nan"), float("inf")):
            assert call(lib, eps=eps) == INVALID
        assert call(lib, cos=None) == INVALID and call(lib, sin=None) == INVALID
        assert call(lib, table=-1) == INVALID and call(lib, pos=None, period=0) == INVALID
        for a in ("q", "k"):
            assert call(lib, **{a: None}) == INVALID and call(lib, **{a: A + 1}) == ALIGN
        for a in ("ldq", "qs", "ldk", "ks"):
            assert call(lib, **{a: -1}) == INVALID
        for a in ("qw", "kw", "cos", "sin"):
            assert call(lib, **{a: A + 2}) == ALIGN
        assert call(lib, pos=E + 4) == ALIGN
    assert _heads(lib, oq=None) == INVALID and _heads(lib, ok=None) == INVALID
    assert _heads(lib, oq=F + 1) == ALIGN and _heads(lib, ok=F + 1) == ALIGN
    assert _heads(lib, tokens=0, q=None, k=None, oq=None, ok=None) == OK
    for a in ("dq", "dk"):
        assert _heads_bwd(lib, **{a: None}) == INVALID and _heads_bwd(lib, **{a: A + 1}) == ALIGN
    for a in ("lddq", "dqs", "lddk", "dks"):
        assert _heads_bwd(lib, **{a: -1}) == INVALID
    for a in ("gq", "gk", "gqw", "gkw"):
        assert _heads_bwd(lib, **{a: A + 1}) == ALIGN
    assert _heads_bwd(lib, ws=None) == INVALID and _heads_bwd(lib, ws=0x710) == ALIGN
    need = ctypes.c_size_t()
    size = lib.muon_norm_rotate_heads_workspace_bytes
    assert size(4, 4, 2, 16, ctypes.byref(need)) == OK and need.value > 0
    assert _heads_bwd(lib, nbytes=need.value - 1) == WORKSPACE
    assert size(4, 4, 2, 16, None) == INVALID and size(-1, 4, 2, 16, ctypes.byref(need)) == INVALID
    assert size(4, 4, 2, 0, ctypes.byref(need)) == SHAPE


def _vocab(lib, tokens=4, vocab=8, dt=0, l=A, ld=8, i=B, scale=1.0, lp=C, lse=D):
    return lib.muon_token_log_probs(tokens, vocab, dt, l, ld, i, scale, lp, lse, None)


def _vocab_bwd(lib, tokens=4, vocab=8, dt=0, d=E, l=A, ld=8, i=B, lse=D, scale=1.0, o=F):
    return lib.muon_token_log_probs_backward(tokens, vocab, dt, d, l, ld, i, lse, scale, o, None)


def test_log_probs_refusals(lib):
    for call in (_vocab, _vocab_bwd):
        assert call(lib, tokens=-1) == INVALID and call(lib, tokens=1 << 31) == SHAPE
        assert call(lib, vocab=0) == SHAPE and call(lib, vocab=(1 << 30) + 1) == SHAPE
        assert call(lib, dt=2) == DTYPE and call(lib, ld=-1) == INVALID
        for scale in (0.0, -1.0, float("nan"), float("inf")):
            assert call(lib, scale=scale) == INVALID
        for a in ("l", "i", "lse"):
            assert call(lib, **{a: None}) == INVALID
        assert call(lib, l=A + 1) == ALIGN and call(lib, i=B + 4) == ALIGN and call(lib, lse=D + 2) == ALIGN
        assert call(lib, tokens=0, l=None, i=None, lse=None) == OK
    assert _vocab(lib, lp=None) == INVALID and _vocab(lib, lp=C + 2) == ALIGN
    assert _vocab_bwd(lib, d=None) == INVALID and _vocab_bwd(lib, o=None) == INVALID
    assert _vocab_bwd(lib, d=E + 2) == ALIGN and _vocab_bwd(lib, o=F + 1) == ALIGN
    assert _vocab_bwd(lib, o=A, ld=16) == INVALID       # in place, with gaps between the rows


def _policy(lib, batch=2, length=4, lp=A, ldl=4, old=B, ldo=4, adv=C, lda=4, r=None, ldr=4, low=0.2, high=0.2,
            kl=0.0, loss=D, k=E, c=F, w=G, ws=0x700, nbytes=1 << 30):
    return lib.muon_policy_loss(batch, length, lp, ldl, old, ldo, adv, lda, r, ldr, None, low, high, kl, 0,
                                loss, k, c, w, ws, nbytes, None)


def _policy_bwd(lib, batch=2, length=4, lp=A, ldl=4, old=B, ldo=4, adv=C, lda=4, r=None, ldr=4, low=0.2,
                high=0.2, kl=0.0, w=G, dl=D, o=E):
    return lib.muon_policy_loss_backward(batch, length, lp, ldl, old, ldo, adv, lda, r, ldr, None, low, high,
                                         kl, w, dl, o, None)


def test_policy_refusals(lib):
    nan, inf = float("nan"), float("inf")
    for call in (_policy, _policy_bwd):
        assert call(lib, batch=-1) == INVALID and call(lib, length=-1) == INVALID
        assert call(lib, batch=1 << 31) == SHAPE and call(lib, length=1 << 31) == SHAPE
        assert call(lib, batch=1 << 20, length=1 << 20) == SHAPE
        for low in (-0.1, 1.0, nan):
            assert call(lib, low=low) == INVALID
        for high in (-0.1, nan, inf):
            assert call(lib, high=high) == INVALID
        assert call(lib, kl=nan) == INVALID and call(lib, kl=inf) == INVALID
        for a in ("ldl", "ldo", "ldr"):
            assert call(lib, **{a: -1}) == INVALID
        for a in ("lp", "old", "adv", "w"):
            assert call(lib, **{a: None}) == INVALID and call(lib, **{a: A + 2}) == ALIGN
        assert call(lib, r=A + 2) == ALIGN
    for a in ("loss", "k", "c"):
        assert _policy(lib, **{a: A + 2}) == ALIGN
    assert _policy(lib, loss=None) == INVALID and _policy(lib, ws=None) == INVALID
    assert _policy(lib, ws=0x710) == ALIGN
    need = ctypes.c_size_t()
    size = lib.muon_policy_loss_workspace_bytes
    assert size(2, 4, ctypes.byref(need)) == OK and need.value > 0
    assert _policy(lib, nbytes=need.value - 1) == WORKSPACE
    assert size(2, 4, None) == INVALID and size(-1, 4, ctypes.byref(need)) == INVALID
    assert _policy_bwd(lib, dl=A + 2) == ALIGN and _policy_bwd(lib, o=A + 2) == ALIGN
    assert _policy_bwd(lib, o=None) == INVALID
    assert _policy_bwd(lib, batch=0, lp=None, old=None, adv=None, w=None, o=None) == OK
    for a in ("lp", "old", "r"):
        ld = {"lp": "ldl", "old": "ldo", "r": "ldr"}[a]
        assert _policy_bwd(lib, **{a: E, ld: 8}) == INVALID     # in place, with gaps between the rows


def test_fault_switch_fails_the_launch(lib, monkeypatch):
    monkeypatch.setenv("MUON_FAULT", "launch")
    for call in (_scan, _scan_bwd, _heads, _heads_bwd, _vocab, _vocab_bwd, _policy, _policy_bwd):
        assert call(lib) == CUDA
    assert _scan(lib, dim=0) == SHAPE      # arguments are still checked first


def test_binding_refuses_host_tensors_and_wrong_types():
    from newton_schulz_05_gb300 import layers
    x = torch.zeros(2, 4, 8)
    with pytest.raises(ValueError):
        layers.gated_scan_forward(x, x)
    with pytest.raises(TypeError):
        layers.gated_scan_forward(x.half(), x.half())
    with pytest.raises(ValueError):
        layers.norm_rotate_heads_forward(x)
    with pytest.raises(TypeError):
        layers.norm_rotate_heads_forward(x.double())
    with pytest.raises(ValueError):
        layers.token_log_probs_forward(x, torch.zeros(2, 4, dtype=torch.int64))
    with pytest.raises(ValueError):
        layers.policy_loss_forward(x[0], x[0], x[0])
    with pytest.raises(TypeError):
        layers.policy_loss_forward(x[0].bfloat16(), x[0], x[0])


def test_rotation_table_is_exact_at_far_positions():
    from newton_schulz_05_gb300.layers import rotation_table
    cos, sin = rotation_table(1 << 17, 8, base=500.0, device="cpu")
    assert cos.shape == sin.shape == (1 << 17, 4) and cos.dtype == torch.float32
    for p in (0, 1, 77777, (1 << 17) - 1):
        for m in range(4):
            angle = p * 500.0 ** (-2 * m / 8)
            assert abs(float(cos[p, m]) - np.cos(angle)) < 1e-7
            assert abs(float(sin[p, m]) - np.sin(angle)) < 1e-7
    with pytest.raises(ValueError):
        rotation_table(4, 3, device="cpu")
