"""Gated linear recurrence and its gradient against the 64-bit recurrence."""
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


def rows_in(t, layout, gen):
    """t as it is, as columns of a wider buffer, or at an odd address."""
    if layout == "dense":
        return t
    shape = t.shape[:-1] + (t.shape[-1] + (5 if layout == "odd" else 16),)
    wide = torch.randn(shape, generator=gen, device="cuda").to(t.dtype)
    at = 3 if layout == "odd" else 8
    wide[..., at:at + t.shape[-1]] = t
    return wide[..., at:at + t.shape[-1]]


def inputs(b, t, d, dtype, seed=0, state=True, starts=None, masked=False, layout="dense"):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    gate, x = (2 * n(b, t, d) + n(d)).to(dtype), n(b, t, d).to(dtype)
    mask = first = None
    if starts:
        first = torch.rand(b, t, generator=gen, device="cuda") < starts
    if masked:
        mask = torch.rand(b, t, generator=gen, device="cuda") > 0.3
        gate[~mask] = float("nan")
        x[~mask] = float("inf")
    return dict(gate=rows_in(gate, layout, gen), x=rows_in(x, layout, gen), state=n(b, d) if state else None,
                starts=first, token_mask=mask), n


def as64(v):
    return {k: None if t is None else ref.f64(t) for k, t in v.items()}


def clean(v):
    """What masked tokens hold, out of the host's way."""
    v = as64(v)
    if v["token_mask"] is not None:
        for k in ("gate", "x"):
            v[k] = np.where(v["token_mask"][..., None] != 0, v[k], 0)
    return v


def check(layers, v, n, mix, dtype):
    o = layers.gated_scan_forward(v["gate"], v["x"], state=v["state"], starts=v["starts"],
                                  token_mask=v["token_mask"], mix=mix)
    w = clean(v)
    h, last, eh, el = ref.scan(w["gate"], w["x"], w["state"], w["starts"], w["token_mask"], mix)
    ref.close(o.h, h, eh, dtype)
    ref.close(o.state, last, el, F32)
    dh, dlast = n(*o.h.shape).to(dtype), n(*o.state.shape)
    g = layers.gated_scan_backward(dh, v["gate"], v["x"], o.h, state=v["state"], dstate=dlast,
                                   starts=v["starts"], token_mask=v["token_mask"], mix=mix)
    (dg, dx, ds), (eg, ex, es) = ref.scan_grad(ref.f64(dh), w["gate"], w["x"], ref.f64(o.h), w["state"],
                                               ref.f64(dlast), w["starts"], w["token_mask"], mix)
    ref.close(g.dgate, dg, eg, dtype)
    ref.close(g.dx, dx, ex, dtype)
    ref.close(g.dstate, ds, es, F32)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("mix", [True, False])
@pytest.mark.parametrize("b,t,d", [
    (1, 1, 1), (2, 1, 64), (5, 1, 72), (300, 1, 40), (1, 2, 8), (3, 3, 7), (2, 4, 64), (2, 5, 130), (1, 7, 256),
    (1, 31, 64), (2, 32, 65), (1, 33, 8), (1, 63, 72), (2, 64, 64), (3, 65, 136), (1, 127, 31), (1, 128, 64),
    (2, 129, 200), (1, 255, 64), (1, 257, 512), (1, 511, 24), (2, 1000, 64), (1, 1025, 1409), (1, 4099, 33),
    (1, 2049, 64), (40, 70, 64), (1, 64, 4096), (2, 17, 2056)])
def test_scan_and_gradient(layers, b, t, d, mix, dtype):
    v, n = inputs(b, t, d, dtype, seed=t)
    check(layers, v, n, mix, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("starts,masked", [(0.02, False), (0.5, False), (1.0, False), (None, True), (0.1, True)])
@pytest.mark.parametrize("b,t,d,layout", [(2, 150, 64, "dense"), (1, 700, 72, "columns"), (3, 261, 33, "odd"),
                                          (2, 3, 128, "dense"), (4, 1, 64, "columns")])
def test_flags_and_strides(layers, b, t, d, layout, starts, masked, dtype):
    for state in (True, False):
        v, n = inputs(b, t, d, dtype, seed=3, state=state, starts=starts, masked=masked, layout=layout)
        check(layers, v, n, True, dtype)
    check(layers, v, n, False, dtype)


# one case for each way the length is cut up: blocks of one, four and eight warps, clusters of
# four and eight, few and many chunks
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout,extra", [("dense", 0), ("columns", 0), ("odd", 1), ("dense", 2), ("dense", 3)])
@pytest.mark.parametrize("b,t,d", [(2, 9, 64), (3, 15, 128), (3, 50, 192), (310, 37, 64), (20, 70, 1024),
                                   (9, 300, 960), (70, 200, 64), (3, 700, 64), (1, 2100, 128)])
def test_flags_however_the_length_is_cut(layers, b, t, d, layout, extra, dtype):
    v, n = inputs(b, t, d + extra, dtype, seed=13, starts=0.05, masked=True, layout=layout)
    check(layers, v, n, (b + t) % 2 == 0, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_halves_of_one_projection(layers, dtype):
    # gate and x side by side, an odd width each: rows and their first elements nowhere aligned
    for b, t, d in ((2, 900, 177), (1, 40, 33), (150, 60, 65)):
        gen = torch.Generator(device="cuda").manual_seed(d)
        n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        both = n(b, t, 2 * d).to(dtype)
        v = dict(gate=both[..., :d], x=both[..., d:], state=None, starts=None, token_mask=None)
        check(layers, v, n, True, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_saturated_gates(layers, dtype):
    # gates of exactly 0 and 1, and far beyond where their exponentials over- or underflow
    v, n = inputs(2, 300, 64, dtype, seed=4)
    v["gate"] = torch.where(torch.rand(2, 300, 64, device="cuda") < 0.5, v["gate"].sign() * 200, v["gate"])
    check(layers, v, n, True, dtype)
    v["gate"].fill_(60.0)       # nothing is taken in: the state stays
    o = layers.gated_scan_forward(v["gate"], v["x"], state=v["state"])
    assert torch.equal(o.state, v["state"])
    v["gate"].fill_(-200.0)     # nothing is kept
    o = layers.gated_scan_forward(v["gate"], v["x"], state=v["state"])
    assert torch.equal(o.h, v["x"]) and torch.equal(o.state, v["x"][:, -1].float())


@pytest.mark.parametrize("t", [50, 3000])
def test_long_memory_converges_to_what_it_is_fed(layers, t):
    # gates of 0.9997: the constant input comes out unchanged however long it runs
    x = torch.full((1, t, 64), 0.7, device="cuda")
    gate = torch.full_like(x, 8.0)
    o = layers.gated_scan_forward(gate, x, state=torch.full((1, 64), 0.7, device="cuda"))
    assert float((o.h - 0.7).abs().max()) < 1e-6


def test_all_tokens_masked_and_no_tokens(layers):
    v, n = inputs(2, 40, 64, F32)
    mask = torch.zeros(2, 40, dtype=torch.bool, device="cuda")
    o = layers.gated_scan_forward(v["gate"], v["x"], state=v["state"], token_mask=mask)
    assert torch.equal(o.state, v["state"]) and torch.equal(o.h, v["state"][:, None].expand(2, 40, 64))
    dl = n(2, 64)
    g = layers.gated_scan_backward(torch.zeros_like(v["x"]), v["gate"], v["x"], o.h, state=v["state"], dstate=dl,
                                   token_mask=mask)
    assert torch.equal(g.dstate, dl) and not g.dx.any() and not g.dgate.any()
    x = torch.empty(2, 0, 64, device="cuda")
    o = layers.gated_scan_forward(x, x, state=v["state"])
    assert o.h.shape == x.shape and torch.equal(o.state, v["state"])
    assert not layers.gated_scan_forward(x, x).state.any()
    g = layers.gated_scan_backward(x, x, x, x, state=v["state"], dstate=dl)
    assert torch.equal(g.dstate, dl) and g.dx.shape == x.shape
    x = torch.empty(0, 5, 64, device="cuda")
    assert layers.gated_scan_forward(x, x).h.shape == x.shape


@pytest.mark.parametrize("t", [6, 400])
def test_what_is_not_finite_stays_in_its_document_and_channel(layers, t):
    v, _ = inputs(2, t, 64, F32, seed=5, state=False)
    starts = torch.zeros(2, t, dtype=torch.bool, device="cuda")
    starts[0, t // 2] = True
    want = layers.gated_scan_forward(v["gate"], v["x"], starts=starts)
    x = v["x"].clone()
    x[0, 1, 7] = float("nan")
    x[0, 2, 9] = float("inf")
    got = layers.gated_scan_forward(v["gate"], x, starts=starts)
    other = torch.ones(64, dtype=torch.bool, device="cuda")
    other[[7, 9]] = False
    assert torch.equal(got.h[1], want.h[1]) and torch.equal(got.h[0][:, other], want.h[0][:, other])
    assert torch.equal(got.h[0, t // 2:], want.h[0, t // 2:]) and torch.equal(got.state, want.state)
    assert bool(got.h[0, 1:t // 2, 7].isnan().all())
    dh = torch.randn_like(x)
    want = layers.gated_scan_backward(dh, v["gate"], v["x"], want.h, starts=starts)
    dh[0, t // 2 + 1, 3] = float("nan")
    got = layers.gated_scan_backward(dh, v["gate"], v["x"], layers.gated_scan_forward(v["gate"], v["x"],
                                     starts=starts).h, starts=starts)
    assert torch.equal(got.dx[1], want.dx[1]) and torch.equal(got.dx[0, :t // 2], want.dx[0, :t // 2])


def test_one_token_at_a_time_is_the_sequence(layers):
    v, _ = inputs(3, 20, 96, F32, seed=6)
    whole = layers.gated_scan_forward(v["gate"], v["x"], state=v["state"])
    state, err = v["state"], 0.0
    for t in range(20):
        o = layers.gated_scan_forward(v["gate"][:, t:t + 1], v["x"][:, t:t + 1], state=state)
        err = max(err, float((o.h[:, 0] - whole.h[:, t]).abs().max()))
        state = o.state
    assert err < 2e-6 and float((state - whole.state).abs().max()) < 2e-6


def test_more_leading_dimensions_and_shapes_refused(layers):
    x = torch.randn(2, 3, 5, 8, device="cuda")
    gate = torch.randn_like(x)
    s = torch.randn(2, 3, 8, device="cuda")
    o = layers.gated_scan_forward(gate, x, state=s)
    p = layers.gated_scan_forward(gate.view(6, 5, 8), x.view(6, 5, 8), state=s.view(6, 8))
    assert o.state.shape == s.shape and torch.equal(o.h.view(6, 5, 8), p.h) and torch.equal(o.state.view(6, 8), p.state)
    one = layers.gated_scan_forward(gate[0, 0], x[0, 0])
    assert one.h.shape == (5, 8) and one.state.shape == (8,)
    flat = s.view(6, 8).clone().requires_grad_()        # the batch in one dimension
    (g,) = torch.autograd.grad(layers.gated_scan(gate, x, state=flat).h.sum(), flat)
    assert g.shape == (6, 8) and bool((g > 0).all())
    for bad in (dict(state=s.view(3, 2, 8)), dict(state=s.transpose(0, 1)), dict(state=s.view(-1)),
                dict(starts=torch.zeros(5, 6, dtype=torch.bool, device="cuda")),
                dict(token_mask=torch.zeros(2, 5, 3, dtype=torch.bool, device="cuda"))):
        with pytest.raises(ValueError):
            layers.gated_scan_forward(gate, x, **bad)
    with pytest.raises(TypeError):
        layers.gated_scan_forward(gate.bfloat16(), x)
    with pytest.raises(TypeError):
        layers.gated_scan_forward(gate, x, state=s.bfloat16())
    with pytest.raises(TypeError):
        layers.gated_scan_forward(gate, x, starts=torch.zeros(2, 3, 5, device="cuda"))
    with pytest.raises(ValueError):
        layers.gated_scan_forward(gate[0, 0, 0], x[0, 0, 0])
    with pytest.raises(ValueError):
        layers.gated_scan_forward(gate[:1], x)


@pytest.mark.parametrize("mix", [True, False])
def test_differentiable(layers, mix):
    v, n = inputs(2, 70, 24, F32, seed=7, starts=0.05, masked=True)
    w = clean(v)
    leaves = [v[k].clone().requires_grad_() for k in ("gate", "x", "state")]
    # neither gate nor x as rows: a transposed view
    args = [leaves[0].transpose(0, 1).contiguous().transpose(0, 1), leaves[1], leaves[2]]
    o = layers.gated_scan(args[0], args[1], state=args[2], starts=v["starts"], token_mask=v["token_mask"], mix=mix)
    ch, cl = n(2, 70, 24), n(2, 24)
    got = torch.autograd.grad((o.h * ch).sum() + (o.state * cl).sum(), leaves)
    want, err = ref.scan_grad(ref.f64(ch), w["gate"], w["x"], ref.f64(o.h), w["state"], ref.f64(cl), w["starts"],
                              w["token_mask"], mix)
    for g, e, r in zip(got, want, err):
        ref.close(g, e, r, F32)
    # only what is asked for, and from one output alone
    o = layers.gated_scan(v["gate"], leaves[1], mix=mix, token_mask=v["token_mask"])
    (g,) = torch.autograd.grad(o.state.sum(), leaves[1])
    assert bool(g[v["token_mask"]].isfinite().all())
    with pytest.raises(RuntimeError):
        (g,) = torch.autograd.grad((layers.gated_scan(v["gate"], leaves[1], mix=mix).h ** 2).sum(), leaves[1],
                                   create_graph=True)
        g.sum().backward()


def test_equal_bits_each_time_and_rows_past_the_end_untouched(layers):
    v, n = inputs(3, 777, 200, BF16, seed=8, starts=0.01)
    call = lambda: layers.gated_scan_forward(v["gate"], v["x"], state=v["state"], starts=v["starts"])  # noqa: E731
    a = call()
    dh = n(3, 777, 200).bfloat16()
    grad = lambda: layers.gated_scan_backward(dh, v["gate"], v["x"], a.h, state=v["state"], starts=v["starts"])  # noqa: E731
    g = grad()
    for _ in range(3):
        assert all(torch.equal(s, t) for s, t in zip(call(), a)) and all(torch.equal(s, t) for s, t in zip(grad(), g))


def test_state_updated_in_place_through_the_c_abi(layers):
    lib = muon().load()
    v, _ = inputs(4, 1, 64, F32, seed=9)
    want = layers.gated_scan_forward(v["gate"], v["x"], state=v["state"])
    h = torch.empty_like(v["x"])
    s = v["state"]
    guard = torch.full((4 * 64 + 64,), 7.0, device="cuda")
    guard[:256] = s.view(-1)
    p = guard.data_ptr()
    assert lib.muon_gated_scan(4, 1, 64, 1, v["gate"].data_ptr(), 64, v["x"].data_ptr(), 64, p, None, None, 1,
                               h.data_ptr(), p, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(guard[:256].view(4, 64), want.state) and torch.equal(h, want.h)
    assert bool((guard[256:] == 7).all())
