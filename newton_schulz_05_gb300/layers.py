"""Training operators around the optimizer step: layer norm (alone, or behind
dropout and the residual add), dropout from a counter-based generator, and the
expert router with its balance loss, each with its gradient.

They produce what MuonWithAdamW.step consumes: the 1-D gradients of norm scales
and biases (the AdamW path), and the router gradient and per-expert token sets
of [E, M, N] expert stacks (the Muon path).  Every computation runs in libmuon's
kernels (muon_layer_norm, muon_dropout, muon_route and their gradients in
include/muon.h, which states the formulas); this module marshals tensors.

Two levels:
  * layer_norm, dropout_add_layer_norm, dropout, route: differentiable
    (torch.autograd), inputs of any strides;
  * *_forward / *_backward: one library call each, outputs as named tuples.

Activations and logits are bf16 or fp32 CUDA tensors whose last dimension is
dense and whose leading dimensions are rows at one stride.  Calls run on the
current stream, or on `stream`: then outputs belong to that stream, and the
caller orders it after whatever produced the inputs.  Nothing is kept between
calls.  Dropout takes an explicit `seed` and `offset`; RandomCounter hands out
offsets that never overlap.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import MUON_BF16, MUON_F32, _check, load

__all__ = ["layer_norm", "dropout_add_layer_norm", "dropout", "route", "RandomCounter",
           "layer_norm_forward", "layer_norm_backward", "dropout_forward", "dropout_backward",
           "route_forward", "route_backward", "NormOut", "NormGrad", "RouteOut"]

_DT = {torch.bfloat16: MUON_BF16, torch.float32: MUON_F32}


class NormOut(NamedTuple):
    y: torch.Tensor
    sum: torch.Tensor      # what was normed: x itself without residual and dropout
    mean: torch.Tensor     # fp32, one a row
    rstd: torch.Tensor


class NormGrad(NamedTuple):
    dx: torch.Tensor
    dresidual: torch.Tensor            # dx itself without dropout
    dweight: Optional[torch.Tensor]
    dbias: Optional[torch.Tensor]


class RouteOut(NamedTuple):
    weights: torch.Tensor    # [tokens, k] fp32 combine weights, 0 at a missing pick
    index: torch.Tensor      # [tokens, k] int32 experts, -1 at a missing pick
    counts: torch.Tensor     # [experts + 1] int32: picks of each expert, then routed tokens
    mean_prob: torch.Tensor  # [experts] fp32
    loss: torch.Tensor       # fp32 scalar


class RandomCounter:
    """Offsets of dropout calls that share a seed: take(n) returns the offset
    of a call over n elements and moves past the counters it uses."""

    def __init__(self, seed: int, offset: int = 0):
        self.seed, self.offset = seed, offset

    def take(self, numel: int) -> int:
        at = self.offset
        self.offset += (numel + 7) // 8
        return at


def _dtype(t: torch.Tensor, what: str) -> int:
    dt = _DT.get(t.dtype)
    if dt is None:
        raise TypeError("%s must be bf16 or fp32, got %s" % (what, t.dtype))
    return dt


def _rows(t: torch.Tensor, what: str):
    """(rows, cols, row stride) of a tensor of rows; ValueError when it is
    not one."""
    if not t.is_cuda:
        raise ValueError("%s is not on a CUDA device" % what)
    shape = t.shape
    if not shape:
        raise ValueError("%s needs at least one dimension" % what)
    cols = shape[-1]
    if len(shape) == 2 and (cols <= 1 or t.stride(1) == 1):
        return shape[0], cols, t.stride(0)
    if t.is_contiguous():
        return (t.numel() // cols if cols else 0), cols, cols
    stride, rows, ld = t.stride(), 1, None
    for d in range(len(shape) - 2, -1, -1):       # leading dims, innermost first
        if shape[d] == 1:
            continue
        if ld is None:
            ld = stride[d]
        elif stride[d] != ld * rows:
            raise ValueError("the leading dimensions of %s are not rows at one stride" % what)
        rows *= shape[d]
    if cols > 1 and stride[-1] != 1:
        raise ValueError("the last dimension of %s is not dense" % what)
    return rows, cols, cols if ld is None else ld


def _as_rows(t: torch.Tensor) -> torch.Tensor:
    """t, or a dense copy when its strides are not those of rows."""
    try:
        _rows(t, "")
        return t
    except ValueError:
        return t.contiguous()


def _vector(t, cols: int, like: torch.Tensor, what: str) -> Optional[int]:
    if t is None:
        return None
    if t.dim() != 1 or t.shape[0] != cols or not t.is_contiguous():
        raise ValueError("%s must be a dense vector of %d elements" % (what, cols))
    if t.device != like.device:
        raise ValueError("%s is not on the device of the rows" % what)
    return t.data_ptr()


def _same(t: torch.Tensor, like: torch.Tensor, what: str):
    """Row stride of `t`, which must match `like` in shape, type and device."""
    if t.shape != like.shape or t.device != like.device:
        raise ValueError("%s must have shape %s on %s" % (what, tuple(like.shape), like.device))
    if t.dtype != like.dtype:
        raise TypeError("%s must be %s, got %s" % (what, like.dtype, t.dtype))
    return _rows(t, what)[2]


def _flat(t: torch.Tensor, numel: int, dtype, like: torch.Tensor, what: str) -> int:
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (what, dtype, t.dtype))
    if t.numel() != numel or not t.is_contiguous() or t.device != like.device:
        raise ValueError("%s must be dense with %d elements on %s" % (what, numel, like.device))
    return t.data_ptr()


def _on(stream, fn, args, kw):
    """fn on another stream: outputs are allocated there, and the inputs'
    memory is not reused before the stream has run the call."""
    with torch.cuda.stream(stream):
        out = fn(*args, **kw)
    for t in list(args) + list(kw.values()):
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    return out


def _here(t: torch.Tensor) -> int:
    """The current stream's handle on the device of t, which must be the
    current device."""
    if t.get_device() != torch.cuda.current_device():
        raise ValueError("tensors are on cuda:%d, the current device is cuda:%d"
                         % (t.get_device(), torch.cuda.current_device()))
    return torch.cuda.current_stream().cuda_stream


def _scratch(fn, rows: int, cols: int, like: torch.Tensor) -> torch.Tensor:
    need = ctypes.c_size_t()
    _check(fn(rows, cols, ctypes.byref(need)), "workspace_bytes")
    return torch.empty(need.value, dtype=torch.uint8, device=like.device)


def layer_norm_forward(x, weight=None, bias=None, *, eps: float = 1e-5, residual=None,
                       p: float = 0.0, seed: int = 0, offset: int = 0, stream=None) -> NormOut:
    """muon_layer_norm: y = norm(residual + dropout(x)) * weight + bias over
    the last dimension.  weight and bias are of one type, bf16 or fp32."""
    if stream is not None:
        return _on(stream, layer_norm_forward, (x, weight, bias),
                   dict(eps=eps, residual=residual, p=p, seed=seed, offset=offset))
    dt = _dtype(x, "x")
    rows, cols, ld = _rows(x, "x")
    wdt = MUON_F32
    if weight is not None or bias is not None:
        wdt = _dtype(weight if weight is not None else bias, "weight and bias")
        if weight is not None and bias is not None and weight.dtype != bias.dtype:
            raise TypeError("weight and bias must be of one type")
    wp, bp = _vector(weight, cols, x, "weight"), _vector(bias, cols, x, "bias")
    handle = _here(x)
    rp, ldr, total, tp = None, 0, x, None
    if residual is not None:
        ldr = _same(residual, x, "residual")
        rp = residual.data_ptr()
    if rp is not None or p != 0.0:
        total = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        tp = total.data_ptr()
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    rstd = torch.empty_like(mean)
    _check(load().muon_layer_norm(rows, cols, dt, wdt, x.data_ptr(), ld, rp, ldr, wp, bp, eps, p,
                                  seed, offset, tp, y.data_ptr(), mean.data_ptr(),
                                  rstd.data_ptr(), handle), "muon_layer_norm")
    return NormOut(y, total, mean, rstd)


def layer_norm_backward(dy, sum, mean, rstd, weight=None, *, dsum=None, p: float = 0.0,
                        seed: int = 0, offset: int = 0, need_weight: bool = True,
                        need_bias: bool = True, stream=None) -> NormGrad:
    """muon_layer_norm_backward: gradients of x, of the residual, and (where
    needed) of weight and bias, in the weight's type (fp32 without a weight).
    `sum`, mean and rstd are the forward pass's; dsum is the gradient that
    reaches `sum` past the norm; p, seed and offset are the forward pass's."""
    if stream is not None:
        return _on(stream, layer_norm_backward, (dy, sum, mean, rstd, weight),
                   dict(dsum=dsum, p=p, seed=seed, offset=offset, need_weight=need_weight,
                        need_bias=need_bias))
    L = load()
    dt = _dtype(dy, "dy")
    rows, cols, ld = _rows(dy, "dy")
    lds = _same(sum, dy, "sum")
    mp = _flat(mean, rows, torch.float32, dy, "mean")
    vp = _flat(rstd, rows, torch.float32, dy, "rstd")
    wdtype = torch.float32 if weight is None else weight.dtype
    wdt = MUON_F32 if weight is None else _dtype(weight, "weight")
    wp = _vector(weight, cols, dy, "weight")
    handle = _here(dy)
    dp, ldd = None, 0
    if dsum is not None:
        ldd = _same(dsum, dy, "dsum")
        dp = dsum.data_ptr()
    dx = torch.empty(dy.shape, dtype=dy.dtype, device=dy.device)
    dres, drp = dx, None
    if p != 0.0:
        dres = torch.empty(dy.shape, dtype=dy.dtype, device=dy.device)
        drp = dres.data_ptr()
    dw = db = wsp = None
    nbytes = 0
    if need_weight or need_bias:
        dw = torch.empty(cols, dtype=wdtype, device=dy.device) if need_weight else None
        db = torch.empty(cols, dtype=wdtype, device=dy.device) if need_bias else None
        ws = _scratch(L.muon_layer_norm_workspace_bytes, rows, cols, dy)
        wsp, nbytes = ws.data_ptr(), ws.numel()
    _check(L.muon_layer_norm_backward(
        rows, cols, dt, wdt, dy.data_ptr(), ld, sum.data_ptr(), lds, mp, vp, wp, dp, ldd, p, seed,
        offset, dx.data_ptr(), drp, None if dw is None else dw.data_ptr(),
        None if db is None else db.data_ptr(), wsp, nbytes, handle), "muon_layer_norm_backward")
    return NormGrad(dx, dres, dw, db)


def dropout_forward(x, p: float, *, seed: int, offset: int = 0, residual=None, out=None,
                    stream=None) -> torch.Tensor:
    """muon_dropout: residual + dropout(x) over dense tensors; `out` may be x
    or residual itself."""
    if stream is not None:
        return _on(stream, dropout_forward, (x, p),
                   dict(seed=seed, offset=offset, residual=residual, out=out))
    dt = _dtype(x, "x")
    n = x.numel()
    xp = _flat(x, n, x.dtype, x, "x")
    if not x.is_cuda:
        raise ValueError("x is not on a CUDA device")
    handle = _here(x)
    rp = None
    if residual is not None:
        if residual.shape != x.shape:
            raise ValueError("residual must have shape %s" % (tuple(x.shape),))
        rp = _flat(residual, n, x.dtype, x, "residual")
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    elif out.shape != x.shape:
        raise ValueError("out must have shape %s" % (tuple(x.shape),))
    op = _flat(out, n, x.dtype, x, "out")
    _check(load().muon_dropout(n, dt, xp, rp, p, seed, offset, op, handle), "muon_dropout")
    return out


def dropout_backward(dy, p: float, *, seed: int, offset: int = 0, out=None,
                     stream=None) -> torch.Tensor:
    """Gradient of dropout_forward's x (the residual's is dy itself)."""
    return dropout_forward(dy, p, seed=seed, offset=offset, out=out, stream=stream)


def _mask_ptr(token_mask, tokens: int, like: torch.Tensor) -> Optional[int]:
    if token_mask is None:
        return None
    if token_mask.dtype not in (torch.bool, torch.uint8):
        raise TypeError("token_mask must be bool or uint8, got %s" % token_mask.dtype)
    return _flat(token_mask, tokens, token_mask.dtype, like, "token_mask")


def route_forward(logits, k: int, *, token_mask=None, normalize: bool = True,
                  stream=None) -> RouteOut:
    """muon_route over logits [..., experts]: the k largest of each token,
    their combine weights, per-expert counts, mean probabilities and the
    balance loss.  token_mask (bool or uint8, one a token): tokens that count."""
    if stream is not None:
        return _on(stream, route_forward, (logits, k),
                   dict(token_mask=token_mask, normalize=normalize))
    L = load()
    dt = _dtype(logits, "logits")
    tokens, experts, ld = _rows(logits, "logits")
    handle = _here(logits)
    dev = logits.device
    mp = _mask_ptr(token_mask, tokens, logits)
    ws = _scratch(L.muon_route_workspace_bytes, tokens, experts, logits)
    shape = logits.shape[:-1] + (max(k, 0),)
    weights = torch.empty(shape, dtype=torch.float32, device=dev)
    index = torch.empty(shape, dtype=torch.int32, device=dev)
    counts = torch.empty(experts + 1, dtype=torch.int32, device=dev)
    mean_prob = torch.empty(experts, dtype=torch.float32, device=dev)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    _check(L.muon_route(tokens, experts, k, dt, logits.data_ptr(), ld, mp, 1 if normalize else 0,
                        weights.data_ptr(), index.data_ptr(), counts.data_ptr(),
                        mean_prob.data_ptr(), loss.data_ptr(), ws.data_ptr(), ws.numel(), handle),
           "muon_route")
    return RouteOut(weights, index, counts, mean_prob, loss)


def route_backward(logits, index, counts, *, dweights=None, dloss=None, token_mask=None,
                   normalize: bool = True, stream=None) -> torch.Tensor:
    """muon_route_backward: gradient of the logits from those of the combine
    weights and of the loss (an fp32 scalar on the device); index and counts
    are route_forward's."""
    if stream is not None:
        return _on(stream, route_backward, (logits, index, counts),
                   dict(dweights=dweights, dloss=dloss, token_mask=token_mask,
                        normalize=normalize))
    dt = _dtype(logits, "logits")
    tokens, experts, ld = _rows(logits, "logits")
    handle = _here(logits)
    if not index.dim() or index.shape[:-1] != logits.shape[:-1]:
        raise ValueError("index must have one row of picks a token")
    k = index.shape[-1]
    ip = _flat(index, tokens * k, torch.int32, logits, "index")
    cp = _flat(counts, experts + 1, torch.int32, logits, "counts")
    wp = None if dweights is None else _flat(dweights, tokens * k, torch.float32, logits, "dweights")
    lp = None if dloss is None else _flat(dloss, 1, torch.float32, logits, "dloss")
    mp = _mask_ptr(token_mask, tokens, logits)
    dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    _check(load().muon_route_backward(tokens, experts, k, dt, logits.data_ptr(), ld, mp,
                                      1 if normalize else 0, ip, cp, wp, lp, dlogits.data_ptr(),
                                      handle), "muon_route_backward")
    return dlogits


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, bias, eps, p, seed, offset):
        o = layer_norm_forward(x, weight, bias, eps=eps, residual=residual, p=p, seed=seed,
                               offset=offset)
        ctx.save_for_backward(o.sum, o.mean, o.rstd, weight)
        ctx.drop = dict(p=p, seed=seed, offset=offset)
        ctx.bias_dtype = None if bias is None else bias.dtype
        ctx.set_materialize_grads(False)
        if residual is None and p == 0.0:
            return o.y, None
        return o.y, o.sum

    @staticmethod
    def backward(ctx, dy, dsum):
        total, mean, rstd, weight = ctx.saved_tensors
        if dy is None and dsum is None:
            return (None,) * 8
        dy = torch.zeros_like(total) if dy is None else _as_rows(dy)
        dsum = None if dsum is None else _as_rows(dsum)
        need_w, need_b = ctx.needs_input_grad[2], ctx.needs_input_grad[3]
        g = layer_norm_backward(dy, total, mean, rstd, weight, dsum=dsum, need_weight=need_w,
                                need_bias=need_b, **ctx.drop)
        db = g.dbias
        if db is not None and db.dtype != ctx.bias_dtype:    # a bias without a weight
            db = db.to(ctx.bias_dtype)
        return (g.dx, g.dresidual if ctx.needs_input_grad[1] else None, g.dweight, db,
                None, None, None, None)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5) -> torch.Tensor:
    """Differentiable layer norm over the last dimension."""
    return _LayerNorm.apply(_as_rows(x), None, weight, bias, eps, 0.0, 0, 0)[0]


def dropout_add_layer_norm(x, residual, weight=None, bias=None, *, p: float, seed: int,
                           offset: int = 0, eps: float = 1e-5):
    """Differentiable (y, s) with s = residual + dropout(x), y = layer norm of
    s: the end of one sublayer and the norm in front of the next."""
    if x.shape != residual.shape:
        raise ValueError("residual must have shape %s" % (tuple(x.shape),))
    return _LayerNorm.apply(_as_rows(x), _as_rows(residual), weight, bias, eps, p, seed, offset)


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, offset):
        ctx.drop = dict(p=p, seed=seed, offset=offset)
        return dropout_forward(x, p, seed=seed, offset=offset, residual=residual)

    @staticmethod
    def backward(ctx, dy):
        dx = dropout_backward(dy.contiguous(), **ctx.drop) if ctx.needs_input_grad[0] else None
        return dx, dy if ctx.needs_input_grad[1] else None, None, None, None


def dropout(x, p: float, *, seed: int, offset: int = 0, residual=None) -> torch.Tensor:
    """Differentiable residual + dropout(x); the flags are recomputed in the
    backward pass from seed and offset."""
    return _Dropout.apply(x.contiguous(), None if residual is None else residual.contiguous(), p,
                          seed, offset)


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, token_mask, normalize):
        o = route_forward(logits, k, token_mask=token_mask, normalize=normalize)
        ctx.save_for_backward(logits, o.index, o.counts, token_mask)
        ctx.normalize = normalize
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(o.index, o.counts, o.mean_prob)
        return o.weights, o.index, o.counts, o.mean_prob, o.loss

    @staticmethod
    def backward(ctx, dweights, _index, _counts, _mean_prob, dloss):
        if dweights is None and dloss is None:
            return None, None, None, None
        logits, index, counts, mask = ctx.saved_tensors
        d = route_backward(logits, index, counts, token_mask=mask, normalize=ctx.normalize,
                           dweights=None if dweights is None else dweights.contiguous(),
                           dloss=None if dloss is None else dloss.contiguous())
        return d, None, None, None


def route(logits, k: int, *, token_mask=None, normalize: bool = True) -> RouteOut:
    """Differentiable router: gradients flow to the logits from the combine
    weights and from the balance loss."""
    mask = None if token_mask is None else token_mask.contiguous()
    return RouteOut(*_Route.apply(_as_rows(logits), k, mask, normalize))
