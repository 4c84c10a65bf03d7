"""Training operators around the optimizer step: layer norm (alone, or behind
dropout and the residual add), dropout from a counter-based generator, and the
expert router with its balance loss, each with its gradient.

They produce what MuonWithAdamW.step consumes: the 1-D gradients of norm scales
and biases (the AdamW path), and the router gradient and per-expert token sets
of [E, M, N] expert stacks (the Muon path).  Every computation runs in libmuon's
kernels (muon_layer_norm, muon_dropout, muon_route and their gradients in
include/muon.h, which states the formulas); this module and its compiled half
(csrc/binding.cpp) check and marshal tensors.

Two levels:
  * layer_norm, dropout_add_layer_norm, dropout, route: differentiable once
    (torch.autograd), inputs of any strides;
  * *_forward / *_backward: one library call each, outputs as named tuples.

Activations and logits are bf16 or fp32 CUDA tensors whose last dimension is
dense and whose leading dimensions are rows at one stride.  Calls run on the
current stream, or on `stream`: then outputs belong to that stream, and the
caller orders it after whatever produced the inputs.  Nothing is kept between
calls.  Dropout takes an explicit `seed` and `offset`; RandomCounter hands out
offsets that never overlap.  A captured CUDA graph replays the seed and offset it
was captured with: the same elements are dropped at every replay.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import _check, load
from .build import binding_path

__all__ = ["layer_norm", "dropout_add_layer_norm", "dropout", "route", "RandomCounter",
           "layer_norm_forward", "layer_norm_backward", "dropout_forward", "dropout_backward",
           "route_forward", "route_backward", "NormOut", "NormGrad", "RouteOut"]

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
    of a call over n elements and moves past the counters it uses.

    Under activation checkpointing the forward pass runs again during the
    backward pass and must drop the same elements, so its offsets are taken
    outside of the checkpointed function and passed in.  take() raises where it
    is called during a backward pass: the offset would be another than the first
    run's, and the gradients wrong without a sign of it."""

    def __init__(self, seed: int, offset: int = 0):
        self.seed, self.offset = seed, offset

    def take(self, numel: int) -> int:
        if torch._C._current_graph_task_id() != -1:
            raise RuntimeError("RandomCounter.take() in a backward pass: a recomputed forward pass "
                               "would drop other elements than the first run; take the offset outside "
                               "of the checkpointed function and pass it in")
        at = self.offset
        self.offset += (numel + 7) // 8
        return at


_bound = None


def _b():
    """The compiled half (built by newton_schulz_05_gb300.build.build()), which
    checks tensors, allocates outputs and calls libmuon."""
    global _bound
    if _bound is None:
        lib = load()
        path = binding_path()
        if not os.path.exists(path):
            raise RuntimeError("the binding is not built at %s: run newton_schulz_05_gb300.build.build()"
                               % path)
        spec = importlib.util.spec_from_file_location(__package__ + "._binding", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind({name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
                     for name in ("muon_layer_norm", "muon_layer_norm_backward",
                                  "muon_layer_norm_workspace_bytes", "muon_dropout", "muon_route",
                                  "muon_route_workspace_bytes", "muon_route_backward")})
        _bound = module
    return _bound


def _as_rows(t: torch.Tensor) -> torch.Tensor:
    """t, or a dense copy when its strides are not those of rows."""
    return t if _b().is_rows(t) else t.contiguous()


def _on(stream, fn, args, kw):
    """fn on another stream: outputs are allocated there, and the inputs'
    memory is not reused before the stream has run the call."""
    with torch.cuda.stream(stream):
        out = fn(*args, **kw)
    for t in list(args) + list(kw.values()):
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    return out


def layer_norm_forward(x, weight=None, bias=None, *, eps: float = 1e-5, residual=None,
                       p: float = 0.0, seed: int = 0, offset: int = 0, stream=None) -> NormOut:
    """muon_layer_norm: y = norm(residual + dropout(x)) * weight + bias over
    the last dimension.  weight and bias are of one type, bf16 or fp32."""
    if stream is not None:
        return _on(stream, layer_norm_forward, (x, weight, bias),
                   dict(eps=eps, residual=residual, p=p, seed=seed, offset=offset))
    r = (_bound or _b()).layer_norm_forward(x, weight, bias, eps, residual, p, seed, offset)
    if type(r) is int:
        _check(r, "muon_layer_norm")
    y, total, mean, rstd = r
    return NormOut(y, x if total is None else total, mean, rstd)


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
    r = (_bound or _b()).layer_norm_backward(dy, sum, mean, rstd, weight, dsum, p, seed, offset,
                                             need_weight, need_bias)
    if type(r) is int:
        _check(r, "muon_layer_norm_backward")
    dx, dres, dw, db = r
    return NormGrad(dx, dx if dres is None else dres, dw, db)


def dropout_forward(x, p: float, *, seed: int, offset: int = 0, residual=None, out=None,
                    stream=None) -> torch.Tensor:
    """muon_dropout: residual + dropout(x) over dense tensors; `out` may be x
    or residual itself.  Writing to `out` counts as an in-place change of it: a
    backward pass that saved it raises, and while gradients are recorded an
    `out` that requires grad is refused."""
    if stream is not None:
        return _on(stream, dropout_forward, (x, p),
                   dict(seed=seed, offset=offset, residual=residual, out=out))
    r = (_bound or _b()).dropout(x, p, seed, offset, residual, out)
    if type(r) is int:
        _check(r, "muon_dropout")
    return r


def dropout_backward(dy, p: float, *, seed: int, offset: int = 0, out=None,
                     stream=None) -> torch.Tensor:
    """Gradient of dropout_forward's x (the residual's is dy itself)."""
    return dropout_forward(dy, p, seed=seed, offset=offset, out=out, stream=stream)


def route_forward(logits, k: int, *, token_mask=None, normalize: bool = True,
                  stream=None) -> RouteOut:
    """muon_route over logits [..., experts]: the k largest of each token,
    their combine weights, per-expert counts, mean probabilities and the
    balance loss.  token_mask (bool or uint8, one a token, in the shape of the
    logits' leading dimensions or as one dimension): tokens that count."""
    if stream is not None:
        return _on(stream, route_forward, (logits, k),
                   dict(token_mask=token_mask, normalize=normalize))
    r = (_bound or _b()).route_forward(logits, k, token_mask, normalize)
    if type(r) is int:
        _check(r, "muon_route")
    return RouteOut._make(r)


def route_backward(logits, index, counts, *, dweights=None, dloss=None, token_mask=None,
                   normalize: bool = True, stream=None) -> torch.Tensor:
    """muon_route_backward: gradient of the logits from those of the combine
    weights and of the loss (an fp32 scalar on the device); index and counts
    are route_forward's."""
    if stream is not None:
        return _on(stream, route_backward, (logits, index, counts),
                   dict(dweights=dweights, dloss=dloss, token_mask=token_mask,
                        normalize=normalize))
    r = (_bound or _b()).route_backward(logits, index, counts, dweights, dloss, token_mask, normalize)
    if type(r) is int:
        _check(r, "muon_route_backward")
    return r


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
    @once_differentiable
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
    @once_differentiable
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
    @once_differentiable
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
