"""Training operators around the optimizer step: layer norm (alone, or behind
dropout and the residual add), dropout from a counter-based generator, the
expert router with its balance loss; and over sequences a gated linear
recurrence, the norms of query and key heads with the rotation of positions, log
probabilities of given tokens and the clipped policy loss on them.  Each comes
with its gradient.

They produce what MuonWithAdamW.step consumes: the 1-D gradients of norm scales
and biases (the AdamW path), and what the gradients of the matrices between them
are made from (the Muon path).  Every computation runs in libmuon's kernels
(include/muon.h states the formulas); this module and its compiled half
(csrc/binding.cpp) check and marshal tensors.

Two levels:
  * layer_norm, dropout_add_layer_norm, dropout, route, gated_scan,
    norm_rotate_heads, token_log_probs, policy_loss: differentiable once
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
           "route_forward", "route_backward", "NormOut", "NormGrad", "RouteOut",
           "gated_scan", "norm_rotate_heads", "rotation_table", "token_log_probs", "policy_loss",
           "gated_scan_forward", "gated_scan_backward", "norm_rotate_heads_forward",
           "norm_rotate_heads_backward", "token_log_probs_forward", "token_log_probs_backward",
           "policy_loss_forward", "policy_loss_backward", "ScanOut", "ScanGrad", "HeadsOut",
           "HeadsGrad", "LogProbsOut", "PolicyOut"]

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


class ScanOut(NamedTuple):
    h: torch.Tensor          # the state behind each token, in x's type
    state: torch.Tensor      # [..., dim] fp32: the state behind the last token


class ScanGrad(NamedTuple):
    dgate: Optional[torch.Tensor]
    dx: Optional[torch.Tensor]
    dstate: Optional[torch.Tensor]     # of the state before the first token


class HeadsOut(NamedTuple):
    q: torch.Tensor
    k: Optional[torch.Tensor]


class HeadsGrad(NamedTuple):
    dq: Optional[torch.Tensor]
    dk: Optional[torch.Tensor]
    dq_weight: Optional[torch.Tensor]
    dk_weight: Optional[torch.Tensor]


class LogProbsOut(NamedTuple):
    log_probs: torch.Tensor  # fp32, one a token, 0 for an ignored one
    lse: torch.Tensor        # fp32: logarithm of the softmax's sum


class PolicyOut(NamedTuple):
    loss: torch.Tensor       # fp32 scalars: the loss,
    kl: torch.Tensor         # its KL term before kl's factor,
    clipped: torch.Tensor    # the share of clipped tokens
    weights: torch.Tensor    # [...] fp32: weight of each token of a sequence


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


_ENTRY_POINTS = (
    "muon_layer_norm", "muon_layer_norm_backward", "muon_layer_norm_workspace_bytes", "muon_dropout",
    "muon_route", "muon_route_workspace_bytes", "muon_route_backward", "muon_gated_scan",
    "muon_gated_scan_backward", "muon_norm_rotate_heads", "muon_norm_rotate_heads_backward",
    "muon_norm_rotate_heads_workspace_bytes", "muon_token_log_probs", "muon_token_log_probs_backward",
    "muon_policy_loss", "muon_policy_loss_backward", "muon_policy_loss_workspace_bytes")

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
                     for name in _ENTRY_POINTS})
        _bound = module
    return _bound


def _as_rows(t: torch.Tensor) -> torch.Tensor:
    """t, or a dense copy when its strides are not those of rows."""
    return t if _b().is_rows(t) else t.contiguous()


def _dense(t):
    """A dense tensor; what is none passes, for the binding to refuse (None: to take)."""
    return t.contiguous() if isinstance(t, torch.Tensor) else t


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
    return _LayerNorm.apply(_as_rows(x), None, _dense(weight), _dense(bias), eps, 0.0, 0, 0)[0]


def dropout_add_layer_norm(x, residual, weight=None, bias=None, *, p: float, seed: int,
                           offset: int = 0, eps: float = 1e-5):
    """Differentiable (y, s) with s = residual + dropout(x), y = layer norm of
    s: the end of one sublayer and the norm in front of the next."""
    if x.shape != residual.shape:
        raise ValueError("residual must have shape %s" % (tuple(x.shape),))
    return _LayerNorm.apply(_as_rows(x), _as_rows(residual), _dense(weight), _dense(bias), eps, p, seed,
                            offset)


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


# ---------------------------------------------------------------- over sequences

def gated_scan_forward(gate, x, *, state=None, starts=None, token_mask=None, mix: bool = True,
                       stream=None) -> ScanOut:
    """muon_gated_scan over x [..., tokens, dim]: h = a p + (1 - a) x (or a p + x
    without `mix`) with a = sigmoid(gate) and p the state before the token, 0
    where the token starts over.  state: [..., dim] fp32, the state before the
    first token.  starts, token_mask: bool or uint8, one a token; masked tokens
    pass the state on."""
    if stream is not None:
        return _on(stream, gated_scan_forward, (gate, x),
                   dict(state=state, starts=starts, token_mask=token_mask, mix=mix))
    r = (_bound or _b()).gated_scan_forward(gate, x, state, starts, token_mask, mix)
    if type(r) is int:
        _check(r, "muon_gated_scan")
    return ScanOut._make(r)


def gated_scan_backward(dh, gate, x, h, *, state=None, dstate=None, starts=None, token_mask=None,
                        mix: bool = True, need_gate: bool = True, need_x: bool = True,
                        need_state: bool = True, stream=None) -> ScanGrad:
    """muon_gated_scan_backward: gradients of gate, x and the state before the
    first token from those of h and (dstate) of the last state; h and the
    flags are the forward pass's.  x is not read without `mix` and may be None."""
    if stream is not None:
        return _on(stream, gated_scan_backward, (dh, gate, x, h),
                   dict(state=state, dstate=dstate, starts=starts, token_mask=token_mask, mix=mix,
                        need_gate=need_gate, need_x=need_x, need_state=need_state))
    r = (_bound or _b()).gated_scan_backward(dh, gate, x, h, state, dstate, starts, token_mask, mix,
                                             need_gate, need_x, need_state)
    if type(r) is int:
        _check(r, "muon_gated_scan_backward")
    return ScanGrad._make(r)


class _GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, x, state, starts, token_mask, mix):
        o = gated_scan_forward(gate, x, state=state, starts=starts, token_mask=token_mask, mix=mix)
        ctx.save_for_backward(gate, x if mix else None, o.h, state, starts, token_mask)
        ctx.mix = mix
        ctx.set_materialize_grads(False)
        return o.h, o.state

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dstate):
        if dh is None and dstate is None:
            return (None,) * 6
        gate, x, h, state, starts, token_mask = ctx.saved_tensors
        need = ctx.needs_input_grad
        g = gated_scan_backward(torch.zeros_like(h) if dh is None else _as_rows(dh), gate, x, h,
                                state=state, dstate=None if dstate is None else dstate.contiguous(),
                                starts=starts, token_mask=token_mask, mix=ctx.mix, need_gate=need[0],
                                need_x=need[1], need_state=need[2])
        ds = None if g.dstate is None else g.dstate.view(state.shape)      # batch in one dimension or several
        return g.dgate, g.dx, ds, None, None, None


def gated_scan(gate, x, *, state=None, starts=None, token_mask=None, mix: bool = True) -> ScanOut:
    """Differentiable gated linear recurrence: gradients flow to gate, x and
    state, from h and from the last state."""
    dense = [_dense(t) for t in (state, starts, token_mask)]
    return ScanOut(*_GatedScan.apply(_as_rows(gate), _as_rows(x), *dense, mix))


def rotation_table(length: int, rotary: int, *, base: float = 10000.0, device="cuda"):
    """(cos, sin) of the angles position * base ** (-2 m / rotary), [length, rotary / 2]
    fp32, from 64-bit angles: a program makes it once and hands it to
    norm_rotate_heads."""
    if rotary < 0 or rotary % 2:
        raise ValueError("rotary must be even and not negative, got %d" % rotary)
    pairs = torch.arange(rotary // 2, dtype=torch.float64, device=device)
    angle = torch.arange(length, dtype=torch.float64, device=device)[:, None] * \
        base ** (-2.0 * pairs / max(rotary, 1))
    return angle.cos().float(), angle.sin().float()


def norm_rotate_heads_forward(q, k=None, q_weight=None, k_weight=None, *, cos=None, sin=None,
                              positions=None, eps: float = 1e-6, neighbours: bool = False,
                              stream=None) -> HeadsOut:
    """muon_norm_rotate_heads: RMS norm of each head of q and k [..., heads, dim]
    over its elements, times the weights [dim], and the rotation of the first
    2 * cos.shape[1] elements by the angles of the tokens' positions (rows of
    cos and sin [table, pairs]; int64, one a token; without them a token's index
    in the last dimension of the tokens).  Pairs are elements m and m + pairs, or
    2 m and 2 m + 1 (neighbours).  A token whose position is outside of the table is
    none: its heads are 0."""
    if stream is not None:
        return _on(stream, norm_rotate_heads_forward, (q, k, q_weight, k_weight),
                   dict(cos=cos, sin=sin, positions=positions, eps=eps, neighbours=neighbours))
    r = (_bound or _b()).norm_rotate_heads_forward(q, k, q_weight, k_weight, cos, sin, positions, eps,
                                                   neighbours)
    if type(r) is int:
        _check(r, "muon_norm_rotate_heads")
    return HeadsOut._make(r)


def norm_rotate_heads_backward(dq, dk, q, k=None, q_weight=None, k_weight=None, *, cos=None, sin=None,
                               positions=None, eps: float = 1e-6, neighbours: bool = False,
                               need_q: bool = True, need_k: bool = True, need_q_weight: bool = True,
                               need_k_weight: bool = True, stream=None) -> HeadsGrad:
    """muon_norm_rotate_heads_backward: gradients of q, k and (where needed) of
    the weights, in the weights' type (fp32 without weights), from those of the
    forward pass's outputs; everything else as in the forward pass."""
    if stream is not None:
        return _on(stream, norm_rotate_heads_backward, (dq, dk, q, k, q_weight, k_weight),
                   dict(cos=cos, sin=sin, positions=positions, eps=eps, neighbours=neighbours,
                        need_q=need_q, need_k=need_k, need_q_weight=need_q_weight,
                        need_k_weight=need_k_weight))
    r = (_bound or _b()).norm_rotate_heads_backward(q, k, q_weight, k_weight, cos, sin, positions, eps,
                                                    neighbours, dq, dk, need_q, need_k, need_q_weight,
                                                    need_k_weight)
    if type(r) is int:
        _check(r, "muon_norm_rotate_heads_backward")
    return HeadsGrad._make(r)


def _as_heads(t: torch.Tensor) -> torch.Tensor:
    """t, or a dense copy when its strides are not those of heads of tokens."""
    return t if _b().is_heads(t) else t.contiguous()


class _NormRotateHeads(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, cos, sin, positions, eps, neighbours):
        o = norm_rotate_heads_forward(q, k, q_weight, k_weight, cos=cos, sin=sin, positions=positions,
                                      eps=eps, neighbours=neighbours)
        ctx.save_for_backward(q, k, q_weight, k_weight, cos, sin, positions)
        ctx.how = dict(eps=eps, neighbours=neighbours)
        ctx.set_materialize_grads(False)
        return o.q, o.k

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        if dq is None and dk is None:
            return (None,) * 9
        q, k, q_weight, k_weight, cos, sin, positions = ctx.saved_tensors
        need = ctx.needs_input_grad
        dq = torch.zeros_like(q) if dq is None else _as_heads(dq)
        if k is not None:
            dk = torch.zeros_like(k) if dk is None else _as_heads(dk)
        g = norm_rotate_heads_backward(dq, dk, q, k, q_weight, k_weight, cos=cos, sin=sin,
                                       positions=positions, need_q=need[0], need_k=need[1],
                                       need_q_weight=need[2], need_k_weight=need[3], **ctx.how)
        return g.dq, g.dk, g.dq_weight, g.dk_weight, None, None, None, None, None


def norm_rotate_heads(q, k=None, q_weight=None, k_weight=None, *, cos=None, sin=None, positions=None,
                      eps: float = 1e-6, neighbours: bool = False) -> HeadsOut:
    """Differentiable norms of query and key heads with the rotation of
    positions."""
    dense = [_dense(t) for t in (q_weight, k_weight, cos, sin, positions)]
    return HeadsOut(*_NormRotateHeads.apply(_as_heads(q), None if k is None else _as_heads(k), *dense, eps,
                                            neighbours))


def token_log_probs_forward(logits, tokens, *, scale: float = 1.0, stream=None) -> LogProbsOut:
    """muon_token_log_probs: log softmax(scale * logits) [..., vocab] at the
    given tokens (int64, one a row), and the logarithm of the softmax's sum.  A
    token outside of the vocabulary (-100, say) is ignored: 0."""
    if stream is not None:
        return _on(stream, token_log_probs_forward, (logits, tokens), dict(scale=scale))
    r = (_bound or _b()).token_log_probs_forward(logits, tokens, scale)
    if type(r) is int:
        _check(r, "muon_token_log_probs")
    return LogProbsOut._make(r)


def token_log_probs_backward(dlog_probs, logits, tokens, lse, *, scale: float = 1.0, out=None,
                             stream=None) -> torch.Tensor:
    """muon_token_log_probs_backward: gradient of the logits.  `out` may be
    the logits themselves, which it then replaces; writing to it counts as an
    in-place change, and while gradients are recorded an `out` that requires
    grad is refused."""
    if stream is not None:
        return _on(stream, token_log_probs_backward, (dlog_probs, logits, tokens, lse),
                   dict(scale=scale, out=out))
    r = (_bound or _b()).token_log_probs_backward(dlog_probs, logits, tokens, lse, scale, out)
    if type(r) is int:
        _check(r, "muon_token_log_probs_backward")
    return r


class _TokenLogProbs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, scale):
        o = token_log_probs_forward(logits, tokens, scale=scale)
        ctx.save_for_backward(logits, tokens, o.lse)
        ctx.scale = scale
        ctx.mark_non_differentiable(o.lse)
        ctx.set_materialize_grads(False)
        return o.log_probs, o.lse

    @staticmethod
    @once_differentiable
    def backward(ctx, dlog_probs, _lse):
        if dlog_probs is None:
            return None, None, None
        logits, tokens, lse = ctx.saved_tensors
        return token_log_probs_backward(dlog_probs.contiguous(), logits, tokens, lse,
                                        scale=ctx.scale), None, None


def token_log_probs(logits, tokens, *, scale: float = 1.0) -> torch.Tensor:
    """Differentiable log probabilities of given tokens, fp32, one a row.  Minus
    their mean is the cross entropy."""
    return _TokenLogProbs.apply(_as_rows(logits), tokens.contiguous(), scale)[0]


def policy_loss_forward(log_probs, old_log_probs, advantages, *, ref_log_probs=None, token_mask=None,
                        clip_low: float = 0.2, clip_high: float = 0.2, kl: float = 0.0,
                        by_sequence: bool = False, stream=None) -> PolicyOut:
    """muon_policy_loss over fp32 [..., tokens]: the clipped surrogate of the
    ratios exp(log_probs - old_log_probs) times the advantages (one a token, or
    one a sequence) plus kl times the KL estimate against ref_log_probs, as
    a mean over all tokens that count, or over sequences of the means over
    theirs.  token_mask (bool or uint8, one a token): tokens that count."""
    if stream is not None:
        return _on(stream, policy_loss_forward, (log_probs, old_log_probs, advantages),
                   dict(ref_log_probs=ref_log_probs, token_mask=token_mask, clip_low=clip_low,
                        clip_high=clip_high, kl=kl, by_sequence=by_sequence))
    r = (_bound or _b()).policy_loss_forward(log_probs, old_log_probs, advantages, ref_log_probs,
                                             token_mask, clip_low, clip_high, kl, by_sequence)
    if type(r) is int:
        _check(r, "muon_policy_loss")
    return PolicyOut._make(r)


def policy_loss_backward(log_probs, old_log_probs, advantages, weights, *, dloss=None,
                         ref_log_probs=None, token_mask=None, clip_low: float = 0.2,
                         clip_high: float = 0.2, kl: float = 0.0, stream=None) -> torch.Tensor:
    """muon_policy_loss_backward: gradient of log_probs; weights are the
    forward pass's, dloss an fp32 scalar on the device (None: 1)."""
    if stream is not None:
        return _on(stream, policy_loss_backward, (log_probs, old_log_probs, advantages, weights),
                   dict(dloss=dloss, ref_log_probs=ref_log_probs, token_mask=token_mask,
                        clip_low=clip_low, clip_high=clip_high, kl=kl))
    r = (_bound or _b()).policy_loss_backward(log_probs, old_log_probs, advantages, ref_log_probs,
                                              token_mask, clip_low, clip_high, kl, weights, dloss)
    if type(r) is int:
        _check(r, "muon_policy_loss_backward")
    return r


class _PolicyLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, log_probs, old, advantages, ref, token_mask, clip_low, clip_high, kl, by_sequence):
        ctx.how = dict(clip_low=clip_low, clip_high=clip_high, kl=kl)
        o = policy_loss_forward(log_probs, old, advantages, ref_log_probs=ref, token_mask=token_mask,
                                by_sequence=by_sequence, **ctx.how)
        ctx.save_for_backward(log_probs, old, advantages, ref, token_mask, o.weights)
        ctx.mark_non_differentiable(o.kl, o.clipped, o.weights)
        ctx.set_materialize_grads(False)
        return o.loss, o.kl, o.clipped, o.weights

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, _kl, _clipped, _weights):
        if dloss is None:
            return (None,) * 9
        log_probs, old, advantages, ref, token_mask, weights = ctx.saved_tensors
        return (policy_loss_backward(log_probs, old, advantages, weights, dloss=dloss.contiguous(),
                                     ref_log_probs=ref, token_mask=token_mask, **ctx.how),) + (None,) * 8


def policy_loss(log_probs, old_log_probs, advantages, *, ref_log_probs=None, token_mask=None,
                clip_low: float = 0.2, clip_high: float = 0.2, kl: float = 0.0,
                by_sequence: bool = False) -> PolicyOut:
    """Differentiable clipped policy loss: gradients flow from the loss to
    log_probs; old and reference log probabilities and advantages are constants."""
    rows = [_as_rows(t) for t in (log_probs, old_log_probs)]
    advantages = _as_rows(advantages) if advantages.shape == log_probs.shape else advantages.contiguous()
    ref = None if ref_log_probs is None else _as_rows(ref_log_probs)
    mask = _dense(token_mask)
    return PolicyOut(*_PolicyLoss.apply(*rows, advantages, ref, mask, clip_low, clip_high, kl, by_sequence))
