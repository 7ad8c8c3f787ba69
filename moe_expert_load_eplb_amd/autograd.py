"""The router, the experts' products and their join as differentiable functions
of torch.

Thin wrappers: forward and backward are the calls of the package, chained as a
training step chains them.  ``route`` carries gradients through the weights and
the balance loss to the logits; ``expert_linear`` (8-bit blocks) and
``expert_linear16`` (16 bits) through the product to the rows and to the weights;
``combine`` through the weighted sum to the experts' rows and to the router's
weights.  None has a second derivative: asking for one raises RuntimeError.
"""
from __future__ import annotations

import torch

from . import (combine_rows, combine_rows_backward, expert_matmul, expert_matmul16, expert_wgrad, expert_wgrad16,
               gate_backward, gate_loss, quantize_columns, quantize_rows, quantize_weights)


class _Final(torch.autograd.Function):
    """A gradient that depends on `through`: the same values, but differentiating them fails."""

    @staticmethod
    def forward(ctx, grad, *through):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("route, the expert_linears and combine have no second derivative")


def _final(grad, *through):
    # under create_graph the gradient would come back as a constant, and its share of a second derivative as zero
    return _Final.apply(grad, *through) if grad is not None and torch.is_grad_enabled() else grad


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, K, seg, alpha, options):
        out = gate_loss(logits, K, seg, alpha, **options)
        ids, weights, loss, counts, prob, tokens = out
        ctx.save_for_backward(logits, ids, seg, counts, tokens, options.get("mask"))
        ctx.alpha = alpha
        ctx.how = {k: options[k] for k in ("scoring", "normalize", "scale") if k in options}
        ctx.mark_non_differentiable(ids, counts, prob, tokens)
        ctx.set_materialize_grads(False)
        return out

    @staticmethod
    def backward(ctx, _ids, d_weights, d_loss, _counts, _prob, _tokens):
        logits, ids, seg, counts, tokens, mask = ctx.saved_tensors
        if d_weights is None and d_loss is None:
            return None, None, None, None, None
        dx = gate_backward(logits, ids, None if d_weights is None else d_weights.contiguous(), mask=mask, seg=seg,
                           alpha=ctx.alpha, counts=counts, tokens=tokens,
                           d_loss=None if d_loss is None else d_loss.contiguous(), **ctx.how)
        return _final(dx, logits, d_weights, d_loss), None, None, None, None


def route(logits: torch.Tensor, K: int, seg: torch.Tensor, alpha: float, **options):
    """gate_loss, differentiable in logits through weights and loss (the choice
    and the counts are held fixed).  Returns (ids, weights, loss, counts, prob,
    tokens)."""
    return _Route.apply(logits, K, seg, alpha, options)


class _ExpertLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets, rows, place, K, x_grad):
        # the transposed weights are the operand of the gradient of x only
        wq, ws, wqt, wst = quantize_weights(w, transpose=True) if x_grad else (*quantize_weights(w), None, None)
        y = expert_matmul(*quantize_rows(x), wq, ws, offsets, rows=rows, K=K, dtype=x.dtype)
        ctx.save_for_backward(x, wqt, wst, offsets, rows, place)
        ctx.K, ctx.w = K, w              # w itself is not read again, only named to a second derivative
        return y

    @staticmethod
    def backward(ctx, dy):
        x, wqt, wst, offsets, rows, place = ctx.saved_tensors
        dy = dy.contiguous()
        dx = dw = None
        if ctx.needs_input_grad[0]:
            # a token's rows are summed in 32 bits, in the order of its choices, and rounded once
            dx = expert_matmul(*quantize_rows(dy), wqt, wst, offsets, dtype=x.dtype if rows is None else torch.float32)
            if rows is not None:
                dx = dx[place.long()].view(x.shape[0], ctx.K, x.shape[1]).sum(1).to(x.dtype)
        if ctx.needs_input_grad[1]:
            dw = expert_wgrad(*quantize_columns(dy, offsets), *quantize_columns(x, offsets, rows=rows, K=ctx.K), offsets,
                              dtype=ctx.w.dtype)
        return _final(dx, dy, ctx.w), _final(dw, dy, x), None, None, None, None, None


def expert_linear(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, rows: torch.Tensor | None = None,
                  place: torch.Tensor | None = None, K: int = 1) -> torch.Tensor:
    """Every grouped row times the transposed weights of its expert, in 8-bit
    blocks, differentiable in x and w.

    x [T, C], w [G, N, C], C a multiple of 16, and N too where x needs a
    gradient; offsets, rows and place: one layer of group_rows' outputs (offsets,
    order, place), rows and place together.  Without them x is in grouped order
    itself.  Returns [R, N]."""
    if x.dim() != 2 or w.dim() != 3 or w.shape[2] != x.shape[1]:
        raise ValueError("x [T, C] and w [G, N, C] expected")
    if x.shape[1] % 16 != 0:
        raise ValueError(f"C must be a multiple of 16, got {x.shape[1]}")
    x_grad = x.requires_grad and torch.is_grad_enabled()
    if w.shape[1] % 16 != 0 and x_grad:
        raise ValueError(f"N must be a multiple of 16 for the gradient of x, got {w.shape[1]}")
    if (rows is None) != (place is None):
        raise ValueError("rows and place go together")
    if rows is not None and rows.shape[0] != x.shape[0] * K:
        raise ValueError(f"rows must be [{x.shape[0] * K}]")
    return _ExpertLinear.apply(x, w, offsets, rows, place, K, x_grad)


MOST_CHOICES = 64            # of a token, in combine_rows


def _index(t: torch.Tensor, name: str, like: torch.Tensor) -> None:
    """Refuses what a backward pass could not use as an index array beside `like`."""
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be torch.int32, got {t.dtype}")
    if t.device != like.device:
        raise ValueError(f"{name} must be on {like.device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class _ExpertLinear16(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets, rows, place, K):
        ctx.save_for_backward(x, w, offsets, rows, place)
        ctx.K = K
        return expert_matmul16(x, w, offsets, rows=rows, K=K)

    @staticmethod
    def backward(ctx, dy):
        x, w, offsets, rows, place = ctx.saved_tensors
        dy = dy.contiguous()
        if dy.data_ptr() % 16 != 0:      # the products' rows start at 16 bytes; a part of a larger gradient starts anywhere
            dy = dy.clone()
        dx = dw = None
        if ctx.needs_input_grad[0]:
            # a token's rows are summed in 32 bits, in the order of its choices, and rounded once
            dx = expert_matmul16(dy, w, offsets, transpose=True, dtype=x.dtype if rows is None else torch.float32)
            if rows is not None:
                dx = combine_rows(dx, place.view(x.shape[0], ctx.K), None, dtype=x.dtype)
        if ctx.needs_input_grad[1]:
            dw = expert_wgrad16(dy, x, offsets, rows=rows, K=ctx.K, dtype=w.dtype)
        return _final(dx, dy, w), _final(dw, dy, x), None, None, None, None


def expert_linear16(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, rows: torch.Tensor | None = None,
                    place: torch.Tensor | None = None, K: int = 1) -> torch.Tensor:
    """Every grouped row times the transposed weights of its expert, in 16 bits
    with 32-bit sums, differentiable in x and w.

    x [T, C], w [G, N, C] of one type, bfloat16 or float16, C a multiple of 8, and
    N too where x or w needs a gradient; offsets, rows and place: one layer of
    group_rows' outputs (offsets, order, place), rows and place together (K at
    most 64 where x needs a gradient).  Without them x is in grouped order itself.
    Returns [R, N]."""
    if x.dim() != 2 or w.dim() != 3 or w.shape[2] != x.shape[1]:
        raise ValueError("x [T, C] and w [G, N, C] expected")
    if x.shape[1] % 8 != 0:
        raise ValueError(f"C must be a multiple of 8, got {x.shape[1]}")
    if w.shape[1] % 8 != 0 and torch.is_grad_enabled() and (x.requires_grad or w.requires_grad):
        raise ValueError(f"N must be a multiple of 8 for the gradients, got {w.shape[1]}")
    if (rows is None) != (place is None):
        raise ValueError("rows and place go together")
    if rows is not None and (rows.shape[0] != x.shape[0] * K or place.numel() != x.shape[0] * K):
        raise ValueError(f"rows and place must be [{x.shape[0] * K}]")
    if rows is not None and x.requires_grad and torch.is_grad_enabled():
        if K > MOST_CHOICES:
            raise ValueError(f"K must be at most {MOST_CHOICES} for the gradient of x, got {K}")
        if place.dim() > 1 and (place.dim() > 2 or place.shape != (x.shape[0], K) and max(place.shape) != place.numel()):
            raise ValueError(f"place must be [{x.shape[0] * K}], got {list(place.shape)}")
        _index(place, "place", x)
    return _ExpertLinear16.apply(x, w, offsets, rows, place, K)


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, place, order, dtype):
        # y is read again for the gradient of the weights only; without it its type and shape are kept
        ctx.save_for_backward(y if ctx.needs_input_grad[1] else y.new_empty(()).expand(y.shape), weights, place, order)
        return combine_rows(y, place, weights, dtype=dtype)

    @staticmethod
    def backward(ctx, d_out):
        y, weights, place, order = ctx.saved_tensors
        dy, dw = combine_rows_backward(d_out.contiguous(), y, place, order, weights)
        return (_final(dy, d_out, weights) if ctx.needs_input_grad[0] else None,
                _final(dw, d_out, y) if ctx.needs_input_grad[1] else None, None, None, None)


def combine(y: torch.Tensor, weights: torch.Tensor, place: torch.Tensor, order: torch.Tensor,
            dtype: torch.dtype | None = None) -> torch.Tensor:
    """The experts' rows joined to tokens, out[t] = sum over k of weights[t, k] *
    y[place[t, k]], differentiable in y and weights.

    y [T * K, C]; weights [T, K] float32; place and order: one layer of
    group_rows' outputs.  Returns [T, C] in ``dtype`` (y's without)."""
    if y.dim() != 2 or weights.dim() != 2 or y.shape[0] != weights.numel():
        raise ValueError("y [T * K, C] and weights [T, K] expected")
    if place.numel() != weights.numel() or order.numel() != weights.numel():
        raise ValueError(f"place and order must be [{weights.numel()}]")
    if torch.is_grad_enabled() and (y.requires_grad or weights.requires_grad):
        _index(order, "order", y)
    return _Combine.apply(y, weights, place, order, dtype)
