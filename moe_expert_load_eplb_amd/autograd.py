"""The router and the experts' product as differentiable functions of torch.

Thin wrappers: forward and backward are the calls of the package, chained as a
training step chains them.  ``route`` carries gradients through the weights and
the balance loss to the logits; ``expert_linear`` through the product to the
rows and to the weights.  Neither has a second derivative: asking for one raises
RuntimeError.
"""
from __future__ import annotations

import torch

from . import (expert_matmul, expert_wgrad, gate_backward, gate_loss, quantize_columns, quantize_rows,
               quantize_weights)


class _Final(torch.autograd.Function):
    """A gradient that depends on `through`: the same values, but differentiating them fails."""

    @staticmethod
    def forward(ctx, grad, *through):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("route and expert_linear have no second derivative")


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
