"""What autograd.py itself does, on a machine without a GPU: the package's calls
are replaced by plain torch ones on host tensors, with the same arguments and
outputs (no 8-bit rounding)."""
from __future__ import annotations

import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "moe_expert_load_eplb_amd", "libeplb.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libeplb.so not built")


@pytest.fixture
def plain(monkeypatch):
    """The module with plain calls behind it; plain.calls: what was called."""
    from moe_expert_load_eplb_amd import autograd as m
    calls = []

    def weights_of(x, ids):
        s = torch.sigmoid(x.detach()).gather(1, ids.long())
        return s / s.sum(1, keepdim=True)

    def gate_loss(x, K, seg, alpha):
        ids = x.detach().topk(K, dim=1).indices.int()
        n, E = x.shape
        counts = torch.bincount(ids.flatten(), minlength=E).view(1, E).int()
        prob = torch.softmax(x.detach(), 1).mean(0, keepdim=True)
        return ids, weights_of(x, ids), alpha * (counts * prob).sum(1), counts, prob, torch.tensor([n], dtype=torch.int32)

    def gate_backward(x, ids, d_weights, **how):
        return torch.ones_like(x)

    def quantize_rows(x):
        return x.detach(), None

    def quantize_weights(w, transpose=False):
        calls.append("transposed" if transpose else "weights")
        w = w.detach()
        return (w, None, w.transpose(1, 2), None) if transpose else (w, None)

    def expert_matmul(q, s, w, ws, offsets, rows=None, K=1, dtype=None):
        calls.append("matmul")
        src = q if rows is None else q[rows.long() // K]
        y = torch.zeros((src.shape[0], w.shape[1]))
        for g in range(w.shape[0]):
            a, b = int(offsets[g]), int(offsets[g + 1])
            y[a:b] = src[a:b] @ w[g].t()
        return y.to(dtype)

    def quantize_columns(x, offsets, rows=None, K=1):
        return (x if rows is None else x[rows.long() // K]).detach().t(), None

    def expert_wgrad(dy, ds, x, xs, offsets, dtype=None):
        calls.append("wgrad")
        cut = [(int(offsets[g]), int(offsets[g + 1])) for g in range(offsets.shape[0] - 1)]
        return torch.stack([dy[:, a:b] @ x[:, a:b].t() for a, b in cut]).to(dtype)

    for f in (gate_loss, gate_backward, quantize_rows, quantize_weights, expert_matmul, quantize_columns, expert_wgrad):
        monkeypatch.setattr(m, f.__name__, f)
    m.calls = calls
    yield m
    del m.calls


def operands(N=32, C=48, x_grad=True, w_grad=True):
    g = torch.Generator().manual_seed(N + C)
    x = torch.randn((20, C), generator=g).requires_grad_(x_grad)
    w = torch.randn((2, N, C), generator=g).requires_grad_(w_grad)
    return x, w, torch.tensor([0, 7, 20], dtype=torch.int32)


def test_first_derivatives(plain):
    x, w, off = operands()
    dy = torch.randn((20, 32), generator=torch.Generator().manual_seed(1))
    got = torch.autograd.grad(plain.expert_linear(x, w, off), (x, w), dy)
    want = torch.autograd.grad(torch.cat([x[:7] @ w[0].t(), x[7:] @ w[1].t()]), (x, w), dy)
    for a, b in zip(got, want):
        torch.testing.assert_close(a, b)
    rows = torch.randperm(40, generator=torch.Generator().manual_seed(2))
    place = torch.empty_like(rows)
    place[rows] = torch.arange(40)
    off = torch.tensor([0, 11, 40], dtype=torch.int32)
    dy = torch.randn((40, 32), generator=torch.Generator().manual_seed(3))
    got = torch.autograd.grad(plain.expert_linear(x, w, off, rows.int(), place.int(), 2), (x, w), dy)
    taken = x[rows // 2]
    want = torch.autograd.grad(torch.cat([taken[:11] @ w[0].t(), taken[11:] @ w[1].t()]), (x, w), dy)
    for a, b in zip(got, want):
        torch.testing.assert_close(a, b)


def test_second_derivatives_are_refused(plain):
    """Neither function has one: asking for it fails, beside other paths too,
    rather than leave its share out.  (The product is linear in each operand: a
    gradient does depend on the other one, and on the output's gradient.)"""
    x = torch.randn((10, 8), generator=torch.Generator().manual_seed(1)).requires_grad_(True)
    seg = torch.tensor([0, 10], dtype=torch.int32)
    for pick in (1, 2):
        out = plain.route(x, 2, seg, 0.1)[pick]
        for scale in (torch.ones_like(out), torch.ones_like(out).requires_grad_(True)):
            d, = torch.autograd.grad(out, x, scale, create_graph=True, retain_graph=True)
            with pytest.raises(RuntimeError, match="second derivative"):
                torch.autograd.grad((d ** 2).sum() + (x ** 2).sum(), x)
    x, w, off = operands()
    y = plain.expert_linear(x, w, off)
    for scale in (torch.ones_like(y), torch.ones_like(y).requires_grad_(True)):
        for first, others in ((x, [w]), (w, [x])):
            d, = torch.autograd.grad(y, first, scale, create_graph=True, retain_graph=True)
            for second in others + [scale] * scale.requires_grad:
                with pytest.raises(RuntimeError, match="second derivative"):
                    torch.autograd.grad((d ** 2).sum() + (second ** 2).sum(), second)
            same, = torch.autograd.grad((d ** 2).sum() + (first ** 2).sum(), first)
            assert torch.equal(same, 2 * first)
    d, = torch.autograd.grad(y, x, torch.ones_like(y))      # without a graph: as ever
    assert not d.requires_grad


def test_widths_that_the_products_refuse(plain):
    """The contraction of a product is a multiple of 16: C of the forward pass, N
    of the gradient of x.  What cannot be done is said before anything is done,
    and what can be is done."""
    x, w, off = operands(N=32, C=40)
    with pytest.raises(ValueError, match="multiple of 16"):
        plain.expert_linear(x, w, off)
    x, w, off = operands(N=100, C=48)
    with pytest.raises(ValueError, match="multiple of 16"):
        plain.expert_linear(x, w, off)
    assert plain.calls == []
    with torch.no_grad():
        assert plain.expert_linear(x, w, off).shape == (20, 100)
    assert plain.expert_linear(x.detach(), w.detach(), off).shape == (20, 100)
    dw, = torch.autograd.grad(plain.expert_linear(x.detach(), w, off).sum(), w)
    assert dw.shape == w.shape


def test_operands_that_do_not_match(plain):
    x, w, off = operands()
    for bad in ((x[0], w, off), (x, w[0], off), (x, w[:, :, :32], off), (x.view(40, 24), w, off)):
        with pytest.raises(ValueError, match=r"x \[T, C\] and w \[G, N, C\]"):
            plain.expert_linear(*bad)


def test_transposed_weights_only_for_the_gradient_of_x(plain):
    """They are as large as the weights: made and kept where that gradient is taken."""
    for x_grad, w_grad, grad_mode, want in ((True, True, True, "transposed"), (True, False, True, "transposed"),
                                            (False, True, True, "weights"), (False, False, True, "weights"),
                                            (True, True, False, "weights")):
        x, w, off = operands(x_grad=x_grad, w_grad=w_grad)
        plain.calls.clear()
        with torch.set_grad_enabled(grad_mode):
            y = plain.expert_linear(x, w, off)
        assert plain.calls == [want, "matmul"], (x_grad, w_grad, grad_mode)
        assert y.requires_grad == (grad_mode and (x_grad or w_grad))
        if y.requires_grad:
            used = [t for t in (x, w) if t.requires_grad]
            got = torch.autograd.grad(y, used, torch.ones_like(y))
            assert [g.shape for g in got] == [t.shape for t in used]
            assert plain.calls[2:] == ["matmul"] * x_grad + ["wgrad"] * w_grad
