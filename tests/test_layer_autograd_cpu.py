"""What expert_linear16 and combine do themselves, on a machine without a GPU: the
package's calls are replaced by plain torch ones on host tensors, with the same
arguments and outputs."""
from __future__ import annotations

import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "moe_expert_load_eplb_amd", "libeplb.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libeplb.so not built")


@pytest.fixture
def plain(monkeypatch):
    from moe_expert_load_eplb_amd import autograd as m
    calls = []

    def cut(offsets):
        return [(int(offsets[g]), int(offsets[g + 1])) for g in range(offsets.shape[0] - 1)]

    def expert_matmul16(x, w, offsets, rows=None, K=1, transpose=False, dtype=None):
        calls.append("transposed" if transpose else "product")
        x, w = x.detach(), w.detach()
        src = x if rows is None else x[rows.long() // K]
        parts = [src[a:b] @ (w[g] if transpose else w[g].t()) for g, (a, b) in enumerate(cut(offsets))]
        return torch.cat(parts).to(torch.promote_types(dtype or x.dtype, x.dtype))

    def expert_wgrad16(dy, x, offsets, rows=None, K=1, dtype=None):
        calls.append("wgrad")
        x = x.detach()
        src = x if rows is None else x[rows.long() // K]
        return torch.stack([dy[a:b].t() @ src[a:b] for a, b in cut(offsets)]).to(dtype)

    def combine_rows(y, place, weights, dtype=None):
        calls.append("sum" if weights is None else "combine")
        T, K = place.shape if weights is None else weights.shape
        rows = y.detach()[place.reshape(-1).long()].view(T, K, -1)
        return (rows if weights is None else rows * weights.detach().unsqueeze(2)).sum(1).to(dtype or y.dtype)

    def combine_rows_backward(d_out, y, place, order, weights):
        calls.append("combine backward")
        T, K = weights.shape
        i = order.long()
        dy = weights.detach().reshape(-1)[i].unsqueeze(1) * d_out[i // K]
        return dy.to(y.dtype), (y.detach()[place.long()].view(T, K, -1) * d_out.unsqueeze(1)).sum(2)

    for f in (expert_matmul16, expert_wgrad16, combine_rows, combine_rows_backward):
        monkeypatch.setattr(m, f.__name__, f)
    m.calls = calls
    return m


def grouping(T, K, G, seed):
    ids = torch.rand((T, G), generator=torch.Generator().manual_seed(seed)).topk(K, 1).indices.reshape(-1)
    order = ids.argsort(stable=True).int()
    place = torch.empty_like(order)
    place[order.long()] = torch.arange(T * K, dtype=torch.int32)
    offsets = torch.zeros(G + 1, dtype=torch.int32)
    offsets[1:] = torch.bincount(ids, minlength=G).cumsum(0)
    return offsets, order, place


def test_gradients_against_differences(plain):
    T, K, G, N, C = 7, 2, 3, 16, 8
    offsets, order, place = grouping(T, K, G, 1)
    g = torch.Generator().manual_seed(2)
    x, w, v = (torch.randn(s, generator=g, dtype=torch.float64, requires_grad=True) for s in ((T, C), (G, N, C), (T, K)))

    def layer(x, w, v):
        y = plain.expert_linear16(x, w, offsets, order, place, K)
        return plain.combine(y, v, place, order)

    assert torch.autograd.gradcheck(layer, (x, w, v))


def test_calls(plain):
    T, K, G, N, C = 9, 2, 4, 8, 16
    offsets, order, place = grouping(T, K, G, 3)
    x, w = torch.randn(T, C), torch.randn(G, N, C)
    for gx, gw, want in ((True, False, ["transposed", "sum"]), (False, True, ["wgrad"]),
                         (True, True, ["transposed", "sum", "wgrad"])):
        a, b = x.clone().requires_grad_(gx), w.clone().requires_grad_(gw)
        plain.calls.clear()
        y = plain.expert_linear16(a, b, offsets, order, place, K)
        assert plain.calls == ["product"]
        y.sum().backward()
        assert plain.calls[1:] == want
        assert (a.grad is not None) == gx and (b.grad is not None) == gw
    plain.calls.clear()
    a = x[order.long() // K].clone().requires_grad_(True)
    plain.expert_linear16(a, w, offsets).sum().backward()
    assert plain.calls == ["product", "transposed"] and a.grad.dtype == x.dtype


def test_partial_gradients_of_combine(plain):
    T, K, G, C = 5, 3, 4, 6
    _, order, place = grouping(T, K, G, 5)
    y, v = torch.randn(T * K, C), torch.rand(T, K)
    for gy, gv in ((True, False), (False, True)):
        a, b = y.clone().requires_grad_(gy), v.clone().requires_grad_(gv)
        plain.combine(a, b, place, order).sum().backward()
        assert (a.grad is not None) == gy and (b.grad is not None) == gv


def test_no_second_derivative(plain):
    T, K, G, N, C = 6, 2, 3, 8, 8
    offsets, order, place = grouping(T, K, G, 7)
    x, w, v = (torch.randn(s, requires_grad=True) for s in ((T, C), (G, N, C), (T, K)))
    out = plain.combine(plain.expert_linear16(x, w, offsets, order, place, K), v, place, order)
    for p in (x, w, v):
        d, = torch.autograd.grad((out ** 2).sum(), p, create_graph=True)
        with pytest.raises(RuntimeError, match="second derivative"):
            torch.autograd.grad(d.sum(), (x, w, v), allow_unused=True)


def test_refusals(plain):
    offsets, order, place = grouping(4, 2, 3, 9)
    x, w = torch.randn(4, 16), torch.randn(3, 12, 16)
    for bad in (lambda: plain.expert_linear16(x, torch.randn(3, 12, 8), offsets),
                lambda: plain.expert_linear16(torch.randn(4, 12), torch.randn(3, 12, 12), offsets),
                lambda: plain.expert_linear16(x.clone().requires_grad_(True), w, offsets, order, place, 2),
                lambda: plain.expert_linear16(x, w.clone().requires_grad_(True), offsets, order, place, 2),
                lambda: plain.expert_linear16(x, w, offsets, order, None, 2),
                lambda: plain.expert_linear16(x, w, offsets, order, place, 3),
                lambda: plain.expert_linear16(x, w, offsets, order, place[:7], 2),
                lambda: plain.combine(torch.randn(8, 4), torch.rand(4, 3), place, order),
                lambda: plain.combine(torch.randn(8, 4), torch.rand(4, 2), place, order[:7]),
                lambda: plain.combine(torch.randn(8), torch.rand(4, 2), place, order)):
        plain.calls.clear()
        with pytest.raises(ValueError):
            bad()
        assert plain.calls == []
    plain.expert_linear16(x, w, offsets, order, place, 2)            # N is only asked for by the gradients
    with torch.no_grad():
        plain.expert_linear16(x.clone().requires_grad_(True), w, offsets, order, place, 2)
