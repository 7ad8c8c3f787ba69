"""What expert_linear16 and combine refuse before the forward pass because their
backward pass could not do it, and what they hand to their calls, on a machine
without a GPU: the package's calls are replaced by ones that note that they ran."""
from __future__ import annotations

import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "moe_expert_load_eplb_amd", "libeplb.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libeplb.so not built")


@pytest.fixture
def noted(monkeypatch):
    from moe_expert_load_eplb_amd import autograd as m
    calls = []
    monkeypatch.setattr(m, "expert_matmul16", lambda x, w, offsets, rows=None, K=1, transpose=False, dtype=None: (
        calls.append("product"), x.new_zeros(((x if rows is None else rows).shape[0], w.shape[2 if transpose else 1])))[1])
    monkeypatch.setattr(m, "combine_rows", lambda y, place, weights, dtype=None: (
        calls.append("combine"), y.new_zeros(((place if weights is None else weights).shape[0], y.shape[1])))[1])
    m.calls = calls
    return m


def refused(m, call, kind):
    m.calls.clear()
    with pytest.raises(kind):
        call()
    assert m.calls == []


def test_choices_past_what_the_join_takes(noted):
    """The gradient of a token is the join of its rows, which takes 64 of them."""
    for K, fine in ((64, True), (65, False)):
        T, C = 3, 8
        x, w = torch.randn((T, C), requires_grad=True), torch.randn((K, 8, C))
        offsets = torch.arange(K + 1, dtype=torch.int32) * T
        order = torch.arange(T * K, dtype=torch.int32)

        def call():
            return noted.expert_linear16(x, w, offsets, order, order, K)
        if fine:
            call().sum().backward()
            assert x.grad.shape == x.shape
        else:
            refused(noted, call, ValueError)
            with torch.no_grad():
                call()
            noted.expert_linear16(x.detach(), w, offsets, order, order, K)     # asked for by the gradient of x only


def test_index_arrays(noted):
    T, K, C, N, G = 4, 2, 16, 8, 3
    offsets, order = torch.tensor([0, 3, 5, 8], dtype=torch.int32), torch.arange(T * K, dtype=torch.int32)
    x, w = torch.randn((T, C), requires_grad=True), torch.randn((G, N, C))
    y, v = torch.randn((T * K, C), requires_grad=True), torch.rand((T, K))
    strided = torch.zeros((T * K, 2), dtype=torch.int32)[:, 0]
    for bad, kind in ((order.long(), TypeError), (order.float(), TypeError), (strided, ValueError),
                      (order.to("meta"), ValueError)):
        refused(noted, lambda: noted.expert_linear16(x, w, offsets, order, bad, K), kind)
        refused(noted, lambda: noted.combine(y, v, order, bad), kind)
        refused(noted, lambda: noted.combine(y.detach(), v.clone().requires_grad_(True), order, bad), kind)
        noted.expert_linear16(x.detach(), w.clone().requires_grad_(True), offsets, order, bad, K)
        noted.combine(y.detach(), v, order, bad)
        with torch.no_grad():
            noted.expert_linear16(x, w, offsets, order, bad, K)
            noted.combine(y, v, order, bad)
    refused(noted, lambda: noted.expert_linear16(x, w, offsets, order, order.view(K, T), K), ValueError)
    for place in (order, order.view(T, K), order.view(1, T * K)):
        noted.expert_linear16(x, w, offsets, order, place, K).sum().backward()


def test_gradients_that_start_anywhere(noted, monkeypatch):
    """A gradient that is a part of a larger one, as behind a concatenation, may start at any element; what the products
    get starts at 16 bytes and holds the same."""
    seen = []

    def expert_matmul16(x, w, offsets, rows=None, K=1, transpose=False, dtype=None):
        if transpose:
            seen.append(x)
        return x.new_zeros((x.shape[0], w.shape[2 if transpose else 1]))

    def expert_wgrad16(dy, x, offsets, rows=None, K=1, dtype=None):
        seen.append(dy)
        return x.new_zeros((offsets.shape[0] - 1, dy.shape[1], x.shape[1]))

    monkeypatch.setattr(noted, "expert_matmul16", expert_matmul16)
    monkeypatch.setattr(noted, "expert_wgrad16", expert_wgrad16)
    offsets = torch.tensor([0, 2, 5], dtype=torch.int32)
    for ahead in (0, 1, 3, 4, 8):
        x = torch.randn((5, 16)).bfloat16().requires_grad_(True)
        w = torch.randn((2, 8, 16)).bfloat16().requires_grad_(True)
        y = noted.expert_linear16(x, w, offsets)
        whole = torch.randn((ahead + y.numel(),)).bfloat16()
        seen.clear()
        torch.cat([torch.zeros((ahead,), dtype=torch.bfloat16), y.reshape(-1)]).backward(whole)
        assert len(seen) == 2
        for dy in seen:
            assert dy.data_ptr() % 16 == 0 and torch.equal(dy, whole[ahead:].view(5, 8))
