"""The join's backward pass where the weights need no gradient, on a machine without
a GPU: y is neither kept nor handed on, and what does not fit together is refused."""
from __future__ import annotations

import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "moe_expert_load_eplb_amd", "libeplb.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libeplb.so not built")


def test_rows_are_not_kept_without_the_weights_gradient(monkeypatch):
    from moe_expert_load_eplb_amd import autograd as m
    T, K, C = 6, 2, 8
    got = []
    monkeypatch.setattr(m, "combine_rows", lambda y, place, weights, dtype=None: y.new_ones((T, C)))
    monkeypatch.setattr(m, "combine_rows_backward", lambda d_out, y, place, order, weights: (
        got.append(y), (torch.full((T * K, C), 2.0, dtype=y.dtype), torch.full((T, K), 3.0)))[1])
    order = torch.arange(T * K, dtype=torch.int32)
    for type_ in (torch.float32, torch.bfloat16):
        for gv in (False, True):
            y, v = torch.randn((T * K, C)).to(type_).requires_grad_(True), torch.rand((T, K)).requires_grad_(gv)
            kept = []
            with torch.autograd.graph.saved_tensors_hooks(lambda t: (kept.append(t), t)[1], lambda t: t):
                out = m.combine(y, v, order, order)
            assert any(t.data_ptr() == y.data_ptr() for t in kept) == gv
            got.clear()
            out.sum().backward()
            assert (y.grad == 2).all() and (v.grad is not None) == gv and (not gv or (v.grad == 3).all())
            assert got[0].shape == y.shape and got[0].dtype == type_
            assert got[0].untyped_storage().nbytes() == (y.untyped_storage().nbytes() if gv else y.element_size())


def test_binding_refusals():
    import moe_expert_load_eplb_amd as eplb
    T, K, C = 4, 2, 8
    d, w, index = torch.zeros((T, C)), torch.zeros((T, K)), torch.arange(T * K, dtype=torch.int32)
    y = torch.zeros(()).expand(T * K, C)
    with pytest.raises(ValueError, match="GPU"):
        eplb.combine_rows_backward(d, y, index, index, w)
    for out in ((torch.zeros((T * K, C)), torch.zeros((T, K))), (torch.zeros((T * K, C)),)):
        with pytest.raises(ValueError, match="None"):
            eplb.combine_rows_backward(d, y, index, index, w, out=out)
    with pytest.raises(ValueError, match="shapes"):
        eplb.combine_rows_backward(d, y, index, index, w, out=(torch.zeros((T * K, C + 1)), None))
    for strided in (torch.zeros((1, C)).expand(T * K, C), torch.zeros((T * K, 1)).expand(T * K, C)):
        with pytest.raises(ValueError):
            eplb.combine_rows_backward(d, strided, index, index, w)
