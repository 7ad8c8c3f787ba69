"""Shapes of the join's index arrays that the binding refuses, on host tensors
(a machine without a GPU)."""
from __future__ import annotations

import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "moe_expert_load_eplb_amd", "libeplb.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libeplb.so not built")


@pytest.mark.parametrize("T,K", [(6, 2), (1, 4), (5, 1)])
def test_place_of_another_shape(T, K):
    """As many elements as choices, but not a token's next to each other: places of other tokens."""
    import moe_expert_load_eplb_amd as eplb
    y, d, w = torch.zeros((T * K, 8)), torch.zeros((T, 8)), torch.zeros((T, K))
    place = torch.arange(T * K, dtype=torch.int32)
    for good in (place, place.view(T, K), place.view(1, T * K), place.view(T * K, 1)):
        with pytest.raises(ValueError, match="GPU"):
            eplb.combine_rows(y, good, w)
        with pytest.raises(ValueError, match="GPU"):
            eplb.combine_rows_backward(d, y, good, place, w)
    for bad in (place.view(K, T), place.view(T, K, 1), place[1:]):
        if bad.dim() == 2 and max(bad.shape) == T * K:
            continue
        with pytest.raises(ValueError, match="elements"):
            eplb.combine_rows(y, bad, w)
        with pytest.raises(ValueError, match="elements"):
            eplb.combine_rows_backward(d, y, bad, place, w)
