"""The router's sigmoid by its short reciprocal and by the division give equal bits
(needs an MI355X).  A logit below -87 makes its row take the division, so the
same logits are routed with one and without."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

eplb = pytest.importorskip("moe_expert_load_eplb_amd")
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("lo,hi", [(-87.0, -40.0), (-40.0, -10.0), (-10.0, 0.0), (0.0, 20.0)])
def test_reciprocal_is_the_division(lo, hi):
    print("[sigmoid]", lo, hi, flush=True)
    T, E = 1 << 17, 64
    g = torch.Generator(device=DEV).manual_seed(int(hi) + 100)
    x = lo + (hi - lo) * torch.rand((T, E), generator=g, device=DEV)
    x[:, 63] = -1.0
    far = x.clone()
    far[:, 63] = -88.0
    scores = []
    for logits in (x, far):
        ids, w = eplb.gate(logits, E, normalize=False)
        assert (ids.sort(1).values == torch.arange(E, device=DEV)).all()
        scores.append(torch.empty_like(w).scatter_(1, ids.long(), w)[:, :63])
    assert torch.equal(scores[0].view(torch.int32), scores[1].view(torch.int32))
    # and both are 1 / (1 + exp(-x)): an exponential of relative error 2^-22 at most, a sum, a division
    want = torch.sigmoid(x[:, :63].double())
    assert ((scores[0].double() - want).abs() <= 2.0 ** -21 * want).all()
