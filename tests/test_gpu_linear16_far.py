"""The experts' 16-bit products on operands past 2^31 bytes: rows that are taken
from anywhere in them, whole ranges of them, and outputs as long (needs an MI355X
and about 8 GB of its memory).  Each value is a sum of small whole numbers and
compared as it is."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

eplb = pytest.importorskip("moe_expert_load_eplb_amd")
DEV = torch.device("cuda:0")


def note(*a):
    print("[far]", *a, flush=True)


@pytest.fixture(scope="module")
def long_rows():
    g = torch.Generator(device=DEV).manual_seed(1)
    return torch.randint(-3, 4, (1200000, 1024), generator=g, device=DEV, dtype=torch.int8).to(torch.bfloat16)


def test_gathered(long_rows):
    x = long_rows
    X, C = x.shape
    assert X * C * 2 > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(2)
    rows = torch.randint(0, X, (5000,), generator=g, device=DEV, dtype=torch.int32)
    rows[:4] = torch.tensor([X - 1, 0, X - 2, X], dtype=torch.int32)
    off = torch.tensor([0, 3000, 3000, 4990], dtype=torch.int32, device=DEV)
    w = torch.randint(-3, 4, (3, 1040, C), generator=g, device=DEV, dtype=torch.int8).to(torch.bfloat16)
    note("product")
    y = eplb.expert_matmul16(x, w, off, rows=rows, dtype=torch.float32)
    taken = x[rows.long().clamp(max=X - 1)].float()
    taken[3] = 0
    want = torch.zeros_like(y)
    want[:3000], want[3000:4990] = taken[:3000] @ w[0].float().t(), taken[3000:4990] @ w[2].float().t()
    assert torch.equal(y, want)
    note("weight gradient")
    dy = torch.randint(-3, 4, (5000, 264), generator=g, device=DEV, dtype=torch.int8).to(torch.bfloat16)
    dw = eplb.expert_wgrad16(dy, x, off, rows=rows, dtype=torch.float32)
    assert torch.equal(dw[0], dy[:3000].float().t() @ taken[:3000])
    assert torch.equal(dw[2], dy[3000:4990].float().t() @ taken[3000:4990]) and (dw[1] == 0).all()
    note("4-bit weights")
    q, s = eplb.quantize_weights4(w[:, :72].contiguous())              # whole numbers up to 3: exact
    y4 = eplb.expert_matmul4(x, q, s, off, rows=rows, dtype=torch.float32)
    assert torch.equal(y4, want[:, :72])


def test_ranges(long_rows):
    x = long_rows
    X, C = x.shape
    g = torch.Generator(device=DEV).manual_seed(3)
    off = torch.tensor([0, 100, X - 70, X], dtype=torch.int32, device=DEV)
    w = torch.randint(-2, 3, (3, 24, C), generator=g, device=DEV, dtype=torch.int8).to(torch.bfloat16)
    note("product")
    y = eplb.expert_matmul16(x, w, off, dtype=torch.float32)
    for g0, a, b in ((0, 0, 100), (1, 100, 400), (1, X - 400, X - 70), (2, X - 70, X)):
        assert torch.equal(y[a:b], x[a:b].float() @ w[g0].float().t())
    note("weight gradient")
    dy = torch.randint(-2, 3, (X, 16), generator=g, device=DEV, dtype=torch.int8).to(torch.bfloat16)
    dw = eplb.expert_wgrad16(dy, x, off, dtype=torch.float32)
    assert torch.equal(dw[0], dy[:100].float().t() @ x[:100].float())
    assert torch.equal(dw[2], dy[X - 70:].float().t() @ x[X - 70:].float())
    want = torch.zeros((16, C), dtype=torch.float64, device=DEV)
    for a in range(100, X - 70, 100000):
        b = min(a + 100000, X - 70)
        want += (dy[a:b].float().t() @ x[a:b].float()).double()       # whole numbers below 2^24: exact
    assert torch.equal(dw[1].double(), want)
    note("transposed, an output past 2^31 bytes")
    wt = torch.randint(-2, 3, (3, 16, C), generator=g, device=DEV, dtype=torch.int8).to(torch.bfloat16)
    out = eplb.expert_matmul16(dy, wt, off, transpose=True)
    for g0, a, b in ((0, 0, 100), (1, X // 2, X // 2 + 300), (2, X - 70, X)):
        assert torch.equal(out[a:b].float(), dy[a:b].float() @ wt[g0].float())
