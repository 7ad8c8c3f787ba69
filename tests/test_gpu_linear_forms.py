"""Every form of the 16-bit and 4-bit products for few rows, and the large tiles at
groups that end in a rest: HIP path against plain sums in 64 bits (needs an
MI355X).  Which form a case takes is checked on the host, where the rules are.

Tolerances: those of the products of few rows, (C + C / 32 + 16) * 2^-23 * sum |x|
|w| and half a step of the output's type.  They hold for half-precision rows with
4-bit weights in every form: a product of such a value and a 4-bit one has 13 bits
and is exact, each of C additions is off by 2^-23 of what it has, and each 32 of
the row take one multiply-add by their scale."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

eplb = pytest.importorskip("moe_expert_load_eplb_amd")

from layer_forms import LARGE, STREAM  # noqa: E402
from test_gpu_linear_few import DEV, TYPES, check, product, rand, weights  # noqa: E402


def note(*a):
    print("[forms]", *a, flush=True)


def grouping(counts, head, tail, topk):
    """(offsets, rows, source of every row or -1, X) with a row before the first and one past the last among them."""
    R = head + sum(counts) + tail
    off = torch.tensor(head + np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    X = R // topk + 1
    idx = torch.randint(0, X * topk, (R,), generator=torch.Generator().manual_seed(R), dtype=torch.int32)
    if R > 3:
        idx[R // 2], idx[R // 3] = -1, X * topk
    src = torch.where(idx >= 0, idx.long() // topk, -1)
    return off, idx, torch.where(src < X, src, -1), X


def taken(x, src):
    out = torch.zeros((src.numel(), x.shape[1]), dtype=torch.float64)
    out[src >= 0] = x.double()[src[src >= 0]]
    return out


def held(y, xr, values, off, transpose=False):
    """y against the sums of 64 bits, group by group; rows of no group are zeros."""
    inside = torch.zeros(y.shape[0], dtype=torch.bool)
    for i in range(off.numel() - 1):
        a, b = int(off[i]), int(off[i + 1])
        inside[a:b] = True
        w = values[i] if transpose else values[i].t()
        check(y[a:b], xr[a:b] @ w, xr[a:b].abs() @ w.abs(), xr.shape[1], i)
    assert (y.cpu()[~inside] == 0).all()


@pytest.mark.parametrize("dtype,out,long", [("bf16", "f32", False), ("bf16", "f32", True), ("f16", "f32", True),
                                            ("f16", "bf16", False)])
@pytest.mark.parametrize("four,form,counts,head,tail,N,short_c,long_c", STREAM)
def test_few_rows(four, form, counts, head, tail, N, short_c, long_c, dtype, out, long):
    C, topk = (long_c if long else short_c), 2 if sum(counts) % 2 else 1
    note(four, form, counts[:6], head, tail, N, C, dtype, out)
    off, idx, src, X = grouping(counts, head, tail, topk)
    R = idx.numel()
    x = rand((X, C), dtype, N + C)
    wide = torch.full((X, C + 8), float("nan"), dtype=x.dtype)
    wide[:, :C] = x
    w, values = weights(four, len(counts), N, C, dtype, N)
    whole = torch.full((R * N + 128,), 7.0, dtype=TYPES[out], device=DEV)
    y = whole[64:64 + R * N].view(R, N)
    product(four, wide.to(DEV)[:, :C], w, off.to(DEV), rows=idx.to(DEV), K=topk, out=y)
    held(y, taken(x, src), values, off)
    assert (y.cpu()[src < 0] == 0).all() and (whole[:64] == 7).all() and (whole[64 + R * N:] == 7).all()
    again = product(four, x.to(DEV), w, off.to(DEV), rows=idx.to(DEV), K=topk, dtype=TYPES[out])
    assert torch.equal(again, y)


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("four,counts,head,tail,width,K", LARGE)
def test_large_tiles(four, counts, head, tail, width, K, dtype, out):
    note("large", four, counts, head, tail, width, K, dtype, out)
    off, idx, src, X = grouping(counts, head, tail, 2)
    x = rand((X, K), dtype, width + K)
    xr = taken(x, src)
    w, values = weights(four, len(counts), width, K, dtype, width)
    y = product(four, x.to(DEV), w, off.to(DEV), rows=idx.to(DEV), K=2, dtype=TYPES[out])
    held(y, xr, values, off)
    assert (y.cpu()[src < 0] == 0).all()
    if not four:
        wt = rand((len(counts), K, width), dtype, K)
        y = eplb.expert_matmul16(x.to(DEV), wt.to(DEV), off.to(DEV), rows=idx.to(DEV), K=2, transpose=True, dtype=TYPES[out])
        held(y, xr, wt.double(), off, transpose=True)
        assert (y.cpu()[src < 0] == 0).all()


@pytest.mark.parametrize("four,form,counts,head,tail,N,short_c,long_c", STREAM)
def test_infinities_and_nan_of_few_rows(four, form, counts, head, tail, N, short_c, long_c):
    """A row's infinities and NaN reach that row's outputs only, a weight's that output's of its group, as the formula has
    them (0 times an infinity is NaN); what a tile, a stage or a set of outputs has none of is not multiplied with them."""
    note("not finite", four, form)
    G, R, C = len(counts), head + sum(counts) + tail, short_c
    dtype = torch.float16 if four else torch.bfloat16
    off, g = torch.tensor(head + np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32), torch.Generator().manual_seed(N)
    x = torch.randn((R, C), generator=g).to(dtype)
    hit = torch.randint(0, R, (3,), generator=g).tolist()
    x[hit[0], 0], x[hit[1], C - 1], x[hit[2], C // 2] = float("inf"), float("-inf"), float("nan")
    if four:
        w, values = weights(True, G, N, C, "f16", N)
        w[1][:, N - 1, C // 32 - 1], w[1][0, 0, 0] = 255, 255        # NaN
        values[:, N - 1, C - 32:], values[0, 0, :32] = float("nan"), float("nan")
    else:
        values = torch.randn((G, N, C), generator=g).to(dtype)
        values[:, N - 1, C - 1], values[0, 0, 0], values[:, 3, 1], values[:, 4] = float("nan"), float("inf"), 0, 0
        w, values = (values.to(DEV),), values.double()
    y = product(four, x.to(DEV), w, off.to(DEV), dtype=torch.float32).double()
    want = torch.zeros((R, N), dtype=torch.float64, device=DEV)
    xd, values = x.double().to(DEV), values.to(DEV)
    for i in range(G):
        for r in range(int(off[i]), int(off[i + 1])):
            want[r] = (values[i] * xd[r]).sum(1)
    odd = ~torch.isfinite(want)
    assert odd.any() and not odd.all() and torch.equal(~torch.isfinite(y), odd)
    assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(y[odd & ~torch.isnan(y)], want[odd & ~torch.isnan(y)])
