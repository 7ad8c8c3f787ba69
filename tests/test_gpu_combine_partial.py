"""The join's backward pass without the gradient of the weights: the same bits of
the rows' gradient as with it, and nothing else written (needs an MI355X)."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

eplb = pytest.importorskip("moe_expert_load_eplb_amd")
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def note(*a):
    print("[partial]", *a, flush=True)


def case(T, K, C, dtype, d_dtype, seed):
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(T * K, generator=g).int()
    place = torch.empty_like(order)
    place[order.long()] = torch.arange(T * K, dtype=torch.int32)
    y, d = torch.randn((T * K, C), generator=g).to(TYPES[dtype]), torch.randn((T, C), generator=g).to(TYPES[d_dtype])
    return [t.to(DEV) for t in (d, y, place, order, torch.rand((T, K), generator=g) - 0.3)]


# one wave to a token and several, 1 to 64 choices, whole widths, pairs and single elements
@pytest.mark.parametrize("T,K,C,dtype,d_dtype", [
    (1, 1, 1, "f32", "f32"), (5, 9, 8, "bf16", "f16"), (7, 64, 33, "f32", "bf16"), (130, 3, 500, "bf16", "f32"),
    (64, 6, 2050, "f16", "f16"), (9, 17, 5000, "f32", "f32"), (2, 8, 20000, "bf16", "bf16"), (1000, 1, 257, "bf16", "bf16")])
def test_same_rows(T, K, C, dtype, d_dtype):
    note(T, K, C, dtype, d_dtype)
    d, y, place, order, w = case(T, K, C, dtype, d_dtype, T + C)
    for weights, at in ((w, place), (None, place.view(T, K))):
        want, _ = eplb.combine_rows_backward(d, y, at, order, weights)
        like = y.new_empty(()).expand(T * K, C)
        whole = torch.full((T * K * C + 64,), 7.0, dtype=y.dtype, device=DEV)
        out = (whole[32:32 + T * K * C].view(T * K, C), None)
        got = eplb.combine_rows_backward(d, like, at, order, weights, out=out if T * K * C > 1 else None)
        assert torch.equal(got[0], want) and (got[1] is None) == (T * K * C > 1)
        assert (whole[:32] == 7).all() and (whole[32 + T * K * C:] == 7).all()
        assert torch.equal(eplb.combine_rows_backward(d, like, at, order, weights)[0], want)
    # the formula: one rounding of a product that 32 bits round once before
    ref = w.double().view(-1)[order.long()].unsqueeze(1) * d.double()[order.long() // K]
    got = eplb.combine_rows_backward(d, y, place, order, w)[0].double()
    room = ref.abs() * (2.0 ** -24 + torch.finfo(TYPES[dtype]).eps / 2 * (1 + 2.0 ** -24)) + (2.0 ** -25 if dtype == "f16" else 0)
    assert ((got - ref).abs() <= room).all()


def test_lost_rows():
    """Rows that no choice is the only one of get zeros, too."""
    T, K, C = 4, 2, 300
    g = torch.Generator().manual_seed(2)
    d, w = torch.randn((T, C), generator=g), torch.rand((T, K), generator=g)
    place = torch.tensor([0, 0, -1, 5, 99, 6, 2 ** 31 - 1, 7], dtype=torch.int32)
    order = torch.tensor([0, 3, -7, 100, 2 ** 31 - 1, 3, 5, 2], dtype=torch.int32)
    like = torch.empty((), device=DEV).expand(T * K, C)
    out = (torch.full((8, C), 9.0, device=DEV), None)
    assert eplb.combine_rows_backward(*[t.to(DEV) for t in (d, )], like, place.to(DEV), order.to(DEV), w.to(DEV), out=out) is out
    want = torch.zeros((8, C))
    for r, i in ((0, 0), (5, 3), (6, 5)):
        want[r] = w.view(-1)[i] * d[i // 2]
    assert torch.equal(out[0].cpu(), want)


def test_autograd_and_graph():
    """autograd.combine with weights that need no gradient: y's gradient has the bits it has with them; captured and
    replayed as eager."""
    from moe_expert_load_eplb_amd.autograd import combine
    T, K, C = 50, 3, 520
    d, y, place, order, w = case(T, K, C, "bf16", "bf16", 3)
    grads = []
    for gv in (False, True):
        a, v = y.clone().requires_grad_(True), w.clone().requires_grad_(gv)
        combine(a, v, place, order).backward(d)
        grads.append(a.grad)
        assert (v.grad is not None) == gv
    assert torch.equal(*grads)
    ref = w.double().view(-1)[order.long()].unsqueeze(1) * d.double()[order.long() // K]
    assert ((grads[0].double() - ref).abs() <= ref.abs() * (2.0 ** -24 + 2.0 ** -8 * (1 + 2.0 ** -24))).all()
    buf, like = d.clone(), y.new_empty(()).expand(T * K, C)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = eplb.combine_rows_backward(buf, like, place, order, w)[0]
    for i in range(4):
        buf.copy_(d * (i + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, eplb.combine_rows_backward(d * (i + 1), y, place, order, w)[0])
