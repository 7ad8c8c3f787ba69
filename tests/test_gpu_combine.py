"""The experts' rows joined to tokens and the gradients of that: HIP path against
plain sums in 64 bits (needs an MI355X).

Tolerances: n fused multiply-adds in 32 bits are off by at most n * 2^-24 of A =
sum |a| |b| (each rounds once, and no partial sum exceeds A by more than what is
already counted: (n + 2) * 2^-24 * A), an output of fewer bits by its half step
more."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

eplb = pytest.importorskip("moe_expert_load_eplb_amd")
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def note(*a):
    print("[combine]", *a, flush=True)


def check(got, ref, absolute, n, what):
    t = got.dtype
    half = torch.finfo(t).eps / 2
    got = got.double().cpu()
    room = (n + 2) * 2.0 ** -24 * absolute
    room = room + half * (ref.abs() + room) + (2.0 ** -25 if t == torch.float16 else 0.0)
    bad = (got - ref).abs() > room
    assert not bad.any(), (what, bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), ref[bad][:4].tolist())


def case(T, K, C, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    y = torch.randn((T * K, C), generator=g).to(TYPES[dtype])
    order = torch.randperm(T * K, generator=g).int()
    place = torch.empty_like(order)
    place[order.long()] = torch.arange(T * K, dtype=torch.int32)
    w = torch.rand((T, K), generator=g) * 2 - 0.5
    d = torch.randn((T, C), generator=g)
    return y, place, order, w, d


SHAPES = [(1, 1, 1, "f32", "f32"), (1, 8, 4096, "bf16", "bf16"), (3, 2, 7, "f16", "f32"), (5, 9, 8, "bf16", "f16"),
          (64, 6, 2050, "f16", "f16"), (7, 64, 33, "f32", "bf16"), (130, 3, 500, "bf16", "f32"), (9, 17, 5000, "f32", "f32"),
          (300, 4, 16, "f16", "f16"), (2, 8, 20000, "bf16", "bf16"), (1000, 1, 257, "bf16", "bf16"), (33, 5, 1024, "f16", "bf16"),
          (40, 2, 1025, "f32", "f16")]


@pytest.mark.parametrize("T,K,C,dtype,out", SHAPES)
def test_forward(T, K, C, dtype, out):
    note("forward", T, K, C, dtype, out)
    y, place, order, w, _ = case(T, K, C, dtype, T + C)
    got = eplb.combine_rows(y.to(DEV), place.to(DEV), w.to(DEV), dtype=TYPES[out])
    rows = y.double()[place.long()].view(T, K, C)
    wd = w.double().unsqueeze(2)
    check(got, (rows * wd).sum(1), (rows * wd).abs().sum(1), K, "out")
    one = eplb.combine_rows(y.to(DEV), place.view(T, K).to(DEV), None, dtype=TYPES[out])
    check(one, rows.sum(1), rows.abs().sum(1), K, "ones")
    # the order of a sum is that of the choices
    ref = torch.zeros((T, C))
    for k in range(K):
        ref = torch.addcmul(ref.double(), rows[:, k].double(), wd[:, k].double()).float()
    exact = eplb.combine_rows(y.to(DEV), place.to(DEV), w.to(DEV), dtype=torch.float32)
    if dtype != "f32":                       # products of 24 and 11 bits and a 32-bit number: 64 bits round the sum twice
        assert (exact.cpu() - ref).abs().max() <= 2.0 ** -22 * (rows * wd).abs().sum(1).max()


def test_choices_that_are_nowhere():
    """Places outside the rows add nothing, whatever weights and rows hold; a row may be used twice."""
    y = torch.randn((4, 40), generator=torch.Generator().manual_seed(1))
    y[3] = float("nan")
    place = torch.tensor([[0, 2], [-1, 1], [4, -5], [1, 1], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32)
    w = torch.tensor([[0.5, 2.0], [float("nan"), 1.0], [1.0, float("inf")], [1.0, 3.0], [float("nan"), 1.0]])
    out = eplb.combine_rows(y.to(DEV), place.to(DEV), w.to(DEV)).cpu()
    want = torch.stack([0.5 * y[0] + 2 * y[2], y[1], torch.zeros(40), 4 * y[1], torch.zeros(40)])
    torch.testing.assert_close(out, want, rtol=2.0 ** -22, atol=0)
    none = eplb.combine_rows(y[:0].to(DEV), place.to(DEV), w.to(DEV))
    assert none.shape == (5, 40) and (none == 0).all()
    assert eplb.combine_rows(y.to(DEV), place[:0].to(DEV), w[:0].to(DEV)).shape == (0, 40)


@pytest.mark.parametrize("T,K,C,dtype,d_dtype", SHAPES)
def test_backward(T, K, C, dtype, d_dtype):
    note("backward", T, K, C, dtype, d_dtype)
    y, place, order, w, d = case(T, K, C, dtype, T + C)
    d = d.to(TYPES[d_dtype])
    at = [t.to(DEV) for t in (d, y, place, order, w)]
    dy, dw = eplb.combine_rows_backward(*at)
    assert dy.dtype == y.dtype and dw.dtype == torch.float32
    rows = y.double()[place.long()].view(T, K, C)
    dd = d.double().unsqueeze(1)
    check(dw, (rows * dd).sum(2), (rows * dd).abs().sum(2), C, "d_weights")
    i = order.long()
    ref = w.double().view(-1)[i].unsqueeze(1) * d.double()[i // K]
    check(dy, ref, ref.abs(), 1, "d_y")
    again = eplb.combine_rows_backward(*at)
    assert torch.equal(again[0], dy) and torch.equal(again[1], dw)
    ones, _ = eplb.combine_rows_backward(at[0], at[1], at[2].view(T, K), at[3], None)
    check(ones, d.double()[i // K], d.double().abs()[i // K], 1, "ones")


def test_backward_against_differences():
    T, K, C = 5, 3, 24
    y, place, order, w, d = case(T, K, C, "f32", 9)
    dy, dw = eplb.combine_rows_backward(*[t.to(DEV) for t in (d, y, place, order, w)])

    def value(y, w):
        return (eplb.combine_rows(y.to(DEV), place.to(DEV), w.to(DEV)).cpu().double() * d.double()).sum().item()

    h = 2.0 ** -4                            # the call is linear in each: a difference is as exact as its sums
    scale = 2.0 ** -20 * (d.double().abs().sum() * w.abs().max() * (y.abs().max() + 1)).item() / h
    for r, c in ((0, 0), (7, 11), (14, 23)):
        up, down = y.clone(), y.clone()
        up[r, c] += h
        down[r, c] -= h
        assert abs((value(up, w) - value(down, w)) / (2 * h) - dy[r, c].item()) < scale
    for t, k in ((0, 0), (4, 2), (2, 1)):
        up, down = w.clone(), w.clone()
        up[t, k] += h
        down[t, k] -= h
        assert abs((value(y, up) - value(y, down)) / (2 * h) - dw[t, k].item()) < scale


def test_backward_of_arrays_that_are_no_grouping():
    """Every output is written once, whatever place and order hold."""
    T, K, C = 4, 2, 300
    g = torch.Generator().manual_seed(2)
    y, d, w = torch.randn((8, C), generator=g), torch.randn((T, C), generator=g), torch.rand((T, K), generator=g)
    place = torch.tensor([0, 0, -1, 5, 99, 6, 2 ** 31 - 1, 7], dtype=torch.int32)
    order = torch.tensor([0, 3, -7, 100, 2 ** 31 - 1, 3, 5, 2], dtype=torch.int32)
    out = (torch.full((8, C), 9.0, device=DEV), torch.full((T, K), 9.0, device=DEV))
    dy, dw = eplb.combine_rows_backward(*[t.to(DEV) for t in (d, y, place, order, w)], out=out)
    want = torch.zeros((8, C))
    for r, i in ((0, 0), (5, 3), (6, 5)):
        want[r] = w.view(-1)[i] * d[i // 2]
    assert torch.equal(dy.cpu(), want)
    for i in range(8):
        p = int(place[i])
        ref = (d[i // 2].double() * y[p].double()).sum() if 0 <= p < 8 else torch.zeros((), dtype=torch.float64)
        assert abs(dw.view(-1)[i].item() - ref.item()) < 1e-3 and (0 <= p < 8 or dw.view(-1)[i] == 0)


def test_graph_and_streams():
    T, K, C = 200, 4, 1024
    y, place, order, w, d = (t.to(DEV) for t in case(T, K, C, "bf16", 4))
    d = d.bfloat16()

    def step(y):
        return (eplb.combine_rows(y, place, w), *eplb.combine_rows_backward(d, y, place, order, w))

    y2 = (y * 3).contiguous()
    want, other = step(y), step(y2)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            b = step(y2)
        a = step(y)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a + b, want + other))
    buf = y.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(buf)
    for i in range(4):
        buf.copy_(y if i % 2 else y2)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want if i % 2 else other))


@pytest.mark.parametrize("T,K,C,dtype", [(2049, 1, 520, "bf16"), (8301, 2, 100, "f32"), (1027, 3, 1030, "f16"),
                                         (1025, 4, 4104, "bf16"), (8195, 2, 33, "f16")])
def test_many_tokens_of_few_choices(T, K, C, dtype):
    """Several tokens at a time, the last ones fewer: the sums of the same tokens taken alone, bit for bit, and right."""
    note("few choices", T, K, C, dtype)
    y, place, order, w, _ = case(T, K, C, dtype, T + C)
    y, place, w = y.to(DEV), place.to(DEV).view(T, K), w.to(DEV)
    place[5], place[T - 1, K - 1] = -1, T * K
    got = eplb.combine_rows(y, place, w)
    some = torch.cat([torch.arange(40), torch.arange(T - 40, T)]).to(DEV)
    assert torch.equal(eplb.combine_rows(y, place[some].contiguous(), w[some].contiguous()), got[some])
    inside = (place >= 0) & (place < T * K)
    rows = y.double()[place.clamp(0, T * K - 1).long()] * inside.unsqueeze(2) * w.double().unsqueeze(2)
    check(got, rows.sum(1).cpu(), rows.abs().sum(1).cpu(), K, "out")


@pytest.mark.parametrize("C", [520, 66])
@pytest.mark.parametrize("shifted", ["y", "out", "d_out", "d_y", "all"])
def test_arrays_at_odd_elements(C, shifted):
    """16-bit arrays that start between words: the same bits as arrays that do not."""
    T, K = 37, 3
    note("odd elements", C, shifted)
    y, place, order, w, d = (t.to(DEV) for t in case(T, K, C, "bf16", C))
    d = d.bfloat16()

    def at(t, name):
        n = 1 if shifted in (name, "all") else 0
        flat = torch.zeros((t.numel() + 2,), dtype=t.dtype, device=DEV)
        flat[n:n + t.numel()] = t.reshape(-1)
        return flat[n:n + t.numel()].view(t.shape), flat

    want = eplb.combine_rows(y, place, w), *eplb.combine_rows_backward(d, y, place, order, w)
    (ys, _), (ds, _) = at(y, "y"), at(d, "d_out")
    (out, flat_out), (dy, flat_dy) = at(torch.zeros_like(want[0]), "out"), at(torch.zeros_like(want[1]), "d_y")
    eplb.combine_rows(ys, place, w, out=out)
    dw = torch.empty_like(want[2])
    eplb.combine_rows_backward(ds, ys, place, order, w, out=(dy, dw))
    assert torch.equal(out, want[0]) and torch.equal(dy, want[1])
    assert torch.equal(dw, want[2]) or shifted != "out"               # lanes have other elements then
    exact = (y.double()[place.long()].view(T, K, C) * d.double().unsqueeze(1))
    check(dw, exact.sum(2).cpu(), exact.abs().sum(2).cpu(), C, "d_weights")
    for flat, t in ((flat_out, out), (flat_dy, dy)):
        first = t.storage_offset()
        assert (flat[:first] == 0).all() and (flat[first + t.numel():] == 0).all()
