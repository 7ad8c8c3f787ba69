"""The experts' products in 16 bits and with 4-bit weights and the join of their
rows, as a layer uses them: functions of torch with their gradients, served and
trained layers, captured steps (needs an MI355X).

Tolerances.  A sum of n products is off by (n + 16) * 2^-23 of the sum of their
magnitudes at most, and each rounding to bfloat16 by 2^-8 of the value: single
calls are held to these.  A layer rounds x W, silu(a) b, the second product, and
its output, its gradients as often again on the way back: seven in a row at most,
2.7 % in norm; it is held to 3 %."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

eplb = pytest.importorskip("moe_expert_load_eplb_amd")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def note(*a):
    print("[layer]", *a, flush=True)


def grouping(T, K, G, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    ids = torch.rand((T, G), generator=g, device=DEV).topk(K, 1).indices.int()
    return tuple(t[0] for t in eplb.group_rows(ids.view(1, -1), G))


def plain_linear(x, w, offsets, order, K):
    """In 64 bits."""
    rows = x[order.long() // K] if order is not None else x
    cut = offsets.tolist()
    return torch.cat([rows[a:b] @ w[g].t() for g, (a, b) in enumerate(zip(cut, cut[1:]))])


def within(got, ref, absolute, n, what):
    half = torch.finfo(got.dtype).eps / 2
    room = (n + 16) * 2.0 ** -23 * absolute
    room = room + half * (ref.abs() + room) + (2.0 ** -25 if got.dtype == torch.float16 else 0)
    assert got.shape == ref.shape and ((got.double() - ref).abs() <= room).all(), what


@pytest.mark.parametrize("T,K,G,N,C,dtype,grouped", [
    (1, 1, 1, 8, 8, torch.bfloat16, False), (33, 2, 4, 72, 136, torch.float16, True),
    (700, 4, 9, 264, 200, torch.bfloat16, True), (130, 1, 3, 128, 64, torch.float16, False),
    (3, 2, 40, 16, 520, torch.bfloat16, True)])
def test_linear(T, K, G, N, C, dtype, grouped):
    from moe_expert_load_eplb_amd.autograd import expert_linear16
    note("linear", T, K, G, N, C, dtype, grouped)
    offsets, order, place = grouping(T, K, G, T)
    g = torch.Generator(device=DEV).manual_seed(N)
    rows = T if grouped else T * K
    x = torch.randn((rows, C), generator=g, device=DEV).to(dtype).requires_grad_(True)
    w = torch.randn((G, N, C), generator=g, device=DEV).to(dtype).requires_grad_(True)
    dy = torch.randn((T * K, N), generator=g, device=DEV).to(dtype)
    y = expert_linear16(x, w, offsets, order, place, K) if grouped else expert_linear16(x, w, offsets)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    assert dx.dtype == dw.dtype == y.dtype == dtype
    refs = []
    for f in (lambda t: t, torch.abs):
        a, b = (f(t.detach().double()).requires_grad_(True) for t in (x, w))
        r = plain_linear(a, b, offsets, order if grouped else None, K)
        refs.append((r.detach(), *torch.autograd.grad(r, (a, b), f(dy.double()))))
    for got, ref, absolute, n, what in zip((y, dx, dw), *refs, (C, N + K, T * K), ("y", "dx", "dw")):
        within(got.detach(), ref, absolute, n, what)


@pytest.mark.parametrize("T,K,C,dtype,out", [(1, 1, 8, torch.bfloat16, None), (65, 6, 2050, torch.float16, torch.float32),
                                             (300, 8, 96, torch.float32, None), (40, 3, 7, torch.bfloat16, torch.float32)])
def test_combine(T, K, C, dtype, out):
    from moe_expert_load_eplb_amd.autograd import combine
    note("combine", T, K, C, dtype, out)
    _, order, place = grouping(T, K, max(K, 9), C)
    g = torch.Generator(device=DEV).manual_seed(T)
    y = torch.randn((T * K, C), generator=g, device=DEV).to(dtype).requires_grad_(True)
    v = torch.rand((T, K), generator=g, device=DEV).requires_grad_(True)
    o = combine(y, v, place, order, dtype=out)
    assert o.dtype == (out or dtype)
    d = torch.randn(o.shape, generator=g, device=DEV).to(o.dtype)
    dy, dv = torch.autograd.grad(o, (y, v), d)
    refs = []
    for f in (lambda t: t, torch.abs):
        a, b = (f(t.detach().double()).requires_grad_(True) for t in (y, v))
        r = (a[place.long()].view(T, K, C) * b.unsqueeze(2)).sum(1)
        refs.append((r.detach(), *torch.autograd.grad(r, (a, b), f(d.double()))))
    for got, ref, absolute, n, what in zip((o, dy, dv), *refs, (K, 1, C), ("out", "dy", "dv")):
        within(got.detach(), ref, absolute, n, what)


def held_values(held, bits):
    """The weights that a layer holds, in 64 bits."""
    if bits == 16:
        return held[0].double()
    q, s = (t.long() for t in held)
    values = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=DEV)
    code = torch.stack([q & 15, q >> 4], -1).view(*s.shape, 32)
    return (torch.cat([values, -values])[code] * torch.exp2(s.double() - 127).unsqueeze(-1)).view(*s.shape[:2], -1)


def plain_layer(x, ids, weights, up, down):
    out = torch.zeros_like(x)
    for e in range(up.shape[0]):
        t, k = (ids == e).nonzero(as_tuple=True)
        a, b = (x[t] @ up[e].t()).chunk(2, dim=1)
        out = out.index_add(0, t, weights[t, k].unsqueeze(1) * ((torch.nn.functional.silu(a) * b) @ down[e].t()))
    return out


@pytest.mark.parametrize("bits", [16, 4])
def test_serving(example, bits):
    layer = example.MoELayer(seed=3, bits=bits)
    g = torch.Generator(device=DEV).manual_seed(4)
    for step, T in enumerate((1, 7, 64, 700)):
        note("serving", bits, T)
        x = torch.randn((T, layer.C), generator=g, device=DEV).bfloat16()
        y = layer.serve(x)
        ids, w = eplb.gate(layer.logits(x), layer.K, bias=layer.bias, G=layer.G, top_groups=layer.G // 2, group_top=2)
        held = layer.log2phy[0, :, 0].long()                        # every replica of an expert holds the same
        up, down = held_values(layer.up_held, bits)[held], held_values(layer.down_held, bits)[held]
        ref = plain_layer(x.double(), ids, w.double(), up, down)
        assert (y.double() - ref).norm() < 0.03 * ref.norm()
        if step == 1:
            layer.place(layer.load)


def test_training(example):
    layer = example.MoELayer(seed=5, bits=16)
    g = torch.Generator(device=DEV).manual_seed(6)
    T = 300
    x = torch.randn((T, layer.C), generator=g, device=DEV).bfloat16().requires_grad_(True)
    seg = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    params = [x, layer.router.requires_grad_(True), layer.up.requires_grad_(True), layer.down.requires_grad_(True)]
    out, _ = layer.train(x, seg, alpha=0.0)
    d = torch.randn(out.shape, generator=g, device=DEV)
    got = torch.autograd.grad((out * d).sum(), params)
    p64 = [p.detach().double().requires_grad_(True) for p in params]
    with torch.no_grad():
        ids, _ = eplb.gate(layer.logits(x), layer.K, bias=layer.bias, G=layer.G, top_groups=layer.G // 2, group_top=2)
    sel = torch.sigmoid(p64[0] @ p64[1].t()).gather(1, ids.long())
    ref = plain_layer(p64[0], ids, sel / sel.sum(1, keepdim=True), p64[2], p64[3])
    want = torch.autograd.grad((ref * d.double()).sum(), p64)
    assert (out.double() - ref).norm() < 0.03 * ref.norm()
    for a, b, name in zip(got, want, ("x", "router", "up", "down")):
        assert (a.double() - b).norm() < 0.03 * b.norm(), name


def test_captured_step(example):
    """A training step in a graph, replayed on new inputs with eager steps between: the eager step's bits every time."""
    layer = example.MoELayer(seed=7, bits=16)
    g = torch.Generator(device=DEV).manual_seed(8)
    T = 200
    offsets, order, place = grouping(T, layer.K, layer.E, 9)
    weights = torch.rand((T, layer.K), generator=g, device=DEV)
    x = torch.zeros((T, layer.C), dtype=torch.bfloat16, device=DEV)
    d = torch.zeros((T, layer.C), dtype=torch.bfloat16, device=DEV)

    def step():
        h = eplb.expert_matmul16(x, layer.up, offsets, rows=order, K=layer.K)
        y = eplb.expert_matmul16(h[:, :layer.F], layer.down, offsets)
        out = eplb.combine_rows(y, place, weights)
        dy, dv = eplb.combine_rows_backward(d, y, place, order, weights)
        dh = eplb.expert_matmul16(dy, layer.down, offsets, transpose=True)
        dw = eplb.expert_wgrad16(dy, h[:, :layer.F], offsets)
        q = eplb.quantize_weights4(layer.down)
        return out, dv, dh, dw, *q, eplb.expert_matmul4(h[:, :layer.F], *q, offsets)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        d.copy_(torch.randn(d.shape, generator=g, device=DEV))
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_streams():
    """Two products at once on streams of their own."""
    g = torch.Generator(device=DEV).manual_seed(1)
    offsets, order, place = grouping(500, 2, 9, 2)
    x = torch.randn((500, 512), generator=g, device=DEV).bfloat16()
    w = torch.randn((9, 264, 512), generator=g, device=DEV).bfloat16()
    q = eplb.quantize_weights4(w)
    want = eplb.expert_matmul16(x, w, offsets, rows=order, K=2), eplb.expert_matmul4(x, *q, offsets, rows=order, K=2)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(a):
            one = eplb.expert_matmul16(x, w, offsets, rows=order, K=2)
        with torch.cuda.stream(b):
            two = eplb.expert_matmul4(x, *q, offsets, rows=order, K=2)
        torch.cuda.synchronize()
        assert torch.equal(one, want[0]) and torch.equal(two, want[1])
