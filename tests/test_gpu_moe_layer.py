"""The layer of examples/moe_layer.py: served and trained end to end, against
the same layer with unquantised weights in 64 bits (needs an MI355X).

Each 8-bit rounding moves a value by at most 1/16 of itself, 2.6 % rms; the two
products of the layer see four such operands in a row, so outputs and gradients
are held to 12 % in norm, and the routing to the rule."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

eplb = pytest.importorskip("moe_expert_load_eplb_amd")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain(layer, x, ids, weights, router, up, down):
    """The layer for given ids, every expert in turn, in the parameters' precision."""
    out = torch.zeros_like(x)
    for e in range(layer.E):
        t, k = (ids == e).nonzero(as_tuple=True)
        a, b = (x[t] @ up[e].t()).chunk(2, dim=1)
        out = out.index_add(0, t, weights[t, k].unsqueeze(1) * ((torch.nn.functional.silu(a) * b) @ down[e].t()))
    return out


def test_serving(example):
    layer = example.MoELayer(seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    total = torch.zeros((layer.E,), dtype=torch.int64, device="cuda")
    for step in range(4):
        T = (1, 7, 64, 200)[step]
        x = torch.randn((T, layer.C), generator=g, device="cuda").bfloat16()
        y = layer.serve(x)
        ids, w = eplb.gate(layer.logits(x), layer.K, bias=layer.bias, G=layer.G, top_groups=layer.G // 2, group_top=2)
        total += torch.bincount(ids.flatten(), minlength=layer.E)
        assert torch.equal(layer.load[0], total)
        ref = plain(layer, x.double(), ids, w.double(), None, layer.up.double(), layer.down.double())
        assert (y.double() - ref).norm() < 0.12 * ref.norm()
        if step == 1:
            layer.place(layer.load)
            assert layer.logcnt.sum() == layer.P


def test_training(example):
    layer = example.MoELayer(seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    T = 300
    x = torch.randn((T, layer.C), generator=g, device="cuda").bfloat16().requires_grad_(True)
    seg = torch.tensor([0, 120, T], dtype=torch.int32, device="cuda")
    params = [x, layer.router.requires_grad_(True), layer.up.requires_grad_(True), layer.down.requires_grad_(True)]
    out, balance = layer.train(x, seg, alpha=0.5)
    d = torch.randn(out.shape, generator=g, device="cuda")
    got = torch.autograd.grad((out * d).sum() + (balance * torch.tensor([2.0, -1.0], device="cuda")).sum(), params)
    # the same in 64 bits, choice and counts fixed
    p64 = [p.detach().double().requires_grad_(True) for p in params]
    with torch.no_grad():
        ids, w = eplb.gate(layer.logits(x), layer.K, bias=layer.bias, G=layer.G, top_groups=layer.G // 2, group_top=2)
    s = torch.sigmoid(p64[0] @ p64[1].t())
    sel = s.gather(1, ids.long())
    weights = sel / sel.sum(1, keepdim=True)
    share = s / s.sum(1, keepdim=True)
    ref_loss = []
    for lo, hi in ((0, 120), (120, T)):
        f = torch.bincount(ids[lo:hi].flatten(), minlength=layer.E).double() * layer.E / (layer.K * (hi - lo))
        ref_loss.append(0.5 * (f * share[lo:hi].mean(0)).sum())
    ref = plain(layer, p64[0], ids, weights, p64[1], p64[2], p64[3])
    want = torch.autograd.grad((ref * d.double()).sum() + 2 * ref_loss[0] - ref_loss[1], p64)
    torch.testing.assert_close(balance.detach().double(), torch.stack(ref_loss).detach(), rtol=4e-5, atol=0)
    assert (out.double() - ref).norm() < 0.12 * ref.norm()
    for a, b, name in zip(got, want, ("x", "router", "up", "down")):
        assert a.dtype == dict(x=torch.bfloat16, router=torch.float32, up=torch.bfloat16, down=torch.bfloat16)[name]
        assert (a.double() - b).norm() < 0.12 * b.norm(), name


def test_route_partial_gradients(example):
    """Gradients of the loss alone, of the weights alone, and of neither."""
    from moe_expert_load_eplb_amd.autograd import route
    x = torch.randn((50, 16), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).requires_grad_(True)
    seg = torch.tensor([0, 50], dtype=torch.int32, device="cuda")
    ids, w, loss, counts, prob, tokens = route(x, 3, seg, 1.0, scoring="softmax")
    assert not ids.requires_grad and not counts.requires_grad and not prob.requires_grad and tokens.tolist() == [50]
    a = torch.autograd.grad(loss.sum(), x, retain_graph=True)[0]
    b = torch.autograd.grad((w ** 2).sum(), x, retain_graph=True)[0]
    both = torch.autograd.grad(loss.sum() + (w ** 2).sum(), x)[0]
    torch.testing.assert_close(a + b, both, rtol=1e-5, atol=1e-7)
    assert a.abs().sum() > 0 and b.abs().sum() > 0
    assert a.sum(1).abs().max() < 1e-6 and b.sum(1).abs().max() < 1e-6      # softmax is blind to a shift


def test_example_runs(example, capsys):
    example.main()
    lines = capsys.readouterr().out.strip().splitlines()
    losses = [float(l.split("loss ")[1].split(",")[0]) for l in lines if l.startswith("step")]
    assert len(losses) == 5 and losses[-1] < losses[0]
