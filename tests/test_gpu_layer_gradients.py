"""Gradients of expert_linear16 and combine where a program hands them something
less regular: a gradient that starts between 16 bytes, no tokens, the most choices
of a token, weights or rows that need none (needs an MI355X).

Tolerances: those of the single calls, a sum of n products (n + 16) * 2^-23 of the
sum of their magnitudes, and half a step of the output's type."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

eplb = pytest.importorskip("moe_expert_load_eplb_amd")

from test_gpu_layer import DEV, grouping, plain_linear, within  # noqa: E402


def note(*a):
    print("[gradients]", *a, flush=True)


@pytest.mark.parametrize("ahead", [1, 3, 4, 7, 8])
@pytest.mark.parametrize("grouped", [False, True])
def test_gradients_that_start_anywhere(ahead, grouped):
    """The part of a concatenation's gradient: the bits of the same gradient by itself."""
    from moe_expert_load_eplb_amd.autograd import expert_linear16
    note("ahead", ahead, grouped)
    T, K, G, N, C = 37, 2, 5, 72, 136
    offsets, order, place = grouping(T, K, G, 3)
    g = torch.Generator(device=DEV).manual_seed(ahead)
    x = torch.randn((T if grouped else T * K, C), generator=g, device=DEV).bfloat16().requires_grad_(True)
    w = torch.randn((G, N, C), generator=g, device=DEV).bfloat16().requires_grad_(True)
    whole = torch.randn((ahead + T * K * N,), generator=g, device=DEV).bfloat16()
    args = (offsets, order, place, K) if grouped else (offsets,)
    want = torch.autograd.grad(expert_linear16(x, w, *args), (x, w), whole[ahead:].view(T * K, N).clone())
    joined = torch.cat([torch.zeros((ahead,), dtype=torch.bfloat16, device=DEV), expert_linear16(x, w, *args).view(-1)])
    got = torch.autograd.grad(joined, (x, w), whole)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    a, b = (t.detach().double().requires_grad_(True) for t in (x, w))
    ref = torch.autograd.grad(plain_linear(a, b, offsets, order if grouped else None, K), (a, b),
                              whole[ahead:].view(T * K, N).double())
    a, b = (t.detach().double().abs().requires_grad_(True) for t in (x, w))
    absolute = torch.autograd.grad(plain_linear(a, b, offsets, order if grouped else None, K), (a, b),
                                   whole[ahead:].view(T * K, N).double().abs())
    for p, r, m, n in zip(got, ref, absolute, (N + K, T * K)):
        within(p, r, m, n, ahead)


def test_most_choices():
    """64 choices of a token have gradients, 65 are refused before the forward pass where x needs one."""
    from moe_expert_load_eplb_amd.autograd import combine, expert_linear16
    T, N, C = 5, 16, 24
    g = torch.Generator(device=DEV).manual_seed(1)
    for K in (64, 65):
        G = K + 6
        offsets, order, place = grouping(T, K, G, K)
        x = torch.randn((T, C), generator=g, device=DEV).bfloat16().requires_grad_(True)
        w = torch.randn((G, N, C), generator=g, device=DEV).bfloat16().requires_grad_(True)
        if K == 65:
            with pytest.raises(ValueError):
                expert_linear16(x, w, offsets, order, place, K)
            expert_linear16(x.detach(), w, offsets, order, place, K).sum().backward()
            assert x.grad is None and w.grad.shape == w.shape
            continue
        y = expert_linear16(x, w, offsets, order, place, K)
        v = torch.rand((T, K), generator=g, device=DEV).requires_grad_(True)
        out = combine(y, v, place, order, dtype=torch.float32)
        d = torch.randn(out.shape, generator=g, device=DEV)
        dv, = torch.autograd.grad(out, v, d, retain_graph=True)
        ref = (y.detach().double()[place.long()].view(T, K, N) * d.double().unsqueeze(1))
        within(dv, ref.sum(2), ref.abs().sum(2), N, "dv")
        dy = torch.randn((T * K, N), generator=g, device=DEV).bfloat16()
        dx, = torch.autograd.grad(y, x, dy)
        refs = []
        for f in (lambda t: t, torch.abs):
            a = f(x.detach().double()).requires_grad_(True)
            refs.append(torch.autograd.grad(plain_linear(a, f(w.detach().double()), offsets, order, K), a, f(dy.double()))[0])
        within(dx, *refs, N + K, "dx")


def test_no_tokens():
    from moe_expert_load_eplb_amd.autograd import combine, expert_linear16
    K, G, N, C = 2, 4, 16, 24
    none = torch.zeros((0,), dtype=torch.int32, device=DEV)
    offsets = torch.zeros((G + 1,), dtype=torch.int32, device=DEV)
    x = torch.zeros((0, C), dtype=torch.bfloat16, device=DEV, requires_grad=True)
    w = torch.randn((G, N, C), device=DEV).bfloat16().requires_grad_(True)
    v = torch.zeros((0, K), device=DEV, requires_grad=True)
    out = combine(expert_linear16(x, w, offsets, none, none, K), v, none, none)
    out.sum().backward()
    assert out.shape == (0, N) and x.grad.shape == (0, C) and v.grad.shape == (0, K) and (w.grad == 0).all()


@pytest.mark.parametrize("gx,gw,gv", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (1, 0, 1)])
def test_partial_gradients(gx, gw, gv):
    """What is asked for has the bits it has when all are asked for."""
    from moe_expert_load_eplb_amd.autograd import combine, expert_linear16
    T, K, G, N, C = 60, 3, 7, 264, 136
    offsets, order, place = grouping(T, K, G, 5)
    g = torch.Generator(device=DEV).manual_seed(6)
    data = (torch.randn((T, C), generator=g, device=DEV).half(), torch.randn((G, N, C), generator=g, device=DEV).half(),
            torch.rand((T, K), generator=g, device=DEV))

    def step(which):
        leaves = [t.clone().requires_grad_(bool(on)) for t, on in zip(data, which)]
        combine(expert_linear16(*leaves[:2], offsets, order, place, K), leaves[2], place, order).float().square().mean().backward()
        return [t.grad for t in leaves]
    for got, want, on in zip(step((gx, gw, gv)), step((1, 1, 1)), (gx, gw, gv)):
        assert torch.equal(got, want) if on else got is None
