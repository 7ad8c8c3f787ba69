"""Weights in 4-bit floating point and the experts' products with them: HIP path
against the format's definition and plain sums in 64 bits (needs an MI355X).

Codes and scales are compared as they are.  A product of a 16-bit value and what
a code stands for is exact in 32 bits (a half-precision value as two bfloat16
ones: two products, so twice as many additions), and a sum of n products is held
to (n + 16) * 2^-23 * sum |x| |w|, each addition being off by at most 2^-23 of
what it has so far; an output of fewer bits to its half step more."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

eplb = pytest.importorskip("moe_expert_load_eplb_amd")
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
VALUES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def note(*a):
    print("[linear4]", *a, flush=True)


def rand(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * torch.exp2(torch.randint(-3, 4, shape[-1:], generator=g).float())).to(
        TYPES[dtype])


def defined(w):
    """(codes [.., C], scale bytes [.., C / 32]) of the definition, in 64 bits."""
    v = w.double().view(*w.shape[:-1], -1, 32)
    top = v.abs().amax(-1)
    fine = torch.isfinite(v).all(-1)
    e = torch.full(top.shape, -100, dtype=torch.int64)
    for _ in range(240):                                             # the least e >= -100 with top <= 7 * 2^e
        e += fine & (7.0 * torch.exp2(e.double()) < top)
    u = torch.where(fine.unsqueeze(-1), v, 0.0) / torch.exp2(e.double()).unsqueeze(-1)
    a = u.abs()
    far = (a.unsqueeze(-1) - VALUES).abs()
    order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7])                   # ties to the even code
    code = order[far[..., order].argmin(-1)]
    code = code + 8 * (torch.signbit(u) & fine.unsqueeze(-1))
    return code.view(w.shape), torch.where(fine, e + 127, 255)


def packed(code):
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)


def stands_for(q, s):
    """What codes and scales hold, in 64 bits."""
    q, s = q.cpu().long(), s.cpu().long()
    code = torch.stack([q & 15, q >> 4], -1).view(*q.shape[:-1], -1)
    v = torch.cat([VALUES, -VALUES])[code].view(*s.shape, 32)
    scale = torch.where(s == 255, torch.nan, torch.exp2(s.double() - 127))
    return (v * scale.unsqueeze(-1)).view(code.shape)


@pytest.mark.parametrize("G,N,C,dtype", [(1, 1, 32, "f32"), (2, 7, 96, "bf16"), (3, 130, 1056, "f16"), (1, 64, 4096, "bf16"),
                                         (5, 3, 160, "f32")])
def test_quantize(G, N, C, dtype):
    note("quantize", G, N, C, dtype)
    w = rand((G, N, C), dtype, N * C)
    if G > 1:
        w[1, 0, 3], w[0, N - 1, C - 1], w[1, N - 1, 33] = float("nan"), float("inf"), 0.0
        w[0, 0, :32] = 0
        w[1, 1, 32:64] *= 2.0 ** -120 if dtype != "f16" else 2.0 ** -20
    q, s = eplb.quantize_weights4(w.to(DEV))
    code, scale = defined(w)
    assert torch.equal(s.cpu().long(), scale) and torch.equal(q.cpu(), packed(code))
    out = (torch.empty_like(q), torch.empty_like(s))
    assert eplb.quantize_weights4(w.to(DEV), out=out) is out and torch.equal(out[0], q)


def test_quantize_borders():
    """Every midpoint of neighbouring values and its neighbours in 32 bits, both signs; the borders of a scale."""
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 6.5, 7.0])
    near = torch.cat([mids, torch.nextafter(mids, torch.zeros(())), torch.nextafter(mids, torch.full((), 9.0))])
    near = torch.cat([near, -near])
    rows = []
    for e in (-130, -100, -99, -20, 0, 60, 124):
        block = near.clamp(-7, 7).double() * 2.0 ** e
        for i in range(0, block.numel(), 31):
            row = torch.zeros(32, dtype=torch.float64)
            row[:block[i:i + 31].numel()] = block[i:i + 31]
            row[31] = 7.0 * 2.0 ** e                                  # the scale is 2^e exactly (where e >= -100)
            rows.append(row)
    for top in (7.0, 3.5, 1.75, 6.0, 14.0, 0.0, 2.0 ** -120, 3.0e38):
        for t in (top, float(torch.nextafter(torch.tensor(top), torch.tensor(float("inf"))))):
            row = torch.zeros(32, dtype=torch.float64)
            row[5], row[6] = t, -t / 2
            rows.append(row)
    w = torch.stack(rows).float().unsqueeze(0)
    q, s = eplb.quantize_weights4(w.to(DEV))
    code, scale = defined(w)
    assert torch.equal(s.cpu().long(), scale) and torch.equal(q.cpu(), packed(code))


def check(got, ref, absolute, n, what):
    t = got.dtype
    half = torch.finfo(t).eps / 2
    got = got.double().cpu()
    tiny = 2.0 ** -25 if t == torch.float16 else 0.0
    room = (n + 16) * 2.0 ** -23 * absolute
    room = room + half * (ref.abs() + room) + tiny
    past = ref.abs() + room > torch.finfo(t).max
    bad = ((got - ref).abs() > room) & ~past
    assert not bad.any(), (what, bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), ref[bad][:4].tolist())


@pytest.mark.parametrize("counts,head,tail,X,topk,N,C,dtype,out,rows", [
    ([1], 0, 0, 1, 1, 1, 32, "bf16", "bf16", False),
    ([1], 0, 0, 1, 1, 17, 64, "f16", "f32", False),
    ([0], 0, 0, 3, 1, 16, 32, "bf16", "f32", True),
    ([1] * 8, 0, 2, 1, 8, 80, 2048, "bf16", "bf16", True),
    ([1, 0, 1, 2, 1], 1, 0, 4, 2, 4096, 512, "f16", "f16", True),
    ([3, 0, 16], 2, 4, 9, 2, 7, 96, "f16", "f16", True),
    ([17, 31, 32, 33], 0, 1, 60, 4, 200, 224, "bf16", "f32", True),
    ([63, 64, 65, 2], 0, 0, 194, 1, 1391, 160, "f16", "f32", False),
    ([127, 128, 129], 0, 0, 384, 1, 130, 1056, "bf16", "f32", False),
    ([257, 1, 0, 16], 3, 5, 140, 2, 264, 288, "f16", "bf16", True),
    ([1] * 70 + [40], 1, 0, 64, 2, 96, 256, "bf16", "f32", True),
    ([4, 4], 0, 0, 0, 1, 24, 64, "bf16", "bf16", True),
    # tiles of 256 rows: whole ones, pieces of them at the end, and what is behind a group's last 256 rows
    ([700, 257, 0, 900], 3, 6, 933, 2, 4001, 96, "bf16", "bf16", True),
    ([700, 257, 0, 900], 3, 6, 933, 2, 4001, 96, "f16", "f16", True),
    ([2304], 0, 0, 2304, 1, 4000, 224, "f16", "f32", False),
    ([1025, 511], 0, 300, 918, 2, 6000, 64, "bf16", "f16", True),
    ([384, 130, 129, 513, 1], 0, 5, 1162, 1, 5120, 160, "f16", "bf16", True)])
def test_product(counts, head, tail, X, topk, N, C, dtype, out, rows):
    G, R = len(counts), head + sum(counts) + tail
    note("product", counts[:6], head, tail, X, topk, N, C, dtype, out, rows)
    off = torch.tensor(head + np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    g = torch.Generator().manual_seed(R + N)
    x = rand((X, C), dtype, N + C)
    q = torch.randint(0, 256, (G, N, C // 2), generator=g, dtype=torch.uint8)
    s = torch.randint(90, 140, (G, N, C // 32), generator=g, dtype=torch.uint8)
    w = stands_for(q, s)
    src = torch.arange(R)
    idx = None
    if rows:
        idx = torch.randint(0, max(1, X * topk), (R,), generator=g, dtype=torch.int32)
        if R > 3:
            idx[R // 2], idx[R // 3] = -1, X * topk
        src = torch.where(idx >= 0, idx.long() // topk, -1)
    src = torch.where(src < X, src, -1)
    wide = torch.full((X, C + 8), float("nan"), dtype=x.dtype)
    wide[:, 8:] = x
    y = eplb.expert_matmul4(wide.to(DEV)[:, 8:], q.to(DEV), s.to(DEV), off.to(DEV),
                            rows=None if idx is None else idx.to(DEV), K=topk, dtype=TYPES[out])
    xr = torch.zeros((R, C), dtype=torch.float64)
    xr[src >= 0] = x.double()[src[src >= 0]]
    ref, absolute = torch.zeros((R, N), dtype=torch.float64), torch.zeros((R, N), dtype=torch.float64)
    for i in range(G):
        a, b = off[i], off[i + 1]
        ref[a:b] = xr[a:b] @ w[i].t()
        absolute[a:b] = xr[a:b].abs() @ w[i].abs().t()
    check(y, ref, absolute, C * (2 if dtype == "f16" else 1), "y")
    none = src < 0
    none[:head] = True
    none[R - tail:] = True
    assert (y.cpu()[none] == 0).all()


def test_every_scale():
    """One block of ones against every scale byte: exact down to 2^-126, NaN for 255, an infinity past 32 bits."""
    x = torch.ones((1, 32), dtype=torch.bfloat16, device=DEV)
    q = torch.zeros((1, 256, 16), dtype=torch.uint8)
    q[:, :, 0] = 0x2A                                                # -1, 1
    q[:, :, 5] = 0x05                                                # 3
    s = torch.arange(256, dtype=torch.uint8).view(1, 256, 1)
    off = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    y = eplb.expert_matmul4(x, q.to(DEV), s.to(DEV), off, dtype=torch.float32).cpu().double()[0]
    assert torch.isnan(y[255])
    want = 3.0 * torch.exp2(torch.arange(256, dtype=torch.float64) - 127)
    fits = want < 2.0 ** 127.9
    assert torch.equal(y[2:255][fits[2:255]], want[2:255][fits[2:255]])
    assert torch.isinf(y[254]) and (y[:2] <= want[:2]).all()


def test_half_precision_is_exact():
    """Every finite half-precision value passes the product unchanged, and infinities stay infinities."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.float16)
    v = torch.where(torch.isnan(v), torch.zeros((), dtype=torch.float16), v)
    x = torch.zeros((65536, 32), dtype=torch.float16)
    x[:, 7] = v
    q = torch.zeros((1, 4, 16), dtype=torch.uint8)
    q[:, :, 3] = 0x20                                                # element 7: 1
    s = torch.full((1, 4, 1), 127, dtype=torch.uint8)
    off = torch.tensor([0, 65536], dtype=torch.int32, device=DEV)
    y = eplb.expert_matmul4(x.to(DEV), q.to(DEV), s.to(DEV), off, dtype=torch.float32).cpu()
    # an infinity times the other weights, which are 0, is NaN by the formula only where it stands itself
    assert torch.equal(y, v.float().unsqueeze(1).expand(-1, 4))


def test_nan_blocks():
    w = torch.randn((2, 40, 96), generator=torch.Generator().manual_seed(1))
    w[0, 3, 40], w[1, 39, 95] = float("nan"), float("inf")
    q, s = eplb.quantize_weights4(w.to(DEV))
    x = torch.randn((9, 96), device=DEV).bfloat16()
    off = torch.tensor([0, 4, 9], dtype=torch.int32, device=DEV)
    y = eplb.expert_matmul4(x, q, s, off).cpu()
    odd = torch.zeros((9, 40), dtype=torch.bool)
    odd[:4, 3], odd[4:, 39] = True, True
    assert torch.equal(torch.isnan(y), odd)


def test_graph():
    """Weights taken to 4 bits and multiplied in a captured graph, replayed on new inputs."""
    g = torch.Generator(device=DEV).manual_seed(3)
    off = torch.tensor([0, 5, 9, 30], dtype=torch.int32, device=DEV)
    data = [(torch.randn((30, 256), generator=g, device=DEV).half(), torch.randn((3, 72, 256), generator=g, device=DEV))
            for _ in range(3)]
    want = [eplb.expert_matmul4(x, *eplb.quantize_weights4(w), off) for x, w in data]
    x, w = data[0][0].clone(), data[0][1].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = eplb.expert_matmul4(x, *eplb.quantize_weights4(w), off)
    for i in (1, 0, 2, 1):
        x.copy_(data[i][0])
        w.copy_(data[i][1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
