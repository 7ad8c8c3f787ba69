"""The experts' products in 16 bits and their gradients: HIP path against plain
sums in 64 bits (needs an MI355X).

Tolerances: a product of two 16-bit values is exact in 32 bits; a sum of n of
them takes n 32-bit additions, each off by at most 2^-23 of what it has so far
(rounded or cut off), that is of A = sum |x| |w| at most.  So a 32-bit sum is
held to (n + 16) * 2^-23 * A, and an output of fewer bits to its half step more."""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

eplb = pytest.importorskip("moe_expert_load_eplb_amd")
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def note(*a):
    print("[linear16]", *a, flush=True)


def rand(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * torch.exp2(torch.randint(-3, 4, shape[-1:], generator=g).float())).to(
        TYPES[dtype])


def check(got, ref, absolute, n, what):
    t = got.dtype
    half = torch.finfo(t).eps / 2
    got = got.double().cpu()
    tiny = 2.0 ** -25 if t == torch.float16 else 0.0                # half a step below float16's normal numbers
    room = (n + 16) * 2.0 ** -23 * absolute
    room = room + half * (ref.abs() + room) + tiny
    past = ref.abs() + room > torch.finfo(t).max                     # may round to infinity
    bad = ((got - ref).abs() > room) & ~past
    assert not bad.any(), (what, bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), ref[bad][:4].tolist())


def grouping(counts, head, tail):
    return torch.tensor(head + np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32), head + sum(counts) + tail


def sources(R, X, topk, seed, rows):
    """(rows on the host or None, source of every grouped row, -1: none)."""
    if not rows:
        src = torch.arange(R)
        return None, torch.where(src < X, src, -1)
    idx = torch.randint(0, max(1, X * topk), (R,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    if R > 3:
        idx[R // 2] = -1
        idx[R // 3] = X * topk
    src = idx.long() // topk
    return idx, torch.where((idx >= 0) & (src < X), src, -1)


def taken(x, src):
    """Rows src of x in 64 bits, zeros where there is none."""
    out = torch.zeros((src.numel(), x.shape[1]), dtype=torch.float64)
    out[src >= 0] = x.double()[src[src >= 0]]
    return out


CASES = [
    # counts, head, tail, X, topk, N, C, dtype, out, rows
    ([1], 0, 0, 1, 1, 8, 8, "bf16", "bf16", False),
    ([1], 0, 0, 1, 1, 1, 64, "f16", "f32", False),
    ([0], 0, 0, 3, 1, 16, 16, "bf16", "f32", True),
    ([3, 0, 5], 2, 4, 9, 2, 7, 72, "f16", "f16", True),
    ([127, 128, 129], 0, 0, 384, 1, 130, 136, "bf16", "f32", False),
    ([257, 1, 0, 16], 3, 5, 140, 2, 264, 1048, "bf16", "bf16", True),
    ([17, 33, 64, 65, 2], 0, 1, 60, 4, 1391, 200, "f16", "bf16", True),
    ([600], 0, 0, 300, 2, 520, 512, "bf16", "f32", True),
    ([1] * 70 + [40], 1, 0, 64, 2, 96, 264, "f16", "f32", True),
    ([4, 4], 0, 0, 0, 1, 24, 40, "bf16", "bf16", True),
    ([300, 212], 0, 0, 512, 1, 1024, 320, "f16", "f16", False),
    # tiles of 256 rows: whole ones, pieces of them at the end, and what is behind a group's last 256 rows
    ([700, 257, 0, 900], 3, 6, 933, 2, 3801, 72, "bf16", "bf16", True),
    ([2304], 0, 0, 2304, 1, 4097, 136, "f16", "f32", False),
    ([1025, 511], 0, 300, 918, 2, 6000, 64, "bf16", "f16", True),
    ([256 * 9], 0, 0, 2304, 1, 3840, 200, "bf16", "bf16", False),
    ([700, 257, 0, 900], 3, 6, 933, 2, 8001, 72, "bf16", "bf16", True),
    ([2304], 0, 0, 2304, 1, 7433, 136, "f16", "f32", False),
    ([1025, 511], 0, 300, 918, 2, 9000, 64, "bf16", "f16", True),
    ([256 * 9], 0, 0, 2304, 1, 7680, 200, "bf16", "bf16", False),
    ([384, 130, 129, 513, 1], 0, 5, 1162, 1, 9728, 64, "f16", "f16", True),
]


@pytest.mark.parametrize("counts,head,tail,X,topk,N,C,dtype,out,rows", CASES)
def test_product(counts, head, tail, X, topk, N, C, dtype, out, rows):
    off, R = grouping(counts, head, tail)
    note("product", counts[:6], head, tail, X, topk, N, C, dtype, out, rows)
    x, w = rand((X, C), dtype, N + C), rand((len(counts), N, C), dtype, R)
    idx, src = sources(R, X, topk, R + N, rows)
    wide = torch.full((X, C + 16), float("nan"), dtype=x.dtype)      # what lies between the rows is not read
    wide[:, 8:8 + C] = x
    if X > 0 and rows is False:
        wide[int(off[-1]):] = float("inf")                           # rows of no group: nothing of them arrives
    y = torch.full((R, N), 7.0, dtype=TYPES[out], device=DEV)
    i = None if idx is None else idx.to(DEV)
    got = eplb.expert_matmul16(wide.to(DEV)[:, 8:8 + C], w.to(DEV), off.to(DEV), rows=i, K=topk, out=y)
    assert got is y
    xr = taken(x, src)
    ref, absolute = torch.zeros((R, N), dtype=torch.float64), torch.zeros((R, N), dtype=torch.float64)
    for g in range(len(counts)):
        a, b = off[g], off[g + 1]
        ref[a:b] = xr[a:b] @ w[g].double().t()
        absolute[a:b] = xr[a:b].abs() @ w[g].double().abs().t()
    check(got, ref, absolute, C, "y")
    none = src < 0
    none[:head] = True
    none[R - tail:] = True
    assert (got.cpu()[none] == 0).all()
    if X > 0:
        again = eplb.expert_matmul16(x.to(DEV), w.to(DEV), off.to(DEV), rows=i, K=topk, dtype=TYPES[out])
        assert torch.equal(again, got)


@pytest.mark.parametrize("counts,head,tail,X,topk,N,C,dtype,out,rows",
                         [c[:5] + (-(-c[5] // 8) * 8,) + c[6:] for c in CASES[:11]] +
                         [c[:5] + (c[6], -(-c[5] // 8) * 8) + c[7:] for c in CASES[11:]])
def test_product_transposed(counts, head, tail, X, topk, N, C, dtype, out, rows):
    off, R = grouping(counts, head, tail)
    note("transposed", counts[:6], head, tail, X, topk, N, C, dtype, out, rows)
    x, w = rand((X, N), dtype, N + C), rand((len(counts), N, C), dtype, R)
    idx, src = sources(R, X, topk, R + N, rows)
    wide = torch.full((X, N + 8), float("nan"), dtype=x.dtype)
    wide[:, :N] = x
    i = None if idx is None else idx.to(DEV)
    got = eplb.expert_matmul16(wide.to(DEV)[:, :N], w.to(DEV), off.to(DEV), rows=i, K=topk, transpose=True,
                               dtype=TYPES[out])
    xr = taken(x, src)
    ref, absolute = torch.zeros((R, C), dtype=torch.float64), torch.zeros((R, C), dtype=torch.float64)
    for g in range(len(counts)):
        a, b = off[g], off[g + 1]
        ref[a:b] = xr[a:b] @ w[g].double()
        absolute[a:b] = xr[a:b].abs() @ w[g].double().abs()
    check(got, ref, absolute, N, "y")
    assert (got.cpu()[src < 0] == 0).all() and (got.cpu()[:head] == 0).all() and (got.cpu()[R - tail:][:tail] == 0).all()


@pytest.mark.parametrize("counts,head,tail,X,topk,N,C,dtype,out,rows",
                         [c[:5] + (-(-c[5] // 8) * 8,) + c[6:] for c in CASES[:11]] + [
                             # tiles of 256 x 256, with rows and without
                             ([70, 0, 193, 64, 1], 3, 2, 111, 3, 1288, 1800, "bf16", "f32", True),
                             ([300, 100], 0, 0, 400, 1, 2056, 2048, "f16", "f16", False)])
def test_weight_gradient(counts, head, tail, X, topk, N, C, dtype, out, rows):
    off, R = grouping(counts, head, tail)
    note("wgrad", counts[:6], head, tail, X, topk, N, C, dtype, out, rows)
    x, dy = rand((X, C), dtype, N + C), rand((R, N), dtype, R)
    idx, src = sources(R, X, topk, R + N, rows)
    if not rows and X != R:
        pytest.skip("without rows x has the grouped rows")
    lost = dy.clone()
    if rows:
        lost[src < 0] = float("nan")                                 # rows of nothing count for nothing
    lost[:head], lost[R - tail:] = float("inf"), float("inf")
    wide = torch.full((R, N + 24), float("nan"), dtype=dy.dtype)
    wide[:, 16:16 + N] = lost
    i = None if idx is None else idx.to(DEV)
    got = eplb.expert_wgrad16(wide.to(DEV)[:, 16:16 + N], x.to(DEV), off.to(DEV), rows=i, K=topk, dtype=TYPES[out])
    xr, d = taken(x, src), dy.double()
    for g in range(len(counts)):
        a, b = off[g], off[g + 1]
        check(got[g], d[a:b].t() @ xr[a:b], d[a:b].abs().t() @ xr[a:b].abs(), counts[g], g)
        if counts[g] == 0:
            assert (got[g] == 0).all()


def test_infinities_and_nan_stay_in_their_rows():
    """A row's infinity reaches that row's outputs only, a weight's that column's; past the end of a contraction nothing
    is multiplied with them."""
    g = torch.Generator().manual_seed(5)
    x, w = torch.randn((150, 72), generator=g).bfloat16(), torch.randn((1, 140, 72), generator=g).bfloat16()
    x[3, 0], x[140, 71], w[0, 7, 0], w[0, 139, 5] = float("inf"), float("nan"), float("inf"), float("nan")
    off = torch.tensor([0, 150], dtype=torch.int32, device=DEV)
    y = eplb.expert_matmul16(x.to(DEV), w.to(DEV), off).float().cpu()
    odd = torch.zeros((150, 140), dtype=torch.bool)
    odd[3], odd[140], odd[:, 7], odd[:, 139] = True, True, True, True
    assert torch.equal(~torch.isfinite(y), odd)
    keep = torch.arange(150) != 140
    want = torch.sign(x[keep, 0].float()) * float("inf")
    want[3] = float("inf") * float(torch.sign(w[0, 7, 0].float()))
    assert torch.equal(y[keep, 7], want)
    dw = eplb.expert_wgrad16(x[:, :64].contiguous().to(DEV), w[0].t().contiguous()[:, :136].repeat(3, 1)[:150].to(DEV), off)
    assert dw.shape == (1, 64, 136)
    bad = ~torch.isfinite(dw[0].float().cpu())
    assert bad[0].all() and bad[:, 7].all() and not bad[1:, :7].any() and not bad[1:, 8:136].any()


def test_offsets_that_decrease():
    """What such groups get is not defined; what lies outside the output is left alone, and the call ends."""
    x, w = torch.randn((300, 64), device=DEV).bfloat16(), torch.randn((4, 96, 64), device=DEV).bfloat16()
    off = torch.tensor([250, 10, 300, 0, 290], dtype=torch.int32, device=DEV)
    guard = torch.full((300 + 16, 96), 5.0, dtype=torch.bfloat16, device=DEV)
    eplb.expert_matmul16(x, w, off, out=guard[8:308])
    eplb.expert_wgrad16(guard[8:308], x, off)
    torch.cuda.synchronize()
    assert (guard[:8] == 5).all() and (guard[308:] == 5).all()


def test_streams_and_graph():
    """Calls on two streams at once, and a captured training step replayed with the program's own work between."""
    g = torch.Generator(device=DEV).manual_seed(3)
    x, w = torch.randn((400, 192), generator=g, device=DEV).bfloat16(), torch.randn((3, 160, 192), generator=g,
                                                                                    device=DEV).bfloat16()
    dy = torch.randn((400, 160), generator=g, device=DEV).bfloat16()
    off = torch.tensor([0, 100, 180, 400], dtype=torch.int32, device=DEV)

    def step(x, dy):
        return (eplb.expert_matmul16(x, w, off), eplb.expert_matmul16(dy, w, off, transpose=True),
                eplb.expert_wgrad16(dy, x, off))

    want, other = step(x, dy), step(x * 2, dy * 2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    twice = (x * 2, dy * 2)
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            a = step(x, dy)
        with torch.cuda.stream(s2):
            b = step(*twice)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a + b, want + other))
    xs, dys = x.clone(), dy.clone()
    graph = torch.cuda.CUDAGraph()
    step(xs, dys)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = step(xs, dys)
    for i in range(4):
        xs.copy_(x if i % 2 else twice[0])
        dys.copy_(dy if i % 2 else twice[1])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want if i % 2 else other))
        assert step(x, dy)[0].sum() == want[0].sum()
