"""The experts' products for few rows to a group, 16-bit and 4-bit weights: HIP
path against plain sums in 64 bits (needs an MI355X).

The cases go through every number of rows that a tile of this form may have, and
from one set of outputs to a workgroup to eight, K shared and not shared among
its waves.  Tolerances: a product of a 16-bit value and a weight (or, in half
precision, a 4-bit weight without its scale) is exact in 32 bits; a sum of n of
them takes at most n additions and one multiplication by a power of two for every
32, each off by 2^-23 of sum |x| |w| at most: (n + n / 32 + 16) * 2^-23 *
sum |x| |w|, and an output of fewer bits its half step more."""
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
    print("[linear few]", *a, flush=True)


def rand(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * torch.exp2(torch.randint(-3, 4, shape[-1:], generator=g).float())).to(
        TYPES[dtype])


def weights(four, G, N, C, dtype, seed):
    """(what the call takes, the weights in 64 bits)"""
    if not four:
        w = rand((G, N, C), dtype, seed)
        return (w.to(DEV),), w.double()
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 256, (G, N, C // 2), generator=g, dtype=torch.uint8)
    s = torch.randint(100, 131, (G, N, C // 32), generator=g, dtype=torch.uint8)
    code = torch.stack([q.long() & 15, q.long() >> 4], -1).view(G, N, C)
    v = torch.cat([VALUES, -VALUES])[code].view(G, N, C // 32, 32) * torch.exp2(s.double() - 127).unsqueeze(-1)
    return (q.to(DEV), s.to(DEV)), v.view(G, N, C)


def product(four, x, w, off, **kw):
    return eplb.expert_matmul4(x, *w, off, **kw) if four else eplb.expert_matmul16(x, *w, off, **kw)


def check(got, ref, absolute, n, what):
    t = got.dtype
    got = got.double().cpu()
    tiny = 2.0 ** -25 if t == torch.float16 else 0.0                # half a step below float16's normal numbers
    room = (n + n / 32 + 16) * 2.0 ** -23 * absolute
    room = room + torch.finfo(t).eps / 2 * (ref.abs() + room) + tiny
    past = ref.abs() + room > torch.finfo(t).max                     # may round to infinity
    bad = ((got - ref).abs() > room) & ~past
    assert not bad.any(), (what, bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), ref[bad][:4].tolist())


@pytest.mark.parametrize("four,dtype", [(False, "bf16"), (False, "f16"), (True, "bf16"), (True, "f16")])
@pytest.mark.parametrize("counts,head,tail,topk,N,C,out", [
    # a token, wide outputs and narrow ones
    ([0, 1, 0, 1, 1, 0], 0, 0, 3, 24, 64, "f32"),
    ([1] * 8 + [0] * 24, 0, 0, 8, 2049, 96, "f32"),
    ([1] * 16, 0, 0, 2, 6000, 32, "bf16"),
    # up to 16 rows: a run of K longer than a stage, K shared by eight waves, four, two and none
    ([16, 1, 15, 0], 0, 0, 1, 17, 4128, "f32"),
    ([9, 16, 11, 2], 2, 1, 2, 776, 1056, "f16"),
    ([7] * 9, 0, 3, 1, 1391, 544, "f32"),
    ([8] * 33, 1, 0, 2, 1032, 160, "bf16"),
    # up to 32, 64 and (16-bit weights) 128 rows, and more than that in one group of many
    ([28, 31, 17, 32, 33, 2], 0, 0, 2, 700, 288, "f32"),
    ([27, 26, 25, 24, 23, 22, 20, 19], 3, 5, 1, 2600, 64, "f16"),
    ([57, 64, 44, 65, 40], 0, 0, 2, 333, 416, "f32"),
    ([50] * 9, 0, 0, 1, 2050, 96, "bf16"),
    ([80, 96, 101, 70, 85], 0, 2, 1, 520, 224, "f32"),
    ([90, 85, 60, 128, 91, 76, 80, 70], 0, 0, 2, 2100, 64, "f32"),
    ([300, 0, 0, 0, 1, 0, 0, 0], 0, 0, 1, 130, 160, "f32")])
def test_product(four, dtype, counts, head, tail, topk, N, C, out):
    G, R = len(counts), head + sum(counts) + tail
    note("product", four, dtype, counts[:6], head, tail, topk, N, C, out)
    off = torch.tensor(head + np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    X = R // topk + 1
    idx = torch.randint(0, X * topk, (R,), generator=torch.Generator().manual_seed(R), dtype=torch.int32)
    if R > 3:
        idx[R // 2], idx[R // 3] = -1, X * topk
    src = torch.where(idx >= 0, idx.long() // topk, -1)
    src = torch.where(src < X, src, -1)
    x = rand((X, C), dtype, N + C)
    wide = torch.full((X, C + 8), float("nan"), dtype=x.dtype)
    wide[:, :C] = x
    w, values = weights(four, G, N, C, dtype, N)
    whole = torch.full((R * N + 128,), 7.0, dtype=TYPES[out], device=DEV)
    y = product(four, wide.to(DEV)[:, :C], w, off.to(DEV), rows=idx.to(DEV), K=topk, out=whole[64:64 + R * N].view(R, N))
    xr = torch.zeros((R, C), dtype=torch.float64)
    xr[src >= 0] = x.double()[src[src >= 0]]
    ref, absolute = torch.zeros((R, N), dtype=torch.float64), torch.zeros((R, N), dtype=torch.float64)
    for i in range(G):
        a, b = off[i], off[i + 1]
        ref[a:b] = xr[a:b] @ values[i].t()
        absolute[a:b] = xr[a:b].abs() @ values[i].abs().t()
    check(y, ref, absolute, C, "y")
    none = src < 0
    none[:head] = True
    none[R - tail:] = True
    assert (y.cpu()[none] == 0).all() and (whole[:64] == 7).all() and (whole[64 + R * N:] == 7).all()


@pytest.mark.parametrize("four,dtype", [(False, "bf16"), (True, "bf16"), (True, "f16")])
def test_odd_groups(four, dtype):
    """Offsets that decrease or lie outside: nothing is written outside the output."""
    G, N, C, R = 6, 80, 96, 50
    off = torch.tensor([0, 9, 4, 30, 30, -7, 400], dtype=torch.int32)
    x = rand((R, C), dtype, 3)
    w, _ = weights(four, G, N, C, dtype, 4)
    whole = torch.full((R + 8, N), 7.0, dtype=torch.float32, device=DEV)
    product(four, x.to(DEV), w, off.to(DEV), out=whole[4:R + 4])
    note("odd groups", four, dtype)
    torch.cuda.synchronize()
    assert (whole[:4] == 7).all() and (whole[R + 4:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_scale(dtype):
    """Every scale byte, K in several stages: what a 32-bit number can hold is exact, 255 is NaN.  3 * 2^127 (254) is past
    32 bits: an infinity, and against a bfloat16 zero NaN."""
    C = 2080
    x = torch.zeros((2, C), dtype=TYPES[dtype], device=DEV)
    x[1, 40] = 1.0
    q = torch.zeros((1, 256, C // 2), dtype=torch.uint8)
    q[:, :, 20] = 0x05                                               # element 40: 3
    s = torch.full((1, 256, C // 32), 127, dtype=torch.uint8)
    s[0, :, 1] = torch.arange(256, dtype=torch.uint8)
    off = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    y = eplb.expert_matmul4(x, q.to(DEV), s.to(DEV), off, dtype=torch.float32).cpu().double()
    want = 3.0 * torch.exp2(torch.arange(256, dtype=torch.float64) - 127)
    assert torch.isnan(y[:, 255]).all() and (y[0, :254] == 0).all()
    assert torch.equal(y[1, 2:254], want[2:254]) and (y[1, :2] <= want[:2]).all() and torch.isinf(y[1, 254])


def test_replayed():
    """A captured product gives the same bits on every replay, whatever ran between."""
    G, N, C = 9, 520, 1056
    off = torch.tensor([0, 3, 3, 20, 21, 40, 40, 60, 70, 90], dtype=torch.int32, device=DEV)
    x = rand((90, C), "f16", 1).to(DEV)
    w16, _ = weights(False, G, N, C, "f16", 2)
    w4, _ = weights(True, G, N, C, "f16", 3)
    want = product(False, x, w16, off), product(True, x, w4, off)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = product(False, x, w16, off), product(True, x, w4, off)
    for _ in range(3):
        for t in got:
            t.zero_()
        product(True, x[:7], w4, off.clamp(max=7))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
