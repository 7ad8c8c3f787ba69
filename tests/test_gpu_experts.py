"""The 8-bit block quantisers and the experts' products: HIP path against plain
implementations in 64 bits (needs an MI355X).

Quantised values are compared bit for bit with the definition's 32-bit steps.
Tolerances of a product: with A = sum of |x| |w| over the contraction, a sum of
n 32-bit operations is off by at most n * 2^-24 * A, so a 32-bit output is held
to (C + 16) * 2^-24 * A; the 8-bit matrix instruction behind a 16-bit output
keeps at least 13 bits of A's largest block sums, so that is held to 2^-13 * A
plus the rounding of its type."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

eplb = pytest.importorskip("moe_expert_load_eplb_amd")
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
B = 128


def note(*a):
    print("[experts]", *a, flush=True)


def up(n):
    return -(-n // B)


def rand(shape, dtype, seed, spread=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if spread:
        x = x * torch.exp2(torch.randint(-6, 7, shape[-1:], generator=g).float())
    return x.to(TYPES[dtype])


# ------------------------------------------------------------------ the definition, in 32-bit steps on the host
def factors(amax):
    a = torch.clamp(amax.float(), min=2.0 ** -100)
    scale = a * torch.tensor(1.0 / 448.0, dtype=torch.float32)
    return scale, (torch.ones_like(a) / a) * torch.tensor(448.0, dtype=torch.float32)


def quantized(x, rows, cols):
    """x [R, C] on the host in blocks of rows x cols: (values as float32 [R, C], scales)."""
    R, C = x.shape
    q, scale = torch.zeros((R, C)), torch.zeros((-(-R // rows), -(-C // cols)))
    for i in range(scale.shape[0]):
        for j in range(scale.shape[1]):
            b = x[i * rows:(i + 1) * rows, j * cols:(j + 1) * cols].float()
            if not torch.isfinite(b).all():
                scale[i, j] = float("nan")
                continue
            s, f = factors(b.abs().max())
            scale[i, j] = s
            q[i * rows:(i + 1) * rows, j * cols:(j + 1) * cols] = (b * f).to(torch.float8_e4m3fn).float()
    return q, scale


def same(a, b):
    return torch.equal(torch.nan_to_num(a.float().cpu(), nan=-777.0), torch.nan_to_num(b.float(), nan=-777.0))


@pytest.mark.parametrize("R,C,dtype", [(1, 1, "f32"), (3, 127, "bf16"), (5, 128, "f16"), (2, 129, "f32"), (7, 1040, "bf16"),
                                       (33, 500, "f16"), (4, 2048, "f32"), (130, 24, "bf16"), (1, 4096, "bf16")])
def test_quantize_rows(R, C, dtype):
    note("rows", R, C, dtype)
    x = rand((R, C), dtype, R * C)
    x[0, C // 2] = 0.0
    x[R - 1] = 0.0                                               # blocks of zeros
    if R > 2:
        x[1, C - 1] = float("nan")
        x[2, 0] = float("inf")
    if dtype == "f32" and R > 1:
        x[0] *= 1e-38                                            # below the least block maximum
    q, s = eplb.quantize_rows(x.to(DEV))
    rq, rs = quantized(x, 1, B)
    assert same(s, rs) and same(q, rq)
    wide = torch.zeros((R, C + 3), dtype=x.dtype)
    wide[:, 1:1 + C] = x                                         # rows that start at odd addresses
    q, s = eplb.quantize_rows(wide.to(DEV)[:, 1:1 + C])
    assert same(s, rs) and same(q, rq)


def test_quantize_ties_to_even():
    """Every midpoint of two neighbouring 8-bit values."""
    steps = [(8 + m + 0.5) * 2.0 ** e for e in range(-9, 6) for m in range(8)] + [(m + 0.5) * 2.0 ** -9 for m in range(8)]
    v = torch.tensor([x for x in steps if x < 448])
    v = torch.cat([v, -v])
    x = torch.zeros((up(v.numel()), B))
    x.view(-1)[:v.numel()] = v
    x[:, B - 1] = 448.0                                          # scale 1, or the nearest 32-bit number to it
    rq, rs = quantized(x, 1, B)
    q, s = eplb.quantize_rows(x.to(DEV))
    assert same(s, rs) and same(q, rq)


@pytest.mark.parametrize("counts,tail,C,dtype,K", [
    ([1], 0, 1, "f32", 1), ([128], 0, 64, "bf16", 1), ([129, 0, 127], 5, 65, "f16", 2), ([0, 0], 3, 40, "bf16", 1),
    ([5, 300, 0, 128, 1], 0, 200, "bf16", 4), ([1] * 70 + [200], 7, 33, "f32", 2)])
def test_quantize_columns(counts, tail, C, dtype, K):
    G, R = len(counts), sum(counts) + tail
    note("columns", counts[:5], tail, C, dtype, K)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    g = torch.Generator().manual_seed(R)
    X = max(1, R // K)
    x = rand((X, C), dtype, R + C)
    if R > 200:
        x[X // 2, C // 2] = float("inf")
    rows = torch.randint(0, X * K, (R,), generator=g, dtype=torch.int32)
    if R > 4:
        rows[1], rows[3] = -1, X * K + 5                         # rows of nothing
    q, s = eplb.quantize_columns(x.to(DEV), off.to(DEV), rows=rows.to(DEV), K=K)
    assert q.shape == (C, eplb.padded_rows(R, G))
    src = rows.long() // K
    ok = (rows >= 0) & (src < X)
    v = torch.where(ok[:, None], x.float()[src.clamp(0, X - 1)], torch.zeros(()))
    pad = 0
    for i, n in enumerate(counts):
        part = torch.zeros((up(n) * B, C))
        part[:n] = v[off[i]:off[i + 1]]
        rq, rs = quantized(part, B, 1)
        assert same(q.float()[:, pad:pad + part.shape[0]].t(), rq)
        assert same(s[pad // B:(pad + part.shape[0]) // B], rs)
        pad += part.shape[0]
    if K == 1 and tail == 0:
        q2, s2 = eplb.quantize_columns(x.to(DEV), off.to(DEV))
        q3, s3 = eplb.quantize_columns(x.to(DEV), off.to(DEV), rows=torch.arange(R, dtype=torch.int32, device=DEV))
        used = slice(0, pad)
        assert torch.equal(q2[:, used].float(), q3[:, used].float()) and torch.equal(s2[:pad // B], s3[:pad // B])


@pytest.mark.parametrize("G,N,K,dtype", [(1, 1, 1, "f32"), (2, 128, 128, "bf16"), (3, 130, 200, "f16"), (1, 257, 129, "f32"),
                                         (2, 72, 1040, "bf16"), (0, 4, 4, "f32")])
def test_quantize_weights(G, N, K, dtype):
    note("weights", G, N, K, dtype)
    w = rand((G, N, K), dtype, N * K)
    if G > 1:
        w[1, N - 1, K - 1] = float("nan")
        w[0, :B, :B] = 0
    q, s, qt, st = eplb.quantize_weights(w.to(DEV), transpose=True)
    for g in range(G):
        rq, rs = quantized(w[g], B, B)
        assert same(q[g], rq) and same(s[g], rs) and same(qt[g].float().t(), rq) and same(st[g].t(), rs)
    q2, s2 = eplb.quantize_weights(w.to(DEV))
    assert same(q2, q.float().cpu()) and same(s2, s.cpu())


# ------------------------------------------------------------------ products
def dequantized(q, s, rows, cols):
    q, s = q.double().cpu(), s.double().cpu()
    return q * s.repeat_interleave(rows, -2)[..., :q.shape[-2], :].repeat_interleave(cols, -1)[..., :q.shape[-1]]


def check(got, ref, absolute, C, what):
    t = got.dtype
    tol = (C + 16) * 2.0 ** -24 if t == torch.float32 else 2.0 ** -13
    got = got.double().cpu()
    past = ref.abs() >= torch.finfo(t).max * (1 + HALF_ULP[t])      # rounds to infinity in this type
    assert torch.equal(got[past], torch.sign(ref[past]) * torch.inf), what
    got, ref, absolute = got[~past], ref[~past], absolute[~past]
    room = tol * absolute + HALF_ULP[t] * ref.abs() + (2.0 ** -25 if t == torch.float16 else 0.0)
    bad = (got - ref).abs() > room
    assert not bad.any(), (what, bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), ref[bad][:4].tolist())


def product_case(counts, head, tail, X, topk, N, C, out, seed, rows=True):
    """Group sizes, rows before the first and behind the last group."""
    G, R = len(counts), head + sum(counts) + tail
    note("product", counts[:6], head, tail, X, topk, N, C, out, rows)
    off = torch.tensor(head + np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    x, w = rand((X, C), "bf16", seed), rand((G, N, C), "bf16", seed + 1)
    q, s = eplb.quantize_rows(x.to(DEV))
    wq, ws = eplb.quantize_weights(w.to(DEV))
    idx = None
    g = torch.Generator().manual_seed(seed)
    if rows:
        idx = torch.randint(0, max(1, X * topk), (R,), generator=g, dtype=torch.int32)
        if R > 3:
            idx[R // 2] = -1
            idx[R // 3] = X * topk
    y = torch.full((R, N), 7.0, dtype=TYPES[out], device=DEV)
    got = eplb.expert_matmul(q, s, wq, ws, off.to(DEV), rows=None if idx is None else idx.to(DEV), K=topk, out=y)
    xd, wd = dequantized(q, s, 1, B), dequantized(wq, ws, B, B)
    src = torch.arange(R) if idx is None else torch.where(idx >= 0, idx.long() // topk, -1)
    ok = (src >= 0) & (src < X)
    xr = torch.where(ok[:, None], xd[src.clamp(0, max(0, X - 1))], torch.zeros((), dtype=torch.float64)) if X else \
        torch.zeros((R, C), dtype=torch.float64)
    ref, absolute = torch.zeros((R, N), dtype=torch.float64), torch.zeros((R, N), dtype=torch.float64)
    for i in range(G):
        a, b = off[i], off[i + 1]
        ref[a:b] = xr[a:b] @ wd[i].t()
        absolute[a:b] = xr[a:b].abs() @ wd[i].abs().t()
    check(got, ref, absolute, C, (counts, N, C))
    none = torch.ones(R, dtype=torch.bool)
    none[off[0]:off[-1]] = False
    assert (got.cpu()[none | ~ok] == 0).all()


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("counts,head,tail,X,topk,N,C", [
    ([1], 0, 0, 1, 1, 1, 16), ([1], 0, 0, 3, 2, 128, 128), ([2, 0, 1], 0, 1, 4, 2, 100, 144), ([16], 0, 0, 16, 1, 64, 256),
    ([0, 0], 2, 3, 5, 1, 40, 32), ([17, 33, 64, 65], 1, 2, 50, 4, 200, 400), ([127, 128, 129], 0, 0, 100, 3, 257, 272),
    ([300], 0, 0, 300, 1, 391, 1040), ([0, 700, 3, 0, 60], 0, 9, 200, 4, 130, 528), ([1] * 80, 3, 4, 30, 3, 48, 1152),
    ([5, 9, 2, 8], 0, 0, 8, 3, 4096, 2048), ([513, 260], 0, 0, 400, 2, 512, 640)])
def test_matmul(counts, head, tail, X, topk, N, C, out):
    product_case(counts, head, tail, X, topk, N, C, out, N + C)


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_matmul_without_rows(out):
    product_case([40, 100], 0, 10, 150, 1, 300, 384, out, 3, rows=False)
    product_case([140], 0, 0, 140, 1, 96, 4096, out, 4, rows=False)
    product_case([30], 0, 20, 50, 1, 96, 128, out, 5, rows=False)
    product_case([3, 5], 0, 0, 0, 1, 70, 64, out, 6)             # an operand without rows


@pytest.mark.parametrize("M", [1, 3, 16, 31, 48, 64, 90, 128, 200, 256, 300, 384, 700, 1500])
@pytest.mark.parametrize("N,C", [(272, 1040), (1000, 128), (129, 400)])
def test_matmul_rows_of_one_group(M, N, C):
    """Every form of the kernel that the number of rows selects, at sizes that fill no tile."""
    product_case([M], 0, 0, M, 1, N, C, "bf16", M + N, rows=False)


def test_matmul_offsets_out_of_range():
    """Offsets outside 0 .. R are clamped, a group that ends before it starts is empty."""
    x, w = rand((50, 128), "bf16", 1), rand((3, 64, 128), "bf16", 2)
    q, s = eplb.quantize_rows(x.to(DEV))
    wq, ws = eplb.quantize_weights(w.to(DEV))
    wild = eplb.expert_matmul(q, s, wq, ws, torch.tensor([-5, 20, 20, 900], dtype=torch.int32, device=DEV))
    tame = eplb.expert_matmul(q, s, wq, ws, torch.tensor([0, 20, 20, 50], dtype=torch.int32, device=DEV))
    assert torch.equal(wild, tame)


def test_matmul_not_finite():
    """A block that is not finite makes its own outputs NaN and no others."""
    x, w = rand((40, 256), "bf16", 1), rand((2, 200, 256), "bf16", 2)
    x[3, 200] = float("inf")
    w[1, 130, 7] = float("nan")
    q, s = eplb.quantize_rows(x.to(DEV))
    wq, ws = eplb.quantize_weights(w.to(DEV))
    off = torch.tensor([0, 20, 40], dtype=torch.int32, device=DEV)
    for t in (torch.float32, torch.bfloat16):
        bad = torch.isnan(eplb.expert_matmul(q, s, wq, ws, off, dtype=t)).cpu()
        want = torch.zeros((40, 200), dtype=torch.bool)
        want[3] = True
        want[20:, 128:] = True
        assert torch.equal(bad, want)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("counts,tail,N,C", [([1], 0, 1, 1), ([128], 0, 128, 128), ([0, 5], 2, 40, 16), ([300, 0, 129, 7], 0, 130, 200),
                                             ([1000], 3, 257, 65), ([1] * 70, 0, 16, 24), ([640, 64], 0, 300, 520)])
def test_wgrad(counts, tail, N, C, out):
    G, R = len(counts), sum(counts) + tail
    note("wgrad", counts[:5], tail, N, C, out)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    x, dy = rand((R, C), "bf16", R), rand((R, N), "bf16", R + 1)
    xq, xs = eplb.quantize_columns(x.to(DEV), off.to(DEV))
    dq, ds = eplb.quantize_columns(dy.to(DEV), off.to(DEV))
    got = eplb.expert_wgrad(dq, ds, xq, xs, off.to(DEV), dtype=TYPES[out])
    xd, dd = dequantized(xq.t(), xs, B, 1), dequantized(dq.t(), ds, B, 1)
    pad = 0
    for i, n in enumerate(counts):
        m = up(n) * B
        a, b = dd[pad:pad + m], xd[pad:pad + m]
        check(got[i], a.t() @ b, a.abs().t() @ b.abs(), m, (counts, i))
        pad += m


def test_gradients_against_differences():
    """The products' gradients are those of sum(dy * y): differences of the
    64-bit objective along random directions, and the formula, within the
    8-bit rounding of their operands (one part in 16 each, independent)."""
    counts, N, C = [40, 0, 150, 3], 144, 208
    R, G = sum(counts), len(counts)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    x, w, dy = rand((R, C), "f32", 1, False), rand((G, N, C), "f32", 2, False), rand((R, N), "f32", 3, False)
    wq, ws, wqt, wst = eplb.quantize_weights(w.to(DEV), transpose=True)
    dq, ds = eplb.quantize_rows(dy.to(DEV))
    dx = eplb.expert_matmul(dq, ds, wqt, wst, off.to(DEV), dtype=torch.float32).double().cpu()
    xc, dc = eplb.quantize_columns(x.to(DEV), off.to(DEV)), eplb.quantize_columns(dy.to(DEV), off.to(DEV))
    dw = eplb.expert_wgrad(*dc, *xc, off.to(DEV)).double().cpu()

    def objective(x, w):
        return sum(((x[off[i]:off[i + 1]] @ w[i].t()) * dy[off[i]:off[i + 1]].double()).sum() for i in range(G))

    x64, w64 = x.double(), w.double()
    rdx, rdw = torch.zeros_like(x64), torch.zeros_like(w64)
    for i in range(G):
        a, b = off[i], off[i + 1]
        rdx[a:b] = dy[a:b].double() @ w64[i]
        rdw[i] = dy[a:b].double().t() @ x64[a:b]
    # two operands, each off by at most 1/16 and by 2.6 % rms of a value
    assert (dx - rdx).norm() < 0.06 * rdx.norm() and (dw - rdw).norm() < 0.06 * rdw.norm()
    g = torch.Generator().manual_seed(9)
    for grad, ref, at, other in ((dx, rdx, 0, None), (dw, rdw, 1, None)):
        for _ in range(3):
            d = torch.randn(ref.shape, generator=g, dtype=torch.float64)
            hi = objective(x64 + 1e-4 * d, w64) if at == 0 else objective(x64, w64 + 1e-4 * d)
            lo = objective(x64 - 1e-4 * d, w64) if at == 0 else objective(x64, w64 - 1e-4 * d)
            slope = float(hi - lo) / 2e-4
            assert abs(float((ref * d).sum()) - slope) < 1e-6 * float(ref.norm() * d.norm())
            assert abs(float((grad * d).sum()) - slope) < 0.06 * 4 * float(ref.norm())   # 4 deviations


def test_matmul_past_32_bits():
    """Operands and outputs past 2^31 bytes."""
    C, N = 4096, 64
    X = (1 << 31) // C + 1000
    note("large operand", X, C)
    q = torch.zeros((X, C), dtype=torch.uint8, device=DEV)
    s = torch.ones((X, C // B), dtype=torch.float32, device=DEV)
    x = rand((8, C), "bf16", 1, False)
    q[-8:], s[-8:] = (t.view(torch.uint8) if t.dtype == eplb.F8 else t for t in eplb.quantize_rows(x.to(DEV)))
    w = rand((1, N, C), "bf16", 2, False)
    wq, ws = eplb.quantize_weights(w.to(DEV))
    rows = torch.arange(X - 8, X, dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    got = eplb.expert_matmul(q, s, wq, ws, off, rows=rows)
    small = eplb.expert_matmul(*eplb.quantize_rows(x.to(DEV)), wq, ws, off)
    assert torch.equal(got, small) and small.abs().sum() > 0
    del q, s
    R, N, C = 70000, 32768, 32
    note("large output", R, N)
    x, w = rand((R, C), "bf16", 3, False), rand((1, N, C), "bf16", 4, False)
    q, s = eplb.quantize_rows(x.to(DEV))
    wq, ws = eplb.quantize_weights(w.to(DEV))
    y = eplb.expert_matmul(q, s, wq, ws, torch.tensor([0, R], dtype=torch.int32, device=DEV))
    part = eplb.expert_matmul(q[-300:].contiguous(), s[-300:].contiguous(), wq, ws,
                              torch.tensor([0, 300], dtype=torch.int32, device=DEV))
    assert torch.equal(y[-300:], part)


def test_streams_and_graph():
    """The calls on another stream, and replays of a captured graph between the
    program's own work, against the eager results."""
    T, E, K, P, C, N = 48, 32, 4, 40, 256, 192
    g = torch.Generator(device=DEV).manual_seed(3)
    logits = torch.randn((T, E), generator=g, device=DEV)
    x = torch.randn((T, C), generator=g, device=DEV).bfloat16()
    w = torch.randn((E, N, C), generator=g, device=DEV).bfloat16()
    seg = torch.tensor([0, 20, T], dtype=torch.int32, device=DEV)
    wq, ws = eplb.quantize_weights(w)

    def step():
        ids, weights, loss, counts, prob, tokens = eplb.gate_loss(logits, K, seg, 0.1)
        off, order, place = eplb.group_rows(ids.view(1, T, K), E)
        q, s = eplb.quantize_rows(x)
        y = eplb.expert_matmul(q, s, wq, ws, off[0], rows=order[0], K=K)
        dl = eplb.gate_backward(logits, ids, weights, seg=seg, alpha=0.1, counts=counts, tokens=tokens, d_loss=loss)
        xc = eplb.quantize_columns(x, off[0], rows=order[0], K=K)
        yc = eplb.quantize_columns(y, off[0])
        return [ids, weights, loss, counts, off, order, place, y, dl, eplb.expert_wgrad(*yc, *xc, off[0])]

    eager = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        for t in held:
            t.zero_()
        if i == 2:
            logits.copy_(torch.randn((T, E), generator=g, device=DEV))
            eager = [t.clone() for t in step()]
            for t in held:
                t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, held)), i


def test_matmul_large_form():
    """The 8-bit matrix instruction behind large 16-bit products.  Within each
    8 consecutive k its products are aligned to the largest one and what lies
    below 2^-13 of that is lost, at most 7 times; sums of the groups of 8 are
    32-bit: the bound below, computed for a sample of rows and columns."""
    counts, head, tail, N, C = [701, 0, 590], 3, 5, 1101, 6416
    R = head + sum(counts) + tail
    note("large form", counts, N, C)
    off = torch.tensor(head + np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    x, w = rand((R, C), "bf16", 1), rand((3, N, C), "bf16", 2)
    q, s = eplb.quantize_rows(x.to(DEV))
    wq, ws = eplb.quantize_weights(w.to(DEV))
    g = torch.Generator().manual_seed(5)
    rows = torch.randperm(R, generator=g).to(torch.int32)
    rows[50], rows[900] = -1, R
    for t in (torch.bfloat16, torch.float16):
        y = eplb.expert_matmul(q, s, wq, ws, off.to(DEV), rows=rows.to(DEV), dtype=t).double().cpu()
        assert (y[:head] == 0).all() and (y[R - tail:] == 0).all() and (y[50] == 0).all() and (y[900] == 0).all()
        for i, pick in ((0, [3, 4, 130, 258, 259, 300, 703]), (2, [704, 705, 831, 960, 1200, 1293])):
            cols = torch.tensor([0, 1, 31, 32, 127, 128, 255, 256, 511, 700, 1023, 1024, 1099, 1100])
            src = rows[torch.tensor(pick)].long()
            xd = dequantized(q[src.to(DEV)], s[src.to(DEV)], 1, B)
            wd = dequantized(wq[i], ws[i], B, B)[cols]
            p = xd[:, None, :] * wd[None, :, :]
            ref = p.sum(2)
            lost = 7 * 2.0 ** -13 * p.abs().view(*ref.shape, C // 8, 8).amax(3).sum(2)
            room = lost + (C + 16) * 2.0 ** -24 * p.abs().sum(2) + HALF_ULP[t] * (ref.abs() + lost)
            got = y[torch.tensor(pick)][:, cols]
            past = ref.abs() > torch.finfo(t).max * 0.99
            assert ((got - ref).abs()[~past] <= room[~past]).all()


def test_wgrad_large_form():
    counts, N, C = [3000, 1, 4000], 1301, 1104
    R = sum(counts)
    note("large weight gradient", counts, N, C)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    x, dy = rand((R, C), "bf16", 1), rand((R, N), "bf16", 2)
    xq, xs = eplb.quantize_columns(x.to(DEV), off.to(DEV))
    dq, ds = eplb.quantize_columns(dy.to(DEV), off.to(DEV))
    got = eplb.expert_wgrad(dq, ds, xq, xs, off.to(DEV))
    xd, dd = dequantized(xq.t(), xs, B, 1).to(DEV), dequantized(dq.t(), ds, B, 1).to(DEV)
    pad = 0
    for i, n in enumerate(counts):
        m = up(n) * B
        a, b = dd[pad:pad + m], xd[pad:pad + m]
        check(got[i], (a.t() @ b).cpu(), (a.abs().t() @ b.abs()).cpu(), m, i)
        pad += m


@pytest.mark.parametrize("counts", [[1] * 7, [0, 0, 5, 0, 2, 0, 0], [0] * 20 + [19, 0, 1], [0, 1, 0]])
@pytest.mark.parametrize("N,C", [(70, 1024), (200, 2064)])
def test_matmul_few_rows_of_many_groups(counts, N, C):
    """As one token's choices make them, also where they fall on one group."""
    product_case(counts, 0, 0, sum(counts), 1, N, C, "f32", N, rows=False)
    product_case(counts, 0, 0, sum(counts), 1, N, C, "bf16", N + 1, rows=False)


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_matmul_wide_tiles(out):
    """Many rows and 32-bit sums: the tolerance of 32-bit sums, over tiles that
    groups, N and K leave unfilled."""
    product_case([701, 0, 2500], 3, 5, 3300, 1, 1101, 416, out, 7)


def test_matmul_large_tiles():
    """test_matmul_large_form's bound at a size of more tiles."""
    counts, N, C = [1201, 0, 1399], 2310, 1440
    R = sum(counts)
    note("large tiles", counts, N, C)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    x, w = rand((R, C), "bf16", 1), rand((3, N, C), "bf16", 2)
    q, s = eplb.quantize_rows(x.to(DEV))
    wq, ws = eplb.quantize_weights(w.to(DEV))
    t = torch.bfloat16
    y = eplb.expert_matmul(q, s, wq, ws, off.to(DEV), dtype=t).double().cpu()
    for i, pick in ((0, [0, 31, 32, 255, 256, 1023, 1200]), (2, [1201, 1456, 1457, 2224, 2225, 2599])):
        cols = torch.tensor([0, 1, 31, 32, 127, 128, 255, 256, 1000, 2047, 2048, 2303, 2304, 2309])
        src = torch.tensor(pick)
        xd = dequantized(q[src.to(DEV)], s[src.to(DEV)], 1, B)
        wd = dequantized(wq[i], ws[i], B, B)[cols]
        p = xd[:, None, :] * wd[None, :, :]
        ref = p.sum(2)
        lost = 7 * 2.0 ** -13 * p.abs().view(*ref.shape, C // 8, 8).amax(3).sum(2)
        room = lost + (C + 16) * 2.0 ** -24 * p.abs().sum(2) + HALF_ULP[t] * (ref.abs() + lost)
        assert ((y[src][:, cols] - ref).abs() <= room).all()


def test_wgrad_few_rows_of_large_outputs():
    """Large tiles with one block, none, and groups that end inside it."""
    counts, N, C = [0, 1, 130, 0, 64], 1030, 1300
    R = sum(counts)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    x, dy = rand((R, C), "bf16", 1), rand((R, N), "bf16", 2)
    xq, xs = eplb.quantize_columns(x.to(DEV), off.to(DEV))
    dq, ds = eplb.quantize_columns(dy.to(DEV), off.to(DEV))
    got = eplb.expert_wgrad(dq, ds, xq, xs, off.to(DEV))
    xd, dd = dequantized(xq.t(), xs, B, 1), dequantized(dq.t(), ds, B, 1)
    pad = 0
    for i, n in enumerate(counts):
        m = up(n) * B
        a, b = dd[pad:pad + m], xd[pad:pad + m]
        check(got[i], a.t() @ b, a.abs().t() @ b.abs(), m, (counts, i))
        pad += m
