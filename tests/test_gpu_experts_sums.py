"""Sums of the experts' products with a 16-bit output are 32-bit at every size
(needs an MI355X).

Tolerances.  A sum of C 32-bit operations is off by at most (C + 16) * 2^-24 *
A, with A = sum of |x| |w|; then the output is rounded once, by at most half a
unit of its type.  Where every partial sum is a multiple of 0.5 below 2^23 it
has 24 bits at most and nothing may be lost at all."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

eplb = pytest.importorskip("moe_expert_load_eplb_amd")
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
B = 128


def one_scale(*shape):
    return torch.ones(shape, dtype=torch.float32, device=DEV)


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R,N,C", [(1, 64, 1536), (40, 100, 1536), (300, 257, 1536), (2560, 2560, 1536), (4100, 1111, 2064)])
def test_small_terms_beside_large_ones_that_cancel(R, N, C, out):
    """Every other eight of k holds one product of 2^16, the next eight its
    negative; all the others are 0.5, 1 or 2 in magnitude.  The large ones leave
    nothing, so the result is the sum of the small ones, exactly."""
    print("[sums]", R, N, C, out, flush=True)
    g = torch.Generator(device=DEV).manual_seed(R + N)

    def operand(rows, values):
        pick = torch.randint(0, len(values), (rows, C), generator=g, device=DEV)
        return torch.tensor(values, device=DEV)[pick]

    x, w = operand(R, [-2.0, -1.0, 1.0, 2.0]), operand(N, [-1.0, -0.5, 0.5, 1.0])
    x[:, 0::16], x[:, 8::16], w[:, 0::8] = 256.0, -256.0, 256.0
    y = eplb.expert_matmul(x.to(eplb.F8), one_scale(R, -(-C // B)), w.to(eplb.F8).view(1, N, C),
                           one_scale(1, -(-N // B), -(-C // B)), torch.tensor([0, R], dtype=torch.int32, device=DEV),
                           dtype=TYPES[out])
    ref = x.double() @ w.double().t().contiguous()
    assert ref.abs().max() < 2048                       # exact in 32 bits, so that one rounding follows
    assert torch.equal(y, ref.float().to(TYPES[out]))


@pytest.mark.parametrize("out", ["bf16", "f16"])
@pytest.mark.parametrize("counts,N,C", [([3], 70, 400), ([0, 60, 200], 130, 1040), ([700, 0, 2500], 1101, 416),
                                        ([2700], 2500, 1440), ([1500, 0, 1700, 3], 1700, 2400)])
def test_sums_of_16_bit_outputs(counts, N, C, out):
    """Random values over twelve powers of two, at the tolerance of 32-bit sums."""
    print("[sums]", counts, N, C, out, flush=True)
    G, R = len(counts), sum(counts)
    g = torch.Generator(device=DEV).manual_seed(N + C)

    def operand(*shape):
        v = torch.randn(shape, generator=g, device=DEV)
        return v * torch.exp2(torch.randint(-6, 7, shape[-1:], generator=g, device=DEV).float())

    # outputs below a few thousand, inside the range of both types
    q, s = eplb.quantize_rows(operand(R, C) * 0.02)
    wq, ws = eplb.quantize_weights(operand(G, N, C) * 0.02)
    off = torch.tensor([sum(counts[:i]) for i in range(G + 1)], dtype=torch.int32, device=DEV)
    y = eplb.expert_matmul(q, s, wq, ws, off, dtype=TYPES[out]).double()
    x = q.double() * s.double().repeat_interleave(B, 1)[:, :C]
    for i in range(G):
        a, b = int(off[i]), int(off[i + 1])
        w = wq[i].double() * ws[i].double().repeat_interleave(B, 0)[:N].repeat_interleave(B, 1)[:, :C]
        wt = w.t().contiguous()
        ref, sums = x[a:b] @ wt, (C + 16) * 2.0 ** -24 * (x[a:b].abs() @ wt.abs())
        room = sums + HALF_ULP[out] * (ref.abs() + sums) + (2.0 ** -25 if out == "f16" else 0.0)
        assert ((y[a:b] - ref).abs() <= room).all(), (i, float(((y[a:b] - ref).abs() / room).max()))
