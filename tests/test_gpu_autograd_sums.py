"""The gradient of expert_linear's rows: a token's K rows are summed in 32 bits and
rounded once (needs an MI355X).

Tolerance.  A product of N terms and the sum of K of them are N + K 32-bit
operations, off by at most (N + K + 16) * 2^-24 * A with A the sum of all
magnitudes; the result is rounded once, by half a unit of its type."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

eplb = pytest.importorskip("moe_expert_load_eplb_amd")
DEV = torch.device("cuda:0")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
B = 128


@pytest.mark.parametrize("T,K,G,C,N,dtype", [(1, 1, 1, 16, 16, "bf16"), (9, 4, 6, 144, 80, "bf16"), (200, 8, 16, 256, 304, "f16"),
                                             (70, 3, 5, 1040, 144, "f32"), (333, 2, 4, 528, 1024, "bf16")])
def test_gradient_of_a_token(T, K, G, C, N, dtype):
    from moe_expert_load_eplb_amd.autograd import expert_linear
    print("[autograd]", T, K, G, C, N, dtype, flush=True)
    g = torch.Generator(device=DEV).manual_seed(T + C)
    ids = torch.rand((T, G), generator=g, device=DEV).topk(K, dim=1).indices.int()
    ids[T // 2, K - 1] = -1                             # a choice of no expert
    off, order, place = (t[0] for t in eplb.group_rows(ids.view(1, T, K), G))
    x = torch.randn((T, C), generator=g, device=DEV).to(TYPES[dtype]).requires_grad_(True)
    w = torch.randn((G, N, C), generator=g, device=DEV).to(TYPES[dtype])
    dy = torch.randn((T * K, N), generator=g, device=DEV).to(TYPES[dtype])
    dx, = torch.autograd.grad(expert_linear(x, w, off, order, place, K), x, dy)
    assert dx.dtype == TYPES[dtype]
    q, s = eplb.quantize_rows(dy)
    wq, ws = eplb.quantize_weights(w)
    dyd = q.double() * s.double().repeat_interleave(B, 1)[:, :N]
    wd = wq.double() * ws.double().repeat_interleave(B, 1)[:, :N].repeat_interleave(B, 2)[:, :, :C]
    ref, size = (torch.zeros((T, C), dtype=torch.float64, device=DEV) for _ in range(2))
    for e in range(G):
        a, b = int(off[e]), int(off[e + 1])
        token = order[a:b].long() // K
        ref.index_add_(0, token, dyd[a:b] @ wd[e])
        size.index_add_(0, token, dyd[a:b].abs() @ wd[e].abs())
    sums = (N + K + 16) * 2.0 ** -24 * size
    room = sums + HALF_ULP[dtype] * (ref.abs() + sums) + (2.0 ** -25 if dtype == "f16" else 0.0)
    err = (dx.double() - ref).abs()
    assert (err <= room).all(), float((err / room.clamp(min=1e-300)).max())
