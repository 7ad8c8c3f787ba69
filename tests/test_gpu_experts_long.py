"""The weight gradient where an operand's row of padded rows is longer than
2^24 bytes: its rows are then more than 2^32 bytes from the first one of a tile
(needs an MI355X).

The same few rows in long arrays and in short ones have to give equal bits; the
rest of the long arrays is never read."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

eplb = pytest.importorskip("moe_expert_load_eplb_amd")
DEV = torch.device("cuda:0")
B = 128


@pytest.mark.parametrize("G,N,C,Rp", [
    (160, 8, 256, 16843136),     # 255 rows of 16,843,136 bytes: past 2^32 by the large tiles
    (3, 9, 64, 68200064)])       # 63 rows of 68,200,064 bytes, by the small ones
def test_weight_gradient_of_long_rows(G, N, C, Rp):
    print("[long]", G, N, C, Rp, flush=True)
    counts = [130, 0, 100] + [0] * (G - 3)
    R = sum(counts)
    off = torch.tensor([sum(counts[:i]) for i in range(G + 1)], dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(G)
    x = torch.randn((R, C), generator=g, device=DEV).bfloat16()
    dy = torch.randn((R, N), generator=g, device=DEV).bfloat16()
    xq, xs = eplb.quantize_columns(x, off)
    dq, ds = eplb.quantize_columns(dy, off)
    want = eplb.expert_wgrad(dq, ds, xq, xs, off, R=R)
    assert (want[0] != 0).any() and (want[2] != 0).any()

    def lengthened(q, s):
        used = 3 * B                                    # 130 rows take two blocks, 100 one
        lq = torch.zeros((q.shape[0], Rp), dtype=torch.uint8, device=DEV)
        lq[:, :used] = q[:, :used].view(torch.uint8)
        ls = torch.zeros((Rp // B, s.shape[1]), dtype=torch.float32, device=DEV)
        ls[:used // B] = s[:used // B]
        return lq, ls

    got = eplb.expert_wgrad(*lengthened(dq, ds), *lengthened(xq, xs), off, R=R)
    assert torch.equal(got, want)
