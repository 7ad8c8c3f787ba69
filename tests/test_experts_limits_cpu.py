"""Size limits of the quantisers and the experts' products, on a machine without
a GPU: each is refused on the host with the documented code, and a size inside
the limits gets past them (to the refusal of a NULL array behind them)."""
from __future__ import annotations

import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "moe_expert_load_eplb_amd", "libeplb.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libeplb.so not built")

F = [0x100000 * (i + 1) for i in range(16)]    # never dereferenced: every call below fails validation first
ARG, LIMIT = 1, 5
B = 128


@pytest.fixture(scope="module")
def lib():
    import moe_expert_load_eplb_amd as m
    return m.lib


def columns(lib, C, R, G, Rp, q=F[3]):
    return lib.eplb_quantize_columns(F[0], 1, C, 10, C, None, R, 1, F[2], G, Rp, q, F[4], None)


def wgrad(lib, N, K, R, G, Rp, dw=F[5]):
    return lib.eplb_expert_wgrad(F[0], F[1], F[2], F[3], F[4], G, R, Rp, N, K, 0, dw, None)


@pytest.mark.parametrize("Rp", [(1 << 32) + B, 1 << 40, 1 << 56, 1 << 62, (1 << 63) - B])
def test_padded_rows_past_their_limit(lib, Rp):
    """Among them such as make the arrays' bytes wrap in 64 bits."""
    for n in (1, 96, 1 << 10, 1 << 24):
        assert columns(lib, n, 300, 4, Rp) == LIMIT
        assert wgrad(lib, n, 1, 300, 4, Rp) == LIMIT
        assert wgrad(lib, 1, n, 300, 4, Rp) == LIMIT


def test_blocks_of_columns(lib):
    """2^23 - 1 workgroups of 128 rows and 128 columns."""
    most = (1 << 23) - 1
    for C, blocks in ((1, most), (128, most), (129, most // 2), (4096, most // 32)):
        assert columns(lib, C, 300, 4, blocks * B, q=None) == ARG
        assert columns(lib, C, 300, 4, (blocks + 1) * B) == LIMIT


def test_tiles_of_a_weight_gradient(lib):
    """2^23 - 1 workgroups of the tiles that the sizes get: 256 x 128 here."""
    for G, N, K in ((256, 16384, 16384), (8191, 128, 1024 * 256), (1, 128, 1 << 24)):
        assert wgrad(lib, N, K, 300, G, 300 // B * B + G * B, dw=None) == ARG
    for G, N, K in ((8192, 128, 1024 * 256), (8192, 1 << 24, 1 << 24), (1 << 8, 1 << 15, 1 << 15)):
        assert wgrad(lib, N, K, 300, G, 300 // B * B + G * B) == LIMIT
