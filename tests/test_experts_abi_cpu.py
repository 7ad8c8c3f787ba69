"""The entry points of include/eplb_experts.h on a machine without a GPU: all
are exported, the header is C99, and every call refuses bad arguments on the
host with the documented codes before it touches the device."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "eplb_experts.h")
LIB = os.path.join(ROOT, "moe_expert_load_eplb_amd", "libeplb.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libeplb.so not built")

F = [0x100000 * (i + 1) for i in range(16)]    # never dereferenced: every call below fails validation first
ARG, DIV, LIMIT, RANGE = 1, 2, 5, 6


@pytest.fixture(scope="module")
def eplb():
    import moe_expert_load_eplb_amd as m
    return m


def refuses(fn, good, cases):
    for pos, bad, code in cases:
        args = list(good)
        for p, b in zip(pos if isinstance(pos, tuple) else (pos,), bad if isinstance(bad, tuple) else (bad,)):
            args[p] = b
        assert fn(*args) == code, (pos, bad)


def test_exports_and_constants(eplb):
    text = open(HEADER).read()
    names = re.findall(r"^\s*[a-z_0-9]+\s+(eplb_[a-z_0-9]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S), flags=re.M)
    assert len(names) == 12 and set(names) <= set(eplb.EXPORTS)
    for k, v in re.findall(r"#define\s+(EPLB_[A-Z_0-9]+)\s+(\d+)", text):
        assert getattr(eplb, k) == int(v)


def test_header_is_c99(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "eplb_experts.h"\nint main(void) { return eplb_gate_loss_workspace_bytes(0, 0, 1) == -EPLB_E_ARG'
                   " ? 0 : 1; }\n")
    exe = str(tmp_path / "h")
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src),
                    "-o", exe, "-L", os.path.dirname(LIB), "-leplb", "-Wl,-rpath," + os.path.dirname(LIB)], check=True)
    assert subprocess.run([exe]).returncode == 0


def test_gate_refusals(eplb):
    # logits, dtype, ld, T, E, K, scoring, bias, G, top_groups, group_top, normalize, scale, mask, ids, weights, stream
    good = [F[0], 1, 256, 10, 256, 8, 0, F[1], 8, 4, 2, 1, 1.0, F[2], F[3], F[4], None]
    refuses(eplb.lib.eplb_gate, good, [
        (0, None, ARG), (0, F[0] + 1, ARG), (1, 3, ARG), (1, -1, ARG), (2, 255, ARG), (2, 1 << 62, LIMIT), (3, -1, ARG),
        (3, (1 << 25) + 1, LIMIT), (4, 0, ARG), ((2, 4, 8), (4097, 4097, 1), LIMIT), (5, 0, ARG), (5, 65, LIMIT),
        ((4, 5, 8), (4, 5, 1), ARG), (6, 2, ARG), (8, 0, ARG), (8, 7, DIV), (8, 128, LIMIT), (9, 0, ARG), (9, 9, ARG),
        (10, 0, ARG), (10, 3, ARG), ((4, 8, 5), (8, 8, 1), ARG), (14, None, ARG), (15, None, ARG), (14, F[0], ARG),
        (15, F[1] + 4, ARG), (14, F[2] + 9, ARG), (15, F[3] + 4, ARG)])
    assert eplb.lib.eplb_gate(None, 1, 256, 0, 256, 8, 0, None, 1, 1, 1, 1, 1.0, None, None, None, None) == 0


def test_loss_refusals(eplb):
    need = eplb.gate_loss_workspace_bytes(10, 256, 3)
    # ..., mask 13, seg 14, S 15, alpha 16, workspace 17, bytes 18, ids 19, weights, loss, counts, prob, tokens 24
    good = [F[0], 1, 256, 10, 256, 8, 0, None, 8, 4, 2, 1, 1.0, None, F[1], 3, 0.1, F[2], need,
            F[3], F[4], F[5], F[6], F[7], F[8], None]
    refuses(eplb.lib.eplb_gate_loss, good, [
        (0, None, ARG), (8, 7, DIV), (14, None, ARG), (15, 0, ARG), (15, (1 << 20) + 1, LIMIT), (17, None, ARG),
        (17, F[2] + 8, ARG), (18, need - 1, ARG), (19, None, ARG), (20, None, ARG), (21, None, ARG), (22, None, ARG),
        (23, None, ARG), (24, None, ARG), (24, F[1], ARG), (22, F[2] + 16, ARG), (17, F[0], ARG)])
    good = [F[0], 1, 256, 10, 256, F[9], 8, 0, None, F[1], 3, 0.1, F[2], need, F[5], F[6], F[7], F[8], None]
    refuses(eplb.lib.eplb_balance_loss, good, [
        (0, None, ARG), (5, None, ARG), (6, 0, ARG), (6, 65, LIMIT), (7, 5, ARG), (9, None, ARG), (10, 0, ARG),
        (12, None, ARG), (13, need - 1, ARG), (14, None, ARG), (17, None, ARG), (14, F[9] + 4, ARG)])
    for args, code in (((-1, 8, 1), ARG), ((1, 0, 1), ARG), ((1, 8, 0), ARG), ((1, 4097, 1), LIMIT)):
        with pytest.raises(eplb.EplbError) as e:
            eplb.gate_loss_workspace_bytes(*args)
        assert e.value.code == code
    # logits, dtype, ld, T, E, ids 5, K, scoring, normalize, scale, mask 10, d_weights, seg, S, alpha, counts 15, tokens,
    # d_loss, d_logits 18
    good = [F[0], 1, 256, 10, 256, F[1], 8, 0, 1, 1.0, None, F[2], F[3], 3, 0.1, F[4], F[5], F[6], F[7], None]
    refuses(eplb.lib.eplb_gate_backward, good, [
        (0, None, ARG), (5, None, ARG), (12, None, ARG), (13, 0, ARG), (13, (1 << 20) + 1, LIMIT), (15, None, ARG),
        (16, None, ARG), (18, None, ARG), (18, F[7] + 1, ARG), (18, F[0] + 16, ARG), (18, F[2], ARG), (18, F[4], ARG)])


def test_group_refusals(eplb):
    need = eplb.group_rows_workspace_bytes(2, 8192, 288)
    assert need > 0 and eplb.group_rows_workspace_bytes(2, 2048, 288) == 0
    good = [F[0], 2, 8192, 0, 288, F[1], need, F[2], F[3], F[4], None]
    refuses(eplb.lib.eplb_group_rows, good, [
        (0, None, ARG), (1, -1, ARG), (1, (1 << 22) + 1, LIMIT), (2, -1, ARG), (2, 1 << 31, RANGE), (4, 0, ARG),
        (4, 8193, LIMIT), (5, None, ARG), (5, F[1] + 2, ARG), (6, need - 1, ARG), (7, None, ARG), (8, None, ARG),
        (9, None, ARG), (8, F[0], ARG), (9, F[3] + 4, ARG), (1, 1 << 21, LIMIT)])
    assert eplb.lib.eplb_group_rows(None, 0, 100, 0, 8, None, 0, None, None, None, None) == 0


def test_quantize_refusals(eplb):
    good = [F[0], 1, 512, 10, 500, F[1], F[2], None]
    refuses(eplb.lib.eplb_quantize_rows, good, [
        (0, None, ARG), (0, F[0] + 1, ARG), (1, 7, ARG), (2, 499, ARG), (3, -1, ARG), (3, 1 << 31, LIMIT), (4, 0, ARG),
        ((2, 4), (1 << 25, 1 << 25), LIMIT), (5, None, ARG), (6, None, ARG), (5, F[0] + 16, ARG), (6, F[1] + 4, ARG)])
    # x, dtype, ld, X, C, rows 5, R, K, offsets 8, G, Rp 10, q, scale
    good = [F[0], 1, 512, 10, 500, F[1], 40, 4, F[2], 5, 640, F[3], F[4], None]
    refuses(eplb.lib.eplb_quantize_columns, good, [
        (0, None, ARG), (1, 3, ARG), (2, 499, ARG), (3, -1, ARG), (4, 0, ARG), (6, -1, ARG), (7, 0, ARG), (8, None, ARG),
        (9, 0, ARG), (9, 8193, LIMIT), (10, 512, ARG), (10, 641, ARG), (11, None, ARG), (11, F[3] + 8, ARG),
        (12, None, ARG), (11, F[0], ARG), (12, F[2], ARG)])
    good = [F[0], 1, 3, 300, 200, F[1], F[2], F[3], F[4], None]
    refuses(eplb.lib.eplb_quantize_weights, good, [
        (0, None, ARG), (1, 3, ARG), (2, -1, ARG), (2, 8193, LIMIT), (3, 0, ARG), (4, 0, ARG), (5, None, ARG),
        (6, None, ARG), (7, None, ARG), (8, None, ARG), (7, F[1], ARG), (8, F[2] + 4, ARG), ((3, 4), (1 << 24, 1 << 24), LIMIT)])


def test_product_refusals(eplb):
    # q, scale, X, w, w_scale, offsets 5, G, rows 7, R, topk, N 10, K, dtype, y 13
    good = [F[0], F[1], 10, F[2], F[3], F[4], 4, F[5], 20, 2, 96, 256, 1, F[6], None]
    refuses(eplb.lib.eplb_expert_matmul, good, [
        (0, None, ARG), (0, F[0] + 8, ARG), (1, None, ARG), (2, -1, ARG), (3, None, ARG), (3, F[2] + 4, ARG), (4, None, ARG),
        (5, None, ARG), (6, 0, ARG), (6, 8193, LIMIT), (8, -1, ARG), (8, 1 << 31, LIMIT), (9, 0, ARG), (10, 0, ARG),
        (10, (1 << 24) + 1, LIMIT), (11, 0, ARG), (11, 264, ARG), (12, 3, ARG), (13, None, ARG), (13, F[6] + 8, ARG),
        (13, F[0], ARG), (13, F[2] + 4096, ARG), (13, F[5], ARG), ((8, 10), ((1 << 31) - 1, 1 << 24), LIMIT)])
    assert eplb.lib.eplb_expert_matmul(None, None, 0, None, None, None, 1, None, 0, 1, 8, 16, 1, None, None) == 0
    # dy, dy_scale, x, x_scale, offsets 4, G, R 6, Rp, N 8, K, dtype, dw 11
    good = [F[0], F[1], F[2], F[3], F[4], 4, 300, 768, 96, 256, 0, F[5], None]
    refuses(eplb.lib.eplb_expert_wgrad, good, [
        (0, None, ARG), (0, F[0] + 4, ARG), (1, None, ARG), (2, None, ARG), (2, F[2] + 8, ARG), (3, None, ARG), (4, None, ARG), (5, 0, ARG),
        (6, -1, ARG), (7, 640, ARG), (7, 769, ARG), (8, 0, ARG), (9, 0, ARG), (10, 3, ARG), (11, None, ARG),
        (11, F[5] + 8, ARG), (11, F[0], ARG), (11, F[3], ARG)])


def test_binding_refusals(eplb):
    """What the binding itself refuses, on host tensors."""
    import torch
    x = torch.zeros((4, 8))
    with pytest.raises(ValueError, match="GPU"):
        eplb.gate(x, 2)
    with pytest.raises(ValueError, match="GPU"):
        eplb.quantize_rows(x)
    with pytest.raises(TypeError):
        eplb.gate(x.double(), 2)
    with pytest.raises(TypeError):
        eplb.quantize_weights(torch.zeros((1, 4, 4), dtype=torch.int32))
    with pytest.raises(ValueError):
        eplb.group_rows(torch.zeros((4,), dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        eplb.expert_matmul(x, x, torch.zeros((1, 4, 4)), x, torch.zeros((2,), dtype=torch.int32))
    assert eplb.padded_rows(0, 1) == 0 and eplb.padded_rows(1, 1) == 128 and eplb.padded_rows(129, 1) == 256
    assert eplb.padded_rows(8, 32) == 3968
