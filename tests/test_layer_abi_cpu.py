"""The entry points of include/eplb_layer.h on a machine without a GPU: all are
exported, the header is C99, every call refuses bad arguments on the host with
the documented codes before it touches the device, and the binding refuses what
does not fit together."""
from __future__ import annotations

import os
import re
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "eplb_layer.h")
LIB = os.path.join(ROOT, "moe_expert_load_eplb_amd", "libeplb.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libeplb.so not built")

F = [0x10000000 * (i + 1) for i in range(16)]    # never dereferenced: every call below fails validation first
ARG, LIMIT = 1, 5


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


def test_exports(eplb):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^\s*[a-z_0-9]+\s+(eplb_[a-z_0-9]+)\s*\(", text, flags=re.M)
    assert len(names) == 6 and set(names) <= set(eplb.EXPORTS)


def test_header_is_c99(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "eplb_layer.h"\nint main(void) { return eplb_combine_rows(0, 0, 0, 0, 0, 0, 0, 1, 0, 0, 0) == '
                   "EPLB_E_ARG ? 0 : 1; }\n")
    exe = str(tmp_path / "h")
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src),
                    "-o", exe, "-L", os.path.dirname(LIB), "-leplb", "-Wl,-rpath," + os.path.dirname(LIB)], check=True)
    assert subprocess.run([exe]).returncode == 0


def test_matmul16_refusals(eplb):
    # x, dtype, ld 2, X, w 4, offsets, G 6, rows, R 8, topk, N 10, C, transpose 12, y_dtype, y 14
    good = [F[0], 1, 264, 10, F[1], F[2], 4, F[3], 20, 2, 96, 256, 0, 1, F[4], None]
    both = [
        (0, None, ARG), (0, F[0] + 8, ARG), (1, 0, ARG), (1, 3, ARG), (2, 95, ARG), (2, 260, ARG), (3, -1, ARG),
        (3, 1 << 31, LIMIT), (4, None, ARG), (4, F[1] + 8, ARG), (5, None, ARG), (6, 0, ARG), (6, 8193, LIMIT),
        (8, -1, ARG), (8, 1 << 31, LIMIT), (9, 0, ARG), (10, 0, ARG), (11, 0, ARG), (11, 252, ARG),
        (2, (1 << 22) + 8, LIMIT), (13, 3, ARG), (14, None, ARG), (14, F[4] + 8, ARG), (14, F[0], ARG), (14, F[2], ARG),
        (14, F[1] + 4096, ARG), (14, F[3], ARG)]
    refuses(eplb.lib.eplb_expert_matmul16, good, both + [
        (10, (1 << 22) + 1, LIMIT), ((2, 11), (1 << 23, 1 << 23), LIMIT), ((8, 10), ((1 << 31) - 1, 1 << 22), LIMIT)])
    good[12] = 1
    refuses(eplb.lib.eplb_expert_matmul16, good, both + [
        (10, 90, ARG), (11, (1 << 22) + 8, LIMIT), ((8, 11), ((1 << 31) - 1, 1 << 22), LIMIT)])
    assert eplb.lib.eplb_expert_matmul16(None, 1, 8, 0, None, None, 1, None, 0, 1, 8, 8, 0, 1, None, None) == 0


def test_wgrad16_refusals(eplb):
    # dy, dtype, dy_ld 2, R, x 4, ld, X 6, offsets, G 8, rows, topk 10, N, C 12, dw_dtype, dw 14
    good = [F[0], 1, 96, 20, F[1], 256, 10, F[2], 4, F[3], 2, 96, 256, 0, F[4], None]
    refuses(eplb.lib.eplb_expert_wgrad16, good, [
        (0, None, ARG), (0, F[0] + 2, ARG), (1, 0, ARG), (2, 88, ARG), (2, 100, ARG), (2, (1 << 22) + 8, LIMIT), (3, -1, ARG),
        (3, 1 << 31, LIMIT), (4, None, ARG), (4, F[1] + 2, ARG), (5, 248, ARG), (5, 260, ARG), (6, -1, ARG), (7, None, ARG),
        (8, 0, ARG), (8, 8193, LIMIT), (10, 0, ARG), (11, 90, ARG), (12, 250, ARG), (13, 3, ARG), (14, None, ARG),
        (14, F[4] + 4, ARG), (14, F[0], ARG), (14, F[1] + 16, ARG), (14, F[2], ARG),
        ((2, 5, 8, 11, 12), (1 << 22, 1 << 22, 8192, 1 << 22, 1 << 22), LIMIT)])


def test_four_bit_refusals(eplb):
    # w, dtype, G 2, N, C 4, q, scale 6
    good = [F[0], 1, 3, 300, 96, F[1], F[2], None]
    refuses(eplb.lib.eplb_quantize_weights4, good, [
        (0, None, ARG), (0, F[0] + 8, ARG), (1, 3, ARG), (2, -1, ARG), (2, 8193, LIMIT), (3, 0, ARG), (4, 0, ARG), (4, 80, ARG),
        (3, (1 << 22) + 1, LIMIT), (4, (1 << 22) + 32, LIMIT), (5, None, ARG), (5, F[1] + 8, ARG), (6, None, ARG),
        (5, F[0] + 32, ARG), (6, F[1] + 5, ARG), (6, F[0], ARG), ((2, 3, 4), (8192, 1 << 20, 128), LIMIT)])
    assert eplb.lib.eplb_quantize_weights4(None, 0, 0, 4, 32, None, None, None) == 0
    # x, dtype, ld 2, X, q 4, scale, offsets 6, G, rows 8, R, topk 10, N, C 12, y_dtype, y 14
    good = [F[0], 2, 256, 10, F[1], F[2], F[3], 4, F[5], 20, 2, 97, 256, 1, F[4], None]
    refuses(eplb.lib.eplb_expert_matmul4, good, [
        (0, None, ARG), (0, F[0] + 8, ARG), (1, 0, ARG), (2, 248, ARG), (2, 257, ARG), (3, -1, ARG), (4, None, ARG),
        (4, F[1] + 8, ARG), (5, None, ARG), (5, F[2] + 1, ARG), (6, None, ARG), (7, 0, ARG), (7, 8193, LIMIT), (9, -1, ARG),
        (9, 1 << 31, LIMIT), (10, 0, ARG), (11, 0, ARG), (11, (1 << 22) + 1, LIMIT), (12, 240, ARG), (13, -1, ARG),
        (14, None, ARG), (14, F[4] + 8, ARG), (14, F[1], ARG), (14, F[2], ARG), (14, F[5], ARG),
        ((9, 11), ((1 << 31) - 1, 1 << 22), LIMIT)])


def test_combine_refusals(eplb):
    # y, dtype, R 2, C, place 4, weights, T 6, K, out_dtype 8, out
    good = [F[0], 1, 40, 100, F[1], F[2], 10, 4, 1, F[3], None]
    refuses(eplb.lib.eplb_combine_rows, good, [
        (0, None, ARG), (0, F[0] + 1, ARG), (1, 3, ARG), (2, -1, ARG), (2, 1 << 31, LIMIT), (3, 0, ARG),
        (3, (1 << 24) + 1, LIMIT), (4, None, ARG), (4, F[1] + 2, ARG), (5, F[2] + 2, ARG), (6, -1, ARG), (6, 1 << 29, LIMIT),
        (7, 0, ARG), (7, 65, LIMIT), (8, 3, ARG), (9, None, ARG), (9, F[3] + 1, ARG), (9, F[0] + 64, ARG), (9, F[1], ARG),
        (9, F[2], ARG)])
    assert eplb.lib.eplb_combine_rows(None, 1, 0, 8, None, None, 0, 4, 1, None, None) == 0
    # d_out, dtype, y 2, y_dtype, C 4, place, order 6, weights, T 8, K, d_y 10, d_weights
    good = [F[0], 1, F[1], 1, 100, F[2], F[3], F[4], 10, 4, F[5], F[6], None]
    refuses(eplb.lib.eplb_combine_rows_backward, good, [
        (0, None, ARG), (0, F[0] + 1, ARG), (1, 3, ARG), (2, None, ARG), (2, F[1] + 1, ARG), (3, -1, ARG), (4, 0, ARG),
        (4, (1 << 24) + 1, LIMIT), (5, None, ARG), (6, None, ARG), (6, F[3] + 1, ARG), (7, F[4] + 2, ARG), (8, -1, ARG),
        (8, 1 << 29, LIMIT), (9, 0, ARG), (9, 65, LIMIT), (10, None, ARG), (10, F[5] + 1, ARG), (11, F[6] + 2, ARG),
        (10, F[1], ARG), (10, F[0], ARG), (11, F[5] + 400, ARG), (11, F[4], ARG), (10, F[2], ARG)])


def test_binding_refusals(eplb):
    """What the binding itself refuses, on host tensors."""
    x, w = torch.zeros((4, 32), dtype=torch.bfloat16), torch.zeros((2, 8, 32), dtype=torch.bfloat16)
    off = torch.tensor([0, 2, 4], dtype=torch.int32)
    for call in (lambda: eplb.expert_matmul16(x, w, off), lambda: eplb.expert_wgrad16(x, x, off),
                 lambda: eplb.expert_matmul4(x, w, w, off), lambda: eplb.quantize_weights4(w),
                 lambda: eplb.combine_rows(x, off[:2].view(1, 2), None)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for t in (x.float(), x.double(), x.int()):
        with pytest.raises(TypeError):
            eplb.expert_matmul16(t, w, off)
        with pytest.raises(TypeError):
            eplb.expert_wgrad16(t, x, off)
        with pytest.raises(TypeError):
            eplb.expert_matmul4(t, w, w, off)
    with pytest.raises(ValueError, match="weights must be"):
        eplb.combine_rows(x, off, torch.zeros((4,)))
    with pytest.raises(ValueError, match="place must be"):
        eplb.combine_rows(x, off, None)
    with pytest.raises(ValueError, match="elements"):
        eplb.combine_rows(x, off, torch.zeros((4, 2)))
    with pytest.raises(ValueError, match="d_out"):
        eplb.combine_rows_backward(x, x, off, off, torch.zeros((3, 1)))
