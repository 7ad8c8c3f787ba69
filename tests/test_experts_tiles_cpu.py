"""Tile counts of groups that overlap: offsets are data, and however they decrease
the count has to stay a count, as block numbers are made from it.  The device
code's own arithmetic, compiled for the host."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")

SOURCE = r"""
#include <cstdio>
#include <vector>
#include "experts_device.h"
using namespace eplb;

// All tiles of the groups, added in order and as a wave adds them.
static int32_t total(const std::vector<int32_t>& off, int32_t R, int32_t size, bool rest) {
  const int32_t G = (int32_t)off.size() - 1, n = rest ? G + 2 : G;
  int32_t all = 0, lane[64] = {};
  for (int32_t g = 0; g < n; ++g) {
    const Span s = group_span(off.data(), g, G, R);
    all = add_tiles(all, tiles_of(s, size));
    lane[g & 63] = add_tiles(lane[g & 63], tiles_of(s, size));
  }
  for (int d = 32; d > 0; d >>= 1)
    for (int l = 0; l < d; ++l) lane[l] = add_tiles(lane[l], lane[l + d]);
  return lane[0] == all ? all : -1;
}

int main() {
  const int32_t kMax = 2147483647;
  std::vector<int32_t> swing(8193), stairs(8193);
  for (int i = 0; i <= 8192; ++i) swing[i] = i & 1 ? kMax : 0, stairs[i] = i * 200 - 500;
  for (int size : {16, 32, 64, 128})
    for (bool rest : {false, true})
      if (total(swing, kMax, size, rest) != kMax) return 1;
  for (int size : {16, 32, 64, 128}) {
    // rows 0 .. 1638099 of groups (the first two groups and 100 rows lie before 0), 5000 behind them
    int64_t want = (100 + size - 1) / size + (int64_t)8189 * ((200 + size - 1) / size);
    if (total(stairs, 1637900 + 5000, size, false) != want) return 2;
    if (total(stairs, 1637900 + 5000, size, true) != want + (5000 + size - 1) / size) return 3;
  }
  if (total({7, 20, 20, 15, 900}, 50, 16, true) != 1 + 0 + 0 + 3 + 0 + 1) return 4;
  if (total({-3, kMax}, 0, 128, true) != 0 || total({0, 0}, kMax, 128, true) != 16777216) return 5;
  puts("ok");
  return 0;
}
"""


def test_tile_counts(tmp_path):
    src, exe = tmp_path / "tiles.hip", tmp_path / "tiles"
    src.write_text(SOURCE)
    pkg = os.path.join(ROOT, "moe_expert_load_eplb_amd", "csrc")
    subprocess.run([HIPCC, "--offload-host-only", "-O1", "-std=c++17", "-I", pkg, "-I", os.path.join(ROOT, "include"),
                    str(src), "-o", str(exe)], check=True, capture_output=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout == "ok\n"
