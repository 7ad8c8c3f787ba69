"""Which form the products of given sizes take: the host's own rules, compiled by
themselves.  The GPU tests of the forms run the sizes listed here, so that a limit
that moves is seen as a size that has left its form."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from layer_forms import LARGE, STREAM, STREAM_FORMS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include "stream16.h"
using namespace eplb;

// for every R, outputs, groups, 4 bits, transposed: the form that the launches choose (operands below 2^31 bytes)
int main(int argc, char** argv) {
  for (int i = 1; i + 4 < argc; i += 5) {
    const int64_t R = atoll(argv[i]), N = atoll(argv[i + 1]);
    const int32_t G = atoi(argv[i + 2]);
    const bool four = atoi(argv[i + 3]) != 0, transposed = atoi(argv[i + 4]) != 0;
    if (!transposed && stream_suits(R, G)) {
      const StreamPlan p = plan_stream(R, N, G, four);
      printf("stream %d %d\n", p.mt, p.share);
    } else {
      puts(large_suits(R, N, G, four) ? "large" : "small");
    }
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def forms(tmp_path_factory):
    at = tmp_path_factory.mktemp("forms")
    (at / "forms.hip").write_text(SOURCE)
    subprocess.run([HIPCC, "--offload-host-only", "-O1", "-std=c++17", "-I",
                    os.path.join(ROOT, "moe_expert_load_eplb_amd", "csrc"), "-I", os.path.join(ROOT, "include"),
                    str(at / "forms.hip"), "-o", str(at / "forms")], check=True, capture_output=True)

    def ask(sizes):
        args = [str(int(v)) for s in sizes for v in s]
        return subprocess.run([str(at / "forms"), *args], capture_output=True, text=True, check=True).stdout.splitlines()
    return ask


def test_streaming_forms(forms):
    sizes = [(head + sum(counts) + tail, N, len(counts), four, 0) for four, _, counts, head, tail, N, _, _ in STREAM]
    for case, got in zip(STREAM, forms(sizes)):
        assert got == "stream %d %d" % case[1], case
    for four, want in STREAM_FORMS.items():
        assert {c[1] for c in STREAM if c[0] == four} == want


def test_large_tiles(forms):
    for transposed in (0, 1):
        listed = [c for c in LARGE if not (transposed and c[0])]
        sizes = [(head + sum(counts) + tail, width, len(counts), four, transposed)
                 for four, counts, head, tail, width, _ in listed]
        assert forms(sizes) == ["large"] * len(listed)
