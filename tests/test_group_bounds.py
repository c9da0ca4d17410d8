"""Bounds of the grouped kernels' index arithmetic, run on the CPU (no GPU needed): the
functions that the kernels call, compiled for the host."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "w8a8_fp8_block_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

MAIN = r"""
#include <cstdio>
#include "group_tiles.h"
using namespace fp8q;
// Every 128-column half of every 256-column tile of N columns: a row of the N / 128
// scale rows, and its own where it has one.
int main() {
  for (uint32_t blocks = 1; blocks <= 300; ++blocks) {
    const uint32_t N = blocks * kGroup;
    for (uint32_t n0 = 0; n0 < N; n0 += 256)
      for (uint32_t half = 0; half < 2; ++half) {
        const uint32_t row = scale_row(n0, half, N), own = n0 / kGroup + half;
        if (row >= blocks || (own < blocks && row != own)) {
          std::printf("N=%u n0=%u half=%u: row %u of %u\n", N, n0, half, row, blocks);
          return 1;
        }
      }
  }
  return 0;
}
"""


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="no hipcc")
def test_weight_scale_rows(tmp_path):
    src, exe = tmp_path / "bounds.hip", tmp_path / "bounds"
    src.write_text(MAIN)
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
                    "-packed-fp32-ops", "-w", "-I", CSRC, "-I", os.path.join(ROOT, "include"), src, "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
