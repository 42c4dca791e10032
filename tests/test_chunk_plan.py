"""The lengths of pieces of chunk attention's plan, compiled for the host: no choice but those that are
weighed against the workspace's bound may cut a tile."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

DRIVER = r"""
#include <cstdio>
#include "dgt_chunk_plan.h"
using namespace dgt::serve;
static bool sound(uint32_t units) {
  for (uint32_t i = 0; i < kChoices; ++i) {
    const uint32_t len = piece_units(units, i);
    const uint64_t pieces = ((uint64_t)units + len - 1) / len;
    if (len < 1 || (units > 1 && len < 2) || (i == 0 && pieces != 1) || (uint64_t)len * 64 > 0x80000000ull) {
      printf("units %u choice %u: pieces of %u\n", units, i, len);
      return false;
    }
  }
  return true;
}
int main() {
  for (uint32_t units = 1; units < 100000; ++units) if (!sound(units)) return 1;
  for (uint32_t power = 17; power <= 25; ++power)
    for (uint32_t d = 0; d < 2000; ++d) {
      const uint32_t units = (1u << power) - 1000 + d;
      if (units <= 1u << 25 && !sound(units)) return 1;
    }
  puts("ok");
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_the_first_choice_cuts_nothing(tmp_path):
    """Also above 2^24 units, which fp32 does not count; and no piece is longer than 2^31 keys."""
    src, exe = tmp_path / "driver.cpp", str(tmp_path / "driver")
    src.write_text(DRIVER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(ROOT, "decode_gemm_tile_amd", "csrc"), str(src), "-o", exe],
                   check=True, capture_output=True, timeout=120)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout
