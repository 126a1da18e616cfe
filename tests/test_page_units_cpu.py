"""How a release shares out its rows and layers (csrc/page_units.cuh), compiled for the host:
every pair once, also where rows times layers pass 31 and 32 bits."""
import shutil
import subprocess

import pytest

from paged_kv_gqa_append_gb300 import build as B

HARNESS = r"""
#include <cstdio>
#include <initializer_list>
#include <vector>
#define __device__
#define __forceinline__ inline
#include "page_units.cuh"
using namespace pkv;

int main() {
  long bad = 0;
  for (int rows : {1, 2, 7, 64, 300})
    for (int layers : {1, 2, 3, 16, 33, 1000})
      for (int warps : {1, 32, 33, 4864}) {
        std::vector<int> seen((size_t)rows * layers, 0);
        for (int w = 0; w < warps; ++w)
          for (UnitWalk u(w, warps, layers); u.row < rows; u.next()) {
            if (u.row < 0 || u.layer < 0 || u.layer >= layers) return 1;
            ++seen[(size_t)u.row * layers + u.layer];
          }
        for (int n : seen) bad += n != 1;
      }
  // 4096 rows of so many layers: the warps' shares, of units in their order
  for (int layers : {524287, 524288, 524289, 1 << 20, (1 << 20) + 5}) {
    const long long all = 4096ll * layers;
    const int warps = 4864;
    for (int w : {0, 1, 2500, warps - 1}) {
      long long at = w;
      for (UnitWalk u(w, warps, layers); u.row < 4096; u.next(), at += warps)
        bad += u.row != at / layers || u.layer != at % layers;
      bad += at < all || at - warps >= all;
    }
  }
  UnitWalk far(4863, 4864, 1 << 30);
  for (; far.row < 1; far.next()) bad += far.layer < 0 || far.layer >= 1 << 30;
  printf("%ld\n", bad);
  return 0;
}
"""


def test_every_row_and_layer_once(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "units.cpp", tmp_path / "units"
    src.write_text(HARNESS)
    r = subprocess.run([cxx, "-std=c++17", "-O2", "-I", B.CSRC, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True, timeout=300).stdout == "0\n"
