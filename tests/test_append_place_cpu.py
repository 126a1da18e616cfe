"""Where the block-scaled append puts a token (csrc/append_place.cuh), compiled for
the host: whatever cu_new and seq_lens hold, a place that is used lies inside
the sequence, and its rows inside those given."""
import shutil
import subprocess

import pytest

from paged_kv_gqa_append_gb300 import build as B

HARNESS = r"""
#include <cstdint>
#include <initializer_list>
#include <cstdio>
#define __device__
#define __forceinline__ inline
#include "append_place.cuh"
using namespace pkv;

int main() {
  const int T = 7;
  const int rows[] = {INT32_MIN, -9, -1, 0, 1, 2, 3, 5, 6, 7, 8, 99, 1 << 29, INT32_MAX};
  const int lens[] = {INT32_MIN, -7, -1, 0, 1, 2, 3, 6, 7, 8, 31, 32, 33, INT32_MAX};
  long used = 0, bad = 0, missed = 0;
  for (int t = 0; t < T; ++t)
    for (int lo : rows)
      for (int hi : rows)
        for (int len : lens)
          for (int most : {1, 32, INT32_MAX}) {
            Place a{0, 0, t + 1, true, false, false};
            set_place(a, t, T, lo, hi, len, most);
            const bool right = 0 <= lo && lo <= t && t < hi && hi <= T && len >= hi - lo && len <= most;
            missed += right != a.ok;
            if (!a.ok) continue;
            ++used;
            bad += a.pos < 0 || a.pos >= len || a.pos != len - (hi - t) || a.end != hi || a.first != (t == lo);
          }
  printf("%ld %ld %ld\n", used, bad, missed);
  return 0;
}
"""


def test_places_stay_inside_their_sequence(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "place.cpp", tmp_path / "place"
    src.write_text(HARNESS)
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-I", B.CSRC, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    used, bad, missed = map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split())
    assert used > 500 and bad == 0 and missed == 0
