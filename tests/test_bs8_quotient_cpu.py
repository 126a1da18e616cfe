"""The quotient without a division that the block-scaled codes are made from
(csrc/bs8.cuh): the product by the rounded inverse, corrected once by its
remainder, lies on the same side of every point where a code changes as the
IEEE quotient, for bf16 values.

Quotients do not depend on powers of two, so a scale is its significand.  A code
changes at k + 1/2 (int8, and e4m3 below 2^-6 in its steps) and at the odd
16ths of a binade (e4m3); only the bf16 values beside scale * such a point can
come near it.  The test takes every 83rd of the 2^23 significands; with a step
of 1 the harness goes through all of them."""
import shutil
import subprocess

import pytest

HARNESS = r"""
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
static float of(uint32_t u) { float f; memcpy(&f, &u, 4); return f; }
static uint32_t bits(float f) { uint32_t u; memcpy(&u, &f, 4); return u; }
static int side(float y, float b) { return y < b ? -1 : y > b; }
int main(int, char** argv) {
  const long from = atol(argv[1]), step = atol(argv[2]);
  long checks = 0, bad = 0;
  for (long m = from; m < 1 << 23; m += step) {
    const float s = of(0x3F800000u | (uint32_t)m), inv = 1.f / s;
    for (int k = 0; k < 127 + 8; ++k) {
      const float b = k < 127 ? k + 0.5f : (17 + 2 * (k - 127)) / 16.f;
      const uint32_t near = bits((float)((double)b * s)) & 0xFFFF0000u;
      for (int e = -1; e <= 2; ++e) {
        const float x = of(near + (uint32_t)e * 0x10000u);
        const float y = x / s;
        float q = x * inv;
        q = fmaf(fmaf(q, s, -x), -inv, q);
        ++checks;
        bad += side(q, b) != side(y, b);
      }
    }
  }
  printf("%ld %ld\n", checks, bad);
  return 0;
}
"""


def test_the_corrected_product_gives_the_codes_of_the_quotient(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "quotient.cpp", tmp_path / "quotient"
    src.write_text(HARNESS)
    r = subprocess.run([cxx, "-std=c++17", "-O2", "-ffp-contract=off", str(src), "-o", str(exe), "-lm"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    checks, bad = map(int, subprocess.run([str(exe), "0", "83"], capture_output=True, text=True, check=True).stdout.split())
    assert checks > 5e7 and bad == 0
