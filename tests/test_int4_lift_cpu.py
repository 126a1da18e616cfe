"""The 4-bit decode's rules for setting a reference and a lift again (csrc/int4_lift.cuh), compiled
for the host: behind a correction the same scores and rows are not voted on again (a vote that leads
nowhere would come back at every step), also not if they come out a little larger the next time,
weights fit fp16, and the lift leaves as many bits as there are."""
import shutil
import subprocess

import pytest

from paged_kv_gqa_append_gb300 import build as B

HARNESS = r"""
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <random>
using std::ceil;
#define __device__
#define __forceinline__ inline
static unsigned __float_as_uint(float x) { unsigned u; memcpy(&u, &x, 4); return u; }
static float __uint_as_float(unsigned u) { float x; memcpy(&x, &u, 4); return x; }
#include "int4_lift.cuh"
using namespace pkv;

constexpr int kN = 32, kLane = 4;  // slots of a head in a step, and a lane's
struct Head {
  float ref = -1.5e38f, lift = 0x1p126f;
};
struct Rows {
  float x[kN], vs[kN], vl[kN];
};

static bool vote(const Head& h, const Rows& r, float more) {
  bool any = false;
  for (int i = 0; i < kN; i += kLane) {
    float p = 0, y = 0, z = 0;
    for (int j = i; j < i + kLane; ++j) {
      const float q = exp2f(r.x[j] - h.ref) * more;
      p += q;
      y += q * h.lift * r.vs[j];
      z += q * h.lift * r.vl[j];
    }
    any |= i4_votes(p, y, z);
  }
  return any;
}

int main() {
  std::mt19937 g(5);
  std::uniform_real_distribution<float> u(0, 1);
  long votes = 0, again = 0, large = 0, small = 0;
  for (int trial = 0; trial < 200000; ++trial) {
    Head h;
    // scores and rows alike or spread, of any size
    const float spread = trial % 3 ? 6 * u(g) * u(g) : 0, vary = trial % 2 ? 4 * u(g) : 0;
    const float size = exp2f(200 * u(g) - 100), offset = trial % 5 ? 8 : 0, centre = trial % 7 ? 40 * u(g) - 20 : 3;
    for (int step = 0; step < 4; ++step) {
      Rows r;
      const float grown = step > 1 ? exp2f(3 * u(g)) : 1;
      for (int i = 0; i < kN; ++i) {
        r.x[i] = centre + spread * u(g) + (step > 2 ? 2 * u(g) : 0);
        r.vs[i] = size * exp2f(vary * u(g)) * grown;
        r.vl[i] = -offset * r.vs[i];
      }
      if (vote(h, r, 1)) {
        ++votes;
        float top = -INFINITY, most = 0;
        for (float x : r.x) top = fmaxf(top, x);
        const float now = i4_reference(h.ref, top);
        h.lift = fminf(h.lift * exp2f(now - h.ref), 0x1p126f);
        h.ref = now;
        for (int i = 0; i < kN; ++i) most = fmaxf(most, exp2f(r.x[i] - now) * fmaxf(r.vs[i], 0.0625f * fabsf(r.vl[i])));
        const float lift = i4_lift(h.lift, most);
        if (lift < h.lift) small += most * lift < 0x1p12f;
        h.lift = lift;
        again += vote(h, r, 1) || vote(h, r, 1.001f);
      }
      for (int i = 0; i < kN; ++i) large += exp2f(r.x[i] - h.ref) * h.lift * r.vs[i] > 65504.f;
    }
  }
  printf("%ld %ld %ld %ld\n", votes, again, large, small);
  return 0;
}
"""


def test_a_correction_settles(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "lift.cpp", tmp_path / "lift"
    src.write_text(HARNESS)
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-I", B.CSRC, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    votes, again, large, small = map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split())
    assert votes > 200000 and again == 0 and large == 0 and small == 0
