"""The hash table of the logits kernel (csrc/logits_table.cuh), compiled for the
host, with another thread acting between any two accesses of the first."""
import shutil
import subprocess

import pytest

from paged_kv_gqa_append_gb300 import build as B

HARNESS = r"""
#include <cstdio>
#include <cstring>
#define __device__
#define __forceinline__ inline
#include "logits_table.cuh"
using namespace pkv;

struct State {
  uint32_t keys[kSlots];
  int listed, accesses, when, other;   // before access `when` another thread enters token `other`
  void clear() { memset(keys, 0xFF, sizeof(keys)); listed = accesses = 0; when = -1; }
  void enter(uint32_t at) {            // all of it at once
    uint32_t i = first_slot((int)at);
    while (keys[i] != kEmpty && keys[i] != at) i = (i + 1) % kSlots;
    if (keys[i] == kEmpty) { keys[i] = at; ++listed; }
  }
  void step() { if (accesses++ == when) enter((uint32_t)other); }
};
struct Table {
  State* s;
  uint32_t key(uint32_t i) const { s->step(); return s->keys[i]; }
  uint32_t claim(uint32_t i, uint32_t at) const {
    s->step();
    const uint32_t was = s->keys[i];
    if (was == kEmpty) s->keys[i] = at;
    return was;
  }
  bool full() const { s->step(); return s->listed >= kList; }
};

int main() {
  static State s;
  long bad = 0, cases = 0, gone = 0;
  for (int count = kList - 3; count <= kList; ++count)          // a pass of `count` tokens, all of them listed
    for (int last = 0; last < count; ++last)
      for (int other = last, k = 0; k < 2; other = (last + 1) % count, ++k)
        for (int when = 0; when < 12; ++when) {
          s.clear();
          for (int at = 0; at < count; ++at)
            if (at != last && at != other) s.enter((uint32_t)at);
          s.when = when;
          s.other = other;
          bool entered = false;
          const int slot = slot_of(Table{&s}, last, false, entered);
          ++cases;
          gone += !entered;
          bad += slot < 0 || s.keys[slot] != (uint32_t)last;
          int copies = 0;
          for (int i = 0; i < kSlots; ++i) copies += s.keys[i] == (uint32_t)last;
          bad += copies != 1;
        }
  // a pass of more tokens: full says so, and the tokens that are in it are still found
  s.clear();
  for (int at = 0; at < kList; ++at) s.enter((uint32_t)(3 * at));
  for (int at = 0; at < 3 * kList; ++at) {
    bool entered = false;
    const int slot = slot_of(Table{&s}, at, true, entered);
    bad += entered || (at % 3 ? slot >= 0 : slot < 0 || s.keys[slot] != (uint32_t)at);
  }
  printf("%ld %ld %ld\n", bad, cases, gone);
  return 0;
}
"""


def test_a_pass_that_fits_loses_no_token(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "table.cpp", tmp_path / "table"
    src.write_text(HARNESS)
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-I", B.CSRC, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    bad, cases, gone = map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split())
    assert bad == 0 and cases > 90000
    assert gone > 1000                     # the other thread was first in many of them
