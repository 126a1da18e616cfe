// Where a new token of a ragged append goes (bs8_append.cu).  On its own, so that
// the checks also compile for the host, where a test goes through them.
#pragma once

namespace pkv {

// A token's place: its sequence and position; ok only if both can be used.
struct Place {
  int seq, pos, end;      // end: the row behind the sequence's last new token
  bool live, ok, first;   // live: the token belongs to a sequence; first: of its new ones
};

// Row t of T, found in a sequence that brings rows [lo, hi) and then holds `len` tokens,
// at most `most`: a.pos, and a.ok if 0 <= pos < len and t < hi <= T, whatever the
// numbers are (cu_new may not ascend, lengths may be anything).
__device__ __forceinline__ void set_place(Place& a, int t, int T, int lo, int hi, int len, int most) {
  if (lo < 0 || lo > t || hi <= t || hi > T) return;  // not ascending, or beyond the rows given
  a.end = hi;
  const int fresh = hi - lo;
  if (len < fresh || len > most) return;
  a.pos = len - fresh + (t - lo);
  a.ok = true;
  a.first = t == lo;
}

}  // namespace pkv
