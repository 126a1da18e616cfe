// The hash table of changed tokens in the logits kernel (logits.cu): which slot
// a token has.  On its own, so that it also compiles for the host, where a test
// lets other threads act between any two of its accesses.
#pragma once

#include <stdint.h>

namespace pkv {

constexpr int kSlots = 2048;                // of the table
constexpr int kList = 1024;                 // tokens entered; a CTA's threads more may be before all see that it is full
constexpr uint32_t kEmpty = 0xFFFFFFFFu;

__device__ __forceinline__ uint32_t first_slot(int at) { return ((uint32_t)at * 2654435769u) >> 21; }
static_assert(kSlots == 1 << 11, "first_slot");

// The slot of token `at`, entered if it is new (open addressing).  With `may_overflow`
// -1 once kList tokens are entered: then the caller does the pass again over fewer
// tokens, and it does not matter that this one may be among the kList.  A pass of at
// most kList tokens, or of lists of at most kList ids, never fills the table: it does
// not ask, since what it is told may be that others entered this very token last.
// Table: key(i) reads a slot, claim(i, at) enters `at` into an empty one and returns
// what was there, full() says that kList tokens are entered.
template <typename Table>
__device__ __forceinline__ int slot_of(const Table& table, int at, bool may_overflow, bool& entered) {
  uint32_t i = first_slot(at);
  for (int tries = 0; tries < kSlots; ++tries, i = (i + 1) & (kSlots - 1)) {
    uint32_t k = table.key(i);
    if (k == (uint32_t)at) return (int)i;
    if (k != kEmpty) continue;
    if (may_overflow && table.full()) return -1;
    k = table.claim(i, (uint32_t)at);
    entered = k == kEmpty;
    if (entered || k == (uint32_t)at) return (int)i;
  }
  return -1;
}

}  // namespace pkv
