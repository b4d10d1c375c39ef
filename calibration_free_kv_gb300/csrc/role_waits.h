// Hand-offs between the warp roles of block_cache_kernel, apart from the instructions that they are
// made of: plain C++, so that the host can run them with copies and barriers of its own.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KVARN_ROLE __device__ __forceinline__
#define KVARN_ROLLED _Pragma("unroll 1")  // a wait is in every role: its code is kept short
#else
#define KVARN_ROLE inline
#define KVARN_ROLLED
#endif

namespace kvarn {
namespace blk {

// The copies a loader has issued into a ring of `slots` slots.  Copy i goes to slot i % slots and
// completes phase i / slots of that slot's barrier; a page whose copy is not issued takes no place.
struct CopyRing {
  int slots;
  int issued = 0, slot = 0;
  uint32_t phase = 0;
  KVARN_ROLE explicit CopyRing(int n) : slots(n) {}
  KVARN_ROLE void next() {  // the copy into `slot` has been issued
    ++issued;
    if (++slot == slots) {
      slot = 0;
      phase ^= 1u;
    }
  }
  // wait(slot, parity) for every copy that may be in flight; whether all of them landed
  template <class Wait>
  KVARN_ROLE bool drain(Wait wait) const {
    bool all = true;
    KVARN_ROLLED for (int i = issued > slots ? issued - slots : 0; i < issued; ++i)
      if (!wait(i % slots, (uint32_t)(i / slots) & 1u)) all = false;
    return all;
  }
};

// A wait for a page's copy or MMAs.  poll() asks the barrier; issued() says whether the MMA warp it
// waits for has issued the page (true where no MMA is waited for).  The barrier alone is not enough:
// a completion that never came leaves its phase behind, and a phase one behind reads as complete for
// a page that is not issued yet.  The role would run ahead and arrive twice at a named barrier that
// its partner has not passed.  When the wait runs out, abort() is called and the role goes on all the
// same: every role runs through all its pages, so that no named barrier is left waiting, and the
// call's results are flagged.  From then on a wait ends once the page is issued, which keeps the
// roles within two pages of each other as the completed MMAs would.
// A wait runs out after kWaitNs of wall time; kEndNs ends it even if the page is still not issued
// (the roles that issue it give up their own waits in between, so this is not reached).
constexpr uint64_t kWaitNs = 2000000000ull, kEndNs = 10000000000ull;
template <class Poll, class Issued, class Aborted, class Abort, class Now>
KVARN_ROLE void wait_page(Poll poll, Issued issued, Aborted aborted, Abort abort, Now now) {
  uint64_t t0 = 0;
  KVARN_ROLLED for (uint32_t n = 1; n != 0; ++n) {
    const bool go = issued();  // read ahead of the poll, whose latency covers it
    if (poll() && go) return;
    if ((n & 255u) != 0) continue;
    const uint64_t t = now();
    if (t0 == 0) t0 = t;
    if (t - t0 >= kWaitNs) abort();
    if (aborted() && go) return;
    if (t - t0 >= kEndNs) return;
  }
}

// A wait for work that may rightly last as long as a segment: it gives up, and returns false, once
// progress() (pages issued) has not moved for kNoProgressNs.
constexpr uint64_t kNoProgressNs = 4000000000ull;
template <class Poll, class Progress, class Now>
KVARN_ROLE bool wait_progress(Poll poll, Progress progress, Now now) {
  if (poll()) return true;
  int seen = progress();
  uint64_t t0 = now();
  KVARN_ROLLED for (uint32_t n = 1; n != 0; ++n) {
    if (poll()) return true;
    if ((n & 255u) != 0) continue;
    const int at = progress();
    const uint64_t t = now();
    if (at != seen) {
      seen = at;
      t0 = t;
    } else if (t - t0 >= kNoProgressNs) {
      return false;
    }
  }
  return false;
}

// The query warps publish segments 0, 1, .. and every role takes them in order.  A role that gave up
// waiting must not end alone: the others meet it at named barriers, which nothing bounds.  So the
// number of published segments and the end are one word: publishing takes it from k to k + 1 in one
// step, a role that gives up sets kGateClosed, which freezes the number, and every role ends after
// the same segments, whichever of the two came first.
constexpr uint32_t kGateClosed = 1u << 31;
template <class Cas>
KVARN_ROLE bool gate_publish(Cas cas, int k) {  // cas(expected, desired) returns the value before
  return cas((uint32_t)k, (uint32_t)k + 1u) == (uint32_t)k;
}
// Whether segment k is there for a role that has waited for it (or given up and closed the gate).
KVARN_ROLE bool gate_open(uint32_t gate, int k) {
  return (gate & kGateClosed) == 0u || (gate & ~kGateClosed) > (uint32_t)k;
}

}  // namespace blk
}  // namespace kvarn
