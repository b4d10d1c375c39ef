// Hand-offs between the warp roles of block_cache_kernel, apart from the instructions that they are
// made of: plain C++, so that the host can run them with copies and barriers of its own.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KVARN_ROLE __device__ __forceinline__
#else
#define KVARN_ROLE inline
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
    for (int i = issued > slots ? issued - slots : 0; i < issued; ++i)
      if (!wait(i % slots, (uint32_t)(i / slots) & 1u)) all = false;
    return all;
  }
};

}  // namespace blk
}  // namespace kvarn
