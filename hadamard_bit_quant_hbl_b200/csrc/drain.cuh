// Which copies a warp still has to wait for once a bounded wait has run out: none may be landing in shared
// memory, or counting on a barrier there, when the CTA exits. Plain counting, which the host can compile too.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define HBL_COUNT __host__ __device__ __forceinline__
#else
#define HBL_COUNT inline
#endif

namespace hbl {

// Copies counted on one barrier, each started after the one before it has been waited for: number i (from 0)
// completes phase i, whose parity is i & 1.
struct LoneCopies {
  uint32_t started = 0;
  HBL_COUNT void start() { ++started; }
  HBL_COUNT uint32_t parity() const { return (started - 1u) & 1u; }  // of the newest one's phase
  // wait(parity) for the newest one, which may still be landing
  template <typename W>
  HBL_COUNT void drain(W wait) const {
    if (started > 0) wait(parity());
  }
};

// Copies through a ring of N barriers, started and used in the same order, at most N started ahead of the
// oldest one that has not been used.
template <int N>
struct RingCopies {
  int stage = 0;        // of the oldest one not used, and the parity of its phase
  uint32_t parity = 0;
  int ahead = 0;        // how many of them there are
  HBL_COUNT void start() { ++ahead; }
  HBL_COUNT void use() {
    --ahead;
    if (++stage == N) {
      stage = 0;
      parity ^= 1u;
    }
  }
  // wait(stage, parity) for each that may still be landing
  template <typename W>
  HBL_COUNT void drain(W wait) {
    while (ahead > 0) {
      wait(stage, parity);
      use();
    }
  }
};

}  // namespace hbl
