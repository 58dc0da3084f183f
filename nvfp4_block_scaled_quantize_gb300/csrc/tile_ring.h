// Position of one thread in a ring of STAGES tile buffers that one thread of the CTA, the owner,
// fills ahead by asynchronous copies, a barrier each (checkpoint.cu). Plain C++, so that its waits
// can be followed on the host.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define NVFP4_HD __host__ __device__ __forceinline__
#else
#define NVFP4_HD inline
#endif

namespace nvfp4 {

// The tile at the ring's position completes phase `parity` of barrier `stage`. Before the wait for
// it, it and at most the kAhead - 1 tiles after it have been fetched and not waited for.
//
// A wait that gives up leaves the thread `dead`: its later waits are skipped, so that every thread
// still reaches every barrier of the CTA, and the owner fetches no more. The owner waits for the
// copies in flight there and then, while it still stands at the tile that they are counted from:
// the CTA must not leave its shared memory to a copy that is yet to land.
template <int STAGES>
struct TileRing {
  static constexpr int kAhead = STAGES > 1 ? STAGES - 1 : 1;
  int stage = 0;
  uint32_t parity = 0;
  bool dead = false;

  // wait(stage, parity): true once that phase has completed, false after a limit. fetched(i):
  // whether the tile i after this one exists (the owner has then fetched it).
  template <class Wait, class Fetched>
  NVFP4_HD void wait(bool owner, Wait&& wait, Fetched&& fetched) {
    if (dead || wait(stage, parity)) return;
    dead = true;
    if (owner)
      for (int i = 0; i < kAhead; i++)
        if (fetched(i)) {
          const bool wraps = stage + i >= STAGES;
          wait(wraps ? stage + i - STAGES : stage + i, wraps ? parity ^ 1u : parity);
        }
  }
  NVFP4_HD void next() {
    if (++stage == STAGES) {
      stage = 0;
      parity ^= 1u;
    }
  }
};

}  // namespace nvfp4
