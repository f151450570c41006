// ring.cuh -- bookkeeping of a ring of stages in shared memory, apart from any
// CUDA call so that it can be checked on the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define WQL_RING_FN __host__ __device__ __forceinline__
#else
#define WQL_RING_FN inline
#endif

namespace wql {

// Fill i goes to slot i % ring and completes phase i / ring of that slot's
// barrier.  Before its block ends, a thread that has issued copies for fills
// 0 .. fills-1 waits for the last one of every slot (it issued a later one only
// after those before had been used): wait(slot, parity) -> did it complete.
template <typename Wait>
WQL_RING_FN bool drain_ring(int fills, int ring, Wait wait) {
  bool ok = true;
  for (int s = 0; s < ring && s < fills; ++s)
    ok = wait(s, (uint32_t)(((fills - 1 - s) / ring) & 1)) && ok;
  return ok;
}

}  // namespace wql
