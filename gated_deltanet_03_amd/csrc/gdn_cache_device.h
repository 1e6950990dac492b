// Device helpers of the paged cache: which sequence a token row belongs to.
#pragma once

#include "gdn_cache_internal.h"
#include "gdn_device.h"

namespace gdn {

// The sequence of token row t (cu[s] <= t < cu[s + 1]), or -1 behind the last one: 64 offsets at a time, one a
// lane, so a few thousand sequences take two steps.  The whole wave calls it with one t.
__device__ __forceinline__ int find_sequence(const int32_t* __restrict__ cu, int N, int t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = N;                       // the answer is among [lo, lo + n)
  while (true) {
    const int step = (n + 63) / 64;
    const int at = lo + (lane + 1) * step; // lane counts if all sequences before `at` end at or before t
    const bool before = (lane + 1) * step <= n && cu[at < N ? at : N] <= t;
    const int full = __popcll(__ballot(before));
    lo += full * step;
    n = n - full * step < step ? n - full * step : step;
    if (n <= 0) return -1;
    if (step == 1) return cu[lo] <= t ? lo : -1;
  }
}

}  // namespace gdn
