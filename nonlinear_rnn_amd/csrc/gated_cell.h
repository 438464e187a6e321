// The gates of the linear recurrence and the feed-forward product.
#pragma once

#include "prn_device.h"

namespace prn {

// s(x) = 1 / (1 + 2^(-x log2 e)) and s(-x) = 1 - s(x), each to a few 2^-24 of
// itself: the smaller of the two comes from the quotient, the larger one is 1
// less that, so a gate next to 1 is off by its own rounding only (over n steps
// the state keeps their product).
struct Gate {
  float on, off;
};
__device__ __forceinline__ Gate gate_of(float x) {
  const float e = ex2(-kLog2e * x), r = rcp(1.0f + e);
  const bool open = e <= 1.0f;
  const float lo = open ? e * r : r, hi = 1.0f - lo;   // (x = -inf: e = inf, r = 0)
  return {open ? hi : lo, open ? lo : hi};
}

}  // namespace prn
