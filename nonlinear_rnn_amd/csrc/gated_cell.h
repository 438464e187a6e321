// The gates of the linear recurrence and the feed-forward product.
#pragma once

#include "prn_device.h"

namespace prn {

// s(x) = 1 / (1 + 2^(-x log2 e)) and s(-x), each to |x| + 4 times 2^-24 of itself
// (the exponent's rounding, and the power's, the sum's and the quotient's): s(-x)
// is the exponential times the quotient, and s(x) 1 less that where it is the
// larger one, so that a gate next to 1 is off by little more than its own rounding
// (over n steps the state keeps their product).  Neither instruction has results
// below the normal numbers: a gate below 2^-126 is 0, and from 2^126 on the
// quotient is 0 too, where s(-x) is 1.
struct Gate {
  float on, off;
};
__device__ __forceinline__ Gate gate_of(float x) {
  const float e = ex2(-kLog2e * x), r = rcp(1.0f + e);
  const float off = e > 0x1p126f ? 1.0f : e * r;   // of NaN: NaN, both
  return {e <= 1.0f ? 1.0f - off : r, off};
}

}  // namespace prn
