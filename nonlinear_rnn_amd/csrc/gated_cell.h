// The step of the gated linear recurrence, for its scan and its decode step.
#pragma once

#include <type_traits>

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

// The cells of prn_decode_step: x the projected values [f | v] or [f | i | v].
// They are not rounded to the storage type on the way.
template <int G_>
struct CellGated {
  static constexpr int G = G_, S = 1;
  static constexpr __host__ __device__ float scale(int) { return 1.0f; }
  static __device__ __forceinline__ void f(const float* x, const float* s, const float* /*as*/, const float* /*a*/, float* out) {
    const Gate f = gate_of(x[0]);
    const float in = G == 2 ? f.off : gate_of(x[1]).on;
    out[0] = fmaf(f.on, s[0], in * x[G - 1]);
  }
};

// cells without recurrent weights, whose projected values stay in fp32
template <class C> struct IsGated : std::false_type {};
template <int G> struct IsGated<CellGated<G>> : std::true_type {};

}  // namespace prn
