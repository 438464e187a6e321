// Dropout from a counter: launches (dropout.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace prn {

struct DropoutArgs {
  bool bf16;
  int64_t n;
  uint32_t drop;           // of 65536 numbers, those below it drop their element
  float scale;             // of the elements that stay
  uint64_t seed, offset;
  const int64_t* state;    // device (seed, offset) instead, or null
  hipStream_t stream;
};

// residual may be null
void launch_dropout(const DropoutArgs& a, const void* x, const void* residual, void* out);

}  // namespace prn
