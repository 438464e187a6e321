// Products of few rows with a gated end: the feed-forward product and the
// decode step of the gated linear cells (gated_few.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace prn {

// rows x (N, K) against the `parts` rows r, R + r, .. of W (parts R, K) for each of R outputs
struct GatedFewArgs {
  bool bf16;
  int64_t N, R, K;
  const void *x, *W;
  hipStream_t stream;
};

// out (N, R) = act(g) u: two parts
void launch_few_ffn(const GatedFewArgs& a, bool silu, void* out);
// state_out and, where not null, h_out (N, R) from state_in (null: zeros) and the
// parts [f | v] or [f | i | v] with their bias (null: none)
void launch_few_step(const GatedFewArgs& a, int parts, const float* bias, const void* state_in, void* state_out, void* h_out);

}  // namespace prn
