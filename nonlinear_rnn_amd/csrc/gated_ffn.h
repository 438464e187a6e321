// Gated feed-forward product: plan and launches (gated_ffn.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace prn {

struct GatedFfnArgs {
  bool bf16, silu;
  int64_t N, d, F;
  uint8_t* ws;
  hipStream_t stream;
};

// do the launches fit their grids and offsets?
bool gated_ffn_fits(const GatedFfnArgs& a);
bool gated_ffn_backward_fits(const GatedFfnArgs& a);   // those of the gradients alone
size_t gated_ffn_workspace(const GatedFfnArgs& a);
void launch_gated_ffn(const GatedFfnArgs& a, const void* x, const void* W, void* out);
// dx / dW may be null
size_t gated_ffn_backward_workspace(const GatedFfnArgs& a);
void launch_gated_ffn_backward(const GatedFfnArgs& a, const void* x, const void* W, const void* dout, void* dx, void* dW);

}  // namespace prn
