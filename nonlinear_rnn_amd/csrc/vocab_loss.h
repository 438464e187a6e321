// Softmax cross entropy over a vocabulary: plan and launches (vocab_loss.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace prn {

struct LossArgs {
  bool bf16;          // storage of x, W, dx, dW
  int target_bytes;   // 4 or 8
  int64_t N, V, d;
  float scale;
  int64_t ignore;
  uint8_t* ws;
  hipStream_t stream;
};

// do the tiles of every launch fit one grid?
bool loss_fits(const LossArgs& a);
size_t loss_workspace(const LossArgs& a);
size_t loss_backward_workspace(const LossArgs& a);

// loss, lse: N fp32
void launch_loss(const LossArgs& a, const void* x, const void* W, const void* targets, float* loss, float* lse);
// dx / dW may be null; dlse may be null
void launch_loss_backward(const LossArgs& a, const void* x, const void* W, const void* targets, const float* lse,
                          const float* dloss, const float* dlse, void* dx, void* dW);

}  // namespace prn
