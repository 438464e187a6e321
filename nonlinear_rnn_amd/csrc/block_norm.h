// Norms at a block boundary with gate and residual scale: launches (block_norm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace prn {

constexpr int64_t kBlockNormMaxWidth = 8192;

struct BlockNormArgs {
  bool bf16;
  int act;            // PRN_ACT_SILU | PRN_ACT_SIGMOID
  int64_t N, d;
  float eps;
  const float *w_post, *w_pre, *alpha;     // d each, or null
  const void *h, *gate, *x;                // N x d; gate, x may be null
  void *r_out, *n_out;                     // forward
  const void *dr, *dn;                     // backward; dr may be null, dn with w_pre null
  void *dh, *dgate, *dx;                   // may be null
  float *dw_post, *dw_pre, *dalpha;        // may be null
  uint8_t* ws;
  hipStream_t stream;
};

size_t block_norm_backward_workspace(bool bf16, int64_t N, int64_t d);
void launch_block_norm(const BlockNormArgs& a);
void launch_block_norm_backward(const BlockNormArgs& a);

}  // namespace prn
