// Embedding lookup and its gradient: plan and launches (embed.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace prn {

struct EmbedArgs {
  bool bf16;
  int token_bytes;    // 4 or 8
  int64_t N, V, d;
  float scale;
  int64_t pad;
  uint8_t* ws;
  hipStream_t stream;
};

size_t embed_backward_workspace(const EmbedArgs& a);
void launch_embed(const EmbedArgs& a, const void* tokens, const void* table, void* out);
void launch_embed_backward(const EmbedArgs& a, const void* tokens, const void* dout, void* dtable);

}  // namespace prn
